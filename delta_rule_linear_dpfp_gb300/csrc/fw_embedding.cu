// fw_embedding.cu -- the rows of a table that a batch of tokens names, and
// the table's gradient.
//
//   out_n = scale E[id_n];   dE[v] = scale sum over n with id_n = v of dout_n.
// A negative id is padding: zeros out, no gradient.  An id past the table's
// end gives a row of NaN, and no gradient.
//
// Bound by the bytes: each row that is named is read once for every time it is
// named (from L2 where it is named often), each row of the output written once.
//
// The gradient goes by sorted tokens, so that every row is summed in an order that
// depends on the ids alone (no atomics, the same bits in every run), in three kernels:
//  1. One cluster of eight CTAs sorts the pairs (id, n) by id, eight bits at
//     a time from the lowest, each pass stable.  A CTA owns an eighth of the
//     sequence; the counts of the digits are exchanged through distributed
//     shared memory; a warp owns 32 to 256 pairs in a row and ranks equal digits
//     by its lanes' votes on the digits' bits.  The sort is all latency and takes eight SMs:
//     another kernel writes the table's zeros on the others meanwhile.
//  2. A group of threads sums 32 sorted pairs (8 where there are few), run by run:
//     a run that ends on both sides is rounded and written, one that goes on
//     beyond leaves its sum in 32 bits.  Every group reads as many rows as any
//     other, whatever a token's share of the batch is.
//  3. A CTA for each such run adds its parts, its groups of threads taking them
//     in turn, the groups' sums in order.  (One CTA even where one token is the whole
//     batch: 65 536 of D 1024 take 214 us instead of 91.)
#include "fw_common.cuh"
#include "fw_ends.h"
#include "fw_pairs.cuh"

#include <algorithm>

namespace fw {

namespace {

constexpr int kT = 256;

// 8 channels as they were loaded.
template <typename T> struct Raw;
template <> struct Raw<float> {
    float4 a, b;
    FW_DEV void load(const float *p) {
        a = __ldcg(reinterpret_cast<const float4 *>(p));
        b = __ldcg(reinterpret_cast<const float4 *>(p) + 1);
    }
    FW_DEV void add_to(float (&s)[8]) const {
        s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
        s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
    }
};
template <> struct Raw<__nv_bfloat16> {
    uint4 u;
    FW_DEV void load(const __nv_bfloat16 *p) { u = __ldcg(reinterpret_cast<const uint4 *>(p)); }
    FW_DEV void add_to(float (&s)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            s[2 * i] += __uint_as_float(w[i] << 16);
            s[2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

// ------------------------------------------------------------------ lookup
// A group of 2^lg threads takes kAhead rows at a time: their ids, then their
// rows, 8 channels a thread, are requested before any is written.
constexpr int kAhead = 4;
template <typename T>
__global__ void __launch_bounds__(kT, sizeof(T) == 2 ? 6 : 4)
    embedding_kernel(Tokens ids, const T *table, T *out, int64_t N, int V, int D, int lg, float scale) {
    griddep_launch_dependents();
    griddep_wait();
    ids.p = after_wait(ids.p);
    table = after_wait(table);
    const int lane = threadIdx.x & ((1 << lg) - 1), per = kT >> lg;
    const int64_t n0 = ((int64_t)blockIdx.x * per + (threadIdx.x >> lg)) * kAhead;
    int id[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
        id[u] = n0 + u < N ? token_at(ids, n0 + u, V) : -1;
    for (int c = 8 * lane; c < D; c += 8 << lg) {
        Raw<T> v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (id[u] >= 0 && id[u] < V)
                v[u].load(table + (int64_t)id[u] * D + c);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (n0 + u < N) {
                float o[8] = {};
                if (id[u] >= 0 && id[u] < V)
                    v[u].add_to(o);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = id[u] < V ? o[e] * scale : __int_as_float(0x7fffffff);
                store8_stream(out + (n0 + u) * D + c, o);
            }
    }
}

// -------------------------------------------------------------------- sort
constexpr int kCluster = 8, kSortT = 1024, kWarps = kSortT / 32, kPerLane = 8, kTile = kSortT * kPerLane;

FW_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What cluster rank `rank` holds at this CTA's shared location p.
FW_DEV unsigned peer_load(const unsigned *p, unsigned rank) {
    unsigned a = (unsigned)__cvta_generic_to_shared(p), v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

struct SortArgs {
    Tokens ids;
    int N, V, passes;
    int2 *pair[2]; // (key, position), from one to the other and back
    uint4 *zeros;         // a small table, cleared here
    int64_t nzeros;
};

// The live lanes of the warp that hold this lane's digit, by the votes on its eight bits.
FW_DEV unsigned peers(unsigned digit, unsigned live) {
    unsigned same = __ballot_sync(0xffffffffu, live);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
        const bool one = digit >> b & 1;
        const unsigned votes = __ballot_sync(0xffffffffu, one);
        same &= one ? votes : ~votes;
    }
    return same;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortT) sort_tokens_kernel(SortArgs a) {
    __shared__ unsigned hist[256], offset[256], rows[kWarps][256];
    __shared__ unsigned scan[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // (in this order: what starts beside this kernel does so when everything before it is complete)
    griddep_wait();
    griddep_launch_dependents();
    const unsigned rank = blockIdx.x;
    for (int64_t i = (int64_t)rank * kSortT + tid; i < a.nzeros; i += kCluster * kSortT)
        a.zeros[i] = make_uint4(0, 0, 0, 0);
    a.ids.p = after_wait(a.ids.p);
    // this CTA's part of the sequence: a multiple of 32 pairs, or of a tile where it does not fit one
    int64_t part = (((int64_t)a.N + kCluster - 1) / kCluster + 31) / 32 * 32;
    const bool one = part <= kTile;
    if (!one)
        part = (part + kTile - 1) / kTile * kTile;
    const int64_t lo = min((int64_t)a.N, part * rank), hi = min((int64_t)a.N, part * (rank + 1));
    const int per = one ? (int)((part + kSortT - 1) / kSortT) : kPerLane; // pairs of a lane in a tile

    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 8 * pass;
        const int2 *in = pass & 1 ? a.pair[1] : a.pair[0];
        int2 *out = pass & 1 ? a.pair[0] : a.pair[1];
        auto pair_at = [&](int64_t i) {
            if (pass)
                return __ldcg(in + i);
            const int t = token_at(a.ids, i, a.V);
            return make_int2(t < 0 ? a.V : t, (int)i); // padding behind every row
        };
        int key[kPerLane], pos[kPerLane];
        unsigned at[kPerLane]; // rank among the warp's pairs with this digit
        int64_t w0 = 0;
        // a tile's pairs into registers, ranked; rows[w][d] = how many of warp w have digit d
        auto rank_tile = [&](int64_t t0) {
            w0 = t0 + (int64_t)warp * 32 * per + lane;
#pragma unroll
            for (int u = 0; u < kPerLane; ++u) {
                const int64_t i = w0 + 32 * u;
                const bool live = u < per && i < hi;
                const int2 p = live ? pair_at(i) : make_int2(0, 0);
                key[u] = p.x;
                pos[u] = p.y;
            }
            for (int e = lane; e < 256; e += 32)
                rows[warp][e] = 0;
            __syncwarp();
#pragma unroll
            for (int u = 0; u < kPerLane; ++u)
                if (u < per) {
                    const unsigned live = w0 + 32 * u < hi, digit = (unsigned)key[u] >> shift & 255u;
                    const unsigned same = peers(live ? digit : 0u, live);
                    const unsigned seen = rows[warp][digit];
                    at[u] = seen + __popc(same & ((1u << lane) - 1));
                    __syncwarp();
                    if (live && lane == __ffs(same) - 1)
                        rows[warp][digit] = seen + __popc(same);
                    __syncwarp();
                }
            __syncthreads();
        };
        // rows[w][d] = o[d] + what the warps before w have of digit d; returns o + all (threads below 256)
        auto scan_warps = [&](unsigned o) {
#pragma unroll 16
            for (int k = 0; k < kWarps; ++k) {
                const unsigned n = rows[k][tid];
                rows[k][tid] = o;
                o += n;
            }
            return o;
        };
        auto scatter = [&](bool add) {
#pragma unroll
            for (int u = 0; u < kPerLane; ++u)
                if (u < per && w0 + 32 * u < hi) {
                    const unsigned d = (unsigned)key[u] >> shift & 255u;
                    const unsigned o = rows[warp][d] + at[u] + (add ? offset[d] : 0u);
                    out[o] = make_int2(key[u], pos[u]);
                }
        };
        if (one) {
            rank_tile(lo);
            if (tid < 256)
                hist[tid] = scan_warps(0);
        } else {
            if (tid < 256)
                hist[tid] = 0;
            __syncthreads();
            for (int64_t i0 = lo; i0 < hi; i0 += kSortT) {
                const int64_t i = i0 + tid;
                const unsigned live = i < hi, digit = live ? (unsigned)pair_at(i).x >> shift & 255u : 0u;
                const unsigned same = peers(digit, live);
                if (live && lane == __ffs(same) - 1)
                    atomicAdd(hist + digit, __popc(same));
            }
        }
        cluster_sync(); // every CTA's counts stand
        if (tid < 256) {
            unsigned before = 0, all = 0; // of this digit: in the CTAs before, in all
#pragma unroll
            for (unsigned c = 0; c < kCluster; ++c) {
                const unsigned h = peer_load(hist + tid, c);
                before += c < rank ? h : 0u;
                all += h;
            }
            unsigned upto = all; // inclusive sum over the digits
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const unsigned t = __shfl_up_sync(0xffffffffu, upto, o);
                upto += lane >= o ? t : 0u;
            }
            if (lane == 31)
                scan[warp] = upto;
            asm volatile("bar.sync 1, 256;" ::: "memory");
            for (int k = 0; k < warp; ++k)
                upto += scan[k];
            offset[tid] = upto - all + before;
        }
        if (one) {
            __syncthreads();
            scatter(true);
        } else {
            cluster_sync(); // (the counts are read: a CTA may clear its own)
            for (int64_t t0 = lo; t0 < hi; t0 += kTile) {
                rank_tile(t0);
                if (tid < 256)
                    offset[tid] = scan_warps(offset[tid]);
                __syncthreads();
                scatter(false);
                __syncwarp(); // (a warp clears its own row alone)
            }
        }
        cluster_sync(); // the pairs stand, for every CTA; its counts are read
    }
}

// A large table's zeros, beside the sort: no wait at the start (the sort lets this kernel
// start only after its own), and one at the end, so that what follows this kernel follows
// the sort as well.
__global__ void __launch_bounds__(kT) zero_table_kernel(uint4 *zeros, int64_t n) {
    griddep_launch_dependents();
    const int64_t step = (int64_t)gridDim.x * kT;
    int64_t i = (int64_t)blockIdx.x * kT + threadIdx.x;
    for (; i + 3 * step < n; i += 4 * step)
#pragma unroll
        for (int u = 0; u < 4; ++u)
            __stcs(zeros + i + u * step, make_uint4(0, 0, 0, 0));
    for (; i < n; i += step)
        __stcs(zeros + i, make_uint4(0, 0, 0, 0));
    griddep_wait();
}

// -------------------------------------------------------------------- sums
// Rows in flight: 128 bytes a thread.
template <typename T> constexpr int kFlight = sizeof(T) == 2 ? 8 : 4;

struct SumArgs {
    const int2 *pair;     // sorted
    float *part;          // [chunks][2][D]: of the run that comes in, of the one that goes on
    int N, V, D, lg, lgc; // 2^lg threads a group, 2^lgc pairs a chunk
    float scale;
    int accumulate;
};

template <typename T> FW_DEV void write_row(const SumArgs &a, T *to, float (&s)[8]) {
    float old[8] = {};
    if (a.accumulate)
        load8(to, old);
#pragma unroll
    for (int x = 0; x < 8; ++x)
        s[x] = a.accumulate ? fmaf(s[x], a.scale, old[x]) : s[x] * a.scale;
    store8(to, s);
}

template <typename T>
__global__ void __launch_bounds__(kT, 3) chunk_sums_kernel(SumArgs a, const T *dout, T *dtable) {
    griddep_launch_dependents();
    griddep_wait();
    a.pair = after_wait(a.pair);
    dout = after_wait(dout);
    const int t = threadIdx.x & ((1 << a.lg) - 1), lane = threadIdx.x & 31;
    const int64_t k = (int64_t)blockIdx.x * (kT >> a.lg) + (threadIdx.x >> a.lg), i0 = k << a.lgc;
    const int count = (int)min((int64_t)1 << a.lgc, a.N - i0); // (groups are whole warps)
    if (count <= 0)
        return;
    // a lane holds a pair; `n` of them have a row, `ends` are the last of their run here
    const int2 own = lane < count ? __ldcg(a.pair + i0 + lane) : make_int2(-1, 0);
    const int key = own.x, pos = own.y;
    const int left = i0 > 0 ? __ldcg(a.pair + i0 - 1).x : -1;
    const int right = i0 + count < a.N ? __ldcg(a.pair + i0 + count).x : -1;
    const int next = __shfl_down_sync(0xffffffffu, key, 1);
    const bool last = lane == count - 1;
    const int n = __popc(__ballot_sync(0xffffffffu, lane < count && key < a.V)); // (padding is sorted behind)
    const unsigned ends = __ballot_sync(0xffffffffu, lane < n && (last || key != next));
    const bool first_comes_in = __shfl_sync(0xffffffffu, key, 0) == left;
    const int goes_on = __shfl_sync(0xffffffffu, key, count - 1) == right ? count - 1 : -1; // the pair whose run does
    for (int c = 8 * t; c - 8 * t < a.D; c += 8 << a.lg) {
        const bool on = c < a.D;
        float s[8] = {};
        bool comes_in = first_comes_in;
        for (int j0 = 0; j0 < n; j0 += kFlight<T>) {
            Raw<T> v[kFlight<T>];
#pragma unroll
            for (int u = 0; u < kFlight<T>; ++u) {
                const int p = __shfl_sync(0xffffffffu, pos, j0 + u);
                if (on && j0 + u < n)
                    v[u].load(dout + (int64_t)p * a.D + c);
            }
#pragma unroll
            for (int u = 0; u < kFlight<T>; ++u) {
                const int j = j0 + u;
                if (j >= n)
                    break;
                v[u].add_to(s);
                if (ends >> j & 1) {
                    const int id = __shfl_sync(0xffffffffu, key, j);
                    if (on) {
                        if (comes_in || j == goes_on)
                            store8(a.part + (2 * k + (comes_in ? 0 : 1)) * a.D + c, s);
                        else
                            write_row(a, dtable + (int64_t)id * a.D + c, s);
                    }
                    comes_in = false;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        s[x] = 0.f;
                }
            }
        }
    }
}

// The run that begins in chunk k and goes on beyond it: a CTA, its groups of
// threads taking the parts in turn.
template <typename T>
__global__ void __launch_bounds__(kT) join_runs_kernel(SumArgs a, T *dtable) {
    __shared__ float red[kT * 8];
    griddep_launch_dependents();
    griddep_wait();
    a.pair = after_wait(a.pair);
    a.part = after_wait(a.part);
    const int64_t k = blockIdx.x, i0 = k << a.lgc, size = (int64_t)1 << a.lgc;
    if (i0 + size >= a.N)
        return;
    // (all four requested at once)
    const int id = __ldcg(a.pair + i0 + size - 1).x, next = __ldcg(a.pair + i0 + size).x, first = __ldcg(a.pair + i0).x;
    const int before = i0 > 0 ? __ldcg(a.pair + i0 - 1).x : -1;
    if (id >= a.V || next != id || (first == id && before == id))
        return;
    // the chunks after this one that the run comes into: their first pair has its id
    int64_t end = k + 1;
    for (bool more = true; more;) {
        const int64_t i = (end + (threadIdx.x & 31)) << a.lgc;
        const unsigned in = __ballot_sync(0xffffffffu, i < a.N && __ldcg(a.pair + i).x == id);
        const int n = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
        end += n;
        more = n == 32;
    }
    const int t = threadIdx.x & ((1 << a.lg) - 1), g = threadIdx.x >> a.lg, groups = kT >> a.lg;
    for (int c = 8 * t; c - 8 * t < a.D; c += 8 << a.lg) {
        const bool on = c < a.D;
        float s[8] = {};
        constexpr int kU = 8;
        if (on)
            for (int64_t j = k + g; j < end; j += groups * kU) {
                Raw<float> v[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (j + u * groups < end)
                        v[u].load(a.part + (2 * (j + u * groups) + (j + u * groups == k ? 1 : 0)) * a.D + c);
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    if (j + u * groups < end)
                        v[u].add_to(s);
            }
        if (groups > 1) {
            __syncthreads();
            store8(red + threadIdx.x * 8, s);
            __syncthreads();
            if (g == 0)
                for (int o = 1; o < groups; ++o)
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        s[x] += red[((o << a.lg) + t) * 8 + x];
        }
        if (on && g == 0)
            write_row(a, dtable + (int64_t)id * a.D + c, s);
    }
}

// log2 of the threads of a row of D channels, 8 a thread (at most a CTA's).
int group_log2(int D) {
    int lg = 0;
    while ((8 << lg) < D && lg < 8)
        ++lg;
    return lg;
}
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T>
cudaError_t lookup(Tokens ids, const void *table, void *out, int64_t N, int V, int D, float scale, cudaStream_t st) {
    const int lg = group_log2(D), per = (kT >> lg) * kAhead;
    return launch_pdl(embedding_kernel<T>, dim3((unsigned)((N + per - 1) / per)), dim3(kT), 0, st, ids, (const T *)table,
                      (T *)out, N, V, D, lg, scale);
}

// Pairs of a chunk: fewer where the chunks are too few to occupy the SMs otherwise
// (16384 x 1024: 31.9 us with 32, 32.6 with 16, 36.6 with 8, whose open runs leave more sums;
// 65 rows of D 512: 2048 tokens 10.8 us with 8, 12.7 with 32, 4096 12.3 and 12.9, 8192 16.7 and 14.6).
int chunk_log2(int N) { return N <= 8192 ? 3 : 5; }
int64_t chunks_of(int N) { return ((int64_t)N + (1 << chunk_log2(N)) - 1) >> chunk_log2(N); }

template <typename T>
cudaError_t sums(const SumArgs &a, const void *dout, void *dtable, cudaStream_t st) {
    const int64_t chunks = chunks_of(a.N), per = kT >> a.lg;
    const cudaError_t e = launch_pdl(chunk_sums_kernel<T>, dim3((unsigned)((chunks + per - 1) / per)), dim3(kT), 0, st, a,
                                     (const T *)dout, (T *)dtable);
    if (e != cudaSuccess || chunks == 1)
        return e;
    return launch_pdl(join_runs_kernel<T>, dim3((unsigned)(chunks - 1)), dim3(kT), 0, st, a, (T *)dtable);
}

} // namespace

cudaError_t launch_embedding(Tokens ids, const void *table, void *out, int64_t N, int V, int D, float scale, int bf16,
                             cudaStream_t st) {
    return bf16 ? lookup<__nv_bfloat16>(ids, table, out, N, V, D, scale, st)
                : lookup<float>(ids, table, out, N, V, D, scale, st);
}

// the pairs twice, two sums of each chunk
size_t embedding_backward_workspace_bytes(int N, int V, int D) {
    (void)V;
    return 2 * up256(8 * (size_t)N) + 8 * (size_t)chunks_of(N) * D;
}

cudaError_t launch_embedding_backward(Tokens ids, const void *dout, void *dtable, void *workspace, int N, int V, int D,
                                      float scale, int accumulate, int bf16, cudaStream_t st) {
    SortArgs a = {};
    a.ids = ids;
    a.N = N;
    a.V = V;
    while (a.passes < 4 && ((unsigned)V >> (8 * a.passes)) != 0) // keys are 0 .. V
        ++a.passes;
    uint8_t *p = static_cast<uint8_t *>(workspace);
    for (int i = 0; i < 2; ++i) {
        a.pair[i] = reinterpret_cast<int2 *>(p);
        p += up256(8 * (size_t)N);
    }
    // the table's zeros: within the sort, or above a megabyte beside it (4096 tokens of D 512:
    // a table of a quarter of a megabyte 15.0 us within, 15.3 beside, half 15.6 and 15.5, one 16.7 and 15.6,
    // four 26 and 15.6)
    uint4 *zeros = static_cast<uint4 *>(dtable);
    const int64_t nzeros = accumulate ? 0 : (int64_t)V * D / (bf16 ? 8 : 4);
    const bool beside = nzeros > 1 << 16;
    a.zeros = zeros;
    a.nzeros = beside ? 0 : nzeros;
    cudaError_t e = launch_pdl(sort_tokens_kernel, dim3(kCluster), dim3(kSortT), 0, st, a);
    if (e == cudaSuccess && beside)
        e = launch_pdl(zero_table_kernel, dim3(152 * 3), dim3(kT), 0, st, zeros, nzeros);
    if (e != cudaSuccess)
        return e;
    const int lg = std::max(5, group_log2(D)); // (whole warps)
    const SumArgs s = {a.passes & 1 ? a.pair[1] : a.pair[0], reinterpret_cast<float *>(p), N, V, D, lg, chunk_log2(N),
                       scale, accumulate};
    return bf16 ? sums<__nv_bfloat16>(s, dout, dtable, st) : sums<float>(s, dout, dtable, st);
}

} // namespace fw
