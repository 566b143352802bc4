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
// The gradient goes by sorted tokens, so that every row is summed by one
// group of threads in the order of the tokens (no atomics, the same bits in
// every run), in three kernels:
//  1. One cluster of eight CTAs sorts the pairs (id, n) by id, eight bits at
//     a time from the lowest, each pass stable.  A CTA owns an eighth of the
//     sequence; the counts of the digits are exchanged through distributed
//     shared memory; inside a tile of 4096 pairs a warp owns 128 and ranks
//     equal digits by a match among its lanes.  Then begin and end of every
//     id's run are noted by id.
//  2. Where 32 pairs in a row from a multiple of 32 on have one id, their rows
//     are added in 32 bits: a token that makes up a sixteenth of the batch is
//     read by as many CTAs as it fills chunks.
//  3. A group of threads per table row adds what the run has before, in and
//     behind such chunks, and rounds once; rows without a token get zeros.
#include "fw_common.cuh"
#include "fw_ends.h"
#include "fw_pairs.cuh"

#include <algorithm>

namespace fw {

namespace {

constexpr int kT = 256;

FW_DEV void load8_cs(const float *p, float (&o)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}
FW_DEV void load8_cs(const __nv_bfloat16 *p, float (&o)[8]) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// ------------------------------------------------------------------ lookup
// A group of 2^lg threads takes kAhead rows at a time: their ids, then their
// rows, 8 channels a thread, are requested before any is written.
constexpr int kAhead = 4;
template <typename T>
__global__ void __launch_bounds__(kT)
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
        float v[kAhead][8];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (id[u] >= 0 && id[u] < V) {
                load8(table + (int64_t)id[u] * D + c, v[u]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[u][e] = id[u] < 0 ? 0.f : __int_as_float(0x7fffffff);
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (n0 + u < N) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[u][e] = id[u] < 0 ? 0.f : v[u][e] * scale;
                store8(out + (n0 + u) * D + c, v[u]);
            }
    }
}

// -------------------------------------------------------------------- sort
constexpr int kCluster = 8, kSortT = 1024, kWarps = kSortT / 32, kPerLane = 4, kTile = kSortT * kPerLane;

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
    int *key[2], *pos[2]; // the pairs, from one to the other and back
    int *begin, *end;     // [V] of each id's run (0, 0 for none)
};

// The lanes of the warp that hold this lane's digit (among `live` lanes).
FW_DEV unsigned peers(unsigned digit, unsigned live) { return __match_any_sync(0xffffffffu, digit | (live << 8)); }

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kSortT) sort_tokens_kernel(SortArgs a) {
    __shared__ unsigned hist[256], offset[256], rows[kWarps][256];
    __shared__ unsigned scan[8];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    unsigned rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    griddep_launch_dependents();
    griddep_wait();
    a.ids.p = after_wait(a.ids.p);
    for (int64_t v = (int64_t)rank * kSortT + tid; v < a.V; v += kCluster * kSortT)
        a.begin[v] = a.end[v] = 0;
    // this CTA's part of the sequence, in whole tiles
    const int64_t tiles = ((int64_t)a.N + kTile - 1) / kTile, mine = (tiles + kCluster - 1) / kCluster;
    const int64_t lo = min((int64_t)a.N, mine * rank * kTile), hi = min((int64_t)a.N, mine * (rank + 1) * kTile);

    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = 8 * pass;
        const int *key_in = pass & 1 ? a.key[1] : a.key[0], *pos_in = pass & 1 ? a.pos[1] : a.pos[0];
        int *key_out = pass & 1 ? a.key[0] : a.key[1], *pos_out = pass & 1 ? a.pos[0] : a.pos[1];
        auto key_at = [&](int64_t i) {
            if (pass)
                return __ldcg(key_in + i);
            const int t = token_at(a.ids, i, a.V);
            return t < 0 ? a.V : t; // padding behind every row
        };
        if (tid < 256)
            hist[tid] = 0;
        __syncthreads();
        for (int64_t i0 = lo; i0 < hi; i0 += kSortT) {
            const int64_t i = i0 + tid;
            const unsigned live = i < hi, digit = live ? (unsigned)key_at(i) >> shift & 255u : 0u;
            const unsigned same = peers(digit, live);
            if (live && lane == __ffs(same) - 1)
                atomicAdd(hist + digit, __popc(same));
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
        cluster_sync(); // (the counts are read: a CTA may clear its own)
        for (int64_t t0 = lo; t0 < hi; t0 += kTile) {
            for (int e = lane; e < 256; e += 32)
                rows[warp][e] = 0;
            __syncwarp();
            int key[kPerLane], pos[kPerLane];
            unsigned at[kPerLane]; // rank among the warp's pairs with this digit
            const int64_t w0 = t0 + (int64_t)warp * 32 * kPerLane + lane;
#pragma unroll
            for (int u = 0; u < kPerLane; ++u) {
                const int64_t i = w0 + 32 * u;
                key[u] = i < hi ? key_at(i) : 0;
                pos[u] = i < hi ? (pass ? __ldcg(pos_in + i) : (int)i) : 0;
            }
#pragma unroll
            for (int u = 0; u < kPerLane; ++u) {
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
            if (tid < 256) { // where each warp's pairs of this digit begin
                unsigned o = offset[tid];
#pragma unroll 8
                for (int k = 0; k < kWarps; ++k) {
                    const unsigned n = rows[k][tid];
                    rows[k][tid] = o;
                    o += n;
                }
                offset[tid] = o;
            }
            __syncthreads();
#pragma unroll
            for (int u = 0; u < kPerLane; ++u)
                if (w0 + 32 * u < hi) {
                    const unsigned o = rows[warp][(unsigned)key[u] >> shift & 255u] + at[u];
                    key_out[o] = key[u];
                    pos_out[o] = pos[u];
                }
            __syncwarp(); // (a warp clears its own row alone)
        }
        cluster_sync(); // the pairs stand, for every CTA
    }
    const int *key = a.passes & 1 ? a.key[1] : a.key[0];
    for (int64_t i = lo + tid; i < hi; i += kSortT) {
        const int k = __ldcg(key + i);
        if (k < a.V) {
            if (i == 0 || __ldcg(key + i - 1) != k)
                a.begin[k] = (int)i;
            if (i == a.N - 1 || __ldcg(key + i + 1) != k)
                a.end[k] = (int)i + 1;
        }
    }
}

// -------------------------------------------------------------------- sums
constexpr int kChunk = 32;

// The sum of rows pos[i], i = from, from + step, ... < to, 8 channels at c, added to s.
template <typename T>
FW_DEV void add_rows(const T *dout, const int *pos, int from, int to, int step, int D, int c, float (&s)[8]) {
    constexpr int kU = 4; // rows in flight
    int i = from;
    for (; i + (kU - 1) * step < to; i += kU * step) {
        float v[kU][8];
#pragma unroll
        for (int u = 0; u < kU; ++u)
            load8_cs(dout + (int64_t)__ldcg(pos + i + u * step) * D + c, v[u]);
#pragma unroll
        for (int u = 0; u < kU; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[e] += v[u][e];
    }
    for (; i < to; i += step) {
        float v[8];
        load8_cs(dout + (int64_t)__ldcg(pos + i) * D + c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[e] += v[e];
    }
}

// part[k] = the sum of chunk k's rows, where all of its 32 pairs have one id.
template <typename T>
__global__ void __launch_bounds__(kT)
    chunk_sums_kernel(const int *key, const int *pos, const T *dout, float *part, int N, int V, int D, int lg) {
    griddep_launch_dependents();
    griddep_wait();
    key = after_wait(key);
    pos = after_wait(pos);
    dout = after_wait(dout);
    const int lane = threadIdx.x & ((1 << lg) - 1), per = kT >> lg;
    const int k = blockIdx.x * per + (threadIdx.x >> lg);
    if (k >= N / kChunk)
        return;
    const int i0 = k * kChunk;
    const int id = __ldcg(key + i0);
    if (id >= V || __ldcg(key + i0 + kChunk - 1) != id)
        return;
    for (int c = 8 * lane; c < D; c += 8 << lg) {
        float s[8] = {};
        add_rows(dout, pos, i0, i0 + kChunk, 1, D, c, s);
        store8(part + (int64_t)k * D + c, s);
    }
}

// Table rows v0 .. v0 + kRows - 1 of each group of 2^lg threads.
constexpr int kRows = 4;
template <typename T>
__global__ void __launch_bounds__(kT)
    table_rows_kernel(const int *begin, const int *end, const int *pos, const T *dout, const float *part, T *dtable, int V,
                      int D, int lg, float scale, int accumulate) {
    griddep_launch_dependents();
    griddep_wait();
    begin = after_wait(begin);
    end = after_wait(end);
    pos = after_wait(pos);
    dout = after_wait(dout);
    part = after_wait(part);
    const int lane = threadIdx.x & ((1 << lg) - 1), per = kT >> lg;
    const int64_t v0 = ((int64_t)blockIdx.x * per + (threadIdx.x >> lg)) * kRows;
    int b[kRows], e[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        b[u] = v0 + u < V ? __ldcg(begin + v0 + u) : 0;
        e[u] = v0 + u < V ? __ldcg(end + v0 + u) : 0;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        if (v0 + u >= V || (accumulate && b[u] == e[u]))
            continue;
        for (int c = 8 * lane; c < D; c += 8 << lg) {
            float s[8] = {};
            // the whole chunks inside the run, and what is before and behind them
            const int k0 = (b[u] + kChunk - 1) / kChunk, k1 = e[u] / kChunk;
            if (k0 < k1) {
                add_rows(dout, pos, b[u], k0 * kChunk, 1, D, c, s);
                int k = k0;
                for (; k + 3 < k1; k += 4) {
                    float t[4][8];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        load8_cs(part + (int64_t)(k + j) * D + c, t[j]);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            s[x] += t[j][x];
                }
                for (; k < k1; ++k) {
                    float t[8];
                    load8_cs(part + (int64_t)k * D + c, t);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        s[x] += t[x];
                }
                add_rows(dout, pos, k1 * kChunk, e[u], 1, D, c, s);
            } else {
                add_rows(dout, pos, b[u], e[u], 1, D, c, s);
            }
            T *to = dtable + (v0 + u) * D + c;
            float old[8] = {};
            if (accumulate)
                load8(to, old);
#pragma unroll
            for (int x = 0; x < 8; ++x)
                s[x] = accumulate ? fmaf(s[x], scale, old[x]) : s[x] * scale;
            store8(to, s);
        }
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

template <typename T>
cudaError_t sums(const SortArgs &a, const void *dout, void *dtable, float *part, int D, float scale, int accumulate,
                 cudaStream_t st) {
    const int lg = group_log2(D), per = kT >> lg, chunks = a.N / kChunk;
    const int *key = a.key[a.passes & 1], *pos = a.pos[a.passes & 1];
    if (chunks) {
        const cudaError_t e = launch_pdl(chunk_sums_kernel<T>, dim3((chunks + per - 1) / per), dim3(kT), 0, st, key, pos,
                                         (const T *)dout, part, a.N, a.V, D, lg);
        if (e != cudaSuccess)
            return e;
    }
    return launch_pdl(table_rows_kernel<T>, dim3((unsigned)(((int64_t)a.V + per * kRows - 1) / (per * kRows))), dim3(kT), 0, st,
                      (const int *)a.begin, (const int *)a.end, pos, (const T *)dout, (const float *)part, (T *)dtable, a.V,
                      D, lg, scale, accumulate);
}

} // namespace

cudaError_t launch_embedding(Tokens ids, const void *table, void *out, int64_t N, int V, int D, float scale, int bf16,
                             cudaStream_t st) {
    return bf16 ? lookup<__nv_bfloat16>(ids, table, out, N, V, D, scale, st)
                : lookup<float>(ids, table, out, N, V, D, scale, st);
}

// keys and positions twice, begin and end of each id's run, the chunks' sums
size_t embedding_backward_workspace_bytes(int N, int V, int D) {
    return 4 * up256(4 * (size_t)N) + 2 * up256(4 * (size_t)V) + up256(4 * (size_t)(N / kChunk) * D);
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
    auto take = [&](size_t bytes) {
        uint8_t *q = p;
        p += up256(bytes);
        return q;
    };
    for (int i = 0; i < 2; ++i) {
        a.key[i] = reinterpret_cast<int *>(take(4 * (size_t)N));
        a.pos[i] = reinterpret_cast<int *>(take(4 * (size_t)N));
    }
    a.begin = reinterpret_cast<int *>(take(4 * (size_t)V));
    a.end = reinterpret_cast<int *>(take(4 * (size_t)V));
    float *part = reinterpret_cast<float *>(p);
    const cudaError_t e = launch_pdl(sort_tokens_kernel, dim3(kCluster), dim3(kSortT), 0, st, a);
    if (e != cudaSuccess)
        return e;
    return bf16 ? sums<__nv_bfloat16>(a, dout, dtable, part, D, scale, accumulate, st)
                : sums<float>(a, dout, dtable, part, D, scale, accumulate, st);
}

} // namespace fw
