// fw_gated_tc.cu -- the gated delta rule with bf16 tensors on the tcgen05
// tensor cores: chunk preparation and the walk over the chunks, forwards
// (answers, or the states the gradients need) and backwards.
//
// The chunk algebra is that of fw_gated_chunk.cu with the triangular inverse
// multiplied out, so that the serial part of a chunk is two products:
//   forward   W' = T diag(beta e^G) K,          U' = T diag(beta) V,
//             Q' = scale e^G Q - M W',          Y' = M U',
//             U = U' - W' S^T,   Y = Y' + Q' S^T,   S1 = e^{G_C} S + (e^{G_C-G} U)^T K;
//   backward  W" = T^T diag(e^{G_C-G}) K,       X0 = T^T M^T dY,
//             dX = X0 + W" dS1^T,
//             dS = e^{G_C} dS1 + (scale e^G dY)^T Q - (beta e^G dX)^T K.
// Both walks have one shape: D = A Z, a row of values per token, then
// Z = e^{G_C} Z + B^T (weighted values) -- so they are one kernel.
//
// Precision.  K, Q, V and dY are bf16 as given and enter products exactly
// (their unit-length factors are fp32 scalars folded into the other side).
// Every other operand -- T, M, the products above, the state, U, dX -- is an
// fp32 value that enters a product as two bf16 terms, hi + lo, which leaves
// 2^-16 of it at most (2^-17.6 rms); lo x lo is dropped.  Accumulators are
// fp32, the state's master copy is fp32 in registers.  One bf16 term would
// leave 2^-8 in an fp32 state.  The two terms of a B operand sit side by side
// along N, so one MMA reads A once for both.
#include "fw_gated.h"
#include "fw_gated_tc.h"
#include "fw_gated_tiles.cuh"
#include "fw_tc.cuh"

#include <algorithm>

namespace fw {

cudaError_t status_word(unsigned **out); // fw_api.cu
cudaError_t device_sms(int *out);

namespace {

using namespace tc;

constexpr int C = kGatedChunk, NT = kGatedThreads, LC = kGatedLd;
constexpr int NV = 32;    // value channels per walk CTA

// 16 fp32 channels of a row in a "piece" (rows of 64 bytes, the base rows of
// the walk): 16-byte chunk c, placed so that eight rows in a row of lanes meet
// eight different bank groups.
FW_DEV uint32_t piece_chunk(int row, int c) { return (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4)); }

// On pairs of floats: v + o, f v.
template <int N> FW_DEV void add_to(float *v, const float *o) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const float2 d = unpack(pack(v[e], v[e + 1]) + pack(o[e], o[e + 1]));
        v[e] = d.x;
        v[e + 1] = d.y;
    }
}
template <int N> FW_DEV void scaled(float *to, float f, const float *v) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
        const float2 d = unpack(both(f) * pack(v[e], v[e + 1]));
        to[e] = d.x;
        to[e + 1] = d.y;
    }
}

// A descriptor `bytes` further into its tile.
FW_DEV uint64_t at(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }

// ------------------------------------------------------------------ prep
// One CTA per (chunk, value head), two to an SM.  Shared memory: the [K; Q]
// tile (K-major, 128 rows; its first 64 rows also serve as the MN-major K),
// an operand region (M and T as hi and lo tiles, then the stacked 128 x 64
// matrices A1 and A2 in turn), the fp32 A / T work space (A's place is V's,
// then dY's, later), per-token scalars.  What a product leaves goes out by
// warps: 32 rows are staged as 4 KB that lie together in the record too, and
// one lane sends them (stored from registers, a row per lane, every 16 bytes
// cost a sector: 317 us for 4096 chunks of d 128 where this took 249, and takes
// 225 with V requested ahead and the decays on pairs of floats).
struct PrepSmem {
    uint32_t kq, op, at, tt, tok, bar, bytes;
};
__host__ __device__ inline PrepSmem prep_smem(int nkb, int nvb) {
    PrepSmem s;
    s.kq = 0;
    s.op = (uint32_t)nkb * 16384;
    s.at = s.op + 32768;
    const uint32_t work = C * LC * 4 + 4096, v = (uint32_t)nvb * 8192;
    s.tt = s.at + (work > v ? work : v);
    s.tok = s.tt + C * LC * 4;
    s.bar = s.tok + C * 44;
    s.bytes = s.bar + 64 + 1024;
    return s;
}

template <bool BWD, int NKB>
__global__ void __launch_bounds__(NT, 2)
    gated_tc_prep_kernel(GatedArgs a, const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ k,
                         const __nv_bfloat16 *__restrict__ v, const __nv_bfloat16 *__restrict__ g,
                         const __nv_bfloat16 *__restrict__ beta, const __nv_bfloat16 *__restrict__ dy, uint8_t *ws,
                         GatedRecord rec, int c0, int beside, int ahead, int tmem_cols, unsigned *status) {
    constexpr int DKP = 64 * NKB;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nvb = (a.d_v + 63) / 64;
    const PrepSmem o = prep_smem(NKB, nvb);
    uint8_t *kq = sm + o.kq, *op = sm + o.op, *vt = sm + o.at;
    float *At = reinterpret_cast<float *>(sm + o.at), *tmp = At + C * LC, *Tt = reinterpret_cast<float *>(sm + o.tt);
    float *tok = reinterpret_cast<float *>(sm + o.tok);
    float *cw = tok + 8 * C, *cb = cw + C, *cd = cb + C; // -beta e^G rk, beta, e^{G_C-G} rk
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + o.bar);
    uint32_t *slot = reinterpret_cast<uint32_t *>(bar + 1);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, c = c0 + blockIdx.x, bh = blockIdx.y;
    const int b = bh / a.H, h = bh % a.H, kh = b * a.Hk + h / (a.H / a.Hk);
    // `beside`: the preceding kernel is a walk over earlier chunks of this
    // call, which has itself waited for everything before it and writes
    // nothing that is read here.  The grid's last CTA waits for it at its end,
    // so that this kernel does not complete before the walk does.
    const bool last = blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1;
    if (!beside)
        griddep_wait();
    q = after_wait(q);
    k = after_wait(k);
    v = after_wait(v);
    g = after_wait(g);
    beta = after_wait(beta);
    dy = after_wait(dy);
    const int n = min(C, seq_len(a, b) - c * C);
    if (n <= 0) {
        griddep_launch_dependents();
        if (beside && last)
            griddep_wait();
        return;
    }
    if (w == 0) {
        tmem_alloc(slot, (uint32_t)tmem_cols);
        tmem_relinquish(); // or no second CTA is placed on the SM
    }
    if (tid == 32) {
        mbar_init(bar, 1);
        fence_barrier_init();
    }
    if (tid == 64) { // into L2 what the CTA that takes this one's place will read (these are inputs)
        const int64_t next = (int64_t)blockIdx.y * gridDim.x + blockIdx.x + ahead;
        if (next < (int64_t)gridDim.x * gridDim.y) {
            const int nc = c0 + (int)(next % gridDim.x), nbh = (int)(next / gridDim.x);
            const size_t nk = (size_t)(nbh / a.H * a.Hk + nbh % a.H / (a.H / a.Hk)) * a.L + (size_t)nc * C;
            const size_t nv = (size_t)nbh * a.L + (size_t)nc * C;
            const uint32_t rows = (uint32_t)min(C, a.L - nc * C);
            l2_prefetch(k + nk * a.d_k, rows * a.d_k * 2);
            l2_prefetch(q + nk * a.d_k, rows * a.d_k * 2);
            l2_prefetch(v + nv * a.d_v, rows * a.d_v * 2);
            if (BWD)
                l2_prefetch(dy + nv * a.d_v, rows * a.d_v * 2);
        }
    }
    // [K; Q], 16 bytes a thread and step
    {
        constexpr int PER = DKP / 8, STEPS = 2 * C * PER / NT; // chunks per row; 4 or 8 steps
        const __nv_bfloat16 *kg = k + ((size_t)kh * a.L + (size_t)c * C) * a.d_k;
        const __nv_bfloat16 *qg = q + ((size_t)kh * a.L + (size_t)c * C) * a.d_k;
        const int ch = tid % PER;
        uint4 u[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int row = (s * NT + tid) / PER;
            u[s] = make_uint4(0, 0, 0, 0);
            if ((row & 63) < n && ch * 8 < a.d_k)
                u[s] = __ldcg(reinterpret_cast<const uint4 *>((row < C ? kg : qg) + (size_t)(row & 63) * a.d_k) + ch);
        }
        if (w == 1) { // the running sums of g, two tokens a lane
            const size_t t0 = (size_t)bh * a.L + (size_t)c * C;
            float x[2], be[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                x[e] = i < n ? io<__nv_bfloat16>::load(g + t0 + i) : 0.f;
                x[e] = x[e] < kGMin ? kGMin : x[e];
                be[e] = i < n ? io<__nv_bfloat16>::load(beta + t0 + i) : 0.f;
            }
            Pair run, all;
            running_sum(x, lane, run, all);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const Pair G = e ? run : add(run, {-x[1], 0.f});
                float *d = tok + 2 * lane + e;
                d[kGhi] = G.hi;
                d[kGlo] = G.lo;
                d[kBeta] = be[e];
                d[kEG] = expf(G.hi);
                d[kEC] = expf((all.hi - G.hi) + (all.lo - G.lo));
            }
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int row = (s * NT + tid) / PER;
            *reinterpret_cast<uint4 *>(kq + kmajor_chunk(row, ch * 8, 128)) = u[s];
        }
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tm = *slot;
    const uint32_t tGram = tm, tMT = tm + 128, tA1 = tm, tA2 = tm + 128;
    uint32_t phase = 0;
    bool ok = true;
    auto finish = [&]() { // the MMAs issued so far are done
        if (ok)
            ok = mbar_wait(bar, phase, status);
        phase ^= 1;
        tc_fence_after();
    };
    auto hand_over = [&]() { // shared memory written, TMEM read: the next MMAs may go
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    const uint64_t dKmaj = desc_sw128(smem_u32(kq), 16, 1024), dKmn = desc_sw128(smem_u32(kq), 16384, 1024);
    const uint64_t dOp = desc_sw128(smem_u32(op), 16, 1024), dOpMn = desc_sw128(smem_u32(op), 8192, 1024);
    const uint64_t dV = desc_sw128(smem_u32(vt), 8192, 1024);
    uint8_t *out = ws + rec.off(bh, c);
    if (tid == 0) { // K K^T (rows 0-63), Q K^T and Q Q^T: the diagonals are the rows' squared lengths
#pragma unroll
        for (int s = 0; s < 4 * NKB; ++s) {
            const uint64_t d = at(dKmaj, kmajor_step(s, 128));
            mma_bf16(tGram, d, d, idesc_bf16(128, 128, 0, 0), s > 0);
        }
        mma_commit(bar);
        // the K (and Q) image for the walk, straight from the tile
        if (BWD) { // (blocks of 128 rows)
            bulk_s2g(out + rec.K, kq, (uint32_t)NKB * 16384u);
        } else {
#pragma unroll
            for (int kb = 0; kb < NKB; ++kb)
                bulk_s2g(out + rec.K + kb * 8192, kq + kb * 16384, 8192);
        }
        bulk_commit();
    }
    finish();
    const int rr = 32 * (w & 3) + lane, half = w >> 2, i = rr & 63;
    if (half == 0) { // 1 / length (0 for a row of zeros)
        float x[32], ss = 0.f;
        tmem_ld16(tGram + tmem_lane_base(w) + (uint32_t)(32 * w), x);
        tmem_ld16(tGram + tmem_lane_base(w) + (uint32_t)(32 * w + 16), x + 16);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e)
            ss = e == lane ? x[e] : ss;
        ss += a.eps;
        ss = !a.l2norm ? 1.f : ss > 0.f ? 1.f / sqrtf(ss) : ss;
        tok[(rr < C ? kRk : kRq) + i] = ss;
        if (rr < C) {
            const float be = tok[kBeta + i];
            cw[i] = -be * tok[kEG + i] * ss;
            cb[i] = be;
            cd[i] = tok[kEC + i] * ss;
        }
    }
    __syncthreads();
    {
        const float ghi = tok[kGhi + i], glo = tok[kGlo + i];
        const F2 fi = both(rr < C ? tok[kBeta + i] * tok[kRk + i] : a.scale * tok[kRq + i]);
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
            const int j0 = 32 * half + 16 * p;
            float x[16];
            tmem_ld16(tGram + tmem_lane_base(w) + (uint32_t)j0, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                F2 d[2];
                decay4(tok, j0 + e, ghi, glo, d);
                const ulonglong2 rk = *reinterpret_cast<const ulonglong2 *>(tok + kRk + j0 + e);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int j = j0 + e + 2 * u;
                    const float2 t = unpack(fi * F2{u ? rk.y : rk.x} * pack(x[e + 2 * u], x[e + 2 * u + 1]) * d[u]);
                    x[e + 2 * u] = (rr < C ? j < i : j <= i) ? t.x : 0.f;
                    x[e + 2 * u + 1] = (rr < C ? j + 1 < i : j + 1 <= i) ? t.y : 0.f;
                }
            }
            if (rr < C) {
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    *reinterpret_cast<float4 *>(At + i * LC + j0 + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    uint4 hi, lo;
                    split8(x + e, hi, lo);
                    const uint32_t to = kmajor_chunk(i, j0 + e, 64);
                    *reinterpret_cast<uint4 *>(op + to) = hi;
                    *reinterpret_cast<uint4 *>(op + 8192 + to) = lo;
                }
            }
        }
    }
    // V or dY as an MN-major tile of 64-channel blocks: two rows' 16-byte chunks a
    // thread and block, requested and stored apart so that V's way is under the
    // inverse (the first two blocks; a wider V follows when its turn comes)
    auto request_rows = [&](const __nv_bfloat16 *src, int blk, uint4 (&u)[2]) {
        const int r = tid >> 2, ch = 8 * blk + 2 * (tid & 3);
        const uint4 *from = reinterpret_cast<const uint4 *>(src + ((size_t)bh * a.L + (size_t)c * C + r) * a.d_v) + ch;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            u[m] = make_uint4(0, 0, 0, 0);
            if (r < n && (ch + m) * 8 < a.d_v)
                u[m] = __ldcg(from + m);
        }
    };
    auto store_rows = [&](int blk, const uint4 (&u)[2]) {
        const int r = tid >> 2, ch = 8 * blk + 2 * (tid & 3);
#pragma unroll
        for (int m = 0; m < 2; ++m)
            *reinterpret_cast<uint4 *>(vt + kmajor_chunk(r, (ch + m) * 8, 64)) = u[m];
    };
    uint4 v0[2], v1[2];
    request_rows(v, 0, v0);
    if (nvb > 1)
        request_rows(v, 1, v1);
    __syncthreads();
    unit_lower_inverse(At, Tt, tmp);
#pragma unroll
    for (int e = tid; e < C * 8; e += NT) { // T as hi and lo tiles
        const int r = e >> 3, j0 = (e & 7) * 8;
        float x[8];
#pragma unroll
        for (int m = 0; m < 8; m += 4) {
            const float4 t = *reinterpret_cast<const float4 *>(Tt + r * LC + j0 + m);
            x[m] = t.x;
            x[m + 1] = t.y;
            x[m + 2] = t.z;
            x[m + 3] = t.w;
        }
        uint4 hi, lo;
        split8(x, hi, lo);
        const uint32_t to = kmajor_chunk(r, j0, 64);
        *reinterpret_cast<uint4 *>(op + 16384 + to) = hi;
        *reinterpret_cast<uint4 *>(op + 24576 + to) = lo;
    }
    hand_over();
    if (tid == 0) { // M T, or (M T)^T = T^T M^T
#pragma unroll
        for (int t = 0; t < 3; ++t) // hi hi, hi lo, lo hi
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const uint64_t dm = at(dOp, (t == 2 ? 8192u : 0u) + kmajor_step(s, 64));
                const uint64_t dt = at(dOpMn, 16384u + (t == 1 ? 8192u : 0u) + (uint32_t)s * 2048u);
                if (BWD)
                    mma_bf16(tMT, dt, dm, idesc_bf16(128, 64, 1, 0), (t | s) != 0);
                else
                    mma_bf16(tMT, dm, dt, idesc_bf16(128, 64, 0, 1), (t | s) != 0);
            }
        mma_commit(bar);
    }
    finish();
    // Stacked left factors, hi tile then lo tile: rows 0-63 from T, rows
    // 64-127 from MT (TMEM lanes 0-63, so the warps that can read those
    // lanes hold the lower rows) or, for W", from T^T.
    auto factor = [&](bool first, float (&x)[32]) {
        const float *coef = (BWD && first && rr < C ? cd : first ? cw : cb) + 32 * half;
        if (rr >= C) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(Tt + i * LC + 32 * half + e);
                x[e] = t.x;
                x[e + 1] = t.y;
                x[e + 2] = t.z;
                x[e + 3] = t.w;
            }
        } else if (BWD && first) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
                x[e] = Tt[(32 * half + e) * LC + i];
        } else {
            tmem_ld16(tMT + tmem_lane_base(w) + (uint32_t)(32 * half), x);
            tmem_ld16(tMT + tmem_lane_base(w) + (uint32_t)(32 * half + 16), x + 16);
            tmem_ld_wait();
            if (BWD)
                return;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(coef + e);
            x[e] *= f.x;
            x[e + 1] *= f.y;
            x[e + 2] *= f.z;
            x[e + 3] *= f.w;
        }
    };
    auto put = [&](const float (&x)[32]) {
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
            uint4 hi, lo;
            split8(x + e, hi, lo);
            const uint32_t to = kmajor_chunk(rr ^ 64, 32 * half + e, 128);
            *reinterpret_cast<uint4 *>(op + to) = hi;
            *reinterpret_cast<uint4 *>(op + 16384 + to) = lo;
        }
    };
    auto multiply = [&](uint32_t d, uint64_t db, uint32_t id) {
        if (tid == 0) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    mma_bf16(d, at(dOp, (uint32_t)(t * 16384 + s * 32)), at(db, (uint32_t)s * 2048u), id, (t | s) != 0);
            mma_commit(bar);
        }
    };
    float x2[32];
    factor(true, x2);
    put(x2);
    hand_over();
    multiply(tA1, dKmn, idesc_bf16(128, DKP, 0, 1)); // [-W'; ...] or [-W'; W"]
    store_rows(0, v0); // A's place
    if (nvb > 1)
        store_rows(1, v1);
    for (int blk = 2; blk < nvb; ++blk) {
        request_rows(v, blk, v0);
        store_rows(blk, v0);
    }
    factor(false, x2);
    finish();
    put(x2);
    hand_over();
    const uint32_t idv = idesc_bf16(128, a.d_v, 0, 1);
    multiply(tA2, dV, idv);
    if (tid < C) { // the walks' scalars
        const float *d = tok + tid;
        float *sf = reinterpret_cast<float *>(out + rec.scalF);
        sf[tid] = d[kEC] * d[kRk];
        if (tid == 0)
            sf[C] = tok[kEG + C - 1];
        if (BWD) {
            float *sr = reinterpret_cast<float *>(out + rec.scalR);
            sr[tid] = -d[kBeta] * d[kEG] * d[kRk];
            sr[C + tid] = a.scale * d[kEG] * d[kRq];
            if (tid == 0)
                sr[2 * C] = tok[kEG + C - 1];
            float *st = reinterpret_cast<float *>(out + rec.tok) + tid;
#pragma unroll
            for (int e = 0; e <= kEC; e += C)
                st[e] = d[e];
        }
    }
    finish();
    // rows [r0, r0 + R) of the product as pieces [16 channels][R rows][16]
    // fp32: a warp stages two pieces of its rows at a time and sends them
    uint8_t *mine = (NKB == 2 ? kq : vt) + w * 4096; // (NKB 2: these rows of K and Q are this warp's own)
    auto sent = [&]() { // what this warp sent has left its place
        if (lane == 0)
            bulk_wait_read();
        __syncwarp();
    };
    // (`two`: the images' hi terms have left or are leaving the operand region,
    // and every other pair of pieces goes there: one copy may be on its way)
    auto rows_out = [&](size_t to, int R, int r0, bool two) {
        if (rr < r0 || rr >= r0 + R)
            return;
        for (int p0 = half; p0 < a.d_v / 16; p0 += 4) {
            uint8_t *place = two && (p0 & 4) ? op + w * 4096 : mine;
            if (two) {
                if (lane == 0)
                    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                __syncwarp();
            } else {
                sent();
            }
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
                const int p = p0 + 2 * e;
                if (p >= a.d_v / 16)
                    break;
                float x[16];
                tmem_ld16(tA2 + tmem_lane_base(w) + (uint32_t)(16 * p), x);
                tmem_ld_wait();
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    *reinterpret_cast<float4 *>(place + 2048 * e + piece_chunk(lane, m)) =
                        make_float4(x[4 * m], x[4 * m + 1], x[4 * m + 2], x[4 * m + 3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (p0 + 2 * e < a.d_v / 16)
                        bulk_s2g(out + to + ((size_t)(p0 + 2 * e) * R + 32 * (w & 3) - r0) * 64, place + 2048 * e, 2048);
                bulk_commit();
            }
        }
    };
    // the first product's rows as images: per 64-wide block 64 hi rows, then
    // the same 64 rows' lo terms
    auto images_out = [&]() {
        uint8_t *hi_at = NKB == 2 ? op + w * 4096 : op + (rr < C ? 0 : 16384),
                *lo_at = NKB == 2 ? vt + w * 4096 : hi_at + 8192;
#pragma unroll 1
        for (int p = 0; p < DKP / 32; ++p) {
            const int c0 = half * (DKP / 2) + 16 * p;
            float x[16];
            tmem_ld16(tA1 + tmem_lane_base(w) + (uint32_t)c0, x);
            tmem_ld_wait();
            if (!BWD && rr >= C) {
                const float f = a.scale * tok[kEG + i] * tok[kRq + i];
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    float y[8];
                    widen8(*reinterpret_cast<const uint4 *>(kq + kmajor_chunk(rr, c0 + e, 128)), y);
#pragma unroll
                    for (int m = 0; m < 8; ++m)
                        x[e + m] = fmaf(f, y[m], x[e + m]);
                }
            }
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                uint4 hi, lo;
                split8(x + e, hi, lo);
                const uint32_t to = kmajor_chunk(NKB == 2 ? lane : i, (c0 + e) & 63, 64); // (one 64-wide block)
                *reinterpret_cast<uint4 *>(hi_at + to) = hi;
                *reinterpret_cast<uint4 *>(lo_at + to) = lo;
            }
        }
        fence_async_smem();
        if (NKB == 2) { // this warp's rows of block `half`
            __syncwarp();
            if (lane == 0) {
                uint8_t *to = out + (rr < C ? rec.A : rec.A2) + half * 16384 + (w & 1) * 4096;
                bulk_s2g(to, hi_at, 4096);
                bulk_s2g(to + 8192, lo_at, 4096);
                bulk_commit();
            }
        } else { // two warps share a row
            __syncthreads();
            if (tid == 0) {
                bulk_s2g(out + rec.A, op, 32768); // (A2 lies behind A)
                bulk_commit();
            }
        }
    };
    if (tid == 0)
        bulk_wait_read(); // the K (and Q) image has left
    __syncthreads();
    if (!BWD) {
        images_out();
        rows_out(rec.base, 128, 0, NKB == 2);
    } else {
        for (int blk = 0; blk < min(nvb, 2); ++blk)
            request_rows(dy, blk, blk ? v1 : v0);
        rows_out(rec.base, C, 0, false);
        if (NKB == 1) { // V's place holds both these rows and dY
            sent();
            __syncthreads();
        }
        store_rows(0, v0); // V's place
        if (nvb > 1)
            store_rows(1, v1);
        for (int blk = 2; blk < nvb; ++blk) {
            request_rows(dy, blk, v0);
            store_rows(blk, v0);
        }
        hand_over();
        multiply(tA2, dV, idv);
        finish();
        images_out();
        rows_out(rec.base2, C, C, NKB == 2);
    }
    if (lane == 0)
        bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (w == 0)
        tmem_dealloc(tm, (uint32_t)tmem_cols);
    if (beside && last)
        griddep_wait();
}

// ------------------------------------------------------------------ walk
// One CTA per (value head, TP tiles of 32 value channels).  An MMA of 128 rows takes the
// same time for any N up to 128 here (66 cycles), so the serial product has
// the hi and the lo rows of its 64 x d_k factor stacked as its 128 rows, 8
// MMAs of it for d_k 128, against [Z hi | Z lo] side by side; the answers'
// product follows while the values are on their way, and the state's product
// after that.  (One tile of W' and Q' rows, hi then lo, had 16 MMAs on the
// serial path: 1.6 us a chunk instead of 1.45.  Two threads issuing half of the
// product each, into accumulators of their own, were no faster: the MMAs, not
// their issue, take the time.)
//
// Eight worker warps a tile.  Of a tile's, warps 0, 1, 4, 5 read the hi rows'
// result, warps 2, 3, 6, 7 the lo rows' of the same tokens (a warp reaches 32
// of the 128 TMEM lanes); the two swap halves of their 16 channels through
// shared memory and each finishes 8 channels.  Thread (row 32 (w % 4) + lane, 16 channels) also
// holds 16 values of the fp32 state (row = key channel).  One more warp's first
// lane issues the MMAs and another's asks for the records, each part as soon
// as the product that last read its place is done, so that none of that is on
// a worker's path.  Workers tell them by two mbarriers that the state's or
// the values' tile is written; commits tell workers that a product is done.
// (tests/test_gated_walk_order.py goes through every order of these steps.)
//
// TP: with one tile a CTA the chain of a chunk is shortest; two tiles read the
// records half as often, which is what counts once there are more CTAs than
// SMs (the backward at B8 H16 L2048, 1024 CTAs with one tile: 955 us with one
// tile, its walks 341, at 9 TB/s out of L2; 893 with two; 715 to 805, by the
// machine, with the faster preparation and gradients of now, the walks 288).  Two
// tiles for d_k > 64 are 18 warps of 96 registers, which spill 24 bytes.
enum { kFwd = 0, kKeep = 1, kRev = 2 };
constexpr int walk_threads(int TP) { return NT * TP + 64; }

template <int MODE, int NKB, int TP> struct Walk {
    static constexpr int RB = MODE == kRev ? 128 : 64;     // tokens the B^T tile holds
    static constexpr int RV = MODE == kFwd ? 128 : 64;     // base rows: U', then Y'
    static constexpr uint32_t A = NKB * 16384 * (MODE == kFwd ? 2 : 1), B = NKB * RB * 128,
                              SCAL = MODE == kRev ? 528 : 512;
    static constexpr uint32_t b = A, base = b + B, rec = base + TP * RV * 128;
    // A product of one 64-wide block reads one more (its rows go unused): what
    // follows in this order covers it.
    static constexpr uint32_t z = 2 * rec, u = z + TP * NKB * 8192, scal = u + TP * RB * 128, bar = scal + 2 * SCAL,
                              bytes = bar + 128 + 1024;
    static_assert(rec + b + B + (NKB == 1 ? B : 0) <= bar && bytes <= 232448, "reads stay inside shared memory");
    static constexpr uint32_t cols = TP * (MODE == kFwd ? 256 : 128); // TMEM: a tile's values, state, answers: 64 each
};

template <int MODE, int NKB, int TP>
FW_DEV void walk(const GatedArgs &a, const __nv_bfloat16 *__restrict__ dy, const float *__restrict__ Z0,
                 float *__restrict__ Zf, __nv_bfloat16 *__restrict__ y, uint8_t *ws, const GatedRecord &rec, int c0,
                 int c1, unsigned *status) {
    using L = Walk<MODE, NKB, TP>;
    constexpr int DKP = 64 * NKB, WORKERS = 8 * TP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *zt = sm + L::z, *ut = sm + L::u;
    uint64_t *fullA = reinterpret_cast<uint64_t *>(sm + L::bar), *fullB = fullA + 2, *m1 = fullA + 4, *m2 = fullA + 5,
             *my = fullA + 6, *zr = fullA + 8, *ur = fullA + 9;
    uint32_t *slot = reinterpret_cast<uint32_t *>(fullA + 10);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, sl = blockIdx.x, bh = blockIdx.y, n0 = sl * TP * NV;
    const int b = bh / a.H;
    griddep_wait();
    dy = after_wait(dy);
    Z0 = after_wait(Z0);
    const int len = seq_len(a, b), nch = max(0, min(c1, (len + C - 1) / C) - c0); // of chunks c0 .. c1 - 1
    if (w == 0) {
        tmem_alloc(slot, L::cols);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (int e = 0; e < 8; ++e)
            mbar_init(fullA + e, 1);
        // A wait knows a phase by its parity, so a role that waits has to see a
        // phase before the next one ends.  The workers and the issuer of the MMAs
        // need one another for that; the forward's copies' warp does not need to
        // be seen by anyone, so it arrives for the state, too, and the answers'
        // product has two barriers, for the chunks in turn (the product after
        // next needs what this warp asks for behind its wait).
        mbar_init(zr, WORKERS + (MODE == kFwd ? 1 : 0));
        mbar_init(ur, WORKERS + (MODE == kFwd ? 0 : 1)); // the state's copy has left its tile
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tm = *slot, tU = tm, tZ = tm + 64 * TP, tY = tm + 128 * TP;
    auto chunk_of = [&](int it) { return c0 + (MODE == kRev ? nch - 1 - it : it); };
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok)
            ok = mbar_wait(bar, parity, status);
    };
    if (w == WORKERS) { // the MMAs
        if (lane == 0) {
            const uint64_t dz = desc_sw128(smem_u32(zt), DKP * 128, 1024),
                           du = desc_sw128(smem_u32(ut), L::RB * 128, 1024);
            const uint64_t dA0 = desc_sw128(smem_u32(sm), 16, 1024);
            const uint64_t dB0 = desc_sw128(smem_u32(sm + L::b), L::RB * 128, 1024);
            for (int it = 0; it < nch; ++it) {
                const uint64_t dA = at(dA0, (uint32_t)(it & 1) * L::rec), dB = at(dB0, (uint32_t)(it & 1) * L::rec);
                wait(fullA + (it & 1), (it >> 1) & 1);
                wait(zr, it & 1);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < 4 * NKB; ++s)
                    mma_bf16(tU, at(dA, kmajor_step(s, 128)), at(dz, (uint32_t)s * 2048u), idesc_bf16(128, 64 * TP, 0, 1),
                             s > 0);
                mma_commit(m1);
                if (MODE == kFwd) {
#pragma unroll
                    for (int s = 0; s < 4 * NKB; ++s)
                        mma_bf16(tY, at(dA, (uint32_t)NKB * 16384u + kmajor_step(s, 128)), at(dz, (uint32_t)s * 2048u),
                                 idesc_bf16(128, 64 * TP, 0, 1), s > 0);
                    mma_commit(my + (it & 1));
                }
                wait(fullB + (it & 1), (it >> 1) & 1);
                wait(ur, it & 1);
                if (!ok)
                    break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < L::RB / 16; ++s)
                    mma_bf16(tZ, at(dB, (uint32_t)s * 2048u), at(du, (uint32_t)s * 2048u), idesc_bf16(128, 64 * TP, 1, 1),
                             s > 0);
                mma_commit(m2);
            }
        }
        __syncwarp();
    } else if (w == WORKERS + 1) { // the copies
        if (lane == 0) {
            const uint32_t pieces = (uint32_t)min(2 * TP, (a.d_v - n0) / 16), tiles = (pieces + 1) / 2;
            auto fetch_a = [&](int it) {
                mbar_arrive_expect_tx(fullA + (it & 1), L::A);
                bulk_g2s(sm + (it & 1) * L::rec, ws + rec.off(bh, chunk_of(it)) + (MODE == kRev ? rec.A2 : rec.A), L::A,
                         fullA + (it & 1));
            };
            auto fetch_b = [&](int it) {
                const uint8_t *src = ws + rec.off(bh, chunk_of(it));
                uint8_t *dst = sm + (it & 1) * L::rec;
                uint64_t *f = fullB + (it & 1);
                const uint32_t base = pieces * L::RV * 64;
                mbar_arrive_expect_tx(f, L::B + L::SCAL + base);
                if (MODE == kKeep) {
#pragma unroll
                    for (int kb = 0; kb < NKB; ++kb)
                        bulk_g2s(dst + L::b + kb * 8192, src + rec.K + kb * 16384, 8192, f);
                } else {
                    bulk_g2s(dst + L::b, src + rec.K, L::B, f);
                }
                bulk_g2s(sm + L::scal + (it & 1) * L::SCAL, src + (MODE == kRev ? rec.scalR : rec.scalF), L::SCAL, f);
                bulk_g2s(dst + L::base, src + (MODE == kRev ? rec.base2 : rec.base) + (size_t)sl * TP * L::RV * 128, base, f);
            };
            if (MODE == kFwd)
                mbar_arrive(zr);
            for (int it = 0; it < min(2, nch); ++it) {
                fetch_a(it);
                fetch_b(it);
            }
            for (int it = 0; it < nch; ++it) {
                wait(zr, it & 1);
                if (!ok)
                    break;
                if (MODE == kFwd)
                    mbar_arrive(zr);
                if (MODE != kFwd) { // the state before this chunk, as it lies
                    bulk_s2g(ws + rec.off(bh, chunk_of(it)) + (MODE == kKeep ? rec.S : rec.dS) + (size_t)sl * TP * DKP * 128,
                             zt, tiles * DKP * 128u);
                    bulk_commit();
                }
                if (it > 0 && it + 1 < nch)
                    fetch_b(it + 1); // the workers are through with the previous chunk
                if (MODE != kFwd) {
                    bulk_wait_read();
                    mbar_arrive(ur);
                } else {
                    wait(my + (it & 1), (it >> 1) & 1);
                }
                if (MODE != kFwd)
                    wait(ur, it & 1); // (they have seen the values' product)
                // (the answers' product ends behind the values')
                if (ok && it + 2 < nch)
                    fetch_a(it + 2);
            }
            if (MODE != kFwd)
                bulk_wait_all();
            if (!ok) // a wait gave up: let the records that were asked for land first
                for (int e = 0; e < 4; ++e)
                    (void)mbar_wait(fullA + e, 0, status);
        }
        __syncwarp();
    } else {
        const int rr = 32 * (w & 3) + lane, hf = w >> 2, i = rr & 63, c8 = (w >> 1) & 1; // c8: which 8 of the 16 channels
        const int tile = hf >> 1, h2 = hf & 1; // which tile, which half of it
        const bool mine = n0 + 16 * hf < a.d_v; // these 16 channels exist (d_v is a multiple of 16)
        const bool zrow = 32 * (w & 3) < DKP;   // this warp holds rows of the state
        const uint32_t lb = tmem_lane_base(w) + (uint32_t)(64 * tile + 16 * h2);
        uint8_t *zt_ = zt + tile * DKP * 128, *ut_ = ut + tile * L::RB * 128;
        float z[16], x[8], y8[8], t0[16], t1[16];
        uint4 even[2], odd[2]; // kRev, lo rows' warps: dY's rows of the next two chunks
        auto read_dy = [&](int it, uint4 (&ahead)[2]) {
            const int c = chunk_of(it);
            const bool in = mine && i < min(C, len - c * C);
            const uint4 *from = reinterpret_cast<const uint4 *>(
                dy + ((size_t)bh * a.L + (size_t)c * C + (in ? i : 0)) * a.d_v + (in ? n0 + 16 * hf : 0));
            ahead[0] = in ? __ldcg(from) : make_uint4(0, 0, 0, 0);
            ahead[1] = in ? __ldcg(from + 1) : make_uint4(0, 0, 0, 0);
        };
        auto put8 = [&](uint8_t *tile, int row, int c, const float *v) { // 8 channels (chunk c of 4) of a pair tile's row
            uint4 hi, lo;
            split8(v, hi, lo);
            *reinterpret_cast<uint4 *>(tile + pair_chunk(row, c)) = hi;
            *reinterpret_cast<uint4 *>(tile + pair_chunk(row, c + 4)) = lo;
        };
        auto written = [&](uint64_t *bar) { // this warp's rows of a tile are written, its TMEM reads done
            fence_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar);
        };
        // this thread's 8 channels of a product: hi rows' sum plus lo rows',
        // added to v; the two warps swap in the 2 KB of base rows that were theirs
        auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + (w & 1) + 2 * hf) : "memory"); }; // warps w, w ^ 2
        auto product = [&](uint32_t t, uint8_t *place, float (&v)[8]) {
            float4 *give = reinterpret_cast<float4 *>(place) + c8 * 64 + lane;
            const float4 *take = reinterpret_cast<const float4 *>(place) + (c8 ^ 1) * 64 + lane;
            tmem_ld16(t + lb, t0);
            if (c8 == 0)
                tmem_ld16(t + lb + 32u, t1);
            tmem_ld_wait();
            if (c8 == 0) {
                add_to<16>(t0, t1);
                give[0] = make_float4(t0[8], t0[9], t0[10], t0[11]);
                give[32] = make_float4(t0[12], t0[13], t0[14], t0[15]);
            } else {
                give[0] = make_float4(t0[0], t0[1], t0[2], t0[3]);
                give[32] = make_float4(t0[4], t0[5], t0[6], t0[7]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    t0[e] = t0[8 + e];
            }
            add_to<8>(v, t0);
            meet();
            const float4 p = take[0], q = take[32];
            const float o8[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
            add_to<8>(v, o8);
        };
        auto base8 = [&](const uint8_t *r, int row, float (&v)[8]) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
                if (mine)
                    p = *reinterpret_cast<const float4 *>(r + L::base + hf * (L::RV * 64) + piece_chunk(row, 2 * c8 + e));
                v[4 * e] = p.x;
                v[4 * e + 1] = p.y;
                v[4 * e + 2] = p.z;
                v[4 * e + 3] = p.w;
            }
        };
#pragma unroll
        for (int e = 0; e < 16; ++e)
            z[e] = Z0 && mine && rr < a.d_k ? __ldcg(Z0 + ((size_t)bh * a.d_v + n0 + 16 * hf + e) * a.d_k + rr) : 0.f;
        if (zrow) {
            put8(zt_, rr, 2 * h2, z);
            put8(zt_, rr, 2 * h2 + 1, z + 8);
        }
        written(zr);
        if (MODE == kRev && c8) {
            if (nch > 0)
                read_dy(0, even);
            if (nch > 1)
                read_dy(1, odd);
        }
        auto step = [&](int it, uint4 (&ahead)[2]) {
            const int c = chunk_of(it), n = min(C, len - c * C);
            uint8_t *r = sm + (it & 1) * L::rec, *place = r + L::base + hf * (L::RV * 64) + (w & 1) * 2048;
            uint8_t *gr = ws + rec.off(bh, c);
            wait(fullB + (it & 1), (it >> 1) & 1);
            const float *scal = reinterpret_cast<const float *>(sm + L::scal + (it & 1) * L::SCAL);
            const float whole = scal[MODE == kRev ? 2 * C : C], f = scal[i];
            if (MODE == kRev && c8) { // dY's rows do not wait for the product
                const float fy = scal[C + i];
                widen8(ahead[0], reinterpret_cast<float(&)[8]>(t0[0]));
                widen8(ahead[1], reinterpret_cast<float(&)[8]>(t0[8]));
                scaled<16>(t0, fy, t0);
                put8(ut_, C + i, 2 * h2, t0);
                put8(ut_, C + i, 2 * h2 + 1, t0 + 8);
                if (it + 2 < nch)
                    read_dy(it + 2, ahead);
            }
            base8(r, i, x);
            if (MODE == kFwd)
                base8(r, C + i, y8);
            meet(); // both have read their base rows
            wait(m1, it & 1);
            tc_fence_after();
            product(tU, place, x);
            scaled<8>(t0, f, x);
            put8(ut_, i, 2 * h2 + c8, t0);
            written(ur);
            if (MODE == kFwd) {
                wait(my + (it & 1), (it >> 1) & 1);
                tc_fence_after();
                product(tY, place + 4096, y8);
                if (mine && i < n)
                    store8(y + ((size_t)bh * a.L + (size_t)c * C + i) * a.d_v + n0 + 16 * hf + 8 * c8, y8);
            } else if (sl * TP + tile < rec.ns) { // U, or dX, for the gradients: a pair tile's row
                put8(gr + (MODE == kKeep ? rec.U : rec.dX) + (size_t)(sl * TP + tile) * 8192, i, 2 * h2 + c8, x);
            }
            wait(m2, it & 1);
            tc_fence_after();
            if (zrow) {
                tmem_ld16(tZ + lb, t0);
                tmem_ld16(tZ + lb + 32u, t1);
                tmem_ld_wait();
                add_to<16>(t0, t1);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 d = unpack(fma2(both(whole), pack(z[e], z[e + 1]), pack(t0[e], t0[e + 1])));
                    z[e] = d.x;
                    z[e + 1] = d.y;
                }
                put8(zt_, rr, 2 * h2, z);
                put8(zt_, rr, 2 * h2 + 1, z + 8);
            }
            written(zr);
        };
        if constexpr (MODE == kRev) { // by twos, so that each dY row has registers of its own
            for (int it = 0; it < nch; it += 2) {
                step(it, even);
                if (it + 1 < nch)
                    step(it + 1, odd);
            }
        } else {
            for (int it = 0; it < nch; ++it)
                step(it, even);
        }
        if (Zf && mine && rr < a.d_k)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                Zf[((size_t)bh * a.d_v + n0 + 16 * hf + e) * a.d_k + rr] = z[e];
        if (MODE == kFwd && c1 == rec.nch) { // no token, no answer
            const size_t c16 = min(NV, a.d_v - n0) / 8, cnt = (size_t)(a.L - len) * c16;
            for (size_t e = tid; e < cnt; e += NT)
                *reinterpret_cast<uint4 *>(y + ((size_t)bh * a.L + len + e / c16) * a.d_v + n0 + 8 * (e % c16)) =
                    make_uint4(0, 0, 0, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (w == 0)
        tmem_dealloc(tm, L::cols);
}

template <int NKB>
__global__ void __launch_bounds__(walk_threads(1))
    gated_tc_walk_kernel(GatedArgs a, const float *__restrict__ W0, float *__restrict__ Wf,
                         __nv_bfloat16 *__restrict__ y, uint8_t *ws, GatedRecord rec, int c0, int c1, unsigned *status) {
    walk<kFwd, NKB, 1>(a, nullptr, W0, Wf, y, ws, rec, c0, c1, status);
}
// The backward's two walks need only the preparation, not each other: one
// launch (B4 H8 L512, 64 CTAs each: 13 us and 15 us in two launches).
template <int NKB, int TP>
__global__ void __launch_bounds__(walk_threads(TP))
    gated_tc_both_walks_kernel(GatedArgs a, const __nv_bfloat16 *__restrict__ dy, const float *__restrict__ W0,
                               const float *__restrict__ dWf, float *__restrict__ dW0, uint8_t *ws, GatedRecord rec,
                               unsigned *status) {
    if (blockIdx.z == 0)
        walk<kRev, NKB, TP>(a, dy, dWf, dW0, nullptr, ws, rec, 0, rec.nch, status);
    else
        walk<kKeep, NKB, TP>(a, nullptr, W0, nullptr, nullptr, ws, rec, 0, rec.nch, status);
}

template <bool BWD, int NKB>
cudaError_t launch_prep(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                        const void *beta, const void *dy, void *ws, const GatedRecord &rec, int c0, int c1, bool beside,
                        int num_sms, unsigned *status, cudaStream_t st) {
    using bf = __nv_bfloat16;
    auto *kern = gated_tc_prep_kernel<BWD, NKB>;
    const uint32_t smem = prep_smem(NKB, (a.d_v + 63) / 64).bytes;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, allowed);
    if (e != cudaSuccess)
        return e;
    // 128 columns for A1's product, d_v for A2's (MT's 64 lie there first)
    const int cols = a.d_v <= 128 ? 256 : 512;
    return launch_pdl(kern, dim3(c1 - c0, a.B * a.H), dim3(NT), smem, st, a, (const bf *)q, (const bf *)k,
                      (const bf *)v, (const bf *)g, (const bf *)beta, (const bf *)dy, (uint8_t *)ws, rec, c0,
                      (int)beside, 2 * num_sms, cols, status);
}

// Chunks in a segment of the forward.  Where the walk's CTAs leave most SMs
// idle, a sequence is cut into segments and the preparation of one runs on the
// idle SMs beside the walk over the one before.  The length wanted is a whole
// number of waves of preparing CTAs (two an SM) and at least kMinSegment
// chunks, since each segment costs the walk a start; the sequence is then cut
// into equal segments, as many as come nearest to that length, so that none
// is a stump.  A segment may so be a few chunks longer or shorter than wanted,
// and its last wave of preparing CTAs partly empty (B2 H8 L2048: 16 chunks
// where a wave holds 15).  The first is prepared by every SM and is as long as
// the others all the same.  (16 heads, 16 381 tokens, d 128: 624 us in
// one piece, 506 in segments of 22 chunks, 742 in segments of 11; B2 H8 L2048,
// d_v 64: 85 us in one piece, 77 in two of 16.  With a faster preparation and
// pairs of floats the two take 468 and 72 us.)
constexpr int kMinSegment = 12;
int segment_chunks(const GatedArgs &a, const GatedRecord &rec, int num_sms) {
    const int64_t heads = (int64_t)a.B * a.H, walkers = heads * rec.ns;
    if (2 * walkers > num_sms)
        return rec.nch;
    const int wave = (int)std::max<int64_t>(1, 2 * (num_sms - walkers) / heads);
    const int seg = (kMinSegment + wave - 1) / wave * wave, n = (rec.nch + seg / 2) / seg;
    return n < 2 ? rec.nch : (rec.nch + n - 1) / n;
}

template <int NKB>
cudaError_t forward(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g, const void *beta,
                    const float *W0, float *Wf, void *y, void *ws, const GatedRecord &rec, int num_sms,
                    unsigned *status, cudaStream_t st) {
    auto *kern = gated_tc_walk_kernel<NKB>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(kern, allowed);
    const int seg = segment_chunks(a, rec, num_sms);
    float *between = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + rec.off((int64_t)a.B * a.H, 0));
    for (int c0 = 0; c0 < rec.nch && e == cudaSuccess; c0 += seg) {
        const int c1 = std::min(rec.nch, c0 + seg);
        e = launch_prep<false, NKB>(a, q, k, v, g, beta, nullptr, ws, rec, c0, c1, c0 > 0, num_sms, status, st);
        if (e == cudaSuccess)
            e = launch_pdl(kern, dim3(rec.ns, a.B * a.H), dim3(walk_threads(1)), Walk<kFwd, NKB, 1>::bytes, st, a,
                           c0 == 0 ? W0 : between, c1 == rec.nch ? Wf : between, (__nv_bfloat16 *)y, (uint8_t *)ws, rec,
                           c0, c1, status);
    }
    return e;
}

template <int NKB, int TP>
cudaError_t launch_both(const GatedArgs &a, const float *W0, const void *dy, const float *dWf, float *dW0, void *ws,
                        const GatedRecord &rec, unsigned *status, cudaStream_t st) {
    auto *kern = gated_tc_both_walks_kernel<NKB, TP>;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, allowed);
    if (e != cudaSuccess)
        return e;
    constexpr uint32_t smem = Walk<kRev, NKB, TP>::bytes;
    static_assert(smem >= Walk<kKeep, NKB, TP>::bytes, "one launch, the larger of the two");
    return launch_pdl(kern, dim3((rec.ns + TP - 1) / TP, a.B * a.H, 2), dim3(walk_threads(TP)), smem, st, a,
                      (const __nv_bfloat16 *)dy, W0, dWf, dW0, (uint8_t *)ws, rec, status);
}

template <int NKB>
cudaError_t walks(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g, const void *beta,
                  const float *W0, const void *dy, const float *dWf, float *dW0, void *ws, const GatedRecord &rec,
                  int num_sms, unsigned *status, cudaStream_t st) {
    cudaError_t e = launch_prep<true, NKB>(a, q, k, v, g, beta, dy, ws, rec, 0, rec.nch, false, num_sms, status, st);
    if (e != cudaSuccess)
        return e;
    if (rec.ns > 1 && 2 * (int64_t)rec.ns * a.B * a.H > num_sms)
        return launch_both<NKB, 2>(a, W0, dy, dWf, dW0, ws, rec, status, st);
    return launch_both<NKB, 1>(a, W0, dy, dWf, dW0, ws, rec, status, st);
}

} // namespace

cudaError_t gated_tc_forward(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                             const void *beta, const float *W0, float *Wf, void *y, void *ws, cudaStream_t st) {
    unsigned *status = nullptr;
    int sms = 0;
    cudaError_t e = status_word(&status);
    if (e == cudaSuccess)
        e = device_sms(&sms);
    if (e != cudaSuccess)
        return e;
    const GatedRecord rec = gated_forward_record(a.L, a.d_k, a.d_v);
    return rec.nkb == 1 ? forward<1>(a, q, k, v, g, beta, W0, Wf, y, ws, rec, sms, status, st)
                        : forward<2>(a, q, k, v, g, beta, W0, Wf, y, ws, rec, sms, status, st);
}

cudaError_t gated_tc_walks(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                           const void *beta, const float *W0, const void *dy, const float *dWf, float *dW0, void *ws,
                           cudaStream_t st) {
    unsigned *status = nullptr;
    int sms = 0;
    cudaError_t e = status_word(&status);
    if (e == cudaSuccess)
        e = device_sms(&sms);
    if (e != cudaSuccess)
        return e;
    const GatedRecord rec = gated_backward_record(a.L, a.d_k, a.d_v);
    return rec.nkb == 1 ? walks<1>(a, q, k, v, g, beta, W0, dy, dWf, dW0, ws, rec, sms, status, st)
                        : walks<2>(a, q, k, v, g, beta, W0, dy, dWf, dW0, ws, rec, sms, status, st);
}

} // namespace fw
