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
#include "fw_tc.cuh"

#include <algorithm>

namespace fw {

cudaError_t status_word(unsigned **out); // fw_api.cu

namespace {

using namespace tc;

constexpr int C = kGatedChunk;
constexpr int NT = 256;
constexpr int NV = 32;    // value channels per walk CTA
constexpr int LC = C + 4; // row stride of an fp32 C x C tile
constexpr float kGMin = -200.f; // e^g is 0 in fp32 below this

FW_DEV int seq_len(const GatedArgs &a, int b) {
    return a.lengths ? min(max(__ldcg(a.lengths + b), 0), a.L) : a.L;
}

// 8 fp32 values as 8 hi and 8 lo bf16 terms.
FW_DEV void split8(const float *x, uint4 &hi, uint4 &lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
        l[e] = pack_bf16x2(x[2 * e] - __uint_as_float(h[e] << 16),
                           x[2 * e + 1] - __uint_as_float(h[e] & 0xffff0000u));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

FW_DEV void widen8(uint4 u, float (&o)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// A "pair tile": rows of 128 bytes, 32 channels' hi terms then their lo
// terms, swizzled as the descriptors of fw_tc.cuh expect.  16-byte chunk c.
FW_DEV uint32_t pair_chunk(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

// (I + A)^-1 of the strictly lower triangular A (row stride LC): forward
// substitution in the four 16 x 16 diagonal blocks, one thread a column, then
// two doublings T21 = -T22 (A21 T11).
FW_DEV void unit_lower_inverse(const float *A, float *T, float *tmp) {
    const int tid = threadIdx.x;
    for (int e = tid; e < C * C; e += NT)
        if ((e >> 6) >> 4 < (e & 63) >> 4)
            T[(e >> 6) * LC + (e & 63)] = 0.f;
    if (tid < C) {
        const int b0 = tid & ~15, j = tid & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == j ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < i; ++m)
                s = fmaf(-A[(b0 + i) * LC + b0 + m], x[m], s);
            x[i] = s;
            T[(b0 + i) * LC + b0 + j] = s;
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 16; h <= 32; h *= 2) {
        const int per = h * h, n = (C / (2 * h)) * per;
        for (int e = tid; e < n; e += NT) {
            const int p = e / per, i = (e % per) / h, j = e % h, r0 = p * 2 * h;
            float s = 0.f;
#pragma unroll 8
            for (int m = 0; m < h; ++m)
                s = fmaf(A[(r0 + h + i) * LC + r0 + m], T[(r0 + m) * LC + r0 + j], s);
            tmp[p * per + i * h + j] = s;
        }
        __syncthreads();
        for (int e = tid; e < n; e += NT) {
            const int p = e / per, i = (e % per) / h, j = e % h, r0 = p * 2 * h;
            float s = 0.f;
#pragma unroll 8
            for (int m = 0; m < h; ++m)
                s = fmaf(T[(r0 + h + i) * LC + r0 + h + m], tmp[p * per + m * h + j], s);
            T[(r0 + h + i) * LC + r0 + j] = -s;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------ prep
// One CTA per (chunk, value head).  Shared memory: the [K; Q] tile (K-major,
// 128 rows; its first 64 rows also serve as the MN-major K), an operand
// region (M and T as hi and lo tiles, then the stacked 128 x 64 matrices A1
// and A2 in turn), the fp32 A / T work space (A's place is V's, then dY's,
// once the inverse is done), per-token scalars.
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
    s.bar = s.tok + C * 32;
    s.bytes = s.bar + 64 + 1024;
    return s;
}

template <bool BWD>
__global__ void __launch_bounds__(NT, 2)
    gated_tc_prep_kernel(GatedArgs a, const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ k,
                         const __nv_bfloat16 *__restrict__ v, const __nv_bfloat16 *__restrict__ g,
                         const __nv_bfloat16 *__restrict__ beta, const __nv_bfloat16 *__restrict__ dy, uint8_t *ws,
                         GatedRecord rec, int tmem_cols, unsigned *status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nkb = rec.nkb, dkp = 64 * nkb, nvb = (a.d_v + 63) / 64;
    const PrepSmem o = prep_smem(nkb, nvb);
    uint8_t *kq = sm + o.kq, *op = sm + o.op, *vt = sm + o.at;
    float *At = reinterpret_cast<float *>(sm + o.at), *tmp = At + C * LC, *Tt = reinterpret_cast<float *>(sm + o.tt);
    float *tok = reinterpret_cast<float *>(sm + o.tok); // per token: G hi, G lo, rk, beta, rq, e^G, e^{G_C-G}, -
    uint64_t *bar = reinterpret_cast<uint64_t *>(sm + o.bar);
    uint32_t *slot = reinterpret_cast<uint32_t *>(bar + 1);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, c = blockIdx.x, bh = blockIdx.y;
    const int b = bh / a.H, h = bh % a.H, kh = b * a.Hk + h / (a.H / a.Hk);
    griddep_wait();
    const int n = min(C, seq_len(a, b) - c * C);
    if (n <= 0) {
        griddep_launch_dependents();
        return;
    }
    if (w == 0)
        tmem_alloc(slot, (uint32_t)tmem_cols);
    if (tid == 32) {
        mbar_init(bar, 1);
        fence_barrier_init();
    }
    // [K; Q], 16 bytes a thread and step; the row's lanes add its squares
    {
        const __nv_bfloat16 *kg = k + ((size_t)kh * a.L + (size_t)c * C) * a.d_k;
        const __nv_bfloat16 *qg = q + ((size_t)kh * a.L + (size_t)c * C) * a.d_k;
        const int per = dkp / 8, steps = 2 * C * per / NT; // chunks per row; 4 or 8 steps
        const int ch = tid % per;
        uint4 u[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const int row = (s * NT + tid) / per;
            u[s] = make_uint4(0, 0, 0, 0);
            if (s < steps && (row & 63) < n && ch * 8 < a.d_k)
                u[s] = __ldcg(reinterpret_cast<const uint4 *>((row < C ? kg : qg) + (size_t)(row & 63) * a.d_k) + ch);
        }
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            if (s >= steps)
                break;
            const int row = (s * NT + tid) / per;
            *reinterpret_cast<uint4 *>(kq + kmajor_chunk(row, ch * 8, 128)) = u[s];
            float x[8], ss = 0.f;
            widen8(u[s], x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                ss = fmaf(x[e], x[e], ss);
            for (int m = per / 2; m > 0; m >>= 1)
                ss += __shfl_xor_sync(0xffffffffu, ss, m);
            if (ch == 0) {
                ss += a.eps;
                tok[(row & 63) * 8 + (row < C ? 2 : 4)] = !a.l2norm ? 1.f : ss > 0.f ? 1.f / sqrtf(ss) : ss;
            }
        }
    }
    if (w == 1) { // the running sums of g in 64 bits, two tokens a lane
        const size_t t0 = (size_t)bh * a.L + (size_t)c * C;
        double s[2];
        float be[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * lane + e;
            const float x = i < n ? io<__nv_bfloat16>::load(g + t0 + i) : 0.f;
            s[e] = x < kGMin ? kGMin : x;
            be[e] = i < n ? io<__nv_bfloat16>::load(beta + t0 + i) : 0.f;
        }
        s[1] += s[0];
        double run = s[1];
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, run, m);
            if (lane >= m)
                run += up;
        }
        const double before = run - s[1], all = __shfl_sync(0xffffffffu, run, 31);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const double G = before + s[e];
            float *d = tok + (2 * lane + e) * 8;
            d[0] = (float)G;
            d[1] = (float)(G - (double)(float)G);
            d[3] = be[e];
            d[5] = expf((float)G);
            d[6] = expf((float)(all - G));
            d[7] = 0.f;
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
    const uint32_t kq_s = smem_u32(kq), op_s = smem_u32(op), vt_s = smem_u32(vt);
    uint8_t *out = ws + rec.off(bh, c);
    if (tid == 0) { // K K^T (rows 0-63) and Q K^T
        const uint32_t id = idesc_bf16(128, 64, 0, 0);
        for (int s = 0; s < 4 * nkb; ++s) {
            const uint64_t d = desc_sw128(kq_s + kmajor_step(s, 128), 16, 1024);
            mma_bf16(tGram, d, d, id, s > 0);
        }
        mma_commit(bar);
        // the K (and Q) image for the walk, straight from the tile
        if (BWD) {
            bulk_s2g(out + rec.KQ, kq, (uint32_t)nkb * 16384u);
        } else {
            for (int kb = 0; kb < nkb; ++kb)
                bulk_s2g(out + rec.K + kb * 8192, kq + kb * 16384, 8192);
        }
        bulk_commit();
    }
    finish();
    const int rr = 32 * (w & 3) + lane, half = w >> 2, i = rr & 63;
    {
        const float4 di = *reinterpret_cast<const float4 *>(tok + i * 8);
        const float fi = rr < C ? di.w * di.z : a.scale * tok[i * 8 + 4];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int j0 = 32 * half + 16 * p;
            float x[16];
            tmem_ld16(tGram + tmem_lane_base(w) + (uint32_t)j0, x);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int j = j0 + e;
                const float4 dj = *reinterpret_cast<const float4 *>(tok + j * 8);
                const bool in = rr < C ? j < i : j <= i;
                x[e] = in ? fi * dj.z * x[e] * expf((di.x - dj.x) + (di.y - dj.y)) : 0.f;
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
                    const uint32_t at = kmajor_chunk(i, j0 + e, 64);
                    *reinterpret_cast<uint4 *>(op + at) = hi;
                    *reinterpret_cast<uint4 *>(op + 8192 + at) = lo;
                }
            }
        }
    }
    __syncthreads();
    unit_lower_inverse(At, Tt, tmp);
    for (int e = tid; e < C * 8; e += NT) { // T as hi and lo tiles
        const int r = e >> 3, j0 = (e & 7) * 8;
        uint4 hi, lo;
        split8(Tt + r * LC + j0, hi, lo);
        const uint32_t at = kmajor_chunk(r, j0, 64);
        *reinterpret_cast<uint4 *>(op + 16384 + at) = hi;
        *reinterpret_cast<uint4 *>(op + 24576 + at) = lo;
    }
    hand_over();
    if (tid == 0) { // M T, or (M T)^T = T^T M^T
        for (int t = 0; t < 3; ++t) { // hi hi, hi lo, lo hi
            const uint32_t m = op_s + (t == 2 ? 8192u : 0u), tt = op_s + 16384u + (t == 1 ? 8192u : 0u);
            for (int s = 0; s < 4; ++s) {
                const uint64_t dm = desc_sw128(m + kmajor_step(s, 64), 16, 1024);
                const uint64_t dt = desc_sw128(tt + (uint32_t)s * 2048u, 8192, 1024);
                if (BWD)
                    mma_bf16(tMT, dt, dm, idesc_bf16(128, 64, 1, 0), (t | s) != 0);
                else
                    mma_bf16(tMT, dm, dt, idesc_bf16(128, 64, 0, 1), (t | s) != 0);
            }
        }
        mma_commit(bar);
    }
    auto load_rows = [&](const __nv_bfloat16 *src) { // V or dY, MN-major 64-channel blocks
        const __nv_bfloat16 *sg = src + ((size_t)bh * a.L + (size_t)c * C) * a.d_v;
        for (int e = tid; e < C * nvb * 8; e += NT) {
            const int r = e / (nvb * 8), ch = e % (nvb * 8);
            uint4 u = make_uint4(0, 0, 0, 0);
            if (r < n && ch * 8 < a.d_v)
                u = __ldcg(reinterpret_cast<const uint4 *>(sg + (size_t)r * a.d_v) + ch);
            *reinterpret_cast<uint4 *>(vt + kmajor_chunk(r, ch * 8, 64)) = u;
        }
    };
    load_rows(v);
    finish();
    // Stacked left factors, hi tile then lo tile: rows 0-63 from T, rows
    // 64-127 from MT (TMEM lanes 0-63, so the warps that can read those
    // lanes write the lower rows) or, for W", from T^T.
    auto put = [&](int row, int j0, const float *x) {
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
            uint4 hi, lo;
            split8(x + e, hi, lo);
            const uint32_t at = kmajor_chunk(row, j0 + e, 128);
            *reinterpret_cast<uint4 *>(op + at) = hi;
            *reinterpret_cast<uint4 *>(op + 16384 + at) = lo;
        }
    };
    auto build = [&](bool first) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int j0 = 32 * half + 16 * p;
            float x[16];
            if (rr >= C) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float *d = tok + (j0 + e) * 8;
                    x[e] = Tt[i * LC + j0 + e] * (first ? -d[3] * d[5] * d[2] : d[3]);
                }
            } else if (BWD && first) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float *d = tok + (j0 + e) * 8;
                    x[e] = Tt[(j0 + e) * LC + i] * d[6] * d[2];
                }
            } else {
                tmem_ld16(tMT + tmem_lane_base(w) + (uint32_t)j0, x);
                tmem_ld_wait();
                if (!BWD) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float *d = tok + (j0 + e) * 8;
                        x[e] *= first ? -d[3] * d[5] * d[2] : d[3];
                    }
                }
            }
            put(rr ^ 64, j0, x);
        }
    };
    auto multiply = [&](uint32_t d, uint32_t bsrc, uint32_t lbo, int N) {
        if (tid == 0) {
            const uint32_t id = idesc_bf16(128, N, 0, 1);
            for (int t = 0; t < 2; ++t)
                for (int s = 0; s < 4; ++s)
                    mma_bf16(d, desc_sw128(op_s + (uint32_t)t * 16384u + (uint32_t)s * 32u, 16, 1024),
                             desc_sw128(bsrc + (uint32_t)s * 2048u, lbo, 1024), id, (t | s) != 0);
            mma_commit(bar);
        }
    };
    build(true);
    hand_over();
    multiply(tA1, kq_s, 16384, dkp); // [-W'; ...] or [-W'; W"]
    finish();
    build(false);
    hand_over();
    multiply(tA2, vt_s, 8192, a.d_v);
    // meanwhile the first product's rows as hi and lo images
    for (int p = half; p < dkp / 16; p += 2) {
        const int c0 = 16 * p;
        float x[16];
        tmem_ld16(tA1 + tmem_lane_base(w) + (uint32_t)c0, x);
        tmem_ld_wait();
        if (!BWD && rr >= C) {
            const float f = a.scale * tok[i * 8 + 5] * tok[i * 8 + 4];
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
            uint8_t *to;
            size_t lo_at;
            if (BWD) {
                to = out + (rr < C ? rec.AF : rec.AR) + kmajor_chunk(i, c0 + e, 64);
                lo_at = (size_t)nkb * 8192;
            } else {
                to = out + rec.A + kmajor_chunk(rr, c0 + e, 128);
                lo_at = (size_t)nkb * 16384;
            }
            *reinterpret_cast<uint4 *>(to) = hi;
            *reinterpret_cast<uint4 *>(to + lo_at) = lo;
        }
    }
    if (tid < C) { // the walks' scalars
        const float *d = tok + tid * 8;
        float *sf = reinterpret_cast<float *>(out + rec.scalF);
        sf[tid] = d[6] * d[2];
        if (tid == 0)
            sf[C] = tok[(C - 1) * 8 + 5];
        if (BWD) {
            float *sr = reinterpret_cast<float *>(out + rec.scalR);
            sr[tid] = -d[3] * d[5] * d[2];
            sr[C + tid] = a.scale * d[5] * d[4];
            if (tid == 0)
                sr[2 * C] = tok[(C - 1) * 8 + 5];
            float4 *st = reinterpret_cast<float4 *>(out + rec.tok) + 2 * tid;
            st[0] = reinterpret_cast<const float4 *>(d)[0];
            st[1] = reinterpret_cast<const float4 *>(d)[1];
        }
    }
    finish();
    auto rows_out = [&](size_t base, int rows, int row, bool on) { // [slice][rows][32] fp32
        for (int p = half; p < a.d_v / 16; p += 2) {
            float x[16];
            tmem_ld16(tA2 + tmem_lane_base(w) + (uint32_t)(16 * p), x);
            tmem_ld_wait();
            if (on) {
                float4 *to = reinterpret_cast<float4 *>(out + base) + ((size_t)(p >> 1) * rows + row) * 8 + (p & 1) * 4;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    to[e] = make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
            }
        }
    };
    if (!BWD) {
        rows_out(rec.base, 128, rr, true);
    } else {
        rows_out(rec.baseU, C, i, rr < C);
        load_rows(dy); // V's place
        hand_over();
        multiply(tA2, vt_s, 8192, a.d_v);
        finish();
        rows_out(rec.baseX, C, i, rr >= C);
    }
    if (tid == 0)
        bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (w == 0) {
        tmem_relinquish();
        tmem_dealloc(tm, (uint32_t)tmem_cols);
    }
}

// ------------------------------------------------------------------ walk
// One CTA per (value head, 32 value channels); thread (row 32 (w % 4) + lane,
// 16 channels) holds 16 values of the state (row = key channel) and handles
// 16 values of a token's row between the products.  Two records are in
// flight; the values' base rows and dY are read a chunk ahead.
enum { kFwd = 0, kKeep = 1, kRev = 2 };

struct WalkSmem {
    uint32_t b, scal, rec, z, u, bar, bytes; // b, scal: offsets inside a record
};
template <int MODE> __host__ __device__ inline WalkSmem walk_smem(int nkb) {
    WalkSmem s;
    s.b = (uint32_t)nkb * (MODE == kFwd ? 32768 : 16384);
    s.scal = s.b + (uint32_t)nkb * (MODE == kRev ? 16384 : 8192);
    s.rec = s.scal + 1024;
    s.z = 2 * s.rec;
    s.u = s.z + (uint32_t)nkb * 8192;
    s.bar = s.u + (MODE == kRev ? 16384 : 8192);
    // a 128-row MMA reads 8 KB past a tile of 64 rows: into what follows, or into this slack
    s.bytes = s.bar + 64 + 8192 + 1024;
    return s;
}

template <int MODE>
__global__ void __launch_bounds__(NT)
    gated_tc_walk_kernel(GatedArgs a, const __nv_bfloat16 *__restrict__ dy, const float *__restrict__ Z0,
                         float *__restrict__ Zf, __nv_bfloat16 *__restrict__ y, uint8_t *ws, GatedRecord rec,
                         unsigned *status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int nkb = rec.nkb, dkp = 64 * nkb;
    const WalkSmem o = walk_smem<MODE>(nkb);
    uint8_t *zt = sm + o.z, *ut = sm + o.u;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + o.bar), *m1 = full + 2, *m2 = full + 3;
    uint32_t *slot = reinterpret_cast<uint32_t *>(full + 4);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, sl = blockIdx.x, bh = blockIdx.y, n0 = sl * NV;
    const int b = bh / a.H;
    const int rr = 32 * (w & 3) + lane, hf = w >> 2, i = rr & 63;
    const bool mine = n0 + 16 * hf < a.d_v; // these 16 channels exist (d_v is a multiple of 16)
    const bool zrow = 32 * (w & 3) < dkp;   // this warp holds rows of the state
    griddep_wait();
    const int len = seq_len(a, b), nch = (len + C - 1) / C;
    if (w == 0)
        tmem_alloc(slot, 128);
    if (tid == 32) {
        for (int e = 0; e < 4; ++e)
            mbar_init(full + e, 1);
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tm = *slot, tD1 = tm, tD2 = tm + 64;
    auto chunk_of = [&](int it) { return MODE == kRev ? nch - 1 - it : it; };
    auto fetch = [&](int it) { // thread 0: a chunk's record
        const uint8_t *src = ws + rec.off(bh, chunk_of(it));
        uint8_t *dst = sm + (it & 1) * o.rec;
        uint64_t *f = full + (it & 1);
        if (MODE == kFwd) { // A, K and the scalars are one piece
            const uint32_t bytes = (uint32_t)nkb * 40960u + 512u;
            mbar_arrive_expect_tx(f, bytes);
            bulk_g2s(dst, src + rec.A, bytes, f);
        } else if (MODE == kKeep) {
            mbar_arrive_expect_tx(f, (uint32_t)nkb * 24576u + 512u);
            bulk_g2s(dst, src + rec.AF, (uint32_t)nkb * 16384u, f);
            for (int kb = 0; kb < nkb; ++kb)
                bulk_g2s(dst + o.b + kb * 8192, src + rec.KQ + kb * 16384, 8192, f);
            bulk_g2s(dst + o.scal, src + rec.scalF, 512, f);
        } else {
            mbar_arrive_expect_tx(f, (uint32_t)nkb * 32768u + 1024u);
            bulk_g2s(dst, src + rec.AR, (uint32_t)nkb * 16384u, f);
            bulk_g2s(dst + o.b, src + rec.KQ, (uint32_t)nkb * 16384u, f);
            bulk_g2s(dst + o.scal, src + rec.scalR, 1024, f);
        }
    };
    float z[16], next[16]; // the state's rows; the next chunk's base row (or dY row)
    auto ahead = [&](int it) {
        const int c = chunk_of(it);
        const uint8_t *r = ws + rec.off(bh, c);
        if (MODE == kRev && rr >= C) {
            const int n = min(C, len - c * C);
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                float x[8] = {};
                if (mine && i < n)
                    load8(dy + ((size_t)bh * a.L + (size_t)c * C + i) * a.d_v + n0 + 16 * hf + e, x);
#pragma unroll
                for (int m = 0; m < 8; ++m)
                    next[e + m] = x[m];
            }
            return;
        }
        const size_t base = MODE == kFwd ? rec.base : MODE == kKeep ? rec.baseU : rec.baseX;
        const int rows = MODE == kFwd ? 128 : C;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (mine && rr < rows)
                x = __ldcg(reinterpret_cast<const float4 *>(r + base) + ((size_t)sl * rows + rr) * 8 + hf * 4 + e);
            next[4 * e] = x.x;
            next[4 * e + 1] = x.y;
            next[4 * e + 2] = x.z;
            next[4 * e + 3] = x.w;
        }
    };
    auto put = [&](uint8_t *tile, int row, const float *x) { // 16 channels of a pair tile's row
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            uint4 hi, lo;
            split8(x + 8 * e, hi, lo);
            *reinterpret_cast<uint4 *>(tile + pair_chunk(row, 2 * hf + e)) = hi;
            *reinterpret_cast<uint4 *>(tile + pair_chunk(row, 4 + 2 * hf + e)) = lo;
        }
    };
    if (tid == 0)
        for (int it = 0; it < min(2, nch); ++it)
            fetch(it);
    if (nch > 0)
        ahead(0);
#pragma unroll
    for (int e = 0; e < 16; ++e)
        z[e] = Z0 && mine && rr < a.d_k
                   ? __ldcg(Z0 + ((size_t)bh * a.d_v + n0 + 16 * hf + e) * a.d_k + rr)
                   : 0.f;
    if (zrow)
        put(zt, rr, z);
    bool ok = true;
    const uint32_t zt_s = smem_u32(zt), ut_s = smem_u32(ut);
    for (int it = 0; it < nch; ++it) {
        const int c = chunk_of(it), n = min(C, len - c * C);
        uint8_t *r = sm + (it & 1) * o.rec;
        const uint32_t r_s = smem_u32(r);
        uint8_t *gr = ws + rec.off(bh, c);
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        if (ok)
            ok = mbar_wait(full + (it & 1), (it >> 1) & 1, status);
        if (tid == 0 && ok) {
            tc_fence_after();
            constexpr int R = MODE == kFwd ? 128 : 64; // rows of the A tile
            for (int t = 0; t < 2; ++t) // hi rows times [Z hi | Z lo], lo rows times Z hi
                for (int s = 0; s < 4 * nkb; ++s)
                    mma_bf16(tD1, desc_sw128(r_s + (uint32_t)(t * nkb * R * 128) + kmajor_step(s, R), 16, 1024),
                             desc_sw128(zt_s + (uint32_t)s * 2048u, 8192, 1024), idesc_bf16(128, t ? 32 : 64, 0, 1),
                             (t | s) != 0);
            mma_commit(m1);
        }
        if (MODE != kFwd && tid == 32) { // the state before this chunk, as it lies
            bulk_s2g(gr + (MODE == kKeep ? rec.S : rec.dS) + (size_t)sl * dkp * 128, zt, (uint32_t)dkp * 128u);
            bulk_commit();
        }
        const float *scal = reinterpret_cast<const float *>(r + o.scal);
        const float whole = scal[MODE == kRev ? 2 * C : C];
        float x[16], t0[16], t1[16];
        if (MODE == kRev && rr >= C) { // dY's rows do not wait for the product
            const float f = scal[C + i];
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[e] = f * next[e];
            put(ut, rr, x);
        }
        if (ok)
            ok = mbar_wait(m1, it & 1, status);
        tc_fence_after();
        if (MODE == kFwd || rr < C) {
            tmem_ld16(tD1 + tmem_lane_base(w) + (uint32_t)(16 * hf), t0);
            tmem_ld16(tD1 + tmem_lane_base(w) + (uint32_t)(32 + 16 * hf), t1);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[e] = next[e] + (t0[e] + t1[e]);
            if (rr < C) {
                const float f = scal[i];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    t0[e] = f * x[e];
                put(ut, i, t0);
            }
        }
        if (MODE != kFwd && tid == 32)
            bulk_wait_read(); // the stored state has left its tile
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0 && ok) {
            tc_fence_after();
            constexpr int R = MODE == kRev ? 128 : 64; // rows of the B^T tile
            for (int s = 0; s < R / 16; ++s)
                mma_bf16(tD2, desc_sw128(r_s + o.b + (uint32_t)s * 2048u, R * 128, 1024),
                         desc_sw128(ut_s + (uint32_t)s * 2048u, 8192, 1024), idesc_bf16(128, 64, 1, 1), s > 0);
            mma_commit(m2);
        }
        if (MODE == kFwd && rr >= C) {
            if (mine && i < n) {
                uint4 *to = reinterpret_cast<uint4 *>(y + ((size_t)bh * a.L + (size_t)c * C + i) * a.d_v + n0 + 16 * hf);
                float p[8];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int m = 0; m < 8; ++m)
                        p[m] = x[8 * e + m];
                    store8(reinterpret_cast<__nv_bfloat16 *>(to + e), p);
                }
            }
        } else if (MODE != kFwd && rr < C) { // U, or dX, for the gradients: a pair tile's row
            put(gr + (MODE == kKeep ? rec.U : rec.dX) + (size_t)sl * 8192, i, x);
        }
        if (it + 1 < nch)
            ahead(it + 1);
        if (ok)
            ok = mbar_wait(m2, it & 1, status);
        tc_fence_after();
        if (tid == 0 && ok && it + 2 < nch)
            fetch(it + 2);
        if (zrow) {
            tmem_ld16(tD2 + tmem_lane_base(w) + (uint32_t)(16 * hf), t0);
            tmem_ld16(tD2 + tmem_lane_base(w) + (uint32_t)(32 + 16 * hf), t1);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                z[e] = fmaf(whole, z[e], t0[e] + t1[e]);
            put(zt, rr, z);
        }
    }
    if (Zf && mine && rr < a.d_k)
#pragma unroll
        for (int e = 0; e < 16; ++e)
            Zf[((size_t)bh * a.d_v + n0 + 16 * hf + e) * a.d_k + rr] = z[e];
    if (MODE == kFwd) { // no token, no answer
        const int nv = min(NV, a.d_v - n0);
        const size_t c8 = nv / 8, cnt = (size_t)(a.L - len) * c8;
        for (size_t e = tid; e < cnt; e += NT)
            *reinterpret_cast<uint4 *>(y + ((size_t)bh * a.L + len + e / c8) * a.d_v + n0 + 8 * (e % c8)) =
                make_uint4(0, 0, 0, 0);
    }
    if (!ok && tid == 0) // a wait gave up: let the records that were asked for land first
        for (int e = 0; e < 2; ++e)
            (void)mbar_wait(full + e, 0, status);
    if (MODE != kFwd && tid == 32)
        bulk_wait_all();
    tc_fence_before();
    __syncthreads();
    if (w == 0) {
        tmem_relinquish();
        tmem_dealloc(tm, 128);
    }
}

template <typename K> cudaError_t allow_smem(K *kern, size_t bytes) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    return e;
}

template <bool BWD>
cudaError_t launch_prep(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                        const void *beta, const void *dy, void *ws, const GatedRecord &rec, unsigned *status,
                        cudaStream_t st) {
    using bf = __nv_bfloat16;
    const uint32_t smem = prep_smem(rec.nkb, (a.d_v + 63) / 64).bytes;
    cudaError_t e = allow_smem(gated_tc_prep_kernel<BWD>, smem);
    if (e != cudaSuccess)
        return e;
    // 128 columns for A1's product, d_v for A2's (MT's 64 lie there first)
    const int cols = a.d_v <= 128 ? 256 : 512;
    return launch_pdl(gated_tc_prep_kernel<BWD>, dim3(rec.nch, a.B * a.H), dim3(NT), smem, st, a, (const bf *)q,
                      (const bf *)k, (const bf *)v, (const bf *)g, (const bf *)beta, (const bf *)dy, (uint8_t *)ws, rec,
                      cols, status);
}

template <int MODE>
cudaError_t launch_walk(const GatedArgs &a, const void *dy, const float *Z0, float *Zf, void *y, void *ws,
                        const GatedRecord &rec, unsigned *status, cudaStream_t st) {
    using bf = __nv_bfloat16;
    const uint32_t smem = walk_smem<MODE>(rec.nkb).bytes;
    cudaError_t e = allow_smem(gated_tc_walk_kernel<MODE>, smem);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(gated_tc_walk_kernel<MODE>, dim3(rec.ns, a.B * a.H), dim3(NT), smem, st, a, (const bf *)dy, Z0,
                      Zf, (bf *)y, (uint8_t *)ws, rec, status);
}

} // namespace

cudaError_t gated_tc_forward(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                             const void *beta, const float *W0, float *Wf, void *y, void *ws, cudaStream_t st) {
    unsigned *status = nullptr;
    cudaError_t e = status_word(&status);
    if (e != cudaSuccess)
        return e;
    const GatedRecord rec = gated_forward_record(a.L, a.d_k, a.d_v);
    e = launch_prep<false>(a, q, k, v, g, beta, nullptr, ws, rec, status, st);
    if (e != cudaSuccess)
        return e;
    return launch_walk<kFwd>(a, nullptr, W0, Wf, y, ws, rec, status, st);
}

cudaError_t gated_tc_walks(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                           const void *beta, const float *W0, const void *dy, const float *dWf, float *dW0, void *ws,
                           cudaStream_t st) {
    unsigned *status = nullptr;
    cudaError_t e = status_word(&status);
    if (e != cudaSuccess)
        return e;
    const GatedRecord rec = gated_backward_record(a.L, a.d_k, a.d_v);
    e = launch_prep<true>(a, q, k, v, g, beta, dy, ws, rec, status, st);
    if (e == cudaSuccess)
        e = launch_walk<kKeep>(a, nullptr, W0, nullptr, nullptr, ws, rec, status, st);
    if (e == cudaSuccess)
        e = launch_walk<kRev>(a, dy, dWf, dW0, nullptr, ws, rec, status, st);
    return e;
}

} // namespace fw
