// fw_gated_grad_tc.cu -- the gradients of a chunk's tokens in the gated delta
// rule (bf16 tensors), from what the two walks left: U, dX, the chunk's first
// state S and the gradient dS' of its last one.
//
// With the names of fw_gated_chunk.cu, and everything in unit keys and
// queries:
//   a = scale e^G (dY S) + E K,   h = e^G (dX S) + F K,
//   w = e^{G_C-G} (U dS') + E^T Q - F^T diag(beta) K,
//   E = lower(scale D dY U^T),    F = strict_lower(D dX U^T),
//   dq = a,  dk = w - beta h,  dV = beta dX,  dbeta_i = dX_i.V_i - k_i.h_i,
//   dg_t = e^{G_C} <S, dS'> + sum_{i >= t} R_i + sum_{j < t} W_j + sum_{i >= t > j} P_ij:
//   what a token reads of S (R), writes to dS' (W), and the pairs with E and F (P).
//
// Six products on the tensor cores, each fp32 operand as two bf16 terms (see
// fw_gated_tc.cu; one term's 2^-9 would show beside the outputs' rounding):
//   [Q; K] K^T, for P;
//   [dY; dX] S and [dY; dX] U^T (128 rows: dY, then dX) and U dS', summed over
//   32-channel slices as the walks stored them, two slices in flight;
//   then [E; F] K and [E; F]^T [Q; K].
// One CTA per (chunk, key head) goes through the value heads that share the
// key, so dq and dk are sums in a fixed order.
//
// What bounds it: for d_k > 64 one CTA an SM (tensor memory, shared memory),
// and a head's 224 KB (d 128) come in four slices of which two fit.  B8 H16
// L2048, two value heads a key head: 325 us, 3.0 TB/s (299 without the sums
// over P, which dg cannot do without); without them a head takes 19 700
// cycles: 10 300 of slices (their copies), 1 100 for the last product, 2 600
// for E and F, 1 500 for the second products, 3 600 for the sums.  It took
// 28 600 when the next slice was asked for after a product had been issued
// instead of when its place was free, the next head's after the sums, and dY
// and V came through registers (375 us); 23 300 with the products issued by a
// warp that shared in the work on the slices; 21 000 without pairs of floats.
#include "fw_gated.h"
#include "fw_gated_tc.h"
#include "fw_gated_tiles.cuh"
#include "fw_tc.cuh"

#include <algorithm>

namespace fw {

cudaError_t status_word(unsigned **out); // fw_api.cu

namespace {

using namespace tc;
using bf = __nv_bfloat16;

constexpr int C = kGatedChunk;
// The warps that share 32 rows split their columns: 16 warps, or 8 for d_k <= 64,
// where two CTAs share an SM's registers.
__host__ __device__ constexpr int parts_of(int nkb) { return 2 * nkb; }

// 8 channels (chunk c of 4) of a pair tile's row: hi + lo.
FW_DEV void pair8(const uint8_t *tile, int row, int c, F2 (&o)[4]) {
    F2 l[4];
    widen8(*reinterpret_cast<const uint4 *>(tile + pair_chunk(row, c)), o);
    widen8(*reinterpret_cast<const uint4 *>(tile + pair_chunk(row, c + 4)), l);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = o[e] + l[e];
}

// Shared memory: [Q; K]; two slices (S, U, dS', [dY; dX]), whose place the E
// and F tiles (64 KB) take afterwards; the sums of dq and dk over the value
// heads -- in the place of the E and F tiles, too, where a key head has one
// value head, so that for d_k <= 64 two CTAs fit an SM (B4 H8 L512, 256 CTAs:
// the whole backward 57 us with one an SM, 52 with two); scalars of this head
// and the next; V's rows of two slices, whose place the sums over P take
// afterwards.
struct GradSmem {
    uint32_t slice, s, ds, yx, u, ef, accq, acck, tok, v, red, bar, bytes;
};
__host__ __device__ inline GradSmem grad_smem(int nkb, bool alone) {
    GradSmem o;
    o.ef = (uint32_t)nkb * 16384;
    o.s = 0; // U follows S, so that one product reads both
    o.u = (uint32_t)nkb * 8192;
    o.ds = o.u + 8192;
    o.yx = o.ds + (uint32_t)nkb * 8192;
    o.slice = o.yx + 16384;
    const uint32_t end = o.ef + 2 * o.slice; // (the E and F tiles are shorter)
    o.accq = alone ? o.ef : end;
    o.acck = o.accq + (uint32_t)nkb * 16384;
    // (U as 128 rows reads 8 KB past it, of dS')
    o.tok = alone ? end : o.acck + (uint32_t)nkb * 16384;
    o.v = o.tok + 2 * C * 32;
    o.red = o.v + 2 * C * 64;
    o.bar = o.red + 4 * ((4 * parts_of(nkb) + 2) * C + 16);
    o.bytes = o.bar + 64 + 1024;
    return o;
}

template <int NKB>
__global__ void __launch_bounds__(128 * parts_of(NKB), NKB == 1 ? 2 : 1)
    gated_tc_grad_kernel(GatedArgs a, const bf *__restrict__ v, const bf *__restrict__ dy, bf *__restrict__ dq,
                         bf *__restrict__ dk, bf *__restrict__ dv, bf *__restrict__ dg, bf *__restrict__ dbeta,
                         const uint8_t *ws, GatedRecord rec, unsigned *status) {
    constexpr int PARTS = parts_of(NKB), NT = 128 * PARTS;
    constexpr int DKP = 64 * NKB, HC = DKP / PARTS; // channels per thread of a row
    constexpr uint32_t kCols = 256 * NKB;               // TMEM: three products of DKP columns, one of 64
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const GradSmem o = grad_smem(NKB, a.H == a.Hk);
    uint8_t *kq = sm, *ef = sm + o.ef;
    float *tok = reinterpret_cast<float *>(sm + o.tok);
    float *red = reinterpret_cast<float *>(sm + o.red);
    // one value per part: q.a and k.h of what is read of S, k.h in all, W; then dX.V, the pairs across, <S, dS'>
    float *r_qa = red, *r_k0 = red + PARTS * C, *r_kh = red + 2 * PARTS * C, *r_w = red + 3 * PARTS * C,
          *r_xv = red + 4 * PARTS * C, *r_c = r_xv + C, *r_ss = r_c + C;
    // P's sums: over the columns of a block of 16 before a token, of a warp's rows from it on, and whole rows of a block
    float *p_part = reinterpret_cast<float *>(sm + o.v), *p_row = p_part + 4 * C;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + o.bar), *done = full + 2, *kqb = full + 4, *mm = full + 5;
    uint32_t *slot = reinterpret_cast<uint32_t *>(full + 6);
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, c = blockIdx.x, bk = blockIdx.y;
    const int b = bk / a.Hk, grp = a.H / a.Hk, ns = rec.ns;
    const int rr = 32 * (w & 3) + lane, part = w >> 2, i = rr & 63;
    // One thread asks for the slices and issues the products.  Of 16 warps its
    // warp is left out of the work on the slices, which runs meanwhile.
    constexpr int BOSS = NKB == 2 ? 15 : 0;
    constexpr int ADDER = NKB == 2 ? 14 : 2; // the warp that adds up P (it has less to do than one of rows 0 - 63)
    const bool boss = tid == 32 * BOSS;
    griddep_wait();
    v = after_wait(v);
    dy = after_wait(dy);
    const int n = min(C, seq_len(a, b) - c * C), rows = min(C, a.L - c * C); // tokens; rows in memory
    const size_t krow = ((size_t)bk * a.L + (size_t)c * C) * a.d_k;
    if (n <= 0) { // behind the sequence's end: no gradient
        griddep_launch_dependents();
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int e = tid; e < rows * a.d_k / 8; e += NT) {
            reinterpret_cast<uint4 *>(dq + krow)[e] = zero;
            reinterpret_cast<uint4 *>(dk + krow)[e] = zero;
        }
        for (int m = 0; m < grp; ++m) {
            const size_t r0 = (size_t)(bk * grp + m) * a.L + (size_t)c * C;
            for (int e = tid; e < rows * a.d_v / 8; e += NT)
                reinterpret_cast<uint4 *>(dv + r0 * a.d_v)[e] = zero;
            for (int e = tid; e < rows; e += NT) {
                io<bf>::store(dg + r0 + e, 0.f);
                io<bf>::store(dbeta + r0 + e, 0.f);
            }
        }
        return;
    }
    bool ok = true;
    auto record = [&](int m) { return ws + rec.off((int64_t)bk * grp + m, c); };
    auto fetch = [&](const uint8_t *src, int s, int g) { // boss: slice s of a record, as the g-th of all
        uint8_t *dst = ef + (g & 1) * o.slice;
        uint64_t *f = full + (g & 1);
        mbar_arrive_expect_tx(f, (uint32_t)(NKB * 16384 + 16384));
        bulk_g2s(dst + o.s, src + rec.S + (size_t)s * NKB * 8192, NKB * 8192, f);
        bulk_g2s(dst + o.ds, src + rec.dS + (size_t)s * NKB * 8192, NKB * 8192, f);
        bulk_g2s(dst + o.yx + 8192, src + rec.dX + (size_t)s * 8192, 8192, f);
        bulk_g2s(dst + o.u, src + rec.U + (size_t)s * 8192, 8192, f);
    };
    // 256 threads: a row and 8 of 32 channels of dY, dX, V; seven of the other warps, if any: <S, dS'>
    const bool rowed = tid < 256, squared = NT == 256 || (!rowed && w != BOSS);
    const int yr = (tid >> 2) & 63, yc = tid & 3;
    int gs = 0; // slices seen
    auto row_at = [&](int m, int s) { // dY's and V's 8 channels of slice s, value head m
        return ((size_t)(bk * grp + m) * a.L + (size_t)c * C + yr) * a.d_v + 32 * s + 8 * yc;
    };
    auto row_in = [&](int s) { return 32 * s + 8 * yc < a.d_v && yr < n; };
    auto request = [&](int m, int s, int g) { // into slice g's place; dY has no lo terms
        if (rowed) {
            uint8_t *yx = ef + (g & 1) * o.slice + o.yx;
            const bool in = row_in(s);
            const size_t at = in ? row_at(m, s) : 0;
            copy16(yx + pair_chunk(yr, yc), dy + at, in);
            copy16(sm + o.v + (g & 1) * (C * 64) + tid * 16, v + at, in);
            *reinterpret_cast<uint4 *>(yx + pair_chunk(yr, yc + 4)) = make_uint4(0, 0, 0, 0);
        }
    };
    // a head's first two slices and its scalars: asked for as soon as their
    // places are free, the next head's while this one's last sums are taken
    auto begin = [&](int m) {
        const uint8_t *src = record(m);
        if (boss && ok) {
            // generic reads and writes of the place end before the copies into it
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            fetch(src, 0, gs);
            if (ns > 1)
                fetch(src, 1, gs + 1);
        }
        request(m, 0, gs);
        if (ns > 1)
            request(m, 1, gs + 1);
        if (tid < 2 * C)
            copy16(sm + o.tok + (m & 1) * (C * 32) + tid * 16, src + rec.tok + tid * 16, true);
    };
    if (boss) {
        for (int e = 0; e < 5; ++e)
            mbar_init(full + e, 1);
        mbar_init(mm, 2); // the products; P's sums have been read
        fence_barrier_init();
    }
    begin(0);
    if (boss) {
        mbar_arrive_expect_tx(kqb, NKB * 16384);
        for (int kb = 0; kb < NKB; ++kb) { // (the record has the keys first)
            const uint8_t *src = record(0) + rec.K + kb * 16384;
            bulk_g2s(kq + kb * 16384, src + 8192, 8192, kqb);
            bulk_g2s(kq + kb * 16384 + 8192, src, 8192, kqb);
        }
    }
    if (w == 0) {
        tmem_alloc(slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_launch_dependents();
    const uint32_t tm = *slot, tA = tm, tB = tm + DKP, tW = tB + 64, tE = tW + DKP;
    const uint32_t lb = tmem_lane_base(w);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok)
            ok = mbar_wait(bar, parity, status);
    };
    const uint32_t kq_s = smem_u32(kq), ef_s = smem_u32(ef);
    // a thread's part of the sums over the value heads: row i, channels part * HC ..
    float4 *accq = reinterpret_cast<float4 *>(sm + o.accq) + (size_t)part * (HC / 4) * C + i;
    float4 *acck = reinterpret_cast<float4 *>(sm + o.acck) + (size_t)part * (HC / 4) * C + i;
    for (int m = 0; m < grp; ++m) {
        const size_t r0 = (size_t)(bk * grp + m) * a.L + (size_t)c * C;
        tok = reinterpret_cast<float *>(sm + o.tok) + (m & 1) * (C * 8);
        F2 xv2 = both(0.f), ss2 = both(0.f);
        for (int s = 0; s < ns; ++s, ++gs) {
            uint8_t *sl = ef + (gs & 1) * o.slice;
            asm volatile("cp.async.wait_all;" ::: "memory"); // this thread's parts of this slice's rows (and tok)
            wait(full + (gs & 1), (gs >> 1) & 1);
            if (s == 0)
                __syncthreads(); // tok
            if (rowed) {
                F2 x[4], y[4];
                float t[8];
                pair8(sl + o.yx + 8192, yr, yc, x);
                widen8(*reinterpret_cast<const uint4 *>(sm + o.v + (gs & 1) * (C * 64) + tid * 16), y);
                const F2 be = both(tok[kBeta + yr]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    xv2 = fma2(x[e], y[e], xv2);
                    const float2 d = unpack(x[e] * be);
                    t[2 * e] = d.x;
                    t[2 * e + 1] = d.y;
                }
                if (row_in(s))
                    store8(dv + row_at(m, s), t);
            }
            if (squared) {
#pragma unroll
                for (int p = tid % 256; p < DKP * 4; p += NT == 256 ? 256 : 224) {
                    F2 x[4], y[4];
                    pair8(sl + o.s, p >> 2, p & 3, x);
                    pair8(sl + o.ds, p >> 2, p & 3, y);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        ss2 = fma2(x[u], y[u], ss2);
                }
            }
            fence_async_smem();
            tc_fence_before();
            __syncthreads();
            if (s >= 1 && s + 1 < ns) { // the other place's slice is done: its successor
                wait(done + ((gs + 1) & 1), ((gs - 1) >> 1) & 1);
                request(m, s + 1, gs + 1);
            }
            if (boss && s == 0 && m == 0)
                wait(kqb, 0);
            if (boss && ok) {
                tc_fence_after();
                if (s == 0) { // [Q; K] K^T, where the later products' E^T [Q; K] will be
#pragma unroll
                    for (int e = 0; e < 4 * NKB; ++e)
                        mma_bf16(tE, desc_sw128(kq_s + kmajor_step(e, 128), 16, 1024),
                                 desc_sw128(kq_s + 8192 + kmajor_step(e, 128), 16, 1024), idesc_bf16(128, 64, 0, 0), e > 0);
                }
                const uint32_t base = ef_s + (uint32_t)(gs & 1) * o.slice;
                for (int t = 0; t < 3; ++t) { // hi hi, hi lo, lo hi
                    const uint32_t ta = t == 2 ? 64u : 0u, tb = t == 1 ? 64u : 0u;
                    for (int e = 0; e < 2; ++e) {
                        const uint64_t yx = desc_sw128(base + o.yx + ta + e * 32, 16, 1024);
                        const uint32_t acc = (s | t | e) != 0;
                        mma_bf16(tA, yx, desc_sw128(base + o.s + tb + e * 32, 16, 1024), // S and U: tA and tB
                                 idesc_bf16(128, DKP + 64, 0, 0), acc);
                        mma_bf16(tW, desc_sw128(base + o.u + ta + e * 32, 16, 1024),
                                 desc_sw128(base + o.ds + tb + e * 32, 16, 1024), idesc_bf16(128, DKP, 0, 0), acc);
                    }
                }
                mma_commit(done + (gs & 1));
                if (s + 2 < ns) { // this place's next slice, as soon as it may come
                    wait(done + (gs & 1), (gs >> 1) & 1);
                    if (ok)
                        fetch(record(m), s + 2, gs + 2);
                }
            }
        }
        // every product of this head's slices (one commit covers those before it)
        wait(done + ((gs - 1) & 1), ((gs - 1) >> 1) & 1);
        tc_fence_after();
        if (m == 0)
            wait(kqb, 0);
        float xv = sum(xv2), ss = sum(ss2);
        xv += __shfl_xor_sync(0xffffffffu, xv, 1);
        xv += __shfl_xor_sync(0xffffffffu, xv, 2);
        if (rowed && yc == 0)
            r_xv[yr] = xv;
        ss = warp_sum(ss);
        if (lane == 0)
            r_ss[w] = ss;
        const float be = tok[kBeta + i], rk = tok[kRk + i], rq = tok[kRq + i];
        // E and F, as [E; F] rk_j (K-major) and as [E rq_i; F (-beta rk_i)]
        {
            const float ghi = tok[kGhi + i], glo = tok[kGlo + i];
            const F2 fr = both(rr < C ? rq : -be * rk), fs = both(rr < C ? a.scale : 1.f);
#pragma unroll
            for (int p = 0; p < 64 / PARTS; p += 16) {
                const int j0 = 64 / PARTS * part + p;
                float x[16], y[16];
                tmem_ld16(tB + lb + (uint32_t)j0, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    F2 d[2];
                    decay4(tok, j0 + e, ghi, glo, d);
                    const ulonglong2 rj = *reinterpret_cast<const ulonglong2 *>(tok + kRk + j0 + e);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int j = j0 + e + 2 * u;
                        float2 t = unpack(fs * pack(x[e + 2 * u], x[e + 2 * u + 1]) * d[u]);
                        t.x = (rr < C ? j <= i : j < i) ? t.x : 0.f;
                        t.y = (rr < C ? j + 1 <= i : j + 1 < i) ? t.y : 0.f;
                        const float2 s = unpack(pack(t.x, t.y) * F2{u ? rj.y : rj.x}), r = unpack(pack(t.x, t.y) * fr);
                        x[e + 2 * u] = s.x;
                        x[e + 2 * u + 1] = s.y;
                        y[e + 2 * u] = r.x;
                        y[e + 2 * u + 1] = r.y;
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    uint4 hi, lo;
                    const uint32_t to = kmajor_chunk(rr, j0 + e, 128);
                    split8(x + e, hi, lo);
                    *reinterpret_cast<uint4 *>(ef + to) = hi;
                    *reinterpret_cast<uint4 *>(ef + 16384 + to) = lo;
                    split8(y + e, hi, lo);
                    *reinterpret_cast<uint4 *>(ef + 32768 + to) = hi;
                    *reinterpret_cast<uint4 *>(ef + 49152 + to) = lo;
                }
                // P (x fr [Q; K] K^T below the diagonal), added up along the row: y[e] is
                // what lies before token j0 + e + 1, if that is not behind the row's own
                tmem_ld16(tE + lb + (uint32_t)j0, y);
                tmem_ld_wait();
                const float fp = unpack(fr).x;
                float run = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const bool below = j0 + e < i;
                    run += below ? x[e] * fp * y[e] : 0.f;
                    y[e] = below ? run : 0.f;
                }
                p_row[(j0 >> 4) * 2 * C + rr] = run;
                // over the warp's rows: halves of the values against halves of the lanes
#pragma unroll
                for (int h = 8; h > 0; h >>= 1) {
                    const bool up = lane & (2 * h);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < h) {
                            const float give = up ? y[e] : y[e + h], keep = up ? y[e + h] : y[e];
                            y[e] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * h);
                        }
                }
                y[0] += __shfl_xor_sync(0xffffffffu, y[0], 1);
                if ((lane & 1) == 0 && j0 + (lane >> 1) + 1 < C)
                    p_part[(w & 3) * C + j0 + (lane >> 1) + 1] = y[0];
            }
        }
        float x[HC]; // rows of a (rr < 64) or h
        const float eg = tok[kEG + i], fs = rr < C ? a.scale * eg : eg;
#pragma unroll
        for (int p = 0; p < HC; p += 16) {
            float t[16];
            tmem_ld16(tA + lb + (uint32_t)(part * HC + p), t);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                x[p + e] = fs * t[e];
        }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        if (boss && ok) {
            tc_fence_after();
            for (int t = 0; t < 2; ++t)
                for (int s = 0; s < 4; ++s)
                    mma_bf16(tA, desc_sw128(ef_s + (uint32_t)t * 16384u + (uint32_t)s * 32u, 16, 1024),
                             desc_sw128(kq_s + 8192u + (uint32_t)s * 2048u, 16384, 1024), idesc_bf16(128, DKP, 0, 1),
                             (t | s) != 0);
            for (int s = 0; s < 8; ++s) // rows 0 - 63 from the hi terms, 64 - 127 from the lo terms
                mma_bf16(tE, desc_sw128(ef_s + 32768u + (uint32_t)s * 2048u, 16384, 1024),
                         desc_sw128(kq_s + (uint32_t)s * 2048u, 16384, 1024), idesc_bf16(128, DKP, 1, 1), s != 0);
            mma_commit(mm);
        }
        if (w == ADDER) { // the pairs across each token, two tokens a lane
            float c2[2], b2[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                c2[e] = 0.f;
                const int t = 2 * lane + e;
                if (t > 0)
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        c2[e] += p_part[p * C + t];
            }
#pragma unroll
            for (int p = 0; p < 3; ++p) { // whole blocks of columns before a token's own
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    b2[e] += p_row[p * 2 * C + 2 * lane + e] + p_row[p * 2 * C + C + 2 * lane + e];
                const float from1 = lanes_after(b2[0] + b2[1], lane) + b2[1];
                if ((2 * lane - 1) >> 4 == p + 1)
                    c2[0] += from1 + b2[0];
                if ((2 * lane) >> 4 == p + 1)
                    c2[1] += from1;
            }
            r_c[2 * lane] = c2[0];
            r_c[2 * lane + 1] = c2[1];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(mm);
        }
        // what is read of S (rows of a meet Q, rows of h meet K), and W
        auto kq_row = [&](int row, int p, F2 (&u)[4]) {
            widen8(*reinterpret_cast<const uint4 *>(kq + kmajor_chunk(row, part * HC + p, 128)), u);
        };
        {
            F2 read2 = both(0.f);
#pragma unroll
            for (int p = 0; p < HC; p += 8) {
                F2 u[4];
                kq_row(rr, p, u);
#pragma unroll
                for (int m2 = 0; m2 < 4; ++m2)
                    read2 = fma2(u[m2], pack(x[p + 2 * m2], x[p + 2 * m2 + 1]), read2);
            }
            (rr < C ? r_qa : r_k0)[part * C + i] = sum(read2) * (rr < C ? rq : rk);
        }
        if (rr < C) {
            F2 w2 = both(0.f);
#pragma unroll
            for (int p = 0; p < HC; p += 16) {
                float t[16];
                tmem_ld16(tW + lb + (uint32_t)(part * HC + p), t);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    F2 u[4];
                    kq_row(C + i, p + e, u);
#pragma unroll
                    for (int m2 = 0; m2 < 4; ++m2)
                        w2 = fma2(u[m2], pack(t[e + 2 * m2], t[e + 2 * m2 + 1]), w2);
                }
            }
            r_w[part * C + i] = sum(w2) * rk * tok[kEC + i];
        }
        wait(mm, (uint32_t)m & 1);
        tc_fence_after();
        if (m + 1 < grp) // (the E and F tiles have been read; the sums lie in their place only if grp is 1)
            begin(m + 1);
        {
            F2 dot2 = both(0.f); // k.h, this part's channels
#pragma unroll
            for (int p = 0; p < HC; p += 16) {
                float t[16];
                tmem_ld16(tA + lb + (uint32_t)(part * HC + p), t);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 8) {
                    F2 u[4] = {};
                    if (rr >= C)
                        kq_row(rr, p + e, u);
#pragma unroll
                    for (int m2 = 0; m2 < 8; m2 += 2) {
                        float *xe = x + p + e + m2;
                        const F2 r = pack(xe[0], xe[1]) + pack(t[e + m2], t[e + m2 + 1]);
                        if (rr >= C)
                            dot2 = fma2(u[m2 / 2], r, dot2);
                        const float2 d = unpack(r);
                        xe[0] = d.x;
                        xe[1] = d.y;
                    }
                }
            }
            if (rr >= C)
                r_kh[part * C + i] = sum(dot2) * rk;
        }
        if (rr >= C) { // -beta h, and w's part of the lo terms
#pragma unroll
            for (int p = 0; p < HC; p += 16) {
                float t[16];
                tmem_ld16(tE + lb + (uint32_t)(part * HC + p), t);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 d = unpack(fma2(both(-be), pack(x[p + e], x[p + e + 1]), pack(t[e], t[e + 1])));
                    x[p + e] = d.x;
                    x[p + e + 1] = d.y;
                }
            }
        } else {
#pragma unroll
            for (int p = 0; p < HC; p += 4) {
                float4 t = make_float4(x[p], x[p + 1], x[p + 2], x[p + 3]);
                if (m > 0) {
                    const float4 s = accq[(p / 4) * C];
                    t = make_float4(t.x + s.x, t.y + s.y, t.z + s.z, t.w + s.w);
                }
                accq[(p / 4) * C] = t;
            }
            const F2 ec = both(tok[kEC + i]);
#pragma unroll
            for (int p = 0; p < HC; p += 16) {
                float t[16], u1[16];
                tmem_ld16(tW + lb + (uint32_t)(part * HC + p), t);
                tmem_ld16(tE + lb + (uint32_t)(part * HC + p), u1);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 d = unpack(fma2(ec, pack(t[e], t[e + 1]), pack(u1[e], u1[e + 1])));
                    t[e] = d.x;
                    t[e + 1] = d.y;
                }
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    float4 r = make_float4(t[e], t[e + 1], t[e + 2], t[e + 3]);
                    if (m > 0) {
                        const float4 s = acck[((p + e) / 4) * C];
                        r = make_float4(r.x + s.x, r.y + s.y, r.z + s.z, r.w + s.w);
                    }
                    acck[((p + e) / 4) * C] = r;
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (rr >= C) { // the row's other thread has left its part
#pragma unroll
            for (int p = 0; p < HC; p += 4) {
                const float4 s = acck[(p / 4) * C];
                acck[(p / 4) * C] = make_float4(s.x + x[p], s.y + x[p + 1], s.z + x[p + 2], s.w + x[p + 3]);
            }
        }
        if (w == BOSS) { // dg and dbeta, two tokens a lane
            float R[2], W[2], out[2], z = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = 2 * lane + e;
                float qa = 0.f, k0 = 0.f, kh = 0.f;
                W[e] = 0.f;
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    qa += r_qa[p * C + t];
                    k0 += r_k0[p * C + t];
                    kh += r_kh[p * C + t];
                    W[e] += r_w[p * C + t];
                }
                R[e] = qa - tok[kBeta + t] * k0;
                if (t < n)
                    io<bf>::store(dbeta + r0 + t, r_xv[t] - kh);
            }
#pragma unroll
            for (int e = 0; e < NT / 32; ++e)
                z += r_ss[e];
            gated_decay_grads(tok[kEG + C - 1] * z, R, W, r_c + 2 * lane, lane, out);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (2 * lane + e < n)
                    io<bf>::store(dg + r0 + 2 * lane + e, out[e]);
        }
        for (int e = n * a.d_v / 8 + tid; e < rows * a.d_v / 8; e += NT)
            reinterpret_cast<uint4 *>(dv + r0 * a.d_v)[e] = make_uint4(0, 0, 0, 0);
        for (int t = n + tid; t < rows; t += NT) {
            io<bf>::store(dg + r0 + t, 0.f);
            io<bf>::store(dbeta + r0 + t, 0.f);
        }
    }
    // dq (the threads of rows 64 ..) and dk: back through the unit length
    __syncthreads(); // dg has been read off; red is free
    {
        const float4 *acc = rr < C ? acck : accq;
        const float r = i >= n ? 0.f : tok[(rr < C ? kRk : kRq) + i];
        float dot = 0.f;
#pragma unroll
        for (int p = 0; p < HC; p += 8) {
            float u[8];
            widen8(*reinterpret_cast<const uint4 *>(kq + kmajor_chunk(rr ^ 64, part * HC + p, 128)), u);
            const float4 s = acc[(p / 4) * C], t = acc[(p / 4 + 1) * C];
            dot += u[0] * s.x + u[1] * s.y + u[2] * s.z + u[3] * s.w + u[4] * t.x + u[5] * t.y + u[6] * t.z + u[7] * t.w;
        }
        red[part * 2 * C + rr] = dot * r;
        __syncthreads();
        float f = 0.f;
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
            f += red[p * 2 * C + rr];
        f = a.l2norm ? f * r : 0.f;
        // through shared memory (rows of DKP + 8), so that a row leaves by neighbouring lanes
        uint8_t *place = ef + 2 * NKB * 16384;
        constexpr int PITCH = DKP * 2 + 16;
#pragma unroll
        for (int p = 0; p < HC; p += 8) {
            float u[8];
            widen8(*reinterpret_cast<const uint4 *>(kq + kmajor_chunk(rr ^ 64, part * HC + p, 128)), u);
            const float4 s = acc[(p / 4) * C], t = acc[(p / 4 + 1) * C];
            const float g8[8] = {s.x, s.y, s.z, s.w, t.x, t.y, t.z, t.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                u[e] = i < n ? r * (g8[e] - u[e] * f) : 0.f;
            store8(reinterpret_cast<bf *>(place + rr * PITCH) + part * HC + p, u);
        }
        __syncthreads();
        const int chunks = a.d_k / 8;
        for (int e = tid; e < 2 * rows * chunks; e += NT) {
            const int row = e / chunks, ch = e - row * chunks, to = row < rows ? row : row - rows; // dk's rows, then dq's
            *reinterpret_cast<uint4 *>((row < rows ? dk : dq) + krow + (size_t)to * a.d_k + 8 * ch) =
                *reinterpret_cast<const uint4 *>(place + (row < rows ? row : C + to) * PITCH + 16 * ch);
        }
    }
    if (!ok && boss) // a wait gave up: let what was asked for land first
        for (int e = 0; e < 2; ++e)
            (void)mbar_wait(full + e, 0, status);
    tc_fence_before();
    __syncthreads();
    if (w == 0)
        tmem_dealloc(tm, kCols);
}

template <int NKB>
cudaError_t launch(const GatedArgs &a, const void *v, const void *dy, void *dq, void *dk, void *dv, void *dg,
                   void *dbeta, const void *ws, const GatedRecord &rec, unsigned *status, cudaStream_t st) {
    auto *kern = gated_tc_grad_kernel<NKB>;
    const uint32_t smem = grad_smem(NKB, a.H == a.Hk).bytes;
    static std::atomic<uint64_t> allowed{0};
    const cudaError_t e = allow_smem(kern, allowed);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(kern, dim3(rec.nch, a.B * a.Hk), dim3(128 * parts_of(NKB)), smem, st, a, (const bf *)v,
                      (const bf *)dy, (bf *)dq, (bf *)dk, (bf *)dv, (bf *)dg, (bf *)dbeta, (const uint8_t *)ws, rec,
                      status);
}

} // namespace

cudaError_t gated_tc_grad(const GatedArgs &a, const void *v, const void *dy, void *dq, void *dk, void *dv, void *dg,
                          void *dbeta, const void *ws, cudaStream_t st) {
    unsigned *status = nullptr;
    cudaError_t e = status_word(&status);
    if (e != cudaSuccess)
        return e;
    const GatedRecord rec = gated_backward_record(a.L, a.d_k, a.d_v);
    return rec.nkb == 1 ? launch<1>(a, v, dy, dq, dk, dv, dg, dbeta, ws, rec, status, st)
                        : launch<2>(a, v, dy, dq, dk, dv, dg, dbeta, ws, rec, status, st);
}

} // namespace fw
