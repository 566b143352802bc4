// fw_gated_decode.cu -- the gated delta rule for one token per (batch, value
// head) against a persistent fp32 state W [B, H, d_v, d_k], updated in place.
//
// For each row r of W, with a = exp(g) and unit keys and queries k, q:
//   u_r = beta (v_r - a W[r].k),  W[r] <- a W[r] + u_r k^T,
//   y_r = scale (a W[r].q + u_r (k.q)),
// so both dot products come from one read of the row: every element of W is
// read once and written once, and the step is bound by those bytes.
//
// Mapping: d_k / 4 lanes own a row (16 bytes a lane), a warp 32 / (d_k / 4)
// rows at a time and kRowSets such sets, all of them requested before the
// first is used.  The key and the query sit in the same lanes (4 channels
// each), so their lengths, k.q and the row's two dot products are shuffles
// among the row's lanes: no shared memory and no barrier.
#include "fw_common.cuh"
#include "fw_gated.h"
#include "fw_gated_tiles.cuh"

namespace fw {

namespace {

constexpr int kWarps = 8;
// Row sets a warp and CTAs an SM: enough bytes in flight, and registers for
// them (268 MB of state: 86 us; 8 sets 99, with three CTAs 89; six CTAs 99).
constexpr int kRowSets = 4, kCtasPerSm = 4;

FW_DEV float4 load4(const float *p) { return __ldcg(reinterpret_cast<const float4 *>(p)); }
FW_DEV float4 load4(const __nv_bfloat16 *p) {
    const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(p));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}
FW_DEV float dot4(float4 a, float4 b) { return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, a.x * b.x))); }

// The sum over the G lanes of a row.
template <int G> FW_DEV float row_sum(float x) {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int DK, int SETS, typename T>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm)
    gated_decode_kernel(GatedArgs a, const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
                        const T *__restrict__ g, const T *__restrict__ beta, float *__restrict__ W,
                        T *__restrict__ y) {
    constexpr int G = DK / 4, RPW = 32 / G, ROWS = kWarps * SETS * RPW;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, gl = lane % G;
    const int nrb = (a.d_v + ROWS - 1) / ROWS;
    const int64_t bh = blockIdx.x / nrb;
    const int r0 = (int)(blockIdx.x % nrb) * ROWS;
    const int64_t kh = bh / a.H * a.Hk + bh % a.H / (a.H / a.Hk);
    griddep_launch_dependents();
    if (threadIdx.x == 0) // the rows on their way to L2 while the preceding kernel ends
        l2_prefetch(W + (bh * a.d_v + r0) * DK, (uint32_t)(min(ROWS, a.d_v - r0) * DK * 4));
    griddep_wait();
    W = after_wait(W);
    float4 x[SETS];
    auto row_of = [&](int s) { return r0 + (s * kWarps + w) * RPW + lane / G; };
#pragma unroll
    for (int s = 0; s < SETS; ++s)
        x[s] = row_of(s) < a.d_v ? __ldcs(reinterpret_cast<const float4 *>(W + (bh * a.d_v + row_of(s)) * DK) + gl)
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 kk = load4(after_wait(k) + kh * DK + 4 * gl), qq = load4(after_wait(q) + kh * DK + 4 * gl);
    const float be = io<T>::load(after_wait(beta) + bh), gg = io<T>::load(after_wait(g) + bh);
    const float al = expf(gg < kGMin ? kGMin : gg);
    float vr[SETS];
#pragma unroll
    for (int s = 0; s < SETS; ++s)
        vr[s] = row_of(s) < a.d_v ? io<T>::load(after_wait(v) + bh * a.d_v + row_of(s)) : 0.f;
    float sc = a.scale;
    if (a.l2norm) { // a row of zeros has length 0 and stays zero
        const float nk = row_sum<G>(dot4(kk, kk)) + a.eps, nq = row_sum<G>(dot4(qq, qq)) + a.eps;
        const float rk = nk > 0.f ? 1.f / sqrtf(nk) : nk;
        sc *= nq > 0.f ? 1.f / sqrtf(nq) : nq;
        kk = make_float4(kk.x * rk, kk.y * rk, kk.z * rk, kk.w * rk);
    }
    const float kq = row_sum<G>(dot4(kk, qq));
#pragma unroll
    for (int s = 0; s < SETS; ++s) {
        float4 r = make_float4(al * x[s].x, al * x[s].y, al * x[s].z, al * x[s].w);
        const float sk = row_sum<G>(dot4(r, kk)), sq = row_sum<G>(dot4(r, qq));
        const float u = be * (vr[s] - sk);
        if (row_of(s) < a.d_v) {
            r = make_float4(fmaf(u, kk.x, r.x), fmaf(u, kk.y, r.y), fmaf(u, kk.z, r.z), fmaf(u, kk.w, r.w));
            __stcs(reinterpret_cast<float4 *>(W + (bh * a.d_v + row_of(s)) * DK) + gl, r);
            if (gl == 0)
                io<T>::store(y + bh * a.d_v + row_of(s), sc * fmaf(u, kq, sq));
        }
    }
}

template <int DK, typename T>
cudaError_t launch_t(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g, const void *beta,
                     float *W, void *y, cudaStream_t st) {
    constexpr int SETS = kRowSets, ROWS = kWarps * SETS * (32 / (DK / 4));
    const int64_t n = (int64_t)a.B * a.H * ((a.d_v + ROWS - 1) / ROWS);
    return launch_pdl(gated_decode_kernel<DK, SETS, T>, dim3((unsigned)n), dim3(32 * kWarps), 0, st, a, (const T *)q,
                      (const T *)k, (const T *)v, (const T *)g, (const T *)beta, W, (T *)y);
}

template <typename T>
cudaError_t launch_dk(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g, const void *beta,
                      float *W, void *y, cudaStream_t st) {
    switch (a.d_k) {
    case 16: return launch_t<16, T>(a, q, k, v, g, beta, W, y, st);
    case 32: return launch_t<32, T>(a, q, k, v, g, beta, W, y, st);
    case 64: return launch_t<64, T>(a, q, k, v, g, beta, W, y, st);
    case 128: return launch_t<128, T>(a, q, k, v, g, beta, W, y, st);
    default: return cudaErrorInvalidValue;
    }
}

} // namespace

cudaError_t launch_gated_decode(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                                const void *beta, float *W, void *y, int bf16, cudaStream_t st) {
    return bf16 ? launch_dk<__nv_bfloat16>(a, q, k, v, g, beta, W, y, st)
                : launch_dk<float>(a, q, k, v, g, beta, W, y, st);
}

} // namespace fw
