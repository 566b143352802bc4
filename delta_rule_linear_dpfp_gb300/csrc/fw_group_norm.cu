// fw_group_norm.cu -- the heads' answers on their way to the output map: each
// head's channels normalised for each token (a group norm over channels-last
// rows, one group per head), affine, then an activation, or times the
// activation of a gate.
//
//   n = (x - mean) r,  r = (var + eps)^-1/2 over the d channels of a head,
//   z = n gamma + beta,  out = act(z), or z act(gate).
// Backward, with dz = dout act'(z) (or dout act(gate)) and dn = dz gamma:
//   dx = r (dn - mean(dn) - n mean(dn n)),  dgate = dout z act'(gate),
//   dgamma = sum dz n,  dbeta = sum dz  over every token.
//
// x is head-major [B, H, L, d] (the layout of the attention calls), gate and
// out token-major [B, L, H d] (the output map's input), so the transpose
// costs nothing.  Bound by the bytes: each tensor is read or written once.
//
// Mapping: LPR lanes own a row of d channels, 8 at a time (16 bytes of bf16);
// the statistics are two passes over registers (mean, then the squares of the
// differences) and shuffles among the row's lanes.  A CTA stays on one head,
// so gamma and beta sit in registers and so do the backward's dgamma and
// dbeta until the end: one partial row per CTA, added by a second kernel in a
// fixed order (no atomics).  Two rows of a lane group are in flight at a time,
// and the activations use the fast exponential and division (2^-21 of the
// value), or the arithmetic would cost as much as the bytes.
#include "fw_common.cuh"
#include "fw_gated.h"

#include <algorithm>

namespace fw {

namespace {

constexpr int kT = 256;
enum { kNone = 0, kRelu = 1, kSilu = 2, kGelu = 3 };

// x sigmoid(x) needs no guard: far below 0 the exponential is infinite and the
// quotient 0.
FW_DEV float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// (A variant of the kernels for each: as a branch per element it made them
// bound by instructions, 36 an element and 49 us where the bytes take 30.)
template <int ACT> FW_DEV float act(float x) {
    if (ACT == kRelu)
        return x > 0.f ? x : x != x ? x : 0.f; // NaN stays NaN
    if (ACT == kSilu)
        return x * sigmoid(x);
    if (ACT == kGelu)
        return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
    return x;
}
// act(x) and its derivative.
template <int ACT> FW_DEV void act_grad(float x, float &f, float &df) {
    if (ACT == kRelu) {
        f = act<kRelu>(x);
        df = x > 0.f ? 1.f : 0.f;
    } else if (ACT == kSilu) {
        const float s = sigmoid(x);
        f = x * s;
        df = s * fmaf(x, 1.f - s, 1.f);
    } else if (ACT == kGelu) {
        const float p = 0.5f * (1.f + erff(x * 0.70710678118654752f));
        f = x * p;
        df = fmaf(x * 0.39894228040143268f, __expf(-0.5f * x * x), p);
    } else {
        f = x;
        df = 1.f;
    }
}

template <int LPR> FW_DEV float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// n = (x - mean) r of a row held 8 channels a lane (lanes at or past d hold
// zeros and stay zero); returns r.
template <int LPR> FW_DEV float normalise(float (&x)[8], bool on, float inv_d, float eps) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s += x[e];
    const float mean = row_sum<LPR>(s) * inv_d;
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = on ? x[e] - mean : 0.f;
        ss = fmaf(x[e], x[e], ss);
    }
    const float r = 1.f / sqrtf(fmaf(row_sum<LPR>(ss), inv_d, eps));
#pragma unroll
    for (int e = 0; e < 8; ++e)
        x[e] *= r;
    return r;
}

// 8 channels as they were loaded.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 u;
    FW_DEV void load(const __nv_bfloat16 *p, bool here) {
        u = here ? __ldcs(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
    }
    FW_DEV void widen(float (&o)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[2 * i] = __uint_as_float(w[i] << 16);
            o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    FW_DEV void load(const float *p, bool here) {
        a = here ? __ldcs(reinterpret_cast<const float4 *>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
        b = here ? __ldcs(reinterpret_cast<const float4 *>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    FW_DEV void widen(float (&o)[8]) const {
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
        o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
    }
};

constexpr int U = 2; // rows in flight per lane group

// Where row `row` of (b, l) starts: in x (head-major) and in out (token-major).
struct Rows {
    int64_t x, out;
};
FW_DEV Rows rows_of(const NormArgs &a, unsigned row, int h, int c0) {
    const unsigned b = row / (unsigned)a.L, l = row - b * (unsigned)a.L;
    return {(((int64_t)b * a.H + h) * a.L + l) * a.d + c0, ((int64_t)row * a.H + h) * a.d + c0};
}

template <int LPR, int ACT, bool GATE, typename T>
__global__ void __launch_bounds__(kT)
    group_norm_kernel(NormArgs a, const T *__restrict__ x, const T *__restrict__ gate, const float *__restrict__ gamma,
                      const float *__restrict__ beta, T *__restrict__ out) {
    constexpr unsigned RPC = kT / LPR; // rows per CTA and step
    const int c0 = 8 * (threadIdx.x % LPR), h = blockIdx.y;
    const unsigned slot = threadIdx.x / LPR, rows = (unsigned)(a.B * (int64_t)a.L), step = gridDim.x * RPC;
    const bool on = c0 < a.d;
    const float inv_d = 1.f / (float)a.d;
    griddep_launch_dependents();
    griddep_wait();
    x = after_wait(x);
    gate = after_wait(gate);
    float ga[8] = {}, be[8] = {};
    if (on) {
        load8(gamma + h * a.d + c0, ga);
        load8(beta + h * a.d + c0, be);
    }
    for (unsigned base = blockIdx.x * RPC; base < rows; base += U * step) {
        Raw8<T> rx[U], rg[U];
        Rows at[U];
        bool here[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned row = base + u * step + slot;
            here[u] = on && row < rows;
            at[u] = rows_of(a, here[u] ? row : 0, h, here[u] ? c0 : 0);
            rx[u].load(x + at[u].x, here[u]);
            if (GATE)
                rg[u].load(gate + at[u].out, here[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8], z[8];
            rx[u].widen(v);
            normalise<LPR>(v, here[u], inv_d, a.eps);
            if (GATE)
                rg[u].widen(z);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = fmaf(v[e], ga[e], be[e]);
                v[e] = GATE ? y * act<ACT>(z[e]) : act<ACT>(y);
            }
            if (here[u])
                store8(out + at[u].out, v);
        }
    }
}

template <int LPR, int ACT, bool GATE, typename T>
__global__ void __launch_bounds__(kT)
    group_norm_backward_kernel(NormArgs a, const T *__restrict__ x, const T *__restrict__ gate,
                               const float *__restrict__ gamma, const float *__restrict__ beta,
                               const T *__restrict__ dout, T *__restrict__ dx, T *__restrict__ dgate,
                               float *__restrict__ part) {
    constexpr unsigned RPC = kT / LPR;
    __shared__ float red[2][RPC][8 * LPR];
    const int c0 = 8 * (threadIdx.x % LPR), h = blockIdx.y;
    const unsigned slot = threadIdx.x / LPR, rows = (unsigned)(a.B * (int64_t)a.L), step = gridDim.x * RPC;
    const bool on = c0 < a.d;
    const float inv_d = 1.f / (float)a.d;
    griddep_launch_dependents();
    griddep_wait();
    x = after_wait(x);
    gate = after_wait(gate);
    dout = after_wait(dout);
    float ga[8] = {}, be[8] = {}, dga[8] = {}, dbe[8] = {};
    if (on) {
        load8(gamma + h * a.d + c0, ga);
        load8(beta + h * a.d + c0, be);
    }
    for (unsigned base = blockIdx.x * RPC; base < rows; base += U * step) {
        Raw8<T> rx[U], rg[U], rd[U];
        Rows at[U];
        bool here[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned row = base + u * step + slot;
            here[u] = on && row < rows;
            at[u] = rows_of(a, here[u] ? row : 0, h, here[u] ? c0 : 0);
            rx[u].load(x + at[u].x, here[u]);
            rd[u].load(dout + at[u].out, here[u]);
            if (GATE)
                rg[u].load(gate + at[u].out, here[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float n[8], t[8], dz[8];
            rx[u].widen(n);
            rd[u].widen(dz);
            const float r = normalise<LPR>(n, here[u], inv_d, a.eps);
            if (GATE)
                rg[u].widen(t);
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = fmaf(n[e], ga[e], be[e]);
                float f, df;
                act_grad<ACT>(GATE ? t[e] : z, f, df);
                if (GATE) {
                    t[e] = dz[e] * z * df;
                    dz[e] *= f;
                } else {
                    dz[e] *= df;
                }
                dga[e] = fmaf(dz[e], n[e], dga[e]);
                dbe[e] += dz[e];
                dz[e] *= ga[e];
                s1 += dz[e];
                s2 = fmaf(dz[e], n[e], s2);
            }
            s1 = row_sum<LPR>(s1) * inv_d;
            s2 = row_sum<LPR>(s2) * inv_d;
            if (here[u]) {
                if (GATE)
                    store8(dgate + at[u].out, t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dz[e] = r * (dz[e] - s1 - n[e] * s2);
                store8(dx + at[u].x, dz);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        red[0][slot][c0 + e] = dga[e];
        red[1][slot][c0 + e] = dbe[e];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * a.d; e += kT) {
        const int m = e / a.d, ch = e % a.d;
        float s = 0.f;
        for (unsigned p = 0; p < RPC; ++p)
            s += red[m][p][ch];
        part[(((size_t)m * gridDim.x + blockIdx.x) * gridDim.y + h) * a.d + ch] = s;
    }
}

// dgamma, dbeta: the CTAs' partial rows in order.
__global__ void __launch_bounds__(kT)
    group_norm_params_kernel(const float *__restrict__ part, float *__restrict__ dgamma, float *__restrict__ dbeta,
                             int nparts, int ch) {
    griddep_launch_dependents();
    griddep_wait();
    part = after_wait(part);
    const int e = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    __shared__ float red[kT / 32][33];
    float s = 0.f;
    if (e < 2 * ch)
        for (int p = w; p < nparts; p += kT / 32)
            s += __ldcg(part + ((size_t)(e / ch) * nparts + p) * ch + e % ch);
    red[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w == 0 && e < 2 * ch) {
        s = 0.f;
#pragma unroll
        for (int p = 0; p < kT / 32; ++p)
            s += red[p][threadIdx.x];
        (e < ch ? dgamma : dbeta)[e % ch] = s;
    }
}

// CTAs per head: enough to fill the SMs (kCtas in all), no more than the rows
// give.
constexpr int kCtas = 152 * 8, kBackwardCtas = 152 * 4;
int parts_of(int B, int H, int L, int d, int ctas) {
    int lpr = 1;
    while (8 * lpr < d)
        lpr *= 2;
    const int64_t steps = ((int64_t)B * L + kT / lpr - 1) / (kT / lpr);
    return (int)std::max<int64_t>(1, std::min<int64_t>(steps, (ctas + H - 1) / H));
}

struct Launch {
    const NormArgs &a;
    const void *x, *gate;
    const float *gamma, *beta;
    void *out;
    const void *dout;
    void *dx, *dgate;
    float *part;
    cudaStream_t st;

    template <int LPR, int ACT, bool GATE, typename T> cudaError_t run() const {
        if (dout)
            return launch_pdl(group_norm_backward_kernel<LPR, ACT, GATE, T>,
                              dim3(parts_of(a.B, a.H, a.L, a.d, kBackwardCtas), a.H), dim3(kT), 0, st, a, (const T *)x,
                              (const T *)gate, gamma, beta, (const T *)dout, (T *)dx, (T *)dgate, part);
        return launch_pdl(group_norm_kernel<LPR, ACT, GATE, T>, dim3(parts_of(a.B, a.H, a.L, a.d, kCtas), a.H), dim3(kT), 0, st, a, (const T *)x,
                          (const T *)gate, gamma, beta, (T *)out);
    }
    template <int LPR, int ACT, bool GATE> cudaError_t dtype(int bf16) const {
        return bf16 ? run<LPR, ACT, GATE, __nv_bfloat16>() : run<LPR, ACT, GATE, float>();
    }
    template <int LPR, int ACT> cudaError_t gated(int bf16) const {
        return gate ? dtype<LPR, ACT, true>(bf16) : dtype<LPR, ACT, false>(bf16);
    }
    template <int LPR> cudaError_t width(int bf16) const {
        switch (a.act) {
        case kRelu: return gated<LPR, kRelu>(bf16);
        case kSilu: return gated<LPR, kSilu>(bf16);
        case kGelu: return gated<LPR, kGelu>(bf16);
        default: return gated<LPR, kNone>(bf16);
        }
    }
    cudaError_t go(int bf16) const {
        if (a.d <= 8) return width<1>(bf16);
        if (a.d <= 16) return width<2>(bf16);
        if (a.d <= 32) return width<4>(bf16);
        if (a.d <= 64) return width<8>(bf16);
        if (a.d <= 128) return width<16>(bf16);
        return width<32>(bf16);
    }
};

} // namespace

size_t group_norm_backward_workspace_bytes(int B, int H, int L, int d) {
    return sizeof(float) * 2 * (size_t)parts_of(B, H, L, d, kBackwardCtas) * H * d;
}

cudaError_t launch_group_norm(const NormArgs &a, const void *x, const void *gate, const float *gamma,
                              const float *beta, void *out, int bf16, cudaStream_t st) {
    return Launch{a, x, gate, gamma, beta, out, nullptr, nullptr, nullptr, nullptr, st}.go(bf16);
}

cudaError_t launch_group_norm_backward(const NormArgs &a, const void *x, const void *gate, const float *gamma,
                                       const float *beta, const void *dout, void *dx, void *dgate, float *dgamma,
                                       float *dbeta, void *workspace, int bf16, cudaStream_t st) {
    float *part = static_cast<float *>(workspace);
    cudaError_t e = Launch{a, x, gate, gamma, beta, nullptr, dout, dx, dgate, part, st}.go(bf16);
    if (e != cudaSuccess)
        return e;
    const int ch = a.H * a.d;
    return launch_pdl(group_norm_params_kernel, dim3((2 * ch + 31) / 32), dim3(kT), 0, st, (const float *)part, dgamma,
                      dbeta, parts_of(a.B, a.H, a.L, a.d, kBackwardCtas), ch);
}

} // namespace fw
