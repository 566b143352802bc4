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
// differences) and shuffles among the row's lanes.  A warp holds kFly rows
// per lane group in flight.  In the backward a CTA stays on one head, so a
// lane's channels never change and dgamma, dbeta are sums in its registers
// until the end: one partial row per CTA, added by a second kernel in a fixed
// order (no atomics).
#include "fw_common.cuh"
#include "fw_gated.h"

#include <algorithm>

namespace fw {

namespace {

constexpr int kT = 256;
enum { kNone = 0, kRelu = 1, kSilu = 2, kGelu = 3 };

FW_DEV float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// (The activation is one uniform branch of a kernel that waits for memory, so
// it is an argument and not a variant.)
FW_DEV float act(int kind, float x) {
    if (kind == kRelu)
        return x > 0.f ? x : x != x ? x : 0.f; // NaN stays NaN
    if (kind == kSilu)
        return x * sigmoid(x);
    if (kind == kGelu)
        return 0.5f * x * (1.f + erff(x * 0.70710678118654752f));
    return x;
}
// act(x) and its derivative.
FW_DEV void act_grad(int kind, float x, float &f, float &df) {
    if (kind == kRelu) {
        f = act(kRelu, x);
        df = x > 0.f ? 1.f : 0.f;
    } else if (kind == kSilu) {
        const float s = sigmoid(x);
        f = x * s;
        df = s * fmaf(x, 1.f - s, 1.f);
    } else if (kind == kGelu) {
        const float p = 0.5f * (1.f + erff(x * 0.70710678118654752f));
        f = x * p;
        df = fmaf(x * 0.39894228040143268f, expf(-0.5f * x * x), p);
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

template <int LPR, bool GATE, typename T>
__global__ void __launch_bounds__(kT)
    group_norm_kernel(NormArgs a, const T *__restrict__ x, const T *__restrict__ gate, const float *__restrict__ gamma,
                      const float *__restrict__ beta, T *__restrict__ out) {
    constexpr int RPC = kT / LPR; // rows per CTA and step
    const int c0 = 8 * (threadIdx.x % LPR), slot = threadIdx.x / LPR;
    const bool on = c0 < a.d;
    const float inv_d = 1.f / (float)a.d;
    const int64_t rows = (int64_t)a.B * a.H * a.L;
    griddep_launch_dependents();
    griddep_wait();
    x = after_wait(x);
    gate = after_wait(gate);
    for (int64_t row = (int64_t)blockIdx.x * RPC + slot; row - slot < rows; row += (int64_t)gridDim.x * RPC) {
        const bool here = on && row < rows;
        const int64_t bh = row / a.L, l = row - bh * a.L, b = bh / a.H;
        const int h = (int)(bh - b * a.H);
        const int64_t at = ((b * a.L + l) * a.H + h) * a.d + c0;
        float v[8] = {}, z[8] = {}, ga[8], be[8];
        if (here) {
            load8(x + row * a.d + c0, v);
            if (GATE)
                load8(gate + at, z);
        }
        normalise<LPR>(v, here, inv_d, a.eps);
        if (here) {
            load8(gamma + h * a.d + c0, ga);
            load8(beta + h * a.d + c0, be);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float y = fmaf(v[e], ga[e], be[e]);
                v[e] = GATE ? y * act(a.act, z[e]) : act(a.act, y);
            }
            store8(out + at, v);
        }
    }
}

template <int LPR, bool GATE, typename T>
__global__ void __launch_bounds__(kT)
    group_norm_backward_kernel(NormArgs a, const T *__restrict__ x, const T *__restrict__ gate,
                               const float *__restrict__ gamma, const float *__restrict__ beta,
                               const T *__restrict__ dout, T *__restrict__ dx, T *__restrict__ dgate,
                               float *__restrict__ part) {
    constexpr int RPC = kT / LPR;
    __shared__ float red[2][RPC][8 * LPR];
    const int c0 = 8 * (threadIdx.x % LPR), slot = threadIdx.x / LPR, h = blockIdx.y;
    const bool on = c0 < a.d;
    const float inv_d = 1.f / (float)a.d;
    const int64_t rows = (int64_t)a.B * a.L;
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
    for (int64_t row = (int64_t)blockIdx.x * RPC + slot; row - slot < rows; row += (int64_t)gridDim.x * RPC) {
        const bool here = on && row < rows;
        const int64_t b = row / a.L, l = row - b * a.L;
        const int64_t from = ((b * a.H + h) * a.L + l) * a.d + c0, at = (row * a.H + h) * a.d + c0;
        float n[8] = {}, t[8] = {}, dz[8] = {};
        if (here) {
            load8(x + from, n);
            load8(dout + at, dz);
            if (GATE)
                load8(gate + at, t);
        }
        const float r = normalise<LPR>(n, here, inv_d, a.eps);
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float z = fmaf(n[e], ga[e], be[e]);
            float f, df;
            act_grad(a.act, GATE ? t[e] : z, f, df);
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
        if (here) {
            if (GATE)
                store8(dgate + at, t);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                dz[e] = r * (dz[e] - s1 - n[e] * s2);
            store8(dx + from, dz);
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
        for (int p = 0; p < RPC; ++p)
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

// CTAs per head of the backward: enough to fill the SMs, no more than the
// rows give.
constexpr int kBackwardCtas = 608; // 4 CTAs on each of 152 SMs

int backward_parts(int B, int H, int L, int d) {
    int lpr = 1;
    while (8 * lpr < d)
        lpr *= 2;
    const int64_t steps = ((int64_t)B * L + kT / lpr - 1) / (kT / lpr);
    return (int)std::max<int64_t>(1, std::min<int64_t>(steps, (kBackwardCtas + H - 1) / H));
}

struct Launch {
    const NormArgs &a;
    const void *x, *gate;
    const float *gamma, *beta;
    void *out;
    const void *dout;
    void *dx, *dgate;
    float *part;
    int num_sms;
    cudaStream_t st;

    template <int LPR, bool GATE, typename T> cudaError_t run() const {
        if (dout)
            return launch_pdl(group_norm_backward_kernel<LPR, GATE, T>,
                              dim3(backward_parts(a.B, a.H, a.L, a.d), a.H), dim3(kT), 0, st, a, (const T *)x,
                              (const T *)gate, gamma, beta, (const T *)dout, (T *)dx, (T *)dgate, part);
        const int64_t rows = (int64_t)a.B * a.H * a.L, per = kT / LPR;
        const unsigned grid = (unsigned)std::min<int64_t>((rows + per - 1) / per, (int64_t)num_sms * 8);
        return launch_pdl(group_norm_kernel<LPR, GATE, T>, dim3(grid), dim3(kT), 0, st, a, (const T *)x,
                          (const T *)gate, gamma, beta, (T *)out);
    }
    template <int LPR, bool GATE> cudaError_t dtype(int bf16) const {
        return bf16 ? run<LPR, GATE, __nv_bfloat16>() : run<LPR, GATE, float>();
    }
    template <int LPR> cudaError_t width(int bf16) const { return gate ? dtype<LPR, true>(bf16) : dtype<LPR, false>(bf16); }
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
    return sizeof(float) * 2 * (size_t)backward_parts(B, H, L, d) * H * d;
}

cudaError_t launch_group_norm(const NormArgs &a, const void *x, const void *gate, const float *gamma,
                              const float *beta, void *out, int bf16, int num_sms, cudaStream_t st) {
    return Launch{a, x, gate, gamma, beta, out, nullptr, nullptr, nullptr, nullptr, num_sms, st}.go(bf16);
}

cudaError_t launch_group_norm_backward(const NormArgs &a, const void *x, const void *gate, const float *gamma,
                                       const float *beta, const void *dout, void *dx, void *dgate, float *dgamma,
                                       float *dbeta, void *workspace, int bf16, int num_sms, cudaStream_t st) {
    float *part = static_cast<float *>(workspace);
    cudaError_t e = Launch{a, x, gate, gamma, beta, nullptr, dout, dx, dgate, part, num_sms, st}.go(bf16);
    if (e != cudaSuccess)
        return e;
    const int ch = a.H * a.d;
    return launch_pdl(group_norm_params_kernel, dim3((2 * ch + 31) / 32), dim3(kT), 0, st, (const float *)part, dgamma,
                      dbeta, backward_parts(a.B, a.H, a.L, a.d), ch);
}

} // namespace fw
