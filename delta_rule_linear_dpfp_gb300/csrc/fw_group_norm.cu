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
// fixed order (no atomics).  The next rows are requested before the current ones
// are worked on, and the arithmetic is on pairs of floats with single-instruction
// exponentials and reciprocals, or it would cost as much as the bytes.
#include "fw_common.cuh"
#include "fw_gated.h"
#include "fw_pairs.cuh"

#include <algorithm>

namespace fw {

cudaError_t device_sms(int *out); // fw_api.cu

namespace {

constexpr int kT = 256;
enum { kNone = 0, kRelu = 1, kSilu = 2, kGelu = 3 };

// (A variant of the kernels for each: as a branch per element it made them
// bound by instructions, 36 an element and 49 us where the bytes take 30.)
// The exponential and the reciprocal as single instructions (2^-22 of the
// value, and 2^-24 |x| log2 e for the exponent's own rounding; denormal results
// are 0).  x sigmoid(x) needs no guard: far below 0 the
// exponential is infinite and the reciprocal 0.
FW_DEV float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;
FW_DEV F2 sigmoid(F2 x) {
    const float2 t = unpack(x * both(-kLog2e));
    const float2 e = unpack(pack(ex2(t.x), ex2(t.y)) + both(1.f));
    return pack(rcp(e.x), rcp(e.y));
}
FW_DEV float relu(float x) { return x > 0.f ? x : x != x ? x : 0.f; } // NaN stays NaN
FW_DEV float phi(float x) { return 0.5f * (1.f + erff(x * 0.70710678118654752f)); }
template <int ACT> FW_DEV F2 act(F2 x) {
    const float2 t = unpack(x);
    if (ACT == kRelu)
        return pack(relu(t.x), relu(t.y));
    if (ACT == kSilu)
        return x * sigmoid(x);
    if (ACT == kGelu)
        return x * pack(phi(t.x), phi(t.y));
    return x;
}
// act(x) and its derivative.
template <int ACT> FW_DEV void act_grad(F2 x, F2 &f, F2 &df) {
    const float2 t = unpack(x);
    if (ACT == kRelu) {
        f = pack(relu(t.x), relu(t.y));
        df = pack(t.x > 0.f ? 1.f : 0.f, t.y > 0.f ? 1.f : 0.f);
    } else if (ACT == kSilu) {
        const F2 s = sigmoid(x);
        f = x * s;
        df = fma2(f, fma2(s, both(-1.f), both(1.f)), s); // s (1 + x (1 - s))
    } else if (ACT == kGelu) {
        const F2 p = pack(phi(t.x), phi(t.y));
        const float2 q = unpack(x * x * both(-0.5f * kLog2e));
        f = x * p;
        df = fma2(x * both(0.39894228040143268f), pack(ex2(q.x), ex2(q.y)), p);
    } else {
        f = x;
        df = both(1.f);
    }
}

template <int LPR> FW_DEV float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// x - mean of a row held 8 channels a lane (lanes at or past d hold zeros and
// stay zero); returns r.
template <int LPR> FW_DEV float centre(F2 (&x)[4], bool on, float inv_d, float eps) {
    const F2 mean = both(-inv_d * row_sum<LPR>(sum((x[0] + x[1]) + (x[2] + x[3]))));
#pragma unroll
    for (int e = 0; e < 4; ++e)
        x[e] = on ? x[e] + mean : F2{0};
    const float ss = sum(fma2(x[0], x[0], x[1] * x[1]) + fma2(x[2], x[2], x[3] * x[3]));
    return rsqrtf(fmaf(row_sum<LPR>(ss), inv_d, eps));
}

// 8 channels as they were loaded.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 u;
    FW_DEV void load(const __nv_bfloat16 *p, bool here) {
        u = here ? __ldcs(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
    }
    FW_DEV void widen(F2 (&o)[4]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    FW_DEV void load(const float *p, bool here) {
        a = here ? __ldcs(reinterpret_cast<const float4 *>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
        b = here ? __ldcs(reinterpret_cast<const float4 *>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    FW_DEV void widen(F2 (&o)[4]) const {
        o[0] = pack(a.x, a.y);
        o[1] = pack(a.z, a.w);
        o[2] = pack(b.x, b.y);
        o[3] = pack(b.z, b.w);
    }
};

template <typename T> FW_DEV void store4(T *p, const F2 (&v)[4]) {
    float o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 t = unpack(v[e]);
        o[2 * e] = t.x;
        o[2 * e + 1] = t.y;
    }
    store8(p, o);
}
FW_DEV void load_pairs(const float *p, F2 (&o)[4]) {
    float t[8];
    load8(p, t);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = pack(t[2 * e], t[2 * e + 1]);
}

// A lane group's walk over the rows (b, l) of a head, `step` rows at a time:
// where the row lies in x (head-major) and in out (token-major), by additions.
struct Walk {
    unsigned row, rows, step, l, L, step_l;
    int64_t x, out, dx, dx_wrap, dout;
    FW_DEV Walk(const NormArgs &a, unsigned first, unsigned step_, int h, int c0) {
        row = first;
        rows = (unsigned)(a.B * (int64_t)a.L);
        step = step_;
        L = (unsigned)a.L;
        const unsigned b = row / L, step_b = step / L;
        l = row - b * L;
        step_l = step - step_b * L;
        x = (((int64_t)b * a.H + h) * a.L + l) * a.d + c0;
        out = ((int64_t)row * a.H + h) * a.d + c0;
        dx = ((int64_t)step_b * a.H * a.L + step_l) * a.d;
        dx_wrap = (int64_t)(a.H - 1) * a.L * a.d; // past the end of one sequence: the next one's same head
        dout = (int64_t)step * a.H * a.d;
    }
    FW_DEV bool here() const { return row < rows; }
    FW_DEV void next() {
        row += step;
        l += step_l;
        x += dx;
        out += dout;
        if (l >= L) {
            l -= L;
            x += dx_wrap;
        }
    }
};

template <int LPR, int ACT, bool GATE, typename T>
__global__ void __launch_bounds__(kT, 3)
    group_norm_kernel(NormArgs a, const T *__restrict__ x, const T *__restrict__ gate, const float *__restrict__ gamma,
                      const float *__restrict__ beta, T *__restrict__ out) {
    constexpr unsigned RPC = kT / LPR; // rows per CTA and step
    const int c0 = 8 * (threadIdx.x % LPR), h = blockIdx.y;
    const bool on = c0 < a.d;
    const float inv_d = 1.f / (float)a.d;
    griddep_launch_dependents();
    griddep_wait();
    x = after_wait(x);
    gate = after_wait(gate);
    gamma = after_wait(gamma);
    beta = after_wait(beta);
    F2 ga[4] = {}, be[4] = {};
    if (on) {
        load_pairs(gamma + h * a.d + c0, ga);
        load_pairs(beta + h * a.d + c0, be);
    }
    Walk at(a, blockIdx.x * RPC + threadIdx.x / LPR, gridDim.x * RPC, h, c0);
    constexpr int D = sizeof(T) == 2 ? 2 : 1; // rows requested ahead (64 to 96 bytes a lane)
    Raw8<T> rx[D], rg[D];
    int64_t to[D];
    bool here[D];
    auto request = [&](int u) {
        here[u] = on && at.here();
        to[u] = at.out;
        rx[u].load(x + at.x, here[u]);
        if (GATE)
            rg[u].load(gate + at.out, here[u]);
        at.next();
    };
#pragma unroll
    for (int u = 0; u < D; ++u)
        request(u);
    // (the loop's trip count is the CTA's, so that the shuffles meet)
    for (unsigned base = blockIdx.x * RPC; base < at.rows; base += D * at.step) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            F2 v[4], z[4];
            rx[u].widen(v);
            if (GATE)
                rg[u].widen(z);
            const bool mine = here[u];
            const int64_t o = to[u];
            request(u);
            const F2 r = both(centre<LPR>(v, mine, inv_d, a.eps));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const F2 y = fma2(v[e] * r, ga[e], be[e]);
                v[e] = GATE ? y * act<ACT>(z[e]) : act<ACT>(y);
            }
            if (mine)
                store4(out + o, v);
        }
    }
}

template <int LPR, int ACT, bool GATE, typename T>
__global__ void __launch_bounds__(kT, 2)
    group_norm_backward_kernel(NormArgs a, const T *__restrict__ x, const T *__restrict__ gate,
                               const float *__restrict__ gamma, const float *__restrict__ beta,
                               const T *__restrict__ dout, T *__restrict__ dx, T *__restrict__ dgate,
                               float *__restrict__ part) {
    constexpr unsigned RPC = kT / LPR;
    __shared__ float red[2][RPC][8 * LPR];
    const int c0 = 8 * (threadIdx.x % LPR), h = blockIdx.y;
    const unsigned slot = threadIdx.x / LPR;
    const bool on = c0 < a.d;
    const float inv_d = 1.f / (float)a.d;
    griddep_launch_dependents();
    griddep_wait();
    x = after_wait(x);
    gate = after_wait(gate);
    gamma = after_wait(gamma);
    beta = after_wait(beta);
    dout = after_wait(dout);
    F2 ga[4] = {}, be[4] = {}, dga[4] = {}, dbe[4] = {};
    if (on) {
        load_pairs(gamma + h * a.d + c0, ga);
        load_pairs(beta + h * a.d + c0, be);
    }
    Walk at(a, blockIdx.x * RPC + slot, gridDim.x * RPC, h, c0);
    constexpr int D = sizeof(T) == 2 ? 2 : 1; // rows requested ahead (64 to 96 bytes a lane)
    Raw8<T> rx[D], rg[D], rd[D];
    int64_t to[D], from[D];
    bool here[D];
    auto request = [&](int u) {
        here[u] = on && at.here();
        to[u] = at.out;
        from[u] = at.x;
        rx[u].load(x + at.x, here[u]);
        rd[u].load(dout + at.out, here[u]);
        if (GATE)
            rg[u].load(gate + at.out, here[u]);
        at.next();
    };
#pragma unroll
    for (int u = 0; u < D; ++u)
        request(u);
    for (unsigned base = blockIdx.x * RPC; base < at.rows; base += D * at.step) {
#pragma unroll
        for (int u = 0; u < D; ++u) {
            F2 n[4], t[4], dz[4];
            rx[u].widen(n);
            rd[u].widen(dz);
            if (GATE)
                rg[u].widen(t);
            const bool mine = here[u];
            const int64_t o = to[u], i = from[u];
            request(u);
            // (a row that is not there has no deviation: with eps 0 its r is infinite, and
            // 0 times that would be in the sums over the rows)
            const float r1 = centre<LPR>(n, mine, inv_d, a.eps), r = mine ? r1 : 0.f;
            F2 s1 = {0}, s2 = {0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                n[e] = n[e] * both(r);
                const F2 z = fma2(n[e], ga[e], be[e]);
                F2 f, df;
                act_grad<ACT>(GATE ? t[e] : z, f, df);
                if (GATE) {
                    t[e] = dz[e] * z * df;
                    dz[e] = dz[e] * f;
                } else {
                    dz[e] = dz[e] * df;
                }
                dga[e] = fma2(dz[e], n[e], dga[e]);
                dbe[e] = dbe[e] + dz[e];
                dz[e] = dz[e] * ga[e];
                s1 = s1 + dz[e];
                s2 = fma2(dz[e], n[e], s2);
            }
            const F2 m1 = both(-inv_d * row_sum<LPR>(sum(s1))), m2 = both(-inv_d * row_sum<LPR>(sum(s2)));
            if (mine) {
                if (GATE)
                    store4(dgate + o, t);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    dz[e] = both(r) * fma2(n[e], m2, dz[e] + m1);
                store4(dx + i, dz);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        *reinterpret_cast<float2 *>(&red[0][slot][c0 + 2 * e]) = unpack(dga[e]);
        *reinterpret_cast<float2 *>(&red[1][slot][c0 + 2 * e]) = unpack(dbe[e]);
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

// CTAs per head: what the device's SMs hold at once (three an SM, two in the
// backward: registers), no more than the rows give.  (B16 H8 L2048 d 128: 31.4 us
// in one wave, 33 in two, 37 with four CTAs an SM, whose 64 registers spill; the
// gradients 62 us in one wave, 66 in two, 105 with three CTAs an SM.)
constexpr int kCtasPerSm = 3, kBackwardCtasPerSm = 2;
constexpr int kMostSms = 152; // (a GB300's: the workspace holds the partial rows of so many)
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
    int parts; // CTAs of a head

    template <int LPR, int ACT, bool GATE, typename T> cudaError_t run() const {
        if (dout)
            return launch_pdl(group_norm_backward_kernel<LPR, ACT, GATE, T>, dim3(parts, a.H), dim3(kT), 0, st, a,
                              (const T *)x, (const T *)gate, gamma, beta, (const T *)dout, (T *)dx, (T *)dgate, part);
        return launch_pdl(group_norm_kernel<LPR, ACT, GATE, T>, dim3(parts, a.H), dim3(kT), 0, st, a, (const T *)x,
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
    return sizeof(float) * 2 * (size_t)parts_of(B, H, L, d, kBackwardCtasPerSm * kMostSms) * H * d;
}

cudaError_t launch_group_norm(const NormArgs &a, const void *x, const void *gate, const float *gamma,
                              const float *beta, void *out, int bf16, cudaStream_t st) {
    int sms = 0;
    const cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess)
        return e;
    const int parts = parts_of(a.B, a.H, a.L, a.d, kCtasPerSm * sms);
    return Launch{a, x, gate, gamma, beta, out, nullptr, nullptr, nullptr, nullptr, st, parts}.go(bf16);
}

cudaError_t launch_group_norm_backward(const NormArgs &a, const void *x, const void *gate, const float *gamma,
                                       const float *beta, const void *dout, void *dx, void *dgate, float *dgamma,
                                       float *dbeta, void *workspace, int bf16, cudaStream_t st) {
    float *part = static_cast<float *>(workspace);
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess)
        return e;
    const int parts = parts_of(a.B, a.H, a.L, a.d, kBackwardCtasPerSm * std::min(sms, kMostSms)), ch = a.H * a.d;
    e = Launch{a, x, gate, gamma, beta, nullptr, dout, dx, dgate, part, st, parts}.go(bf16);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(group_norm_params_kernel, dim3((2 * ch + 31) / 32), dim3(kT), 0, st, (const float *)part, dgamma,
                      dbeta, parts, ch);
}

} // namespace fw
