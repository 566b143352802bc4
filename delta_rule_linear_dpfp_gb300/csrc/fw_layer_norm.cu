// fw_layer_norm.cu -- the norm between a model's parts, with the residual sum
// before it, and the gradients.
//
//   s = x + residual,  n = (s - mean) r,  r = (var + eps)^-1/2 over the d
//   channels,  out = n gamma + beta.
// Backward, with dn = dout gamma:
//   ds = r (dn - mean(dn) - n mean(dn n)) + dsum,
//   dgamma = sum dout n,  dbeta = sum dout  over every row.
//
// Bound by the bytes: each tensor is read or written once.
//
// Mapping: G threads own a row, 8 channels each (16 bytes of bf16), all in
// registers.  The statistics take two passes over them: a warp's own mean, then
// the squares of the differences to it; a row of several warps (then G is the
// CTA) combines the warps' (mean, squares) in shared memory, one barrier a row.
// The backward's two means of products go through the same exchange: with the
// warp's own mean m_w they are sum dn and sum dn (s - m_w), and
// sum dn (s - mean) = sum over the warps of the latter + (m_w - mean) sum dn:
// differences of nearby numbers only.  gamma, beta, dgamma and dbeta stay in
// registers: one partial row of the parameters' gradients per CTA, added by a
// second kernel in a fixed order (no atomics).  The next rows are requested before
// the current ones are worked on, and the bf16 backward works on two at a time: the
// chain of shuffles and the barrier are latency that two rows share.
#include "fw_common.cuh"
#include "fw_ends.h"
#include "fw_pairs.cuh"

#include <algorithm>

namespace fw {

namespace {

constexpr int kT = 256; // threads of a CTA whose rows are a warp's or less

// 8 channels as they were loaded.
template <typename T> struct Raw;
template <> struct Raw<__nv_bfloat16> {
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
template <> struct Raw<float> {
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
FW_DEV void singles(const F2 (&v)[4], float (&o)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 t = unpack(v[e]);
        o[2 * e] = t.x;
        o[2 * e + 1] = t.y;
    }
}
FW_DEV void store_pairs(float *p, const F2 (&v)[4]) { // (shared or global)
    float o[8];
    singles(v, o);
    store8(p, o);
}
template <typename T> FW_DEV void stream_pairs(T *p, const F2 (&v)[4]) { // (global)
    float o[8];
    singles(v, o);
    store8_stream(p, o);
}
FW_DEV void param_pairs(const float *p, int c, bool on, float missing, F2 (&o)[4]) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        t[e] = missing;
    if (p && on)
        load8(p + c, t);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = on ? pack(t[2 * e], t[2 * e + 1]) : F2{0};
}

// Sums over the lanes of a row, or over the warp where the row is wider.
template <int G> FW_DEV float lanes_sum(float x) {
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The threads of a row: thread t of G holds channels 8 t .. 8 t + 7.
template <int G> struct Row {
    static constexpr int W = G > 32 ? G / 32 : 1; // warps of a row
    int c;
    bool on;
    float n, inv_n; // the channels of this warp's part of the row
    FW_DEV Row(int t, int d) {
        c = 8 * t;
        on = c < d;
        n = part_size(G > 32 ? t / 32 : 0, d);
        inv_n = n > 0.f ? 1.f / n : 0.f;
    }
    // Channels of the row that warp w holds.
    static FW_DEV float part_size(int w, int d) { return (float)min(max(d - 256 * w, 0), 8 * (G > 32 ? 32 : G)); }
};

// s -> s - (the warp's mean), which is returned with the sum of the squares.
template <int G> FW_DEV float2 centre(F2 (&s)[4], const Row<G> &row) {
    const float mean = row.inv_n * lanes_sum<G>(sum((s[0] + s[1]) + (s[2] + s[3])));
#pragma unroll
    for (int e = 0; e < 4; ++e)
        s[e] = row.on ? s[e] + both(-mean) : F2{0};
    return make_float2(mean, lanes_sum<G>(sum(fma2(s[0], s[0], s[1] * s[1]) + fma2(s[2], s[2], s[3] * s[3]))));
}

// Sum over lanes 0 .. W - 1 of what lane k % W holds.
template <int W> FW_DEV float parts_sum(float x) {
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
        x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int G> struct Walk { // the rows of this group of threads
    int64_t at, step, rows;
    FW_DEV Walk(int64_t rows_) {
        constexpr int kPer = G > 32 ? 1 : kT / G;
        at = (int64_t)blockIdx.x * kPer + (G > 32 ? 0 : threadIdx.x / G);
        step = (int64_t)gridDim.x * kPer;
        rows = rows_;
    }
};

// CTAs of a kernel that fit an SM: 64 registers a thread forward, 128 backward.
template <int G> constexpr int an_sm(bool backward) {
    return (backward ? 512 : 1024) / (G > 32 ? G : kT) > 0 ? (backward ? 512 : 1024) / (G > 32 ? G : kT) : 1;
}

template <int G, bool RES, typename T>
__global__ void __launch_bounds__(G > 32 ? G : kT, an_sm<G>(false))
    layer_norm_kernel(const T *x, const T *residual, const float *gamma, const float *beta, T *out, T *sum_out,
                      int64_t rows, int d, float eps) {
    using R = Row<G>;
    __shared__ float2 part[2][R::W];
    const R row((int)(threadIdx.x % G), d);
    const float inv_d = 1.f / (float)d, size = R::part_size((threadIdx.x & 31) % R::W, d);
    griddep_launch_dependents();
    griddep_wait();
    x = after_wait(x);
    residual = after_wait(residual);
    gamma = after_wait(gamma);
    beta = after_wait(beta);
    F2 ga[4], be[4];
    param_pairs(gamma, row.c, row.on, 1.f, ga);
    param_pairs(beta, row.c, row.on, 0.f, be);
    Walk<G> w(rows);
    Raw<T> rx, rr;
    auto request = [&](int64_t r) {
        const bool here = row.on && r < w.rows;
        rx.load(x + r * d + row.c, here);
        if (RES)
            rr.load(residual + r * d + row.c, here);
    };
    request(w.at);
    int turn = 0;
    // (the trip count is the CTA's, so that the shuffles and barriers meet)
    for (int64_t base = w.at - (G > 32 ? 0 : threadIdx.x / G); base < rows; base += w.step, turn ^= 1) {
        F2 s[4];
        const int64_t at = w.at;
        const bool mine = row.on && at < rows;
        rx.widen(s);
        if (RES) {
            F2 t[4];
            rr.widen(t);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[e] = s[e] + t[e];
            if (mine)
                stream_pairs(sum_out + at * d + row.c, s);
        }
        w.at += w.step;
        request(w.at);
        const float2 st = centre<G>(s, row);
        float shift = 0.f, ss = st.y;
        if (G > 32) {
            if ((threadIdx.x & 31) == 0)
                part[turn][threadIdx.x / 32] = st;
            __syncthreads();
            const float2 p = part[turn][(threadIdx.x & 31) % R::W];
            const float mean = inv_d * parts_sum<R::W>(size * p.x), off = p.x - mean;
            ss = parts_sum<R::W>(fmaf(size * off, off, p.y));
            shift = st.x - mean;
        }
        const F2 r = both(rsqrtf(fmaf(ss, inv_d, eps))), sh = both(shift);
        if (mine) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[e] = fma2((G > 32 ? s[e] + sh : s[e]) * r, ga[e], be[e]);
            stream_pairs(out + at * d + row.c, s);
        }
    }
}

template <int G, bool RES, typename T>
__global__ void __launch_bounds__(G > 32 ? G : kT, an_sm<G>(true))
    layer_norm_backward_kernel(const T *x, const float *gamma, const T *dout, const T *dsum, T *dx, float *partial,
                               int64_t rows, int d, float eps) {
    using R = Row<G>;
    constexpr int U = sizeof(T) == 2 && G < 1024 ? 2 : 1; // rows worked on together (registers)
    __shared__ float4 part[2][U][R::W];
    const R row((int)(threadIdx.x % G), d);
    const float inv_d = 1.f / (float)d, size = R::part_size((threadIdx.x & 31) % R::W, d);
    griddep_launch_dependents();
    griddep_wait();
    x = after_wait(x);
    gamma = after_wait(gamma);
    dout = after_wait(dout);
    dsum = after_wait(dsum);
    F2 ga[4], dga[4] = {}, dbe[4] = {};
    param_pairs(gamma, row.c, row.on, 1.f, ga);
    Walk<G> w(rows);
    Raw<T> rx[U], rd[U], rs[U];
    auto request = [&](int64_t r) { // rows r, r + step, ...
#pragma unroll
        for (int u = 0; u < U; ++u, r += w.step) {
            const bool here = row.on && r < w.rows;
            rx[u].load(x + r * d + row.c, here);
            rd[u].load(dout + r * d + row.c, here);
            if (RES)
                rs[u].load(dsum + r * d + row.c, here);
        }
    };
    request(w.at);
    int turn = 0;
    for (int64_t base = w.at - (G > 32 ? 0 : threadIdx.x / G); base < rows; base += U * w.step, turn ^= 1) {
        F2 s[U][4], dn[U][4], more[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            rx[u].widen(s[u]);
            rd[u].widen(dn[u]);
            if (RES)
                rs[u].widen(more[u]);
        }
        const int64_t at = w.at;
        w.at += U * w.step;
        request(w.at);
        float s1[U], s2[U], ss[U], shift[U];
        float2 st[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            st[u] = centre<G>(s[u], row);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            F2 t1 = {0}, t2 = {0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                dbe[e] = dbe[e] + dn[u][e];
                const F2 g = dn[u][e] * ga[e];
                t1 = t1 + g;
                t2 = fma2(g, s[u][e], t2);
            }
            s1[u] = lanes_sum<G>(sum(t1));
            s2[u] = lanes_sum<G>(sum(t2));
            ss[u] = st[u].y;
            shift[u] = 0.f;
        }
        if (G > 32) {
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int u = 0; u < U; ++u)
                    part[turn][u][threadIdx.x / 32] = make_float4(st[u].x, st[u].y, s1[u], s2[u]);
            __syncthreads();
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float4 p = part[turn][u][(threadIdx.x & 31) % R::W];
                const float mean = inv_d * parts_sum<R::W>(size * p.x), off = p.x - mean;
                ss[u] = parts_sum<R::W>(fmaf(size * off, off, p.y));
                s1[u] = parts_sum<R::W>(p.z);
                s2[u] = parts_sum<R::W>(fmaf(off, p.z, p.w));
                shift[u] = st[u].x - mean;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r0 = at + u * w.step;
            const bool mine = row.on && r0 < rows;
            // (a row that is not there has no deviation: with eps 0 its r is infinite, and
            // 0 times that would be in the sums over the rows)
            const float r1 = mine ? rsqrtf(fmaf(ss[u], inv_d, eps)) : 0.f;
            const F2 r = both(r1), sh = both(shift[u]), m1 = both(-inv_d * s1[u]), m2 = both(-inv_d * s2[u] * r1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const F2 n = (G > 32 ? s[u][e] + sh : s[u][e]) * r;
                dga[e] = fma2(dn[u][e], n, dga[e]);
                const F2 g = r * fma2(n, m2, fma2(dn[u][e], ga[e], m1));
                dn[u][e] = RES ? g + more[u][e] : g;
            }
            if (mine)
                stream_pairs(dx + r0 * d + row.c, dn[u]);
        }
    }
    if (!partial)
        return;
    // one row of dgamma and one of dbeta per CTA
    float *to = partial + (size_t)blockIdx.x * 2 * d;
    if constexpr (G > 32) {
        if (row.on) {
            store_pairs(to + row.c, dga);
            store_pairs(to + d + row.c, dbe);
        }
    } else {
        constexpr int kPer = kT / G, C = 8 * G;
        __shared__ float red[kPer * C];
        for (int m = 0; m < 2; ++m) {
            __syncthreads();
            store_pairs(red + (threadIdx.x / G) * C + row.c, m ? dbe : dga);
            __syncthreads();
            for (int e = threadIdx.x; e < d; e += kT) {
                float t = 0.f;
#pragma unroll
                for (int p = 0; p < kPer; ++p)
                    t += red[p * C + e];
                to[m * d + e] = t;
            }
        }
    }
}

// dgamma, dbeta: the CTAs' partial rows, 32 columns a CTA and the rows dealt to
// its warps; eight of a warp's rows are in flight.
constexpr int kP = 1024;
__global__ void __launch_bounds__(kP)
    layer_norm_params_kernel(const float *partial, float *dgamma, float *dbeta, int nparts, int d) {
    griddep_launch_dependents();
    griddep_wait();
    partial = after_wait(partial);
    const int e = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
    __shared__ float red[kP / 32][33];
    float s = 0.f;
    if (e < 2 * d) {
        const float *p = partial + e;
        int k = w;
        for (; k + 7 * (kP / 32) < nparts; k += 8 * (kP / 32)) {
            float t[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                t[u] = __ldcg(p + (size_t)(k + u * (kP / 32)) * 2 * d);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                s += t[u];
        }
        for (; k < nparts; k += kP / 32)
            s += __ldcg(p + (size_t)k * 2 * d);
    }
    red[w][threadIdx.x & 31] = s;
    __syncthreads();
    if (w == 0 && e < 2 * d) {
        s = 0.f;
#pragma unroll
        for (int p = 0; p < kP / 32; ++p)
            s += red[p][threadIdx.x];
        (e < d ? dgamma : dbeta)[e % d] = s;
    }
}

// Threads of a row of d channels.
int group_of(int d) {
    int g = 8;
    while (8 * g < d)
        g *= 2;
    return g;
}
constexpr int kMostSms = 152; // (a GB300's: the workspace holds the partial rows of so many)
int ctas_of(int64_t rows, int d, int sms, bool backward) {
    const int g = group_of(d), per = g > 32 ? 1 : kT / g;
    const int fit = std::max(1, (backward ? 512 : 1024) / std::max(g, g > 32 ? 1 : kT));
    return (int)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, (int64_t)fit * sms));
}

struct Launch {
    const void *x, *other;
    const float *gamma, *beta;
    const void *dout;
    void *out, *sum;
    float *partial;
    int64_t rows;
    int d;
    float eps;
    int ctas;
    cudaStream_t st;

    template <int G, bool RES, typename T> cudaError_t run() const {
        const dim3 grid(ctas), block(G > 32 ? G : kT);
        if (dout)
            return launch_pdl(layer_norm_backward_kernel<G, RES, T>, grid, block, 0, st, (const T *)x, gamma,
                              (const T *)dout, (const T *)other, (T *)out, partial, rows, d, eps);
        return launch_pdl(layer_norm_kernel<G, RES, T>, grid, block, 0, st, (const T *)x, (const T *)other, gamma, beta,
                          (T *)out, (T *)sum, rows, d, eps);
    }
    template <int G> cudaError_t of(int bf16) const {
        if (other)
            return bf16 ? run<G, true, __nv_bfloat16>() : run<G, true, float>();
        return bf16 ? run<G, false, __nv_bfloat16>() : run<G, false, float>();
    }
    cudaError_t go(int bf16) const {
        switch (group_of(d)) {
        case 8: return of<8>(bf16);
        case 16: return of<16>(bf16);
        case 32: return of<32>(bf16);
        case 64: return of<64>(bf16);
        case 128: return of<128>(bf16);
        case 256: return of<256>(bf16);
        case 512: return of<512>(bf16);
        default: return of<1024>(bf16);
        }
    }
};

} // namespace

size_t layer_norm_backward_workspace_bytes(int64_t rows, int d) {
    return sizeof(float) * 2 * (size_t)ctas_of(rows, d, kMostSms, true) * d;
}

cudaError_t launch_layer_norm(const void *x, const void *residual, const float *gamma, const float *beta, void *out,
                              void *sum, int64_t rows, int d, float eps, int bf16, cudaStream_t st) {
    int sms = 0;
    const cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess)
        return e;
    return Launch{x, residual, gamma, beta, nullptr, out, sum, nullptr, rows, d, eps, ctas_of(rows, d, sms, false), st}
        .go(bf16);
}

cudaError_t launch_layer_norm_backward(const void *x, const float *gamma, const void *dout, const void *dsum, void *dx,
                                       float *dgamma, float *dbeta, void *workspace, int64_t rows, int d, float eps,
                                       int bf16, cudaStream_t st) {
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess)
        return e;
    float *partial = dgamma ? static_cast<float *>(workspace) : nullptr;
    const int ctas = ctas_of(rows, d, std::min(sms, kMostSms), true);
    e = Launch{x, dsum, gamma, nullptr, dout, dx, nullptr, partial, rows, d, eps, ctas, st}.go(bf16);
    if (e != cudaSuccess || !partial)
        return e;
    return launch_pdl(layer_norm_params_kernel, dim3((2 * d + 31) / 32), dim3(kP), 0, st, (const float *)partial, dgamma,
                      dbeta, ctas, d);
}

} // namespace fw
