// fw_vocab_rows.cu -- the vocabulary loss's work by token: the loss of up to four
// answers without tensor cores, a token's log-sum-exp from its parts, and what a
// token brings to the gradients.  The formulas stand at the head of fw_vocab.cu.
#include "fw_vocab.h"

#include <algorithm>

namespace fw {
namespace vocab {

namespace {

constexpr float kQMin = 1e-7f; // q below it (p_t = 1 in 32 bits) divides nothing

// ------------------------------------------------------------ few tokens
// Up to four answers: bound by reading W once, so a product on CUDA cores from
// registers, whose start and end cost less than the tensor cores' (32 000
// entries, D 512: one token 8.9 us, four 11.9, on tensor cores 15 to 17; eight
// would take 17.9, and 27.8 against 22.9 at D 1024).  A warp takes four rows of
// W at a time, its lanes 8 channels each; h sits in shared memory in 32 bits.
// After the lanes' sums have been exchanged each lane keeps the (reference, sum
// of exponentials) of one token over the rows it got.
constexpr int kFewT = 256, kFewRows = 4, kFewStep = kFewT / 32 * kFewRows;
constexpr int kFewValues = 11264; // NT D: 44 KB of shared memory
constexpr int few_an_sm(int nt) { return nt == 1 ? 4 : 2; } // (registers)

// 8 channels as they were loaded, as pairs.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 u;
    FW_DEV void load(const __nv_bfloat16 *p, bool here) {
        u = here ? __ldcs(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
    }
    FW_DEV F2 two(int i) const {
        const uint32_t w = i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
        return pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};
template <> struct Eight<float> {
    float4 a, b;
    FW_DEV void load(const float *p, bool here) {
        a = here ? __ldcs(reinterpret_cast<const float4 *>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
        b = here ? __ldcs(reinterpret_cast<const float4 *>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    FW_DEV F2 two(int i) const { return i == 0 ? pack(a.x, a.y) : i == 1 ? pack(a.z, a.w) : i == 2 ? pack(b.x, b.y) : pack(b.z, b.w); }
};

template <int NT, typename T>
__global__ void __launch_bounds__(kFewT, few_an_sm(NT))
    vocab_few_kernel(const T *h, const T *W, const float *bias, Tokens targets, float2 *part,
                     float *target_z, int N, int V, int D) {
    extern __shared__ float hs[]; // [NT][D]
    __shared__ float2 red[kFewT];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_launch_dependents();
    griddep_wait();
    h = after_wait(h);
    W = after_wait(W);
    bias = after_wait(bias);
    targets.p = after_wait(targets.p);
    for (int i = 8 * tid; i < NT * D; i += 8 * kFewT) {
        float v[8] = {};
        if (i < N * D)
            load8(h + i, v);
        store8(hs + i, v);
    }
    __syncthreads();
    constexpr int n = kFewRows * NT; // a step's values: row r, token t at r NT + t
    static_assert(n <= 32, "a lane keeps one value");
    int mine = 0; // the value that this lane keeps
#pragma unroll
    for (int half = n / 2, o = 16; half > 0; half /= 2, o /= 2)
        mine += lane & o ? half : 0;
    const int t = mine % NT, r0 = mine / NT;
    const bool owner = (lane & (32 / n - 1)) == 0 && t < N; // (of the lanes that end up with the same value)
    const int target = t < N ? token_at(targets, t, V) : -1;
    float top = kNoRef, total = 0.f;
    for (int64_t v0 = ((int64_t)blockIdx.x * (kFewT / 32) + warp) * kFewRows; v0 < V; v0 += (int64_t)gridDim.x * kFewStep) {
        F2 acc[kFewRows][NT] = {};
        const float b = bias && owner && v0 + r0 < V ? __ldcg(bias + v0 + r0) : 0.f;
#pragma unroll 2
        for (int c = 8 * lane; c < D; c += 256) {
            Eight<T> w[kFewRows];
#pragma unroll
            for (int r = 0; r < kFewRows; ++r)
                w[r].load(W + (v0 + r) * D + c, v0 + r < V);
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                const float4 x = *reinterpret_cast<const float4 *>(hs + k * D + c);
                const float4 y = *reinterpret_cast<const float4 *>(hs + k * D + c + 4);
#pragma unroll
                for (int r = 0; r < kFewRows; ++r) {
                    acc[r][k] = fma2(w[r].two(0), pack(x.x, x.y), acc[r][k]);
                    acc[r][k] = fma2(w[r].two(1), pack(x.z, x.w), acc[r][k]);
                    acc[r][k] = fma2(w[r].two(2), pack(y.x, y.y), acc[r][k]);
                    acc[r][k] = fma2(w[r].two(3), pack(y.z, y.w), acc[r][k]);
                }
            }
        }
        float x[n];
#pragma unroll
        for (int i = 0; i < n; ++i)
            x[i] = sum(acc[i / NT][i % NT]);
        int o = 16;
#pragma unroll
        for (int half = n / 2; half > 0; half /= 2, o /= 2) {
            const bool up = lane & o;
#pragma unroll
            for (int j = 0; j < half; ++j) {
                const float give = up ? x[j] : x[j + half], keep = up ? x[j + half] : x[j];
                x[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
        }
#pragma unroll
        for (int o1 = 16 / n; o1 > 0; o1 /= 2)
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], o1);
        if (owner && v0 + r0 < V) {
            const float z = x[0] + b;
            if (v0 + r0 == target) {
                target_z[t] = z; // (kept apart from the others)
            } else if (!(z < kOut)) {
                const float m = fmaxf(top, reference(z));
                total = total * ex2(top - m) + ex2(fmaf(z, kLog2e, -m));
                top = m;
            }
        }
    }
    red[tid] = make_float2(top, total);
    __syncthreads();
    if (warp < N) { // this warp's token: what the lanes that keep it have, of every warp
        top = kNoRef;
        total = 0.f;
        auto join = [&](float2 p) {
            const float m = fmaxf(top, p.x);
            total = total * ex2(top - m) + p.y * ex2(p.x - m);
            top = m;
        };
        if (t == warp && owner)
            for (int w = 0; w < kFewT / 32; ++w)
                join(red[32 * w + lane]);
        for (int o = 16; o > 0; o >>= 1)
            join(make_float2(__shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, total, o)));
        if (lane == 0)
            part[(size_t)blockIdx.x * N + warp] = make_float2(top, total);
    }
}

// ------------------------------------------------------------ small kernels
constexpr int kS = 256;

// A token's parts joined: 32 tokens of a CTA and 32 threads for each, or one
// token and 1024 where there are few (the loss of 128 tokens over 32 000 entries, D 256:
// 12.6 us by one, 13.5 by 32; of 512 18.8 and 16.8, over 8000, D 512, 14.1 and 10.5;
// below 512 the parts of a small vocabulary are joined sooner by 32, too: 128 over 8000
// 11.1 and 10.3).
constexpr int kJ = 1024;
__global__ void __launch_bounds__(kJ)
    join_parts_kernel(const float2 *part, const float *target_z, Tokens targets, float *loss, float *lse, int N, int V,
                      int nparts, int tokens) {
    __shared__ float2 red[kJ];
    griddep_launch_dependents();
    griddep_wait();
    part = after_wait(part);
    target_z = after_wait(target_z);
    targets.p = after_wait(targets.p);
    const int slices = kJ / tokens, i = threadIdx.x % tokens, w = threadIdx.x / tokens;
    const int n = blockIdx.x * tokens + i;
    float top = kNoRef, total = 0.f;
    auto join = [&](float2 p) { // (references are sixteenths: their differences are exact)
        const float m = fmaxf(top, p.x);
        total = total * ex2(top - m) + p.y * ex2(p.x - m);
        top = m;
    };
    if (n < N)
        for (int k = w; k < nparts; k += 8 * slices) {
            float2 p[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                p[u] = k + u * slices < nparts ? __ldcg(part + (size_t)(k + u * slices) * N + n)
                                               : make_float2(kNoRef, 0.f);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                join(p[u]);
        }
    red[threadIdx.x] = make_float2(top, total);
    for (int o = slices / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (w < o) {
            join(red[threadIdx.x + o * tokens]);
            red[threadIdx.x] = make_float2(top, total);
        }
    }
    if (w == 0 && n < N) {
        const int t = token_at(targets, n, V);
        // the sum is that of the other entries: loss = log(1 + sum / exp(z_t)), without a
        // difference of large numbers where the target is all but certain
        const float l = logf(total);
        float a = 0.f, b = 0.f;
        if (t >= V) {
            a = __int_as_float(0x7fffffff);
            b = fmaf(top, kLn2, l);
        } else if (t >= 0) {
            const float z = __ldcg(target_z + n), x = fmaf(-z, kLog2e, top);
            if (x > 64.f) { // (the target's own part is nothing beside them)
                b = fmaf(top, kLn2, l);
                a = z < kOut ? b - z : fmaf(x, kLn2, l); // (x may be past the largest float)
            } else {
                a = log1pf(total * ex2(x));
                b = z + a;
            }
            if (z < kOut && total == 0.f) // every entry is out, the target too
                a = __int_as_float(0x7fffffff);
        }
        loss[n] = a;
        lse[n] = b;
    }
}

// What a token brings to G and to its row of dh: with q = max(-expm1(-loss), kQMin),
//   G = 2^(z log2 e - row.x) row.y off the target, row.z on it; q dloss = row.w,
// all 0 for a token without a gradient.  Folded, row.x takes in log2 q and row.y is what
// its rounding is off by, 1 to within 2^-25 |row.x|: left out of what is rounded to
// bf16 anyway, not of the sums that are kept in 32 bits.
FW_DEV bool row_constants(const Tokens &targets, const float *loss, const float *lse, const float *dloss, bool folded,
                          int n, int V, float4 &row, int &target) {
    const int t = token_at(targets, n, V);
    target = t < V ? t : -1; // (past the vocabulary: the loss is NaN, there is no gradient)
    row = make_float4(0.f, 0.f, 0.f, 0.f);
    if (target < 0)
        return false;
    const float q = -expm1f(-__ldcg(loss + n)), s = __ldcg(lse + n), over = fmaxf(q, kQMin);
    row.x = folded ? fmaf(s, kLog2e, log2f(over)) : reference(s);
    row.y = ex2(fmaf(-s, kLog2e, row.x)) / over; // (what the reference is off by)
    row.z = -q / over;
    row.w = over * __ldcg(dloss + n);
    return true;
}

// The tokens' constants, and w h in bf16 (wh, or null): zeros for the tokens without a
// gradient, whatever h holds there.  With lo_rows, what its rounding leaves follows from
// that row on, rounded as well, and the rows between are zeros.
__global__ void __launch_bounds__(kS)
    rows_kernel(const __nv_bfloat16 *h, Tokens targets, const float *loss, const float *lse, const float *dloss,
                float4 *row, int *row_target, __nv_bfloat16 *wh, int lo_rows, bool folded, int N, int V, int D, int lg) {
    griddep_launch_dependents();
    griddep_wait();
    h = after_wait(h);
    targets.p = after_wait(targets.p);
    loss = after_wait(loss);
    lse = after_wait(lse);
    dloss = after_wait(dloss);
    const int n = (int)(blockIdx.x * (kS >> lg) + (threadIdx.x >> lg)), lane = threadIdx.x & ((1 << lg) - 1);
    if (n >= max(N, wh ? lo_rows : 0))
        return;
    float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
    int target = -1;
    const bool live = n < N && row_constants(targets, loss, lse, dloss, folded, n, V, r, target);
    if (lane == 0 && n < N) {
        row[n] = r;
        row_target[n] = target;
    }
    if (wh)
        for (int c = 8 * lane; c < D; c += 8 << lg) {
            float v[8] = {};
            if (live) {
                load8(h + (size_t)n * D + c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] *= r.w;
            }
            store8(wh + (size_t)n * D + c, v);
            if (lo_rows) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] -= __bfloat162float(__float2bfloat16_rn(v[e]));
                store8(wh + (size_t)(lo_rows + n) * D + c, v);
            }
        }
}

int few_tokens(int N) { return N <= 2 ? N : 4; }

template <int NT, typename T>
cudaError_t go_few(const void *h, const void *W, const float *bias, Tokens targets, float2 *part, float *target_z, int N,
                   int V, int D, cudaStream_t st) {
    return launch_pdl(vocab_few_kernel<NT, T>, dim3(parts_of(N, V, D)), dim3(kFewT), sizeof(float) * NT * D, st,
                      (const T *)h, (const T *)W, bias, targets, part, target_z, N, V, D);
}

} // namespace

bool few(int N, int D) { return N <= 4 && few_tokens(N) * (int64_t)D <= kFewValues; }
int parts_of(int N, int V, int D) {
    return few(N, D) ? std::min((V - 1) / kFewStep + 1, 2 * kPairs * few_an_sm(few_tokens(N))) : (V - 1) / kCols + 1;
}

cudaError_t launch_few(const void *h, const void *W, const float *bias, Tokens targets, float2 *part, float *target_z,
                       int N, int V, int D, int bf16, cudaStream_t st) {
    switch (few_tokens(N)) {
    case 1:
        return bf16 ? go_few<1, __nv_bfloat16>(h, W, bias, targets, part, target_z, N, V, D, st)
                    : go_few<1, float>(h, W, bias, targets, part, target_z, N, V, D, st);
    case 2:
        return bf16 ? go_few<2, __nv_bfloat16>(h, W, bias, targets, part, target_z, N, V, D, st)
                    : go_few<2, float>(h, W, bias, targets, part, target_z, N, V, D, st);
    default:
        return bf16 ? go_few<4, __nv_bfloat16>(h, W, bias, targets, part, target_z, N, V, D, st)
                    : go_few<4, float>(h, W, bias, targets, part, target_z, N, V, D, st);
    }
}

cudaError_t launch_join_parts(const float2 *part, const float *target_z, Tokens targets, float *loss, float *lse, int N,
                              int V, int nparts, cudaStream_t st) {
    const int tokens = N < 512 ? 1 : 32;
    return launch_pdl(join_parts_kernel, dim3((N + tokens - 1) / tokens), dim3(kJ), 0, st, part, target_z, targets, loss,
                      lse, N, V, nparts, tokens);
}

cudaError_t launch_rows(const void *h, Tokens targets, const float *loss, const float *lse, const float *dloss,
                        float4 *row, int *row_target, void *wh, int lo_rows, bool folded, int N, int V, int D, cudaStream_t st) {
    const int lg = group_log2(D), per = kS >> lg, rows = std::max(N, lo_rows);
    return launch_pdl(rows_kernel, dim3((rows + per - 1) / per), dim3(kS), 0, st, (const __nv_bfloat16 *)h, targets, loss,
                      lse, dloss, row, row_target, (__nv_bfloat16 *)wh, lo_rows, folded, N, V, D, lg);
}

} // namespace vocab
} // namespace fw
