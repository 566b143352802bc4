// fw_gated_chunk.cu -- the gated delta rule over a sequence and its
// gradients, in chunks of 64 tokens: fp32 tensors, on CUDA cores (bf16 tensors
// take the same algebra to the tensor cores: fw_gated_tc.cu,
// fw_gated_grad_tc.cu).
//
// The rule, per value head (a_t = exp(g_t)):
//   W_t = a_t W_{t-1} + beta_t (v_t - a_t W_{t-1} k_t) k_t^T,  y_t = scale W_t q_t.
// With G the running sum of g inside a chunk, D_ij = exp(G_i - G_j) for
// j <= i, S the chunk's first state and S' its last, row i of each matrix
// belonging to token i:
//   A = strict_lower(beta_i D_ij k_i.k_j),   T = (I + A)^-1,
//   X = beta (V - e^G K S^T),                U = T X,
//   M = lower(scale D_ij q_i.k_j),           Y = scale e^G Q S^T + M U,
//   S' = e^{G_C} S + (e^{G_C - G} U)^T K.
// Every exponent is a difference of sums taken over later tokens minus
// earlier ones, so nothing overflows for g <= 0 however strong the gate is;
// the sums are formed in 64 bits and kept as a float pair, because a
// difference of two large sums would lose the small one.
//
// Transposed, given dY and dS' (the gradient of the next chunk's state):
//   dU = M^T dY + e^{G_C - G} K dS'^T,       dX = T^T dU,
//   dS = e^{G_C} dS' + (scale e^G dY)^T Q - (beta e^G dX)^T K,
// and per chunk, with E = lower(scale D dY U^T), F = strict_lower(D dX U^T):
//   q-side   a_i = scale e^{G_i} S^T dY_i + sum_j E_ij k_j            (= dq_i)
//   reader   h_i = e^{G_i} S^T dX_i + sum_j F_ij k_j
//   writer   w_j = e^{G_C-G_j} dS'^T U_j + sum_i E_ij q_i - sum_i beta_i F_ij k_i
//   dk = w - beta h,  dV = beta dX,  dbeta_i = dX_i.V_i - k_i.h_i.
// dg_t is the sum of everything that decays by token t, from what was there
// before it to what comes with it or after:
//   dg_t = e^{G_C} <S, dS'> + sum_{i >= t} R_i + sum_{j < t} W_j + sum_{i >= t > j} P_ij,
//   R_i = e^{G_i} (scale q_i.S^T dY_i - beta_i k_i.S^T dX_i),  W_j = e^{G_C-G_j} k_j.dS'^T U_j,
//   P_ij = E_ij q_i.k_j - beta_i F_ij k_i.k_j.
// (As the sums over i >= t of q_i.a_i - beta_i k_i.h_i - k_i.w_i, the pairs on
// one side of t would cancel, and what they leave is all there is where the
// gates are strong, or nothing was there before: 1325 us instead of 1389 for
// the gradients of B8 H16 L512 d 128, and dg wrong by more than its own size
// behind gates of e^-8.)
// Keys and queries scaled to unit length enter as r k with one fp32 r per
// token, and dk = r (dk^ - k^ (k^.dk^)) comes back.
//
// Kernels: prep (per chunk: T, M and the per-token scalars), walk (the chunks
// of a head in order, per slice of 32 value channels: a channel's row of the
// state never meets another), reverse walk (the same backwards), grad (per
// chunk and key head: the sums over its value heads stay in one CTA, so the
// gradients of shared heads have a fixed order).
#include "fw_common.cuh"
#include "fw_gated.h"
#include "fw_gated_tc.h"
#include "fw_gated_tiles.cuh"
#include "fw_pairs.cuh"

#include <algorithm>

namespace fw {

cudaError_t device_sms(int *out); // fw_api.cu

namespace {

constexpr int C = kGatedChunk, NT = kGatedThreads, LC = kGatedLd;
constexpr int NV = 32;   // value channels per slice of the gradient kernel
constexpr int TOK = 8; // floats per token: rk, rq, e^G, e^{G_C-G}, G high, G low, beta, unused

// Workspace, in floats: per chunk of every value head.
struct Ws {
    float *T, *M, *tok, *S, *dS, *U, *dX;
};
struct WsOff {
    size_t T, M, tok, S, dS, U, dX, end;
};
WsOff ws_off(int BH, int L, int d_k, int d_v, bool backward) {
    const size_t n = (size_t)BH * ((L + C - 1) / C);
    WsOff o;
    o.T = 0;
    o.M = o.T + n * C * C;
    o.tok = o.M + n * C * C;
    o.S = o.tok + n * C * TOK;
    if (!backward) {
        o.dS = o.U = o.dX = o.end = o.S;
        return o;
    }
    o.dS = o.S + n * d_v * d_k;
    o.U = o.dS + n * d_v * d_k;
    o.dX = o.U + n * C * d_v;
    o.end = o.dX + n * C * d_v;
    return o;
}
Ws ws_at(void *p, const WsOff &o) {
    float *f = static_cast<float *>(p);
    return {f + o.T, f + o.M, f + o.tok, f + o.S, f + o.dS, f + o.U, f + o.dX};
}

// rows x width of a tensor (row stride lds) into shared memory; rows at or past
// `valid` and channels at or past `cols` are zero (whatever is stored there).
FW_DEV void load_tile(float *dst, int ldd, const float *src, size_t lds, int rows, int valid, int cols, int width) {
    const int c8 = width >> 3;
    for (int e = threadIdx.x; e < rows * c8; e += NT) {
        const int i = e / c8, c = (e % c8) * 8;
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (i < valid && c < cols)
            load8(src + (size_t)i * lds + c, x);
        float4 *d = reinterpret_cast<float4 *>(dst + i * ldd + c);
        d[0] = make_float4(x[0], x[1], x[2], x[3]);
        d[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

FW_DEV float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

// Products of tiles in shared memory, on pairs of floats: one instruction for
// two products (B8 H16 L512 d 128: forward 438 -> 417 us; with few heads the
// walks wait for shared memory and barriers, and it makes no difference).
struct Quad { // 16 bytes as two pairs
    F2 a, b;
};
FW_DEV Quad ldq(const float *p) {
    const ulonglong2 t = *reinterpret_cast<const ulonglong2 *>(p);
    return {{t.x}, {t.y}};
}

// acc[r][s] += sum_k A[r][k] B[s][k] (K a multiple of 4).
template <int R, int S>
FW_DEV void mm_nt(float (&acc)[R][S], const float *A, int lda, int ra, const float *B, int ldb, int rb, int K) {
    F2 t[R][S] = {};
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        Quad a[R], b[S];
#pragma unroll
        for (int r = 0; r < R; ++r)
            a[r] = ldq(A + r * ra * lda + k);
#pragma unroll
        for (int s = 0; s < S; ++s)
            b[s] = ldq(B + s * rb * ldb + k);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int s = 0; s < S; ++s)
                t[r][s] = fma2(a[r].b, b[s].b, fma2(a[r].a, b[s].a, t[r][s]));
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int s = 0; s < S; ++s)
            acc[r][s] += sum(t[r][s]);
}

// Four columns' sums as two pairs.
template <int R> struct Columns {
    F2 t[R][2];
    FW_DEV Columns(const float (&acc)[R][4]) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            t[r][0] = pack(acc[r][0], acc[r][1]);
            t[r][1] = pack(acc[r][2], acc[r][3]);
        }
    }
    FW_DEV void add(int r, float x, const Quad &y) {
        t[r][0] = fma2(both(x), y.a, t[r][0]);
        t[r][1] = fma2(both(x), y.b, t[r][1]);
    }
    FW_DEV void get(float (&acc)[R][4]) const {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 p = unpack(t[r][0]), q = unpack(t[r][1]);
            acc[r][0] = p.x;
            acc[r][1] = p.y;
            acc[r][2] = q.x;
            acc[r][3] = q.y;
        }
    }
};

// acc[r][0..3] += sum_k A[k lda + r ra] B[k ldb .. + 3]: A's rows run along k
// (transposed use).
template <int R>
FW_DEV void mm_tn(float (&acc)[R][4], const float *A, int lda, int ra, const float *B, int ldb, int K) {
    Columns<R> t(acc);
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        const Quad b = ldq(B + k * ldb);
#pragma unroll
        for (int r = 0; r < R; ++r)
            t.add(r, A[k * lda + r * ra], b);
    }
    t.get(acc);
}

// acc[r][0..3] += sum_k A[r][k] B[k ldb .. + 3].
template <int R>
FW_DEV void mm_nn(float (&acc)[R][4], const float *A, int lda, int ra, const float *B, int ldb, int K) {
    Columns<R> t(acc);
#pragma unroll 2
    for (int k = 0; k < K; k += 4) {
        float4 a[R];
#pragma unroll
        for (int r = 0; r < R; ++r)
            a[r] = lds4(A + r * ra * lda + k);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const Quad b = ldq(B + (k + u) * ldb);
#pragma unroll
            for (int r = 0; r < R; ++r)
                t.add(r, u == 0 ? a[r].x : u == 1 ? a[r].y : u == 2 ? a[r].z : a[r].w, b);
        }
    }
    t.get(acc);
}

// A thread's asynchronous copies (copy16) in groups.
FW_DEV void copies_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> FW_DEV void copies_done() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// rows x width (a power of two, given as the logarithm of its quarter) of a
// tensor whose rows at or past `valid` and columns at or past `cols` read as zero.
FW_DEV void copy_tile(float *dst, int ldd, const float *src, size_t lds, int rows, int valid, int cols, int log_w4) {
    for (int e = threadIdx.x; e < rows << log_w4; e += NT) {
        const int i = e >> log_w4, c = (e & ((1 << log_w4) - 1)) * 4;
        const bool in = i < valid && c < cols;
        copy16(dst + i * ldd + c, in ? src + (size_t)i * lds + c : src, in);
    }
}
FW_DEV int log2_of(int x) { return 31 - __clz(x); }

// ------------------------------------------------------------------ prep
__global__ void __launch_bounds__(NT)
    gated_prep_kernel(GatedArgs a, const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ g,
                      const float *__restrict__ beta, Ws ws) {
    extern __shared__ __align__(16) float sm[];
    const int ldk = a.d_k + 4;
    float *kt = sm, *qt = kt + C * ldk, *At = qt + C * ldk, *Tt = At + C * LC, *tmp = Tt + C * LC, *tok = tmp + 1024;
    const int tid = threadIdx.x, c = blockIdx.x, bh = blockIdx.y;
    const int b = bh / a.H, h = bh % a.H, kh = b * a.Hk + h / (a.H / a.Hk);
    griddep_launch_dependents();
    griddep_wait();
    q = after_wait(q);
    k = after_wait(k);
    g = after_wait(g);
    beta = after_wait(beta);
    const int n = min(C, seq_len(a, b) - c * C);
    if (n <= 0)
        return;
    const size_t row0 = (size_t)c * C;
    const int lk4 = log2_of(a.d_k / 4);
    copy_tile(kt, ldk, k + ((size_t)kh * a.L + row0) * a.d_k, a.d_k, C, n, a.d_k, lk4);
    copy_tile(qt, ldk, q + ((size_t)kh * a.L + row0) * a.d_k, a.d_k, C, n, a.d_k, lk4);
    copies_sent();
    if (tid < 32) { // the running sums of g, two tokens a lane
        const size_t t0 = (size_t)bh * a.L + row0;
        float x[2], be[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * tid + e;
            x[e] = i < n ? io<float>::load(g + t0 + i) : 0.f;
            x[e] = x[e] < kGMin ? kGMin : x[e];
            be[e] = i < n ? io<float>::load(beta + t0 + i) : 0.f;
        }
        Pair run, all;
        running_sum(x, tid, run, all);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const Pair G = e ? run : add(run, {-x[1], 0.f});
            float *d = tok + (2 * tid + e) * TOK;
            d[2] = expf(G.hi);
            d[3] = expf((all.hi - G.hi) + (all.lo - G.lo));
            d[4] = G.hi;
            d[5] = G.lo;
            d[6] = be[e];
            d[7] = 0.f;
        }
    }
    copies_done<0>();
    __syncthreads();
    { // 1 / length of each key and query (0 for a row of zeros): two lanes a row, every other 16 bytes
        const int row = tid >> 1;
        const float *x = (row < C ? kt : qt) + (row & 63) * ldk + 4 * (tid & 1);
        float ss = 0.f;
        for (int m = 0; m < a.d_k; m += 8) {
            const float4 t = lds4(x + m);
            ss = fmaf(t.x, t.x, fmaf(t.y, t.y, fmaf(t.z, t.z, fmaf(t.w, t.w, ss))));
        }
        ss += __shfl_xor_sync(0xffffffffu, ss, 1);
        ss += a.eps;
        if ((tid & 1) == 0)
            tok[(row & 63) * TOK + (row >> 6)] = !a.l2norm ? 1.f : ss > 0.f ? 1.f / sqrtf(ss) : ss;
    }
    __syncthreads();
    const size_t ch = (size_t)bh * gridDim.x + c;
    {
        const int ti = (tid & 7) + 8 * ((tid >> 5) & 1), tj = ((tid >> 3) & 3) + 4 * (tid >> 6);
        float akk[4][4] = {}, aqk[4][4] = {};
        mm_nt<4, 4>(akk, kt + ti * ldk, ldk, 16, kt + tj * ldk, ldk, 16, a.d_k);
        mm_nt<4, 4>(aqk, qt + ti * ldk, ldk, 16, kt + tj * ldk, ldk, 16, a.d_k);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int i = ti + 16 * r, j = tj + 16 * s;
                const float *di = tok + i * TOK, *dj = tok + j * TOK;
                const float D = j <= i ? expf((di[4] - dj[4]) + (di[5] - dj[5])) : 0.f;
                At[i * LC + j] = j < i ? di[6] * D * di[0] * dj[0] * akk[r][s] : 0.f;
                ws.M[ch * C * C + i * C + j] = j <= i ? a.scale * D * di[1] * dj[0] * aqk[r][s] : 0.f;
            }
    }
    __syncthreads();
    unit_lower_inverse(At, Tt, tmp);
    for (int e = tid; e < C * C; e += NT)
        ws.T[ch * C * C + e] = Tt[(e >> 6) * LC + (e & 63)];
    for (int e = tid; e < C * TOK; e += NT)
        ws.tok[ch * C * TOK + e] = tok[e];
}

// A walk CTA's channels: 32, or 16 where that still leaves SMs idle (the work
// of a chunk is what a chunk takes then; B1 H4 L333 d 64: 61 us with
// 32, 50 with 16).  A thread's rows of a tile are ti + S r (S = 64 / R, R rows of
// each 64) and its columns 4 tj ..; a warp covers 8 rows by 4 column groups, so
// that both operands' 16-byte reads are one wavefront each (32 rows a warp took
// four for one of them).
template <int NV> struct Tile {
    static constexpr int R = NV / 16, S = C / R, LV = NV + 4, LOG4 = NV == 32 ? 3 : 2;
    static FW_DEV int row(int tid) { return (tid & 7) + 8 * ((tid >> 5) & (8 / R - 1)); }
    static FW_DEV int column(int tid) { return ((tid >> 3) & 3) + 4 * ((tid >> 5) / (8 / R)); }
};

// Z[n][k] <- whole Z[n][k] + sum_t A[t][n] B[t][k] (+ the same of A2, B2):
// the state's 32 x d_k, four rows and four columns a thread.
template <int NV>
FW_DEV void update_state(float *Z, int ldk, float whole, const float *A, const float *B, const float *A2,
                         const float *B2, int d_k) {
    const int kg = d_k / 4, k4 = (threadIdx.x % kg) * 4, n0 = (threadIdx.x / kg) * 4;
    if (n0 >= NV)
        return;
    float s[4][4] = {};
    Columns<4> sums(s);
    for (int src = 0; src < (A2 ? 2 : 1); ++src) {
        const float *a = (src ? A2 : A) + n0, *b = (src ? B2 : B) + k4;
#pragma unroll 4
        for (int t = 0; t < C; ++t) {
            const float4 x = lds4(a + t * Tile<NV>::LV);
            const Quad y = ldq(b + t * ldk);
            sums.add(0, x.x, y);
            sums.add(1, x.y, y);
            sums.add(2, x.z, y);
            sums.add(3, x.w, y);
        }
    }
    sums.get(s);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        float *p = Z + (n0 + r) * ldk + k4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            p[e] = fmaf(whole, p[e], s[r][e]);
    }
}

// ------------------------------------------------------------------ walk
// One CTA per (value head, NV value channels).  A chunk's keys, queries,
// values and scalars are copied a chunk ahead into a second buffer, T and M as
// soon as the chunk before has used its own.  KEEP: the chunks' first states
// and U stay in the workspace for the gradients (no answers then).
template <bool KEEP, int NV>
__global__ void __launch_bounds__(NT)
    gated_walk_kernel(GatedArgs a, const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
                      const float *__restrict__ W0, float *__restrict__ Wf, float *__restrict__ y, Ws ws) {
    using W = Tile<NV>;
    constexpr int R = W::R, LV = W::LV;
    extern __shared__ __align__(16) float sm[];
    const int ldk = a.d_k + 4, nC = (a.L + C - 1) / C, lk4 = log2_of(a.d_k / 4), ahead = 2 * C * ldk + C * LV + C * TOK;
    float *S = sm, *Tt = S + NV * ldk, *Mt = Tt + C * LC, *Ut = Mt + C * LC, *buf = Ut + C * LV; // buf: K, Q, V, tok; twice
    const int tid = threadIdx.x, ti = W::row(tid), tj = W::column(tid), bh = blockIdx.y, n0 = blockIdx.x * NV;
    const int b = bh / a.H, kh = b * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const int nv = min(NV, a.d_v - n0);
    griddep_launch_dependents();
    griddep_wait();
    q = after_wait(q);
    k = after_wait(k);
    v = after_wait(v);
    W0 = after_wait(W0);
    const int len = seq_len(a, b), nch = (len + C - 1) / C;
    const size_t st0 = ((size_t)bh * a.d_v + n0) * a.d_k;
    auto fetch = [&](int c) {
        float *p = buf + (c & 1) * ahead;
        const int n = min(C, len - c * C);
        const size_t t0 = (size_t)c * C, krow = ((size_t)kh * a.L + t0) * a.d_k;
        copy_tile(p, ldk, k + krow, a.d_k, C, n, a.d_k, lk4);
        if (!KEEP)
            copy_tile(p + C * ldk, ldk, q + krow, a.d_k, C, n, a.d_k, lk4);
        copy_tile(p + 2 * C * ldk, LV, v + ((size_t)bh * a.L + t0) * a.d_v + n0, a.d_v, C, n, nv, W::LOG4);
        copy_tile(p + 2 * C * ldk + C * LV, TOK, ws.tok + ((size_t)bh * nC + c) * C * TOK, TOK, C, C, TOK, 1);
    };
    auto fetch_sq = [&](float *dst, const float *src, int c) {
        copy_tile(dst, LC, src + ((size_t)bh * nC + c) * C * C, C, C, C, C, 4);
    };
    load_tile(S, ldk, W0 + st0, a.d_k, NV, W0 ? nv : 0, a.d_k, a.d_k);
    if (nch > 0) {
        fetch(0);
        fetch_sq(Tt, ws.T, 0);
        if (!KEEP)
            fetch_sq(Mt, ws.M, 0);
    }
    copies_sent();
    for (int c = 0; c < nch; ++c) {
        const int n = min(C, len - c * C);
        const size_t ch = (size_t)bh * nC + c, vrow = ((size_t)bh * a.L + (size_t)c * C) * a.d_v + n0;
        float *kq = buf + (c & 1) * ahead, *Xt = kq + 2 * C * ldk, *tok = Xt + C * LV;
        copies_done<0>();
        __syncthreads(); // this chunk is here, and the last one's buffers are free
        if (c + 1 < nch)
            fetch(c + 1);
        if (KEEP)
            for (int e = tid; e < nv << lk4; e += NT)
                *reinterpret_cast<float4 *>(ws.S + ch * a.d_v * a.d_k + (size_t)n0 * a.d_k + 4 * e) =
                    lds4(S + (e >> lk4) * ldk + (e & ((1 << lk4) - 1)) * 4);
        float acc[2 * R][4] = {}; // rows of K, then of Q
        if (KEEP) {
            float pk[R][4] = {};
            mm_nt<R, 4>(pk, kq + ti * ldk, ldk, W::S, S + tj * 4 * ldk, ldk, 1, a.d_k);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    acc[r][s] = pk[r][s];
        } else {
            mm_nt<2 * R, 4>(acc, kq + ti * ldk, ldk, W::S, S + tj * 4 * ldk, ldk, 1, a.d_k);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float *d = tok + (ti + W::S * r) * TOK;
            float *x = Xt + (ti + W::S * r) * LV + tj * 4;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                x[s] = d[6] * (x[s] - d[2] * d[0] * acc[r][s]);
        }
        __syncthreads();
        float u[R][4] = {};
        mm_nn<R>(u, Tt + ti * LC, LC, W::S, Xt + tj * 4, LV, C);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = ti + W::S * r;
            *reinterpret_cast<float4 *>(Ut + i * LV + tj * 4) = make_float4(u[r][0], u[r][1], u[r][2], u[r][3]);
            if (KEEP && tj * 4 < nv)
                *reinterpret_cast<float4 *>(ws.U + (ch * C + i) * a.d_v + n0 + tj * 4) =
                    make_float4(u[r][0], u[r][1], u[r][2], u[r][3]);
        }
        __syncthreads();
        if (c + 1 < nch)
            fetch_sq(Tt, ws.T, c + 1);
        if (!KEEP) {
            float o[R][4];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float *d = tok + (ti + W::S * r) * TOK;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    o[r][s] = a.scale * d[2] * d[1] * acc[R + r][s];
            }
            mm_nn<R>(o, Mt + ti * LC, LC, W::S, Ut + tj * 4, LV, C);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (ti + W::S * r < n && tj * 4 < nv)
                    *reinterpret_cast<float4 *>(y + vrow + (size_t)(ti + W::S * r) * a.d_v + tj * 4) =
                        make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
            __syncthreads();
            if (c + 1 < nch)
                fetch_sq(Mt, ws.M, c + 1);
        }
        copies_sent();
        // rows of U weighted for the state, where X was
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = ti + W::S * r;
            const float f = tok[i * TOK + 3] * tok[i * TOK];
            *reinterpret_cast<float4 *>(Xt + i * LV + tj * 4) =
                make_float4(f * u[r][0], f * u[r][1], f * u[r][2], f * u[r][3]);
        }
        __syncthreads();
        update_state<NV>(S, ldk, tok[(C - 1) * TOK + 2], Xt, kq, nullptr, nullptr, a.d_k);
    }
    copies_done<0>();
    __syncthreads();
    if (!KEEP) {
        if (Wf)
            for (int e = tid; e < nv * a.d_k; e += NT)
                Wf[st0 + e] = S[(e / a.d_k) * ldk + e % a.d_k];
        for (size_t e = tid; e < (size_t)(a.L - len) * nv; e += NT) // no token, no answer
            y[((size_t)bh * a.L + len + e / nv) * a.d_v + n0 + e % nv] = 0.f;
    }
}

// ---------------------------------------------------------- reverse walk
template <int NV>
__global__ void __launch_bounds__(NT)
    gated_reverse_kernel(GatedArgs a, const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ dy,
                         const float *__restrict__ dWf, float *__restrict__ dW0, Ws ws) {
    using W = Tile<NV>;
    constexpr int R = W::R, LV = W::LV;
    extern __shared__ __align__(16) float sm[];
    const int ldk = a.d_k + 4, nC = (a.L + C - 1) / C, lk4 = log2_of(a.d_k / 4), ahead = 2 * C * ldk + C * LV + C * TOK;
    float *D = sm, *Tt = D + NV * ldk, *Mt = Tt + C * LC, *Ut = Mt + C * LC, *buf = Ut + C * LV; // buf: K, Q, dY, tok; twice
    const int tid = threadIdx.x, ti = W::row(tid), tj = W::column(tid), bh = blockIdx.y, n0 = blockIdx.x * NV;
    const int b = bh / a.H, kh = b * a.Hk + (bh % a.H) / (a.H / a.Hk);
    const int nv = min(NV, a.d_v - n0);
    griddep_launch_dependents();
    griddep_wait();
    q = after_wait(q);
    k = after_wait(k);
    dy = after_wait(dy);
    dWf = after_wait(dWf);
    const int len = seq_len(a, b), nch = (len + C - 1) / C;
    const size_t st0 = ((size_t)bh * a.d_v + n0) * a.d_k;
    auto fetch = [&](int c) {
        float *p = buf + (c & 1) * ahead;
        const int n = min(C, len - c * C);
        const size_t t0 = (size_t)c * C, krow = ((size_t)kh * a.L + t0) * a.d_k;
        copy_tile(p, ldk, k + krow, a.d_k, C, n, a.d_k, lk4);
        copy_tile(p + C * ldk, ldk, q + krow, a.d_k, C, n, a.d_k, lk4);
        copy_tile(p + 2 * C * ldk, LV, dy + ((size_t)bh * a.L + t0) * a.d_v + n0, a.d_v, C, n, nv, W::LOG4);
        copy_tile(p + 2 * C * ldk + C * LV, TOK, ws.tok + ((size_t)bh * nC + c) * C * TOK, TOK, C, C, TOK, 1);
    };
    auto fetch_sq = [&](float *dst, const float *src, int c) {
        copy_tile(dst, LC, src + ((size_t)bh * nC + c) * C * C, C, C, C, C, 4);
    };
    load_tile(D, ldk, dWf + st0, a.d_k, NV, dWf ? nv : 0, a.d_k, a.d_k);
    if (nch > 0) {
        fetch(nch - 1);
        fetch_sq(Tt, ws.T, nch - 1);
        fetch_sq(Mt, ws.M, nch - 1);
    }
    copies_sent();
    for (int c = nch - 1; c >= 0; --c) {
        const size_t ch = (size_t)bh * nC + c;
        float *kq = buf + (c & 1) * ahead, *Yt = kq + 2 * C * ldk, *tok = Yt + C * LV;
        copies_done<0>();
        __syncthreads(); // this chunk is here, and the last one's buffers are free
        if (c > 0)
            fetch(c - 1);
        for (int e = tid; e < nv << lk4; e += NT)
            *reinterpret_cast<float4 *>(ws.dS + ch * a.d_v * a.d_k + (size_t)n0 * a.d_k + 4 * e) =
                lds4(D + (e >> lk4) * ldk + (e & ((1 << lk4) - 1)) * 4);
        float u[R][4] = {};
        mm_nt<R, 4>(u, kq + ti * ldk, ldk, W::S, D + tj * 4 * ldk, ldk, 1, a.d_k);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float *d = tok + (ti + W::S * r) * TOK;
#pragma unroll
            for (int s = 0; s < 4; ++s)
                u[r][s] *= d[3] * d[0];
        }
        mm_tn<R>(u, Mt + ti, LC, W::S, Yt + tj * 4, LV, C);
#pragma unroll
        for (int r = 0; r < R; ++r)
            *reinterpret_cast<float4 *>(Ut + (ti + W::S * r) * LV + tj * 4) =
                make_float4(u[r][0], u[r][1], u[r][2], u[r][3]);
        __syncthreads();
        if (c > 0)
            fetch_sq(Mt, ws.M, c - 1);
        float x[R][4] = {};
        mm_tn<R>(x, Tt + ti, LC, W::S, Ut + tj * 4, LV, C);
        __syncthreads();
        if (c > 0)
            fetch_sq(Tt, ws.T, c - 1);
        copies_sent();
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = ti + W::S * r;
            const float *d = tok + i * TOK;
            if (tj * 4 < nv)
                *reinterpret_cast<float4 *>(ws.dX + (ch * C + i) * a.d_v + n0 + tj * 4) =
                    make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
            const float wx = -d[6] * d[2] * d[0], wy = a.scale * d[2] * d[1];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                Ut[i * LV + tj * 4 + s] = wx * x[r][s];
                Yt[i * LV + tj * 4 + s] *= wy;
            }
        }
        __syncthreads();
        update_state<NV>(D, ldk, tok[(C - 1) * TOK + 2], Ut, kq, Yt, kq + C * ldk, a.d_k);
    }
    copies_done<0>();
    __syncthreads();
    if (dW0)
        for (int e = tid; e < nv * a.d_k; e += NT)
            dW0[st0 + e] = D[(e / a.d_k) * ldk + e % a.d_k];
}

// ------------------------------------------------------------------ grad
// One CTA per (chunk, key head); a warp owns 8 tokens (rows 8 w .. 8 w + 7)
// and a lane 4 key channels, so every dot product over the key channels is
// one warp reduction.
__global__ void __launch_bounds__(NT)
    gated_grad_kernel(GatedArgs a, const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
                      const float *__restrict__ dy, float *__restrict__ dq, float *__restrict__ dk, float *__restrict__ dv,
                      float *__restrict__ dg, float *__restrict__ dbeta, Ws ws) {
    extern __shared__ __align__(16) float sm[];
    const int ldk = a.d_k + 4, nC = gridDim.x, lv = NV + 4;
    float *kt = sm, *qt = kt + C * ldk, *accq = qt + C * ldk, *acck = accq + C * a.d_k, *S0 = acck + C * a.d_k,
          *S1 = S0 + NV * ldk, *Yt = S1 + NV * ldk, *Xt = Yt + C * lv, *Ut = Xt + C * lv, *Et = Ut + C * lv,
          *Ft = Et + C * LC, *tok = Ft + C * LC, *red = tok + C * TOK; // red: R [C], W [C], pairs across [C], <S, dS'> per warp [8]
    float *Pt = Yt; // (after the slices)
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, c = blockIdx.x, bk = blockIdx.y;
    const int b = bk / a.Hk, grp = a.H / a.Hk, i0 = 8 * w, kc = 4 * lane;
    const bool on = kc < a.d_k;
    griddep_launch_dependents();
    griddep_wait();
    q = after_wait(q);
    k = after_wait(k);
    v = after_wait(v);
    dy = after_wait(dy);
    const int n = min(C, seq_len(a, b) - c * C);
    const size_t krow = ((size_t)bk * a.L + (size_t)c * C) * a.d_k;
    const int rows = min(C, a.L - c * C); // rows that exist in memory
    if (n <= 0) { // behind the sequence's end: no gradient
        for (int e = tid; e < rows * a.d_k; e += NT) {
            io<float>::store(dq + krow + e, 0.f);
            io<float>::store(dk + krow + e, 0.f);
        }
        for (int m = 0; m < grp; ++m) {
            const size_t r0 = (size_t)(bk * grp + m) * a.L + (size_t)c * C;
            for (int e = tid; e < rows * a.d_v; e += NT)
                io<float>::store(dv + r0 * a.d_v + e, 0.f);
            for (int e = tid; e < rows; e += NT) {
                io<float>::store(dg + r0 + e, 0.f);
                io<float>::store(dbeta + r0 + e, 0.f);
            }
        }
        return;
    }
    load_tile(kt, ldk, k + krow, a.d_k, C, n, a.d_k, a.d_k);
    load_tile(qt, ldk, q + krow, a.d_k, C, n, a.d_k, a.d_k);
    for (int m = 0; m < grp; ++m) {
        const int bh = bk * grp + m;
        const size_t ch = (size_t)bh * nC + c, r0 = (size_t)bh * a.L + (size_t)c * C;
        __syncthreads();
        for (int e = tid; e < C * TOK; e += NT)
            tok[e] = __ldcg(ws.tok + ch * C * TOK + e);
        __syncthreads();
        if (m == 0) { // unit keys and queries (the same for every value head)
            for (int e = tid; e < C * a.d_k; e += NT) {
                const int i = e / a.d_k, x = i * ldk + e % a.d_k;
                kt[x] *= tok[i * TOK];
                qt[x] *= tok[i * TOK + 1];
                accq[e] = acck[e] = 0.f;
            }
        }
        float aq[8][4] = {}, ah[8][4] = {}, aw[8][4] = {}; // rows i0 + r, channels kc ..
        float e_[4][4] = {}, f_[4][4] = {};               // E, F: rows (tid & 15) + 16 r, columns (tid >> 4) + 16 s
        float xv[8] = {}, ss = 0.f;                        // dX_i . V_i (this lane's share), <S, dS'>
        const int ei = tid & 15, ej = tid >> 4;
        for (int n0 = 0; n0 < a.d_v; n0 += NV) {
            const int nv = min(NV, a.d_v - n0);
            __syncthreads();
            load_tile(S0, ldk, ws.S + ch * a.d_v * a.d_k + (size_t)n0 * a.d_k, a.d_k, NV, nv, a.d_k, a.d_k);
            load_tile(S1, ldk, ws.dS + ch * a.d_v * a.d_k + (size_t)n0 * a.d_k, a.d_k, NV, nv, a.d_k, a.d_k);
            load_tile(Yt, lv, dy + r0 * a.d_v + n0, a.d_v, C, n, nv, NV);
            load_tile(Xt, lv, ws.dX + ch * C * a.d_v + n0, a.d_v, C, n, nv, NV);
            load_tile(Ut, lv, ws.U + ch * C * a.d_v + n0, a.d_v, C, n, nv, NV);
            __syncthreads();
            if (on) {
                mm_nn<8>(aq, Yt + i0 * lv, lv, 1, S0 + kc, ldk, NV);
                mm_nn<8>(ah, Xt + i0 * lv, lv, 1, S0 + kc, ldk, NV);
                mm_nn<8>(aw, Ut + i0 * lv, lv, 1, S1 + kc, ldk, NV);
            }
            mm_nt<4, 4>(e_, Yt + ei * lv, lv, 16, Ut + ej * lv, lv, 16, NV);
            mm_nt<4, 4>(f_, Xt + ei * lv, lv, 16, Ut + ej * lv, lv, 16, NV);
            for (int e = tid; e < NV * a.d_k; e += NT) {
                const int x = (e / a.d_k) * ldk + e % a.d_k;
                ss = fmaf(S0[x], S1[x], ss);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int i = i0 + r;
                if (i < n && lane < nv) {
                    const size_t at = (r0 + i) * a.d_v + n0 + lane;
                    const float x = Xt[i * lv + lane];
                    xv[r] = fmaf(x, io<float>::load(v + at), xv[r]);
                    io<float>::store(dv + at, tok[i * TOK + 6] * x);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int i = ei + 16 * r, j = ej + 16 * s;
                const float *di = tok + i * TOK, *dj = tok + j * TOK;
                const float Dd = j <= i ? expf((di[4] - dj[4]) + (di[5] - dj[5])) : 0.f;
                e_[r][s] = j <= i ? a.scale * Dd * e_[r][s] : 0.f;
                f_[r][s] = j < i ? Dd * f_[r][s] : 0.f;
                Et[i * LC + j] = e_[r][s];
                Ft[i * LC + j] = f_[r][s];
            }
        { // P, from the unit keys' and queries' products
            float x[4][4] = {};
            mm_nt<4, 4>(x, qt + ei * ldk, ldk, 16, kt + ej * ldk, ldk, 16, a.d_k);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    e_[r][s] = ej + 16 * s < ei + 16 * r ? e_[r][s] * x[r][s] : 0.f;
                    x[r][s] = 0.f;
                }
            mm_nt<4, 4>(x, kt + ei * ldk, ldk, 16, kt + ej * ldk, ldk, 16, a.d_k);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int i = ei + 16 * r, j = ej + 16 * s;
                    Pt[i * LC + j] = j < i ? fmaf(-tok[i * TOK + 6] * f_[r][s], x[r][s], e_[r][s]) : 0.f;
                }
        }
        ss = warp_sum(ss);
        if (lane == 0)
            red[3 * C + w] = ss;
        __syncthreads();
        { // the pairs across each token: columns' sums over the rows from it on, eight tokens a warp
            float c0 = 0.f, c1 = 0.f;
            for (int i = i0 + 8; i < C; ++i) {
                c0 += Pt[i * LC + lane];
                c1 += Pt[i * LC + lane + 32];
            }
            for (int t = i0 + 7; t >= i0; --t) {
                c0 += Pt[t * LC + lane];
                c1 += Pt[t * LC + lane + 32];
                const float s = warp_sum((lane < t ? c0 : 0.f) + (lane + 32 < t ? c1 : 0.f));
                if (lane == 0)
                    red[2 * C + t] = s;
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) { // R and W
            const float *d = tok + (i0 + r) * TOK;
            float ra = 0.f, rw = 0.f;
            if (on) {
                const float4 kk = lds4(kt + (i0 + r) * ldk + kc), qq = lds4(qt + (i0 + r) * ldk + kc);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    aq[r][e] *= a.scale * d[2];
                    ah[r][e] *= d[2];
                    aw[r][e] *= d[3];
                }
                ra = (qq.x * aq[r][0] + qq.y * aq[r][1] + qq.z * aq[r][2] + qq.w * aq[r][3]) -
                     d[6] * (kk.x * ah[r][0] + kk.y * ah[r][1] + kk.z * ah[r][2] + kk.w * ah[r][3]);
                rw = kk.x * aw[r][0] + kk.y * aw[r][1] + kk.z * aw[r][2] + kk.w * aw[r][3];
            }
            ra = warp_sum(ra);
            rw = warp_sum(rw);
            if (lane == 0) {
                red[i0 + r] = ra;
                red[C + i0 + r] = rw;
            }
        }
        if (on) {
            mm_nn<8>(aq, Et + i0 * LC, LC, 1, kt + kc, ldk, C);
            mm_nn<8>(ah, Ft + i0 * LC, LC, 1, kt + kc, ldk, C);
            mm_tn<8>(aw, Et + i0, LC, 1, qt + kc, ldk, C);
        }
        __syncthreads();
        for (int e = tid; e < C * C; e += NT)
            Ft[(e >> 6) * LC + (e & 63)] *= -tok[(e >> 6) * TOK + 6];
        __syncthreads();
        if (on)
            mm_tn<8>(aw, Ft + i0, LC, 1, kt + kc, ldk, C);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int i = i0 + r;
            const float be = tok[i * TOK + 6];
            float kh = 0.f;
            if (on) {
                const float4 kk = lds4(kt + i * ldk + kc);
                kh = kk.x * ah[r][0] + kk.y * ah[r][1] + kk.z * ah[r][2] + kk.w * ah[r][3];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    accq[i * a.d_k + kc + e] += aq[r][e];
                    acck[i * a.d_k + kc + e] += aw[r][e] - be * ah[r][e];
                }
            }
            kh = warp_sum(kh);
            const float xvs = warp_sum(xv[r]);
            if (lane == 0 && i < n)
                io<float>::store(dbeta + r0 + i, xvs - kh);
        }
        __syncthreads();
        if (tid < 32) { // dg, two tokens a lane
            float z = 0.f;
            for (int x = 0; x < 8; ++x)
                z += red[3 * C + x];
            float x[2];
            gated_decay_grads(tok[(C - 1) * TOK + 2] * z, red + 2 * lane, red + C + 2 * lane, red + 2 * C + 2 * lane, lane, x);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (2 * lane + e < n)
                    io<float>::store(dg + r0 + 2 * lane + e, x[e]);
        }
        for (int e = n * a.d_v + tid; e < rows * a.d_v; e += NT)
            io<float>::store(dv + r0 * a.d_v + e, 0.f);
        for (int i = n + tid; i < rows; i += NT) {
            io<float>::store(dg + r0 + i, 0.f);
            io<float>::store(dbeta + r0 + i, 0.f);
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        const int i = i0 + r;
        if (i >= rows)
            break;
        float4 kk = make_float4(0, 0, 0, 0), qq = kk, gk = kk, gq = kk;
        if (on) {
            kk = lds4(kt + i * ldk + kc);
            qq = lds4(qt + i * ldk + kc);
            gk = lds4(acck + i * a.d_k + kc);
            gq = lds4(accq + i * a.d_k + kc);
        }
        float pk = 0.f, pq = 0.f;
        if (a.l2norm) {
            pk = warp_sum(kk.x * gk.x + kk.y * gk.y + kk.z * gk.z + kk.w * gk.w);
            pq = warp_sum(qq.x * gq.x + qq.y * gq.y + qq.z * gq.z + qq.w * gq.w);
        }
        if (on) {
            const float rk = i < n ? tok[i * TOK] : 0.f, rq = i < n ? tok[i * TOK + 1] : 0.f;
            float *ok = dk + krow + (size_t)i * a.d_k + kc, *oq = dq + krow + (size_t)i * a.d_k + kc;
            io<float>::store(ok, rk * (gk.x - kk.x * pk));
            io<float>::store(ok + 1, rk * (gk.y - kk.y * pk));
            io<float>::store(ok + 2, rk * (gk.z - kk.z * pk));
            io<float>::store(ok + 3, rk * (gk.w - kk.w * pk));
            io<float>::store(oq, rq * (gq.x - qq.x * pq));
            io<float>::store(oq + 1, rq * (gq.y - qq.y * pq));
            io<float>::store(oq + 2, rq * (gq.z - qq.z * pq));
            io<float>::store(oq + 3, rq * (gq.w - qq.w * pq));
        }
    }
}

size_t prep_smem(int d_k) { return sizeof(float) * (2 * C * (d_k + 4) + 2 * C * LC + 1024 + C * TOK); }
size_t walk_smem(int d_k, int nv) {
    return sizeof(float) *
           (nv * (d_k + 4) + 2 * C * LC + C * (nv + 4) + 2 * (2 * C * (d_k + 4) + C * (nv + 4) + C * TOK));
}
// Channels per walk CTA (see Tile).
cudaError_t walk_channels(const GatedArgs &a, int *nv) {
    int sms = 0;
    const cudaError_t e = device_sms(&sms);
    *nv = 2 * (int64_t)a.B * a.H * ((a.d_v + 31) / 32) <= sms ? 16 : 32;
    return e;
}
size_t grad_smem(int d_k) {
    return sizeof(float) * (2 * (C + NV) * (d_k + 4) + 2 * C * d_k + 3 * C * (NV + 4) + 2 * C * LC + C * TOK + 3 * C + 8);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_smem(void (*kern)(KArgs...), std::atomic<uint64_t> &allowed, dim3 grid, size_t smem, cudaStream_t st,
                        Args... args) {
    const cudaError_t e = allow_smem(kern, allowed);
    return e != cudaSuccess ? e : launch_pdl(kern, grid, dim3(NT), smem, st, args...);
}

template <bool KEEP, int NV>
cudaError_t launch_walk(const GatedArgs &a, const float *q, const float *k, const float *v, const float *W0, float *Wf,
                        float *y, const Ws &ws, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    return launch_smem(gated_walk_kernel<KEEP, NV>, allowed, dim3((a.d_v + NV - 1) / NV, a.B * a.H),
                       walk_smem(a.d_k, NV), st, a, q, k, v, W0, Wf, y, ws);
}
template <int NV>
cudaError_t launch_reverse(const GatedArgs &a, const float *q, const float *k, const float *dy, const float *dWf,
                           float *dW0, const Ws &ws, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    return launch_smem(gated_reverse_kernel<NV>, allowed, dim3((a.d_v + NV - 1) / NV, a.B * a.H), walk_smem(a.d_k, NV),
                       st, a, q, k, dy, dWf, dW0, ws);
}

cudaError_t prepare_f32(const GatedArgs &a, const float *q, const float *k, const float *g, const float *beta,
                        const Ws &ws, cudaStream_t st) {
    static std::atomic<uint64_t> allowed{0};
    return launch_smem(gated_prep_kernel, allowed, dim3((a.L + C - 1) / C, a.B * a.H), prep_smem(a.d_k), st, a, q, k, g,
                       beta, ws);
}

cudaError_t forward_f32(const GatedArgs &a, const float *q, const float *k, const float *v, const float *g,
                        const float *beta, const float *W0, float *Wf, float *y, void *workspace, cudaStream_t st) {
    const Ws ws = ws_at(workspace, ws_off(a.B * a.H, a.L, a.d_k, a.d_v, false));
    int nv = 0;
    cudaError_t e = walk_channels(a, &nv);
    if (e == cudaSuccess)
        e = prepare_f32(a, q, k, g, beta, ws, st);
    if (e != cudaSuccess)
        return e;
    return nv == 16 ? launch_walk<false, 16>(a, q, k, v, W0, Wf, y, ws, st)
                    : launch_walk<false, 32>(a, q, k, v, W0, Wf, y, ws, st);
}

cudaError_t backward_f32(const GatedArgs &a, const float *q, const float *k, const float *v, const float *g,
                         const float *beta, const float *W0, const float *dy, const float *dWf, float *dq, float *dk,
                         float *dv, float *dg, float *dbeta, float *dW0, void *workspace, cudaStream_t st) {
    const Ws ws = ws_at(workspace, ws_off(a.B * a.H, a.L, a.d_k, a.d_v, true));
    int nv = 0;
    cudaError_t e = walk_channels(a, &nv);
    if (e == cudaSuccess)
        e = prepare_f32(a, q, k, g, beta, ws, st);
    if (e == cudaSuccess)
        e = nv == 16 ? launch_walk<true, 16>(a, q, k, v, W0, nullptr, nullptr, ws, st)
                     : launch_walk<true, 32>(a, q, k, v, W0, nullptr, nullptr, ws, st);
    if (e == cudaSuccess)
        e = nv == 16 ? launch_reverse<16>(a, q, k, dy, dWf, dW0, ws, st)
                     : launch_reverse<32>(a, q, k, dy, dWf, dW0, ws, st);
    if (e != cudaSuccess)
        return e;
    static std::atomic<uint64_t> allowed{0};
    return launch_smem(gated_grad_kernel, allowed, dim3((a.L + C - 1) / C, a.B * a.Hk), grad_smem(a.d_k), st, a, q, k, v,
                       dy, dq, dk, dv, dg, dbeta, ws);
}

} // namespace

size_t gated_forward_workspace_bytes(int B, int H, int L, int d_k, int d_v, int bf16) {
    if (bf16) {
        const GatedRecord r = gated_forward_record(L, d_k, d_v); // and the state between two segments
        return (size_t)B * H * (r.nch * r.bytes + sizeof(float) * d_v * d_k);
    }
    return sizeof(float) * ws_off(B * H, L, d_k, d_v, false).end;
}
size_t gated_backward_workspace_bytes(int B, int H, int L, int d_k, int d_v, int bf16) {
    if (bf16) {
        const GatedRecord r = gated_backward_record(L, d_k, d_v);
        return (size_t)B * H * r.nch * r.bytes;
    }
    return sizeof(float) * ws_off(B * H, L, d_k, d_v, true).end;
}

cudaError_t launch_gated_forward(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                                 const void *beta, const float *W0, float *Wf, void *y, void *workspace, int bf16,
                                 cudaStream_t st) {
    if (bf16)
        return gated_tc_forward(a, q, k, v, g, beta, W0, Wf, y, workspace, st);
    auto f = [](const void *p) { return static_cast<const float *>(p); };
    return forward_f32(a, f(q), f(k), f(v), f(g), f(beta), W0, Wf, static_cast<float *>(y), workspace, st);
}

cudaError_t launch_gated_backward(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                                  const void *beta, const float *W0, const void *dy, const float *dWf, void *dq,
                                  void *dk, void *dv, void *dg, void *dbeta, float *dW0, void *workspace, int bf16,
                                  cudaStream_t st) {
    if (bf16) {
        const cudaError_t e = gated_tc_walks(a, q, k, v, g, beta, W0, dy, dWf, dW0, workspace, st);
        return e != cudaSuccess ? e : gated_tc_grad(a, v, dy, dq, dk, dv, dg, dbeta, workspace, st);
    }
    auto f = [](const void *p) { return static_cast<const float *>(p); };
    auto o = [](void *p) { return static_cast<float *>(p); };
    return backward_f32(a, f(q), f(k), f(v), f(g), f(beta), W0, f(dy), dWf, o(dq), o(dk), o(dv), o(dg), o(dbeta), dW0,
                        workspace, st);
}

} // namespace fw
