// fw_vocab_f32.cu -- the vocabulary loss of fp32 answers and an fp32 output map,
// and its gradients: the products in fp32 arithmetic on CUDA cores (the formulas
// stand at the head of fw_vocab.cu).
//
// Bound by the fp32 rate.  One kernel forms 128 x 128 tiles of every product, a
// CTA of 256 threads with 8 x 8 sums each as pairs of floats; the contraction goes
// by steps of 16 through two stages of shared memory, the next step's values on
// their way in registers meanwhile.  An operand whose memory runs along the
// contraction is transposed on its way into shared memory, one that runs along the
// output is copied.  A sum of more than 512 terms goes by chunks of so many, added to
// totals in shared memory (LONG): one sum over 16 384 equal channels was off by 2.4e-4 of
// itself, and the gradients at 8192 x 50 001 by 2.8e-6 instead of 4.2e-7; chunks of 256 leave
// 3.4e-7.  The totals cost 1 % of the gradients' time and 6 % of the loss's (4096 x 20 001,
// D 1024: 3.06 ms, 3.23).  The softmax's gradient g is kept in fp32, in pieces of the
// vocabulary; a contraction is split where the tiles are few, and the splits' sums
// are added in order.
#include "fw_vocab.h"

#include <algorithm>

namespace fw {
namespace vocab {

namespace {

constexpr int kT = 256, kTile = 128, kStep = 16, kLd = kTile + 4;
constexpr int kChunk = 32;               // steps of a chunk
constexpr int kTotalBytes = kT * 64 * 4; // the chunks' totals, where there are several

enum Mode {
    kLoss, // h W^T: parts of the logits' log-sum-exp, the targets' logits
    kGrad, // h W^T: g
    kDh,   // g W
    kDw    // g^T h
};

struct Args {
    const float *A, *B;
    int64_t lda, ldb;
    int M, N, K;       // of the product, as far as they are there
    int mt, nt, per;   // tiles; steps of a split
    const float *bias; // kLoss, kGrad: of this piece, or null
    Tokens targets;    // kLoss
    int vocab, v0;     // all entries; the first of this piece
    float2 *part;
    float *target_z;
    const float4 *row; // (row_constants)
    const int *row_target;
    float *out;        // kGrad: g; kDh, kDw: the gradient, or [splits][M][N]
    int64_t ldo, a_split;
    int add;           // kDh: added to what is there
};

// Rows r0 .. r0 + 127, 16 of the contraction from k on, of an operand [rows][k]; 0 past either end.
FW_DEV void load_along(const float *p, int64_t ld, int rows, int K, int r0, int k, float4 (&v)[2]) {
    const int kk = k + 4 * (threadIdx.x & 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = r0 + (threadIdx.x >> 2) + 64 * i;
        v[i] = r < rows && kk < K ? __ldcg(reinterpret_cast<const float4 *>(p + r * ld + kk)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
FW_DEV void store_along(float (&s)[kStep][kLd], const float4 (&v)[2]) {
    const int kk = 4 * (threadIdx.x & 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = (threadIdx.x >> 2) + 64 * i;
        s[kk][r] = v[i].x;
        s[kk + 1][r] = v[i].y;
        s[kk + 2][r] = v[i].z;
        s[kk + 3][r] = v[i].w;
    }
}
// The same of an operand [k][columns]; `live` (or null): rows of it that count.
FW_DEV void load_across(const float *p, int64_t ld, int cols, int K, int c0, int k, const int *live, float4 (&v)[2]) {
    const int c = c0 + 4 * (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int kk = k + (threadIdx.x >> 5) + 8 * i;
        const bool here = kk < K && c < cols && (!live || __ldcg(live + kk) >= 0);
        v[i] = here ? __ldcg(reinterpret_cast<const float4 *>(p + kk * ld + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
FW_DEV void store_across(float (&s)[kStep][kLd], const float4 (&v)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        *reinterpret_cast<float4 *>(&s[(threadIdx.x >> 5) + 8 * i][4 * (threadIdx.x & 31)]) = v[i];
}

FW_DEV float over_row(float x, bool top) { // the maximum or the sum over a row's 16 threads
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        const float y = __shfl_xor_sync(0xffffffffu, x, o);
        x = top ? fmaxf(x, y) : x + y;
    }
    return x;
}

template <Mode MODE, bool LONG> __global__ void __launch_bounds__(kT, 2) vocab_f32_kernel(Args a) {
    __shared__ __align__(16) float As[2][kStep][kLd], Bs[2][kStep][kLd];
    extern __shared__ float4 total[]; // (LONG) [16][kT]: a thread's own
    griddep_launch_dependents();
    griddep_wait();
    a.A = after_wait(a.A);
    a.B = after_wait(a.B);
    a.bias = after_wait(a.bias);
    a.targets.p = after_wait(a.targets.p);
    a.row = after_wait(a.row);
    a.row_target = after_wait(a.row_target);
    a.out = after_wait(a.out);
    const int tiles = a.mt * a.nt, z = blockIdx.x / tiles, t = blockIdx.x - z * tiles;
    const int m0 = (t % a.mt) * kTile, n0 = (t / a.mt) * kTile;
    const int steps = (a.K + kStep - 1) / kStep, s0 = z * a.per, s1 = min(steps, s0 + a.per);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float4 va[2], vb[2];
    auto load = [&](int s) {
        if (MODE == kDw)
            load_across(a.A, a.lda, a.M, a.K, m0, s * kStep, nullptr, va);
        else
            load_along(a.A, a.lda, a.M, a.K, m0, s * kStep, va);
        if (MODE == kLoss || MODE == kGrad)
            load_along(a.B, a.ldb, a.N, a.K, n0, s * kStep, vb);
        else
            load_across(a.B, a.ldb, a.N, a.K, n0, s * kStep, MODE == kDw ? a.row_target : nullptr, vb);
    };
    auto store = [&](int b) {
        if (MODE == kDw)
            store_across(As[b], va);
        else
            store_along(As[b], va);
        if (MODE == kLoss || MODE == kGrad)
            store_along(Bs[b], vb);
        else
            store_across(Bs[b], vb);
    };
    // sums of rows 4 ty .. + 3 and 64 further, columns 4 tx .. + 3 and 64 further
    F2 acc[8][4];
    load(s0);
    store(0);
    __syncthreads();
    int c1;
    for (int c0 = s0; c0 < s1; c0 = c1) {
        c1 = LONG ? min(c0 + kChunk, s1) : s1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = F2{0};
        for (int s = c0; s < c1; ++s) {
            const int b = (s - s0) & 1;
            if (s + 1 < s1)
                load(s + 1);
#pragma unroll
            for (int k = 0; k < kStep; ++k) {
                const float4 a0 = *reinterpret_cast<const float4 *>(&As[b][k][4 * ty]);
                const float4 a1 = *reinterpret_cast<const float4 *>(&As[b][k][64 + 4 * ty]);
                const float4 b0 = *reinterpret_cast<const float4 *>(&Bs[b][k][4 * tx]);
                const float4 b1 = *reinterpret_cast<const float4 *>(&Bs[b][k][64 + 4 * tx]);
                const float x[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
                const F2 y[4] = {pack(b0.x, b0.y), pack(b0.z, b0.w), pack(b1.x, b1.y), pack(b1.z, b1.w)};
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = fma2(both(x[i]), y[j], acc[i][j]);
            }
            if (s + 1 < s1)
                store(b ^ 1);
            __syncthreads();
        }
        if (!LONG || s1 - s0 <= kChunk) // (the one chunk)
            break;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                float4 *const p = total + (2 * i + j / 2) * kT + threadIdx.x;
                if (c0 > s0) {
                    const float4 t = *p;
                    acc[i][j] = acc[i][j] + pack(t.x, t.y);
                    acc[i][j + 1] = acc[i][j + 1] + pack(t.z, t.w);
                }
                if (c1 < s1) {
                    const float2 u = unpack(acc[i][j]), v = unpack(acc[i][j + 1]);
                    *p = make_float4(u.x, u.y, v.x, v.y);
                }
            }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = m0 + 4 * ty + (i < 4 ? i : 60 + i);
        const bool here = row < a.M;
        int target = -1;
        float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
        if (here && MODE == kLoss)
            target = token_at(a.targets, row, a.vocab);
        if (here && MODE == kGrad) {
            target = __ldcg(a.row_target + row);
            c = __ldcg(a.row + row);
        }
        const bool dead = MODE == kDh && here && __ldcg(a.row_target + row) < 0; // (0 whatever W holds)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int col = n0 + 64 * half + 4 * tx;
            const float2 p = unpack(acc[i][2 * half]), q = unpack(acc[i][2 * half + 1]);
            float v[4] = {p.x, p.y, q.x, q.y};
            if (MODE == kLoss || MODE == kGrad) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = col + j < a.N ? v[j] + (a.bias ? __ldcg(a.bias + col + j) : 0.f) : -INFINITY;
            }
            if (MODE == kLoss) {
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (target == col + j && target < a.vocab) { // (kept apart from the others)
                        a.target_z[row] = v[j];
                        v[j] = -INFINITY;
                    }
                    top = fmaxf(top, v[j]);
                }
                const float ref = reference(over_row(top, true));
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum += ex2(fmaf(v[j], kLog2e, -ref));
                sum = over_row(sum, false);
                if (tx == 0 && here && n0 + 64 * half < a.N)
                    a.part[(size_t)((n0 + 64 * half) / kCols) * a.M + row] = make_float2(sum == 0.f ? kNoRef : ref, sum);
            } else if (MODE == kGrad) {
                // (columns past the vocabulary get zeros: the products read whole steps)
                const int k = target < 0 ? -1 : target - a.v0 - col;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = target < 0 ? 0.f : k == j ? c.z * c.w : ex2(fmaf(v[j], kLog2e, -c.x)) * (c.y * c.w);
                if (here)
                    *reinterpret_cast<float4 *>(a.out + row * a.ldo + col) = make_float4(v[0], v[1], v[2], v[3]);
            } else if (here && col < a.N) {
                float4 *to = reinterpret_cast<float4 *>(a.out + z * a.a_split + row * a.ldo + col);
                if (dead)
                    v[0] = v[1] = v[2] = v[3] = 0.f;
                if (a.add) {
                    const float4 old = *to;
                    v[0] += old.x;
                    v[1] += old.y;
                    v[2] += old.z;
                    v[3] += old.w;
                }
                *to = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
    }
}

// out (+)= the splits' sums, in order.
__global__ void __launch_bounds__(kT)
    join_f32_kernel(const float *part, float *out, int64_t values, int splits, int64_t a_split, int add) {
    griddep_launch_dependents();
    griddep_wait();
    part = after_wait(part);
    out = after_wait(out);
    const int64_t i = 4 * ((int64_t)blockIdx.x * kT + threadIdx.x);
    if (i >= values)
        return;
    float4 s = add ? *reinterpret_cast<const float4 *>(out + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int z = 0; z < splits; ++z) {
        const float4 v = __ldcg(reinterpret_cast<const float4 *>(part + z * a_split + i));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    *reinterpret_cast<float4 *>(out + i) = s;
}

// Sums of g's columns over 32 tokens each.
__global__ void __launch_bounds__(kT) colsum_f32_kernel(const float *g, float *colsum, int N, int64_t ldg) {
    griddep_launch_dependents();
    griddep_wait();
    g = after_wait(g);
    const int across = (int)((ldg + kT - 1) / kT), block = blockIdx.x / across;
    const int64_t v = (int64_t)(blockIdx.x - block * across) * kT + threadIdx.x;
    if (v >= ldg)
        return;
    const int n0 = 32 * block;
    float s = 0.f;
#pragma unroll 8
    for (int n = n0; n < min(N, n0 + 32); ++n)
        s += __ldcg(g + n * ldg + v);
    colsum[block * ldg + v] = s;
}

int tiles_of(int64_t n) { return (int)((n + kTile - 1) / kTile); }

// Splits of a contraction of K: as many as bring the CTAs to two an SM, of 256 at least.
struct Splits {
    int n, per;
};
Splits splits_of(int64_t tiles, int K) {
    const int steps = (K + kStep - 1) / kStep;
    int64_t n = std::max<int64_t>(1, std::min<int64_t>(4 * kPairs / tiles, steps / 16));
    const int per = (int)((steps + n - 1) / n);
    return {(steps + per - 1) / per, per};
}

struct Plan {
    int width; // vocabulary entries of a piece (a multiple of 128), and G's row stride
    Splits dh, dw;
    size_t row, row_target, g, dh_part, dw_part, colsum, bytes; // offsets
};
Plan plan_of(int N, int V, int D) {
    Plan p;
    const int vt = tiles_of(V), dt = tiles_of(D);
    const int64_t most = std::max<int64_t>(1, (int64_t)(kPieceBytes / ((size_t)4 * kTile * N)));
    const int64_t pieces = (vt + most - 1) / most;
    p.width = (int)((vt + pieces - 1) / pieces) * kTile;
    p.dh = splits_of((int64_t)tiles_of(N) * dt, std::min(p.width, V));
    p.dw = splits_of((int64_t)(p.width / kTile) * dt, N);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    p.row = take(sizeof(float4) * (size_t)N);
    p.row_target = take(sizeof(int) * (size_t)N);
    p.g = take((size_t)4 * N * p.width);
    p.dh_part = take(p.dh.n > 1 ? (size_t)4 * p.dh.n * N * D : 0);
    p.dw_part = take(p.dw.n > 1 ? (size_t)4 * p.dw.n * p.width * D : 0);
    p.colsum = take((size_t)4 * ((N + 31) / 32) * p.width);
    p.bytes = at;
    return p;
}

template <Mode MODE> cudaError_t launch(Args a, int splits, cudaStream_t st) {
    a.mt = tiles_of(a.M);
    a.nt = tiles_of(a.N);
    const dim3 grid((unsigned)((int64_t)a.mt * a.nt * splits));
    if (a.per <= kChunk)
        return launch_pdl(vocab_f32_kernel<MODE, false>, grid, dim3(kT), 0, st, a);
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(vocab_f32_kernel<MODE, true>, done, kTotalBytes);
    return e != cudaSuccess ? e : launch_pdl(vocab_f32_kernel<MODE, true>, grid, dim3(kT), kTotalBytes, st, a);
}

cudaError_t join(const float *part, float *out, int64_t values, int splits, int64_t a_split, int add, cudaStream_t st) {
    return launch_pdl(join_f32_kernel, dim3((unsigned)((values / 4 + kT - 1) / kT)), dim3(kT), 0, st, part, out, values,
                      splits, a_split, add);
}

} // namespace

cudaError_t loss_products_f32(const float *h, const float *W, const float *bias, Tokens targets, float2 *part,
                              float *target_z, int N, int V, int D, cudaStream_t st) {
    Args a = {};
    a.A = h;
    a.B = W;
    a.lda = a.ldb = D;
    a.M = N;
    a.N = a.vocab = V;
    a.K = D;
    a.per = (D + kStep - 1) / kStep;
    a.bias = bias;
    a.targets = targets;
    a.part = part;
    a.target_z = target_z;
    return launch<kLoss>(a, 1, st);
}

size_t backward_workspace_f32(int N, int V, int D) { return plan_of(N, V, D).bytes; }

cudaError_t backward_f32(const float *h, const float *W, const float *bias, Tokens targets, const float *loss,
                         const float *lse, const float *dloss, float *dh, float *dW, float *dbias, void *workspace, int N,
                         int V, int D, cudaStream_t st) {
    const Plan p = plan_of(N, V, D);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    float4 *row = reinterpret_cast<float4 *>(ws + p.row);
    int *row_target = reinterpret_cast<int *>(ws + p.row_target);
    float *g = reinterpret_cast<float *>(ws + p.g), *dh_part = reinterpret_cast<float *>(ws + p.dh_part);
    float *dw_part = reinterpret_cast<float *>(ws + p.dw_part), *colsum = reinterpret_cast<float *>(ws + p.colsum);
    cudaError_t e = launch_rows(nullptr, targets, loss, lse, dloss, row, row_target, nullptr, 0, false, N, V, D, st);
    for (int v0 = 0; e == cudaSuccess && v0 < V; v0 += p.width) {
        const int nv = std::min(p.width, V - v0), blocks = (N + 31) / 32;
        Args a = {};
        a.A = h;
        a.B = W + (size_t)v0 * D;
        a.lda = a.ldb = D;
        a.M = N;
        a.N = nv;
        a.K = D;
        a.per = (D + kStep - 1) / kStep;
        a.bias = bias ? bias + v0 : nullptr;
        a.vocab = V;
        a.v0 = v0;
        a.row = row;
        a.row_target = row_target;
        a.out = g;
        a.ldo = p.width;
        e = launch<kGrad>(a, 1, st);
        if (e == cudaSuccess && dbias) {
            e = launch_pdl(colsum_f32_kernel, dim3((unsigned)((int64_t)((p.width + kT - 1) / kT) * blocks)), dim3(kT), 0, st,
                           (const float *)g, colsum, N, (int64_t)p.width);
            if (e == cudaSuccess)
                e = launch_join_bias(colsum, dbias + v0, nv, blocks, p.width, st);
        }
        if (e == cudaSuccess && dh) {
            Args q = {};
            q.A = g;
            q.lda = p.width;
            q.B = W + (size_t)v0 * D;
            q.ldb = D;
            q.M = N;
            q.N = D;
            q.K = nv;
            q.per = p.dh.per;
            q.row_target = row_target;
            const int splits = ((nv + kStep - 1) / kStep + q.per - 1) / q.per;
            q.out = p.dh.n > 1 ? dh_part : dh;
            q.ldo = D;
            q.a_split = (int64_t)N * D;
            q.add = p.dh.n == 1 && v0 > 0;
            e = launch<kDh>(q, splits, st);
            if (e == cudaSuccess && p.dh.n > 1)
                e = join(dh_part, dh, (int64_t)N * D, splits, q.a_split, v0 > 0, st);
        }
        if (e == cudaSuccess && dW) {
            Args q = {};
            q.A = g;
            q.lda = p.width;
            q.B = h;
            q.ldb = D;
            q.M = nv;
            q.N = D;
            q.K = N;
            q.per = p.dw.per;
            q.row_target = row_target;
            float *to = dW + (size_t)v0 * D;
            q.out = p.dw.n > 1 ? dw_part : to;
            q.ldo = D;
            q.a_split = (int64_t)p.width * D;
            e = launch<kDw>(q, p.dw.n, st);
            if (e == cudaSuccess && p.dw.n > 1)
                e = join(dw_part, to, (int64_t)nv * D, p.dw.n, q.a_split, 0, st);
        }
    }
    return e;
}

} // namespace vocab
} // namespace fw
