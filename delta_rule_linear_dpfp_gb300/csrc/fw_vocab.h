// fw_vocab.h -- what the vocabulary loss's files share: fw_vocab.cu (bf16, tensor
// cores), fw_vocab_f32.cu (fp32, CUDA cores) and fw_vocab_rows.cu (a token's
// parts and constants, and the form for few tokens).
#pragma once
#include "fw_common.cuh"
#include "fw_ends.h"
#include "fw_pairs.cuh"

namespace fw {
namespace vocab {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
constexpr float kNoRef = -1e30f; // the reference of no entries: below every other
// Logits below it are out of the vocabulary, as those of -infinity are.  (A mask may be any
// low number; from 2^31 on a reference's own rounding is past what an exponential holds.)
constexpr float kOut = -0x1p30f;
constexpr int kCols = 64;        // vocabulary entries of a part of a token's sum
constexpr int kPairs = 76;       // pairs of a GB300's SMs: what splits (and so the workspaces) go by
// Of the softmax's gradient, tokens x a piece of the vocabulary: 512 MB took 3 % longer at D 2048 and
// 5 % at D 512 (8192 x 50 001), and leave half of it in memory at a time.
constexpr size_t kPieceBytes = (size_t)1024 << 20;

#ifdef __CUDACC__
// A reference near x for exponentials: x log2 e to a sixteenth, so that z log2 e less
// the reference takes one rounding (0 where all of them are out: their exponentials are 0).
FW_DEV float reference(float x) { return x < kOut ? 0.f : rintf(x * kLog2e * 16.f) * 0.0625f; }
#endif

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
// log2 of the threads of a row of D channels, 8 a thread (at most a CTA's 256).
inline int group_log2(int D) {
    int lg = 0;
    while ((8 << lg) < D && lg < 8)
        ++lg;
    return lg;
}

// The parts that the products leave of a token, [parts][N] (reference, sum of
// 2^(z log2 e - reference) over the entries other than its target), the targets'
// logits behind them.
int parts_of(int N, int V, int D);
// Up to four answers that fit: the whole product, on CUDA cores.
bool few(int N, int D);
cudaError_t launch_few(const void *h, const void *W, const float *bias, Tokens targets, float2 *part, float *target_z,
                       int N, int V, int D, int bf16, cudaStream_t st);
cudaError_t launch_join_parts(const float2 *part, const float *target_z, Tokens targets, float *loss, float *lse, int N,
                              int V, int nparts, cudaStream_t st);
// The tokens' constants (see row_constants; `folded`: log2 q into row.x) and targets (-1
// for none), and w h in bf16 (or null), with lo_rows in two terms.
cudaError_t launch_rows(const void *h, Tokens targets, const float *loss, const float *lse, const float *dloss,
                        float4 *row, int *row_target, void *wh, int lo_rows, bool folded, int N, int V, int D, cudaStream_t st);

// dbias of a piece from the sums of 32 tokens each ([blocks][ldc]), in order (fw_vocab.cu).
cudaError_t launch_join_bias(const float *colsum, float *dbias, int V, int blocks, int ldc, cudaStream_t st);

// fw_vocab_f32.cu
cudaError_t loss_products_f32(const float *h, const float *W, const float *bias, Tokens targets, float2 *part,
                              float *target_z, int N, int V, int D, cudaStream_t st);
size_t backward_workspace_f32(int N, int V, int D);
cudaError_t backward_f32(const float *h, const float *W, const float *bias, Tokens targets, const float *loss,
                         const float *lse, const float *dloss, float *dh, float *dW, float *dbias, void *workspace, int N,
                         int V, int D, cudaStream_t st);

} // namespace vocab
} // namespace fw
