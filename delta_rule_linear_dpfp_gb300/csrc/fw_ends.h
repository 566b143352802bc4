// fw_ends.h -- host interface of a model's two ends and the norm between its
// parts: the embedding (fw_embedding.cu), the layer norm (fw_layer_norm.cu)
// and the vocabulary loss (fw_vocab.cu), for the argument-checking C ABI in
// fw_ends_api.cu.
#pragma once
#include <cuda_runtime.h>
#ifdef __CUDACC__
#include "fw_common.cuh"
#endif
#include <stddef.h>
#include <stdint.h>

namespace fw {

cudaError_t device_sms(int *out);          // fw_api.cu
cudaError_t status_word(unsigned **out);   // fw_api.cu

// Tokens as a call was given them: 32 or 64 bits each.
struct Tokens {
    const void *p;
    int wide;
};
#ifdef __CUDACC__
// store8 for what is written once and not read by the same call: it is the first to leave L2.
__device__ __forceinline__ void store8_stream(float *p, const float (&v)[8]) {
    __stcs(reinterpret_cast<float4 *>(p), make_float4(v[0], v[1], v[2], v[3]));
    __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8_stream(__nv_bfloat16 *p, const float (&v)[8]) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                    pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
}

// Token i within [0, V), -1 for any negative one, V for any past the end.
__device__ __forceinline__ int token_at(const Tokens &t, int64_t i, int V) {
    const int64_t x = t.wide ? __ldcg(static_cast<const long long *>(t.p) + i) : __ldcg(static_cast<const int *>(t.p) + i);
    return x < 0 ? -1 : x >= V ? V : (int)x;
}
#endif

cudaError_t launch_embedding(Tokens ids, const void *table, void *out, int64_t N, int V, int D, float scale, int bf16,
                             cudaStream_t st);
size_t embedding_backward_workspace_bytes(int N, int V, int D);
cudaError_t launch_embedding_backward(Tokens ids, const void *dout, void *dtable, void *workspace, int N, int V, int D,
                                      float scale, int accumulate, int bf16, cudaStream_t st);

cudaError_t launch_layer_norm(const void *x, const void *residual, const float *gamma, const float *beta, void *out,
                              void *sum, int64_t rows, int d, float eps, int bf16, cudaStream_t st);
size_t layer_norm_backward_workspace_bytes(int64_t rows, int d);
cudaError_t launch_layer_norm_backward(const void *x, const float *gamma, const void *dout, const void *dsum, void *dx,
                                       float *dgamma, float *dbeta, void *workspace, int64_t rows, int d, float eps,
                                       int bf16, cudaStream_t st);

size_t vocab_loss_workspace_bytes(int N, int V, int D);
cudaError_t launch_vocab_loss(const void *h, const void *W, const float *bias, Tokens targets, float *loss, float *lse,
                              void *workspace, int N, int V, int D, int bf16, cudaStream_t st);
size_t vocab_loss_backward_workspace_bytes(int N, int V, int D, int bf16);
cudaError_t launch_vocab_loss_backward(const void *h, const void *W, const float *bias, Tokens targets,
                                       const float *loss, const float *lse, const float *dloss, void *dh, void *dW,
                                       float *dbias, void *workspace, int N, int V, int D, int bf16, cudaStream_t st);

} // namespace fw
