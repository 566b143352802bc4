// fw_gated.h -- host interface of the gated delta rule's kernels
// (fw_gated_chunk.cu, fw_gated_tc.cu, fw_gated_grad_tc.cu, fw_gated_decode.cu)
// and of the group norm's (fw_group_norm.cu), for the argument-checking C ABI
// in fw_gated_api.cu.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fw {

// One call's shape and options (arguments validated by the caller).
struct GatedArgs {
    int B, Hk, H, L, d_k, d_v;
    int l2norm;         // 1: keys and queries scaled to unit length
    float scale, eps;   // of the answers; inside the root of the l2 norm
    const int *lengths; // device [B] or null
};

constexpr int kGatedChunk = 64; // tokens per chunk

size_t gated_forward_workspace_bytes(int B, int H, int L, int d_k, int d_v, int bf16);
size_t gated_backward_workspace_bytes(int B, int H, int L, int d_k, int d_v, int bf16);

cudaError_t launch_gated_forward(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                                 const void *beta, const float *W0, float *W_final, void *y, void *workspace, int bf16,
                                 cudaStream_t st);
cudaError_t launch_gated_backward(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                                  const void *beta, const float *W0, const void *dy, const float *dW_final, void *dq,
                                  void *dk, void *dv, void *dg, void *dbeta, float *dW0, void *workspace, int bf16,
                                  cudaStream_t st);
cudaError_t launch_gated_decode(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                                const void *beta, float *W, void *y, int bf16, cudaStream_t st);

// The group norm (fw_group_norm.cu).
struct NormArgs {
    int B, H, L, d, act;
    float eps;
};
size_t group_norm_backward_workspace_bytes(int B, int H, int L, int d);
cudaError_t launch_group_norm(const NormArgs &a, const void *x, const void *gate, const float *gamma,
                              const float *beta, void *out, int bf16, cudaStream_t st);
cudaError_t launch_group_norm_backward(const NormArgs &a, const void *x, const void *gate, const float *gamma,
                                       const float *beta, const void *dout, void *dx, void *dgate, float *dgamma,
                                       float *dbeta, void *workspace, int bf16, cudaStream_t st);

} // namespace fw
