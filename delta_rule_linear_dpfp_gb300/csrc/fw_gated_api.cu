// fw_gated_api.cu -- the C ABI of the gated delta rule and of the group norm
// behind it (include/fastweight.h): argument checks on the host, then
// dispatch.  Nothing is enqueued unless every check passes.
#include "fastweight.h"
#include "fw_common.cuh"
#include "fw_gated.h"

#include <climits>
#include <cmath>

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool usable(const void *p) { return p && aligned16(p); }
bool dtype_ok(int d) { return d == FW_DTYPE_F32 || d == FW_DTYPE_BF16; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? FW_OK : FW_ERR_CUDA; }

constexpr int64_t kMaxHeads = 65535; // batch x value heads: one grid dimension

int check_gated_shape(int B, int Hk, int H, int L, int d_k, int d_v, int io_dtype) {
    if (B < 0 || Hk <= 0 || H <= 0 || H % Hk || L < 0 || d_k <= 0 || d_v <= 0 || !dtype_ok(io_dtype))
        return FW_ERR_INVALID_ARG;
    if (!(d_k == 16 || d_k == 32 || d_k == 64 || d_k == 128) || d_v % 16 || d_v > 256 || (int64_t)B * H > kMaxHeads ||
        L > INT_MAX - fw::kGatedChunk)
        return FW_ERR_UNSUPPORTED;
    return FW_OK;
}
bool options_ok(int l2norm, float scale, float eps) {
    return (l2norm == 0 || l2norm == 1) && std::isfinite(scale) && std::isfinite(eps) && eps >= 0.f;
}

int check_norm(int B, int H, int L, int d, int act, int io_dtype, float eps) {
    if (B < 0 || H < 0 || L < 0 || d <= 0 || act < FW_ACT_NONE || act > FW_ACT_GELU || !dtype_ok(io_dtype) ||
        !std::isfinite(eps) || eps < 0.f)
        return FW_ERR_INVALID_ARG;
    if (d % 8 || d > 256 || H > kMaxHeads || (int64_t)H * d > INT_MAX / 2 || (int64_t)B * L > INT_MAX)
        return FW_ERR_UNSUPPORTED;
    return FW_OK;
}

cudaError_t set_state(float *to, const float *from, size_t bytes, cudaStream_t st) {
    if (!to || to == from)
        return cudaSuccess;
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(to, 0, bytes, st);
}

} // namespace

extern "C" {

FW_API size_t fw_gated_delta_forward_workspace_size(int B, int Hk, int H, int L, int d_k, int d_v, int io_dtype) {
    if (check_gated_shape(B, Hk, H, L, d_k, d_v, io_dtype) != FW_OK)
        return 0;
    return fw::gated_forward_workspace_bytes(B, H, L, d_k, d_v, io_dtype == FW_DTYPE_BF16);
}

FW_API int fw_gated_delta_forward(const void *q, const void *k, const void *v, const void *g, const void *beta,
                                  const float *W0, float *W_final, void *y, const int32_t *lengths, void *workspace,
                                  size_t workspace_bytes, int B, int Hk, int H, int L, int d_k, int d_v, int l2norm,
                                  float scale, float eps, int io_dtype, void *stream) {
    if (!options_ok(l2norm, scale, eps))
        return FW_ERR_INVALID_ARG;
    const int rc = check_gated_shape(B, Hk, H, L, d_k, d_v, io_dtype);
    if (rc != FW_OK)
        return rc;
    if (B == 0)
        return FW_OK;
    if ((W0 && !aligned16(W0)) || (W_final && !aligned16(W_final)) || (lengths && !aligned16(lengths)))
        return FW_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (L == 0)
        return cuda_status(set_state(W_final, W0, sizeof(float) * (size_t)B * H * d_v * d_k, st));
    if (!usable(q) || !usable(k) || !usable(v) || !usable(g) || !usable(beta) || !usable(y) || !usable(workspace) ||
        workspace_bytes < fw_gated_delta_forward_workspace_size(B, Hk, H, L, d_k, d_v, io_dtype))
        return FW_ERR_INVALID_ARG;
    const fw::GatedArgs a{B, Hk, H, L, d_k, d_v, l2norm, scale, eps, lengths};
    return cuda_status(fw::launch_gated_forward(a, q, k, v, g, beta, W0, W_final, y, workspace,
                                                io_dtype == FW_DTYPE_BF16, st));
}

FW_API size_t fw_gated_delta_backward_workspace_size(int B, int Hk, int H, int L, int d_k, int d_v, int io_dtype) {
    if (check_gated_shape(B, Hk, H, L, d_k, d_v, io_dtype) != FW_OK)
        return 0;
    return fw::gated_backward_workspace_bytes(B, H, L, d_k, d_v, io_dtype == FW_DTYPE_BF16);
}

FW_API int fw_gated_delta_backward(const void *q, const void *k, const void *v, const void *g, const void *beta,
                                   const float *W0, const void *dy, const float *dW_final, void *dq, void *dk, void *dv,
                                   void *dg, void *dbeta, float *dW0, const int32_t *lengths, void *workspace,
                                   size_t workspace_bytes, int B, int Hk, int H, int L, int d_k, int d_v, int l2norm,
                                   float scale, float eps, int io_dtype, void *stream) {
    if (!options_ok(l2norm, scale, eps))
        return FW_ERR_INVALID_ARG;
    const int rc = check_gated_shape(B, Hk, H, L, d_k, d_v, io_dtype);
    if (rc != FW_OK)
        return rc;
    if (B == 0)
        return FW_OK;
    if ((W0 && !aligned16(W0)) || (dW_final && !aligned16(dW_final)) || (dW0 && !aligned16(dW0)) ||
        (lengths && !aligned16(lengths)))
        return FW_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (L == 0) // no token: dL/dW0 = dL/dW_final
        return cuda_status(set_state(dW0, dW_final, sizeof(float) * (size_t)B * H * d_v * d_k, st));
    const void *need[] = {q, k, v, g, beta, dy, dq, dk, dv, dg, dbeta, workspace};
    for (const void *p : need)
        if (!usable(p))
            return FW_ERR_INVALID_ARG;
    if (workspace_bytes < fw_gated_delta_backward_workspace_size(B, Hk, H, L, d_k, d_v, io_dtype))
        return FW_ERR_INVALID_ARG;
    const fw::GatedArgs a{B, Hk, H, L, d_k, d_v, l2norm, scale, eps, lengths};
    return cuda_status(fw::launch_gated_backward(a, q, k, v, g, beta, W0, dy, dW_final, dq, dk, dv, dg, dbeta, dW0,
                                                 workspace, io_dtype == FW_DTYPE_BF16, st));
}

FW_API int fw_gated_delta_decode_step(const void *q, const void *k, const void *v, const void *g, const void *beta,
                                      float *W, void *y, int B, int Hk, int H, int d_k, int d_v, int l2norm,
                                      float scale, float eps, int io_dtype, void *stream) {
    if (!options_ok(l2norm, scale, eps))
        return FW_ERR_INVALID_ARG;
    const int rc = check_gated_shape(B, Hk, H, 1, d_k, d_v, io_dtype);
    if (rc != FW_OK)
        return rc;
    if (B == 0)
        return FW_OK;
    if (!usable(q) || !usable(k) || !usable(v) || !usable(g) || !usable(beta) || !usable(W) || !usable(y))
        return FW_ERR_INVALID_ARG;
    const fw::GatedArgs a{B, Hk, H, 1, d_k, d_v, l2norm, scale, eps, nullptr};
    return cuda_status(fw::launch_gated_decode(a, q, k, v, g, beta, W, y, io_dtype == FW_DTYPE_BF16,
                                               static_cast<cudaStream_t>(stream)));
}

FW_API int fw_group_norm_act(const void *x, const void *gate, const float *gamma, const float *beta, void *out, int B,
                             int H, int L, int d, int act, int io_dtype, float eps, void *stream) {
    const int rc = check_norm(B, H, L, d, act, io_dtype, eps);
    if (rc != FW_OK)
        return rc;
    if (B == 0 || H == 0 || L == 0)
        return FW_OK;
    if (!usable(x) || !usable(gamma) || !usable(beta) || !usable(out) || (gate && !aligned16(gate)))
        return FW_ERR_INVALID_ARG;
    const fw::NormArgs a{B, H, L, d, act, eps};
    return cuda_status(fw::launch_group_norm(a, x, gate, gamma, beta, out, io_dtype == FW_DTYPE_BF16,
                                             static_cast<cudaStream_t>(stream)));
}

FW_API size_t fw_group_norm_act_backward_workspace_size(int B, int H, int L, int d) {
    if (check_norm(B, H, L, d, FW_ACT_NONE, FW_DTYPE_F32, 0.f) != FW_OK || B == 0 || H == 0 || L == 0)
        return 0;
    return fw::group_norm_backward_workspace_bytes(B, H, L, d);
}

FW_API int fw_group_norm_act_backward(const void *x, const void *gate, const float *gamma, const float *beta,
                                      const void *dout, void *dx, void *dgate, float *dgamma, float *dbeta,
                                      void *workspace, size_t workspace_bytes, int B, int H, int L, int d, int act,
                                      int io_dtype, float eps, void *stream) {
    const int rc = check_norm(B, H, L, d, act, io_dtype, eps);
    if (rc != FW_OK)
        return rc;
    if (H == 0)
        return FW_OK;
    if (!usable(dgamma) || !usable(dbeta))
        return FW_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (B == 0 || L == 0) { // no token: the parameters' gradients are zero
        const size_t bytes = sizeof(float) * (size_t)H * d;
        const cudaError_t e = cudaMemsetAsync(dgamma, 0, bytes, st);
        return cuda_status(e != cudaSuccess ? e : cudaMemsetAsync(dbeta, 0, bytes, st));
    }
    if (!usable(x) || !usable(gamma) || !usable(beta) || !usable(dout) || !usable(dx) ||
        (gate && (!aligned16(gate) || !usable(dgate))) || (!gate && dgate) || !usable(workspace) ||
        workspace_bytes < fw_group_norm_act_backward_workspace_size(B, H, L, d))
        return FW_ERR_INVALID_ARG;
    const fw::NormArgs a{B, H, L, d, act, eps};
    return cuda_status(fw::launch_group_norm_backward(a, x, gate, gamma, beta, dout, dx, dgate, dgamma, dbeta,
                                                      workspace, io_dtype == FW_DTYPE_BF16, st));
}

} // extern "C"
