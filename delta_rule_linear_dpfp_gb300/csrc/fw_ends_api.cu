// fw_ends_api.cu -- the C ABI of the embedding, the layer norm and the
// vocabulary loss (include/fastweight.h): argument checks on the host, then
// dispatch.  Nothing is enqueued unless every check passes.  An output or a
// workspace that shares bytes with something else of the call is refused,
// where the header does not allow it: its values would be lost, or depend on
// the order in which CTAs happen to run.
#include "fastweight.h"
#include "fw_ends.h"

#include <climits>
#include <cmath>

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool usable(const void *p) { return p && aligned16(p); }
bool dtype_ok(int d) { return d == FW_DTYPE_F32 || d == FW_DTYPE_BF16; }
// (tokens are read one at a time: a shifted view of a batch's is a usual argument)
bool tokens_ok(const void *p, int type) { return p && (reinterpret_cast<uintptr_t>(p) & (type == FW_INDEX_I64 ? 7u : 3u)) == 0; }
bool index_ok(int i) { return i == FW_INDEX_I32 || i == FW_INDEX_I64; }
// Whether n bytes at p and m at q share none (a null pointer has none).
struct Bytes {
    const void *p;
    size_t n;
};
bool apart(Bytes a, Bytes b) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
    return !p || !q || !a.n || !b.n || (p < q ? q - p >= a.n : p - q >= b.n);
}
bool same_or_apart(Bytes a, Bytes b) { return a.p == b.p || apart(a, b); }
// An output and everything else that a call is given.
template <typename... Others> bool apart(Bytes a, Bytes b, Others... more) { return apart(a, b) && apart(a, more...); }
// Every output apart from every input and from every other output.
template <size_t I, size_t O> bool all_apart(const Bytes (&in)[I], const Bytes (&out)[O]) {
    for (size_t i = 0; i < O; ++i) {
        for (const Bytes &b : in)
            if (!apart(out[i], b))
                return false;
        for (size_t j = 0; j < i; ++j)
            if (!apart(out[i], out[j]))
                return false;
    }
    return true;
}
size_t value_bytes(int io_dtype) { return io_dtype == FW_DTYPE_BF16 ? 2 : 4; }
size_t token_bytes(int index_type) { return index_type == FW_INDEX_I64 ? 8 : 4; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? FW_OK : FW_ERR_CUDA; }

constexpr int kMaxCount = INT_MAX - (1 << 17); // tokens, table rows: their tiles are counted in int
constexpr int kMaxWidth = 65536, kMaxNorm = 8192;

int check_table(int64_t N, int V, int D) {
    if (N < 0 || V <= 0 || D <= 0)
        return FW_ERR_INVALID_ARG;
    return D % 8 || D > kMaxWidth || V > kMaxCount ? FW_ERR_UNSUPPORTED : FW_OK;
}
int check_norm(int64_t rows, int d, float eps) {
    if (rows < 0 || d <= 0 || !std::isfinite(eps) || eps < 0.f)
        return FW_ERR_INVALID_ARG;
    return d % 8 || d > kMaxNorm ? FW_ERR_UNSUPPORTED : FW_OK;
}
int check_loss(int N, int V, int D, int io_dtype) {
    if (!dtype_ok(io_dtype))
        return FW_ERR_INVALID_ARG;
    const int rc = check_table(N, V, D);
    if (rc != FW_OK)
        return rc;
    const int64_t mt = ((int64_t)N + 255) / 256, nt = ((int64_t)V + 255) / 256, dt = ((int64_t)D + 255) / 256;
    const int64_t most = io_dtype == FW_DTYPE_BF16 ? INT_MAX : INT_MAX / 4; // (fp32: tiles of half the edge)
    return N > kMaxCount || mt * nt > most || mt * dt > INT_MAX / 256 || nt * dt > INT_MAX / 256 ? FW_ERR_UNSUPPORTED
                                                                                                    : FW_OK;
}

} // namespace

extern "C" {

FW_API int fw_embedding(const void *ids, const void *table, void *out, int64_t N, int V, int D, float scale,
                        int index_type, int io_dtype, void *stream) {
    if (!index_ok(index_type) || !dtype_ok(io_dtype) || !std::isfinite(scale))
        return FW_ERR_INVALID_ARG;
    const int rc = check_table(N, V, D);
    if (rc != FW_OK)
        return rc;
    if (N > (int64_t)INT_MAX * 4)
        return FW_ERR_UNSUPPORTED;
    if (N == 0)
        return FW_OK;
    const size_t e = value_bytes(io_dtype);
    if (!tokens_ok(ids, index_type) || !usable(table) || !usable(out) ||
        !apart({out, e * N * D}, Bytes{table, e * V * D}, Bytes{ids, token_bytes(index_type) * N}))
        return FW_ERR_INVALID_ARG;
    return cuda_status(fw::launch_embedding({ids, index_type}, table, out, N, V, D, scale, io_dtype == FW_DTYPE_BF16,
                                            static_cast<cudaStream_t>(stream)));
}

FW_API size_t fw_embedding_backward_workspace_size(int64_t N, int V, int D) {
    if (check_table(N, V, D) != FW_OK || N == 0 || N > kMaxCount)
        return 0;
    return fw::embedding_backward_workspace_bytes((int)N, V, D);
}

FW_API int fw_embedding_backward(const void *ids, const void *dout, void *dtable, void *workspace,
                                 size_t workspace_bytes, int64_t N, int V, int D, float scale, int accumulate,
                                 int index_type, int io_dtype, void *stream) {
    if (!index_ok(index_type) || !dtype_ok(io_dtype) || !std::isfinite(scale) || (accumulate != 0 && accumulate != 1))
        return FW_ERR_INVALID_ARG;
    const int rc = check_table(N, V, D);
    if (rc != FW_OK)
        return rc;
    if (N > kMaxCount)
        return FW_ERR_UNSUPPORTED;
    if (!usable(dtable))
        return FW_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t e = value_bytes(io_dtype);
    if (N == 0) // no token: nothing to add, a gradient of zero
        return cuda_status(accumulate ? cudaSuccess : cudaMemsetAsync(dtable, 0, e * V * D, st));
    const size_t need = fw_embedding_backward_workspace_size(N, V, D);
    const Bytes tokens = {ids, token_bytes(index_type) * N}, given = {dout, e * N * D}, scratch = {workspace, need};
    if (!tokens_ok(ids, index_type) || !usable(dout) || !usable(workspace) || workspace_bytes < need ||
        !apart({dtable, e * V * D}, tokens, given, scratch) || !apart(scratch, tokens, given))
        return FW_ERR_INVALID_ARG;
    return cuda_status(fw::launch_embedding_backward({ids, index_type}, dout, dtable, workspace, (int)N, V, D, scale,
                                                     accumulate, io_dtype == FW_DTYPE_BF16, st));
}

FW_API int fw_layer_norm(const void *x, const void *residual, const float *gamma, const float *beta, void *out,
                         void *sum, int64_t rows, int d, float eps, int io_dtype, void *stream) {
    if (!dtype_ok(io_dtype))
        return FW_ERR_INVALID_ARG;
    const int rc = check_norm(rows, d, eps);
    if (rc != FW_OK)
        return rc;
    if (rows == 0)
        return FW_OK;
    const size_t n = value_bytes(io_dtype) * rows * d, p = sizeof(float) * d;
    if (!usable(x) || !usable(out) || !aligned16(residual) || !aligned16(gamma) || !aligned16(beta) || !aligned16(sum) ||
        !residual != !sum)
        return FW_ERR_INVALID_ARG;
    for (const void *to : {out, sum}) // (in place: a row's values are read before they are written)
        if (!same_or_apart({to, n}, {x, n}) || !same_or_apart({to, n}, {residual, n}) ||
            !apart({to, n}, Bytes{gamma, p}, Bytes{beta, p}))
            return FW_ERR_INVALID_ARG;
    if (!apart({out, n}, Bytes{sum, n}))
        return FW_ERR_INVALID_ARG;
    return cuda_status(fw::launch_layer_norm(x, residual, gamma, beta, out, sum, rows, d, eps, io_dtype == FW_DTYPE_BF16,
                                             static_cast<cudaStream_t>(stream)));
}

FW_API size_t fw_layer_norm_backward_workspace_size(int64_t rows, int d) {
    if (check_norm(rows, d, 0.f) != FW_OK || rows == 0)
        return 0;
    return fw::layer_norm_backward_workspace_bytes(rows, d);
}

FW_API int fw_layer_norm_backward(const void *x, const float *gamma, const void *dout, const void *dsum, void *dx,
                                  float *dgamma, float *dbeta, void *workspace, size_t workspace_bytes, int64_t rows,
                                  int d, float eps, int io_dtype, void *stream) {
    if (!dtype_ok(io_dtype))
        return FW_ERR_INVALID_ARG;
    const int rc = check_norm(rows, d, eps);
    if (rc != FW_OK)
        return rc;
    const size_t n = value_bytes(io_dtype) * rows * d, p = sizeof(float) * d;
    const Bytes dg = {dgamma, p}, db = {dbeta, p};
    if (!dgamma != !dbeta || !aligned16(dgamma) || !aligned16(dbeta) || !apart(dg, db))
        return FW_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) { // no token: the parameters' gradients are zero
        if (!dgamma)
            return FW_OK;
        const cudaError_t e = cudaMemsetAsync(dgamma, 0, sizeof(float) * d, st);
        return cuda_status(e != cudaSuccess ? e : cudaMemsetAsync(dbeta, 0, sizeof(float) * d, st));
    }
    const size_t need = dgamma ? fw_layer_norm_backward_workspace_size(rows, d) : 0;
    if (!usable(x) || !usable(dout) || !usable(dx) || !aligned16(gamma) || !aligned16(dsum) ||
        (dgamma && (!usable(workspace) || workspace_bytes < need)))
        return FW_ERR_INVALID_ARG;
    const Bytes to = {dx, n}, ga = {gamma, p}, scratch = {workspace, need};
    for (const void *in : {x, dout, dsum}) // (dx in place of any of them)
        if (!same_or_apart(to, {in, n}) || !apart({in, n}, dg, db, scratch))
            return FW_ERR_INVALID_ARG;
    if (!apart(to, ga, dg, db, scratch) || !apart(scratch, ga, dg, db) || !apart(ga, db) || !same_or_apart(ga, dg))
        return FW_ERR_INVALID_ARG;
    return cuda_status(fw::launch_layer_norm_backward(x, gamma, dout, dsum, dx, dgamma, dbeta, workspace, rows, d, eps,
                                                      io_dtype == FW_DTYPE_BF16, st));
}

FW_API size_t fw_vocab_loss_workspace_size(int N, int V, int D, int io_dtype) {
    if (check_loss(N, V, D, io_dtype) != FW_OK || N == 0)
        return 0;
    return fw::vocab_loss_workspace_bytes(N, V, D);
}

FW_API int fw_vocab_loss(const void *h, const void *W, const float *bias, const void *targets, float *loss, float *lse,
                         void *workspace, size_t workspace_bytes, int N, int V, int D, int index_type, int io_dtype,
                         void *stream) {
    if (!index_ok(index_type))
        return FW_ERR_INVALID_ARG;
    const int rc = check_loss(N, V, D, io_dtype);
    if (rc != FW_OK)
        return rc;
    if (N == 0)
        return FW_OK;
    const size_t need = fw_vocab_loss_workspace_size(N, V, D, io_dtype), e = value_bytes(io_dtype), f = sizeof(float);
    if (!usable(h) || !usable(W) || !aligned16(bias) || !tokens_ok(targets, index_type) || !usable(loss) || !usable(lse) ||
        !usable(workspace) || workspace_bytes < need)
        return FW_ERR_INVALID_ARG;
    const Bytes in[] = {{h, e * N * D}, {W, e * V * D}, {bias, f * V}, {targets, token_bytes(index_type) * N}};
    const Bytes out[] = {{loss, f * N}, {lse, f * N}, {workspace, need}};
    if (!all_apart(in, out))
        return FW_ERR_INVALID_ARG;
    return cuda_status(fw::launch_vocab_loss(h, W, bias, {targets, index_type}, loss, lse, workspace, N, V, D,
                                             io_dtype == FW_DTYPE_BF16, static_cast<cudaStream_t>(stream)));
}

FW_API size_t fw_vocab_loss_backward_workspace_size(int N, int V, int D, int io_dtype) {
    if (check_loss(N, V, D, io_dtype) != FW_OK || N == 0)
        return 0;
    return fw::vocab_loss_backward_workspace_bytes(N, V, D, io_dtype == FW_DTYPE_BF16);
}

FW_API int fw_vocab_loss_backward(const void *h, const void *W, const float *bias, const void *targets,
                                  const float *loss, const float *lse, const float *dloss, void *dh, void *dW,
                                  float *dbias, void *workspace, size_t workspace_bytes, int N, int V, int D,
                                  int index_type, int io_dtype, void *stream) {
    if (!index_ok(index_type))
        return FW_ERR_INVALID_ARG;
    const int rc = check_loss(N, V, D, io_dtype);
    if (rc != FW_OK)
        return rc;
    const size_t need = fw_vocab_loss_backward_workspace_size(N, V, D, io_dtype), e = value_bytes(io_dtype), f = sizeof(float);
    const Bytes in[] = {{h, e * N * D}, {W, e * V * D}, {bias == dbias ? nullptr : bias, f * V},
                        {targets, token_bytes(index_type) * N}, {loss, f * N}, {lse, f * N}, {dloss, f * N}};
    const Bytes out[] = {{dh, e * N * D}, {dW, e * V * D}, {dbias, f * V}, {workspace, need}};
    if (!aligned16(dh) || !aligned16(dW) || !aligned16(dbias) || !all_apart(in, out))
        return FW_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (N == 0) { // no token: gradients of zero
        cudaError_t rc = dW ? cudaMemsetAsync(dW, 0, e * V * D, st) : cudaSuccess;
        if (rc == cudaSuccess && dbias)
            rc = cudaMemsetAsync(dbias, 0, f * V, st);
        return cuda_status(rc);
    }
    if (!usable(h) || !usable(W) || !aligned16(bias) || !tokens_ok(targets, index_type) || !usable(loss) || !usable(lse) ||
        !usable(dloss) || !usable(workspace) || workspace_bytes < need)
        return FW_ERR_INVALID_ARG;
    return cuda_status(fw::launch_vocab_loss_backward(h, W, bias, {targets, index_type}, loss, lse, dloss, dh, dW, dbias,
                                                      workspace, N, V, D, io_dtype == FW_DTYPE_BF16, st));
}

} // extern "C"
