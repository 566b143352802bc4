// fw_gated_tc.h -- what the tensor-core kernels of the gated delta rule leave
// for one another in the workspace, per chunk of each value head.
#pragma once
#include "fw_gated.h"

namespace fw {

// Byte offsets inside a chunk's record.  Images are operand tiles as shared
// memory holds them; "pair tiles" are rows of 128 bytes, 32 channels' hi terms
// then their lo terms.
struct GatedRecord {
    int nkb, ns, nch;            // 64-wide blocks of d_k, 32-wide slices of d_v, chunks
    size_t bytes;                // per chunk
    // Images of 64 hi rows and the same rows' lo terms per 64-wide block: A is
    // -W', A2 is Q' (forward) or W" (backward); K is the chunk's keys, in the
    // backward [keys; queries] per 64-wide block.
    size_t A, A2, K, scalF, scalR;
    size_t base, base2;          // fp32 pieces [d_v / 16][rows][16]: [U'; Y'] (128 rows), or U' and X0 (64 rows)
    size_t U, dX, S, dS, tok;    // pair tiles [ns] of 64 (U, dX) and d_k (S, dS) rows; the tokens' scalars

    __host__ __device__ size_t off(int64_t bh, int c) const { return ((size_t)bh * nch + c) * bytes; }
};

inline GatedRecord gated_shape_record(int L, int d_k, int d_v) {
    GatedRecord r = {};
    r.nkb = d_k <= 64 ? 1 : 2;
    r.ns = (d_v + 31) / 32;
    r.nch = (L + kGatedChunk - 1) / kGatedChunk;
    return r;
}
inline GatedRecord gated_forward_record(int L, int d_k, int d_v) {
    GatedRecord r = gated_shape_record(L, d_k, d_v);
    r.A = 0;
    r.A2 = r.A + (size_t)r.nkb * 16384;
    r.K = r.A2 + (size_t)r.nkb * 16384;
    r.scalF = r.K + (size_t)r.nkb * 8192;
    r.base = r.scalF + 512;
    r.bytes = r.base + (size_t)r.ns * 16384;
    return r;
}
inline GatedRecord gated_backward_record(int L, int d_k, int d_v) {
    GatedRecord r = gated_shape_record(L, d_k, d_v);
    r.A = 0;
    r.A2 = r.A + (size_t)r.nkb * 16384;
    r.K = r.A2 + (size_t)r.nkb * 16384;
    r.scalF = r.K + (size_t)r.nkb * 16384;
    r.scalR = r.scalF + 512;
    r.tok = r.scalR + 1024;
    r.base = r.tok + 2048;
    r.base2 = r.base + (size_t)r.ns * 8192;
    r.U = r.base2 + (size_t)r.ns * 8192;
    r.dX = r.U + (size_t)r.ns * 8192;
    r.S = r.dX + (size_t)r.ns * 8192;
    r.dS = r.S + (size_t)r.ns * r.nkb * 8192;
    r.bytes = r.dS + (size_t)r.ns * r.nkb * 8192;
    return r;
}

cudaError_t gated_tc_forward(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                             const void *beta, const float *W0, float *Wf, void *y, void *ws, cudaStream_t st);
// Preparation and both walks of the backward: U, dX, S, dS and dW0.
cudaError_t gated_tc_walks(const GatedArgs &a, const void *q, const void *k, const void *v, const void *g,
                           const void *beta, const float *W0, const void *dy, const float *dWf, float *dW0, void *ws,
                           cudaStream_t st);
// The gradients of the tokens from what gated_tc_walks left (the keys and
// queries are in the records).
cudaError_t gated_tc_grad(const GatedArgs &a, const void *v, const void *dy, void *dq, void *dk, void *dv, void *dg,
                          void *dbeta, const void *ws, cudaStream_t st);

} // namespace fw
