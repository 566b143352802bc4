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
    size_t A, K, scalF, base;    // forward: [-W'; Q'] hi, lo; K; scalars; [U'; Y'] fp32 pieces [d_v / 16][128][16]
    size_t AF, AR, KQ, scalR;    // backward: -W' and W" hi, lo (64 rows); [K; Q]; scalars
    size_t baseU, baseX;         // U', X0: fp32 pieces [d_v / 16][64][16]
    size_t U, dX, S, dS, tok;    // pair tiles [ns] of 64 (U, dX) and d_k (S, dS) rows; 8 floats a token

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
    r.K = r.A + (size_t)r.nkb * 32768;
    r.scalF = r.K + (size_t)r.nkb * 8192;
    r.base = r.scalF + 512;
    r.bytes = r.base + (size_t)r.ns * 16384;
    return r;
}
inline GatedRecord gated_backward_record(int L, int d_k, int d_v) {
    GatedRecord r = gated_shape_record(L, d_k, d_v);
    r.AF = 0;
    r.AR = r.AF + (size_t)r.nkb * 16384;
    r.KQ = r.AR + (size_t)r.nkb * 16384;
    r.scalF = r.KQ + (size_t)r.nkb * 16384;
    r.scalR = r.scalF + 512;
    r.tok = r.scalR + 1024;
    r.baseU = r.tok + 2048;
    r.baseX = r.baseU + (size_t)r.ns * 8192;
    r.U = r.baseX + (size_t)r.ns * 8192;
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
// The gradients of the tokens from what gated_tc_walks left.
cudaError_t gated_tc_grad(const GatedArgs &a, const void *q, const void *k, const void *v, const void *dy, void *dq,
                          void *dk, void *dv, void *dg, void *dbeta, const void *ws, cudaStream_t st);

} // namespace fw
