// fw_gated_tiles.cuh -- what the gated delta rule's kernels share: where a
// sequence ends, and fp32 values as two bf16 terms in operand tiles.
#pragma once

#include "fw_common.cuh"
#include "fw_gated.h"

namespace fw {

constexpr float kGMin = -200.f; // e^g is 0 in fp32 below this: a gate of -inf is a sum that stays finite

FW_DEV int seq_len(const GatedArgs &a, int b) {
    return a.lengths ? min(max(__ldcg(a.lengths + b), 0), a.L) : a.L;
}

// 8 fp32 values as 8 hi and 8 lo bf16 terms.
FW_DEV void split8(const float *x, uint4 &hi, uint4 &lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
        l[e] = pack_bf16x2(x[2 * e] - __uint_as_float(h[e] << 16),
                           x[2 * e + 1] - __uint_as_float(h[e] & 0xffff0000u));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

FW_DEV void widen8(uint4 u, float (&o)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// A "pair tile": rows of 128 bytes, 32 channels' hi terms then their lo terms,
// swizzled as the descriptors of fw_tc.cuh expect.  16-byte chunk c of a row.
FW_DEV uint32_t pair_chunk(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

} // namespace fw
