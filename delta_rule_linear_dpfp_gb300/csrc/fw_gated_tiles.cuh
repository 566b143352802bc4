// fw_gated_tiles.cuh -- what the gated delta rule's kernels share: where a
// sequence ends, and fp32 values as two bf16 terms in operand tiles.
#pragma once

#include "fw_common.cuh"
#include "fw_gated.h"
#include "fw_pairs.cuh"

namespace fw {

constexpr int kGatedThreads = 256;          // per CTA of the preparing kernels
constexpr int kGatedLd = kGatedChunk + 4;   // row stride of an fp32 chunk x chunk tile
constexpr float kGMin = -200.f; // e^g is 0 in fp32 below this: a gate of -inf is a sum that stays finite

// (called after griddep_wait)
FW_DEV int seq_len(const GatedArgs &a, int b) {
    return a.lengths ? min(max(__ldcg(after_wait(a.lengths) + b), 0), a.L) : a.L;
}

// 16 bytes on their way into shared memory by an asynchronous copy; `in` false: zeros.
FW_DEV void copy16(void *to, const void *from, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from),
                 "r"(in ? 16 : 0)
                 : "memory");
}

// Sums kept as an unevaluated pair of floats (hi + lo, 48 bits).
struct Pair {
    float hi, lo;
};
FW_DEV Pair add(Pair a, Pair b) { // two-sum of the highs, the lows added to what it left
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float h = s + e;
    return {h, e - (h - s)};
}
// Of 64 values, two a lane: the sum up to and with the lane's second, and of all.
FW_DEV void running_sum(const float (&x)[2], int lane, Pair &run, Pair &all) {
    run = add({x[0], 0.f}, {x[1], 0.f});
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const Pair up = {__shfl_up_sync(0xffffffffu, run.hi, m), __shfl_up_sync(0xffffffffu, run.lo, m)};
        if (lane >= m)
            run = add(up, run);
    }
    all = {__shfl_sync(0xffffffffu, run.hi, 31), __shfl_sync(0xffffffffu, run.lo, 31)};
}

// 8 fp32 values as 8 hi and 8 lo bf16 terms.
FW_DEV void split8(const float *x, uint4 &hi, uint4 &lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
        const float2 d = unpack(pack(x[2 * e], x[2 * e + 1]) -
                                pack(__uint_as_float(h[e] << 16), __uint_as_float(h[e] & 0xffff0000u)));
        l[e] = pack_bf16x2(d.x, d.y);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// Of 64 values, two a lane: the sum over the lanes after this one, or before it.
FW_DEV float lanes_after(float x, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float up = __shfl_down_sync(0xffffffffu, x, m);
        x += lane + m < 32 ? up : 0.f;
    }
    x = __shfl_down_sync(0xffffffffu, x, 1);
    return lane < 31 ? x : 0.f;
}
FW_DEV float lanes_before(float x, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float up = __shfl_up_sync(0xffffffffu, x, m);
        x += lane >= m ? up : 0.f;
    }
    x = __shfl_up_sync(0xffffffffu, x, 1);
    return lane > 0 ? x : 0.f;
}
// dg of a lane's two tokens of 64 (the formula at the head of
// fw_gated_chunk.cu): the state's part z, the readers R from a token on, the
// writers W before it, the pairs c across it.  One warp.
FW_DEV void gated_decay_grads(float z, const float *R, const float *W, const float *c, int lane, float (&dg)[2]) {
    const float later = lanes_after(R[0] + R[1], lane), earlier = lanes_before(W[0] + W[1], lane);
    dg[0] = ((later + R[1]) + R[0]) + earlier + (c[0] + z);
    dg[1] = (later + R[1]) + (earlier + W[0]) + (c[1] + z);
}

// The tensor-core kernels' scalars of a chunk's tokens, [7][64]: G (the
// running sum of g) as hi and lo, 1 / |k|, beta, 1 / |q|, e^G, e^{G_C - G}.
enum { kGhi = 0, kGlo = 64, kRk = 128, kBeta = 192, kRq = 256, kEG = 320, kEC = 384 };

// e^{G_i - G_j} of four tokens j; (ghi, glo) is G_i.
FW_DEV void decay4(const float *tok, int j, float ghi, float glo, F2 (&d)[2]) {
    const ulonglong2 h = *reinterpret_cast<const ulonglong2 *>(tok + kGhi + j);
    const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(tok + kGlo + j);
    const F2 hp[2] = {{h.x}, {h.y}}, lp[2] = {{l.x}, {l.y}};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float2 t = unpack(((both(ghi) - hp[e]) + (both(glo) - lp[e])) * both(1.4426950408889634f));
        d[e] = pack(ex2(t.x), ex2(t.y));
    }
}

FW_DEV void widen8(uint4 u, float (&o)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __uint_as_float(w[i] << 16);
        o[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

FW_DEV void widen8(uint4 u, F2 (&o)[4]) {
    float x[8];
    widen8(u, x);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        o[e] = pack(x[2 * e], x[2 * e + 1]);
}

// A "pair tile": rows of 128 bytes, 32 channels' hi terms then their lo terms,
// swizzled as the descriptors of fw_tc.cuh expect.  16-byte chunk c of a row.
FW_DEV uint32_t pair_chunk(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

// s += R rows of a (H / R apart) times four columns of b, over H terms; more
// rows a thread are more products for each value read from shared memory.
template <int H, int R> FW_DEV void block_product(const float *a, int lda, const float *b, int ldb, float (&s)[R][4]) {
#pragma unroll
    for (int m = 0; m < H; m += 4) {
        float f[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float4 t = *reinterpret_cast<const float4 *>(a + r * (H / R) * lda + m);
            f[r][0] = t.x;
            f[r][1] = t.y;
            f[r][2] = t.z;
            f[r][3] = t.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 t = *reinterpret_cast<const float4 *>(b + (m + e) * ldb);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s[r][0] = fmaf(f[r][e], t.x, s[r][0]);
                s[r][1] = fmaf(f[r][e], t.y, s[r][1]);
                s[r][2] = fmaf(f[r][e], t.z, s[r][2]);
                s[r][3] = fmaf(f[r][e], t.w, s[r][3]);
            }
        }
    }
}
// One doubling: T21 = -T22 (A21 T11) in each pair of H x H diagonal blocks, R
// rows and four columns a thread.
template <int H, int R> FW_DEV void double_inverse(const float *A, float *T, float *tmp) {
    constexpr int Q = H / 4, N = (kGatedChunk / (2 * H)) * (H / R) * Q; // threads: pair of blocks, row, four columns
    const int tid = threadIdx.x, p = tid / (H / R * Q), i = (tid / Q) % (H / R), j = (tid % Q) * 4, r0 = p * 2 * H;
    if (tid < N) {
        float s[R][4] = {};
        block_product<H, R>(A + (r0 + H + i) * kGatedLd + r0, kGatedLd, T + r0 * kGatedLd + r0 + j, kGatedLd, s);
#pragma unroll
        for (int r = 0; r < R; ++r)
            *reinterpret_cast<float4 *>(tmp + (p * H + i + r * (H / R)) * H + j) =
                make_float4(s[r][0], s[r][1], s[r][2], s[r][3]);
    }
    __syncthreads();
    if (tid < N) {
        float s[R][4] = {};
        block_product<H, R>(T + (r0 + H + i) * kGatedLd + r0 + H, kGatedLd, tmp + p * H * H + j, H, s);
#pragma unroll
        for (int r = 0; r < R; ++r)
            *reinterpret_cast<float4 *>(T + (r0 + H + i + r * (H / R)) * kGatedLd + r0 + j) =
                make_float4(-s[r][0], -s[r][1], -s[r][2], -s[r][3]);
    }
    __syncthreads();
}

// (I + A)^-1 of the strictly lower triangular A (row stride kGatedLd): forward
// substitution in the four 16 x 16 diagonal blocks, one thread a column, then
// two doublings.
FW_DEV void unit_lower_inverse(const float *A, float *T, float *tmp) {
    const int tid = threadIdx.x;
    for (int e = tid; e < kGatedChunk * kGatedChunk / 4; e += kGatedThreads) {
        const int r = e >> 4, c4 = (e & 15) * 4;
        if (r >> 4 < c4 >> 4)
            *reinterpret_cast<float4 *>(T + r * kGatedLd + c4) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < kGatedChunk) {
        const int b0 = tid & ~15, j = tid & 15;
        const float *Ab = A + b0 * kGatedLd + b0;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == j ? 1.f : 0.f, s2 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(Ab + i * kGatedLd + m);
                s = fmaf(-f.x, x[m], s);
                if (m + 1 < i)
                    s2 = fmaf(-f.y, x[m + 1], s2);
                if (m + 2 < i)
                    s = fmaf(-f.z, x[m + 2], s);
                if (m + 3 < i)
                    s2 = fmaf(-f.w, x[m + 3], s2);
            }
            x[i] = s + s2;
            T[(b0 + i) * kGatedLd + b0 + j] = x[i];
        }
    }
    __syncthreads();
    double_inverse<16, 1>(A, T, tmp);
    double_inverse<32, 2>(A, T, tmp);
}

} // namespace fw
