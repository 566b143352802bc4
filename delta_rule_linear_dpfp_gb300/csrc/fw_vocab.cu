// fw_vocab.cu -- the loss at a model's end: softmax cross entropy of the
// answers h [N, D] over a vocabulary whose output map is W [V, D], with the
// gradients, without the N x V logits.
//
//   z_n = W h_n + b;  lse_n = log sum_v exp z_nv;  loss_n = lse_n - z_n,t
//   g_nv = dloss_n (exp(z_nv - lse_n) - [v = t_n])
//   dh = g W,  dW = g^T h,  db = sum_n g_n
// for the target t_n of token n; tokens whose target is negative are padding
// (no loss, no gradient, whatever h holds).
//
// Bound by the tensor cores: 2 N V D operations forward, 6 N V D backward (the
// logits are formed again).  All four products run on one kernel: a pair of
// CTAs (two SMs) owns 256 x 256 tiles of the output, the operands come by TMA in
// steps of 64 of the contraction, each CTA fetching half of A's rows and half of
// B's, and one thread of the pair issues the MMAs (tcgen05, cta_group::2, fp32
// accumulators in both CTAs' TMEM, 128 rows each).  A tile's accumulator takes
// half of TMEM, so the epilogue of one tile (16 warps in either CTA, 64 columns of
// a row per thread) runs while the next is formed.
//
// Forward: the epilogue turns a row's 64 columns into (reference, sum of
// 2^(z log2 e - reference)), the target's entry left out, and writes the target's
// logit apart; a second kernel joins a token's parts.  Backward, by pieces of the vocabulary of at most 1 GB of
// (bf16) g: one product forms the logits again and its epilogue writes
//   G = (exp(z - lse) - [v = t]) / q,   q = 1 - p_t = -expm1(-loss),
// then dh += G W and dW = G^T (w h) with w = q dloss (dh's rows take w at the
// end, in 32 bits).  What is rounded to bf16 on the way is G, whose largest entry
// is exactly -1 at the target, and w h, element by element: errors that are as
// independent as those of the rounded outputs.  Rounding (p - 1) dloss itself
// would put one relative error of up to 2^-8 into a whole row of dh and dW.  Up to
// 256 tokens, whose contraction is short, and for small vocabularies (second_terms)
// w h goes in as two terms (2^-16 of it left).
#include <cuda.h>

#include <algorithm>

#include "fw_forward_tc.h"
#include "fw_tc.cuh"
#include "fw_vocab.h"

namespace fw {

namespace {

using namespace tc;
using namespace vocab;

constexpr int kEpiWarps = 16;  // each 32 rows x kCols columns of a CTA's 128 x 256
constexpr int kT = 32 * (4 + kEpiWarps); // warp 0: copies, 1: products, 2: TMEM, 4 and on: epilogue
constexpr int kTile = 256;    // rows and columns of a pair's tile
constexpr int kStages = 5;
constexpr int kStageBytes = 32768; // half of A's rows and half of B's, 64 of the contraction
constexpr int kOutOff = kStages * kStageBytes;
constexpr int kOutBytes = kEpiWarps * 4096; // a box of 32 rows x 128 bytes per epilogue warp
constexpr int kBarOff = kOutOff + kOutBytes;
constexpr int kSmem = kBarOff + 256 + 1024;
static_assert(kSmem <= 227 * 1024, "one CTA's shared memory");
// Steps of 64 that an accumulator of logits takes: the tensor core truncates what it
// adds, so that a sum of many terms of one sign falls short (1024 terms in one accumulator:
// by 1.6e-6 of itself, 32 768: by 1.6e-4).  Chunks of 512, which leave 7e-7 at any width, are
// added in the epilogue, where sums are rounded; of 128 1.5e-7.
constexpr int kLogitSteps = 8, kFewLogitSteps = 2, kFewTokens = 256;
// (up to kFewTokens by 128, and w h in two terms: 64 tokens over 50 001 entries, D 1024, 87 us
// for the gradients instead of 81)
// w h in two terms beyond that as well where the entries fit one tile and h has no more values
// than this: a row of dW is then the sum of many tokens', whose roundings come on top of its own
// (2048 x 65, D 512: dW off by 1.7e-3 of itself instead of 2.4e-3, 18.3 us -> 19.9; at the limit,
// 4096 x 65, D 1024, 30.2 -> 30.7; twice as many values 37.0 -> 41.1).  Over more entries a row
// has fewer tokens (1024 x 1000: 1.95e-3, 2048 x 8000: 1.67e-3), and the term costs up to a third.
constexpr int64_t kSecondValues = 1 << 22;
// Those of an accumulator of the gradients' products: 2^20 terms of one sign in one accumulator
// fell short by 4.3e-3 of themselves, more than the output's rounding leaves; by 8192 no shortfall
// is left to be seen (8e-6), at 0 to 0.5 % of the time (8192 x 50 001, D 512: 801 us, 805).
constexpr int kSumSteps = 128;

enum Mode {
    kLoss,    // h W^T: parts of the logits' log-sum-exp, the targets' logits
    kGrad,    // h W^T: G, and its columns' sums
    kProducts // G W and G^T (w h), one after the other: dh's and dW's
};
// What becomes of a product.
enum Out {
    kBf16,     // rounded
    kWeighted, // a row times its token's weight, rounded
    kF32,      // in 32 bits, each split to a place of its own
    kAdd       // ... added to what is there
};

// Division of numbers below 2^31 by a fixed one: n m >> 32 >> s with m = 2^(32 + s) / d
// rounded up and 2^s < d <= 2^(s + 1), which errs by less than n d / 2^(32 + s) < 1 / d.
struct Divisor {
    uint32_t m, s, d;
    Divisor() = default;
    explicit Divisor(int by) : m(0), s(0), d((uint32_t)by) {
        while ((2u << s) < d)
            ++s;
        if (d > 1)
            m = (uint32_t)(((uint64_t)1 << (32 + s)) / d + 1);
    }
#ifdef __CUDACC__
    FW_DEV int of(int n) const { return d > 1 ? (int)(__umulhi((uint32_t)n, m) >> s) : n; }
#endif
};

// One product's tiles, 256 x 256 of the output each, and how they are walked.
struct Product {
    int mt, nt;          // tiles of the output
    int kb, per, splits; // 64-steps of the contraction, and those of a split
    int group;           // tile rows that are walked together, column by column
    Divisor by_split, by_group, by_rows, by_last; // a split's tiles, a group's, a group's rows, the last group's rows
    int b0;              // B's first row
    int a_steps;         // steps after which A begins anew (B goes on: the second terms of its rows)
    int N, V;            // rows and columns of the output that are there
    int out;             // Out (kProducts)
    int rows_a_split;    // kF32, kAdd: rows between the splits' outputs
    int tiles;           // of all splits
};

struct GemmArgs {
    Product of[2];      // (the second: kProducts alone)
    int extra;          // see walk
    int chunk;          // steps of an accumulator
    const float *bias;  // kLoss, kGrad: of this piece, or null
    Tokens targets;
    int vocab;          // all of the vocabulary's entries
    float2 *part;       // kLoss: [ceil(V / 64)][N] (reference, sum)
    float *target_z;    // kLoss: [N]
    const float4 *row;  // kGrad, kWeighted: [N] of each token (see row_constants), and its target, -1 for none
    const int *row_target;
    float *colsum;      // kGrad: [ceil(N / 32)][ldc] or null
    int ldc;
};
struct Maps {
    CUtensorMap a, b, out; // of a product
};

FW_DEV uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
FW_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
FW_DEV uint32_t leader_addr(const void *p) { // the pair's first CTA's location of the same name
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
// A box into this CTA's shared memory, its bytes counted on the leader's barrier.
FW_DEV void tma_load_pair(void *dst, const void *map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}
FW_DEV void tma_store(const void *map, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
}
FW_DEV void tma_add(const void *map, const void *src, int x, int y) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(src)), "r"(x), "r"(y)
                 : "memory");
}
FW_DEV void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// Arrive on `bar` of both CTAs once every MMA issued so far has completed.
FW_DEV void commit_pair(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}
// (relaxed: what it tells of are this warp's reads of TMEM, which have completed; a release
// would hold the warp at a cluster-scope fence)
FW_DEV void arrive_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// (the wait in the same statement: nothing that reads the registers gets between)
FW_DEV void tmem_ld32(uint32_t taddr, float *r) {
    uint32_t u[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
                   "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
                   "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]),
                   "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]),
                   "=r"(u[30]), "=r"(u[31])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i)
        r[i] = __uint_as_float(u[i]);
}

// 16 columns of an accumulator added to z.
FW_DEV void add_tmem(uint32_t taddr, float *z) {
    uint32_t u[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
                   "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int j = 0; j < 16; ++j)
        z[j] += __uint_as_float(u[j]);
}

// Lane l's sum over the warp's lanes of value l of the 32 at x: halves are exchanged and added.
FW_DEV float columns_sum(float *x, int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int j = 0; j < o; ++j) {
            const float give = up ? x[j] : x[j + o], keep = up ? x[j + o] : x[j];
            x[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return x[0];
}

// kLoss, kGrad: both operands' memory runs along the contraction.  kProducts: B's
// runs along the output, and so does A's of the second product.
template <Mode MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kT, 1)
    vocab_gemm_kernel(const __grid_constant__ Maps maps0, const __grid_constant__ Maps maps1,
                      const __grid_constant__ GemmArgs g, unsigned *status) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = (uint64_t *)(smem + kBarOff); // [kStages] (leader's) both CTAs' copies of a step have landed
    uint64_t *empty = full + kStages;              // [kStages] the step's MMAs are done
    uint64_t *ready = empty + kStages;             // [2] a tile's accumulator is complete
    uint64_t *taken = ready + 2;                   // [2] (leader's) ... and has been read by both CTAs
    uint32_t *slot = (uint32_t *)(taken + 2);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(ready + s, 1);
            mbar_init(taken + s, 2 * kEpiWarps);
        }
        fence_barrier_init();
    }
    if (warp == 2) { // (both CTAs' warps: the allocation is the pair's)
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync(); // the barriers stand in both CTAs
    tc_fence_after();
    griddep_launch_dependents();
    griddep_wait();
    const float *const bias = after_wait(g.bias);
    const Tokens targets = {after_wait(g.targets.p), g.targets.wide};
    const float4 *const rows = after_wait(g.row);
    const int *const row_targets = after_wait(g.row_target);
    const uint32_t tm = *slot;

    // Tile i of this pair's walk: of product w, rows mb, columns nb, split z; false past
    // the last.  The first product's tiles are dealt to the pairs in turn, then the
    // second's: `extra` each to the pairs that got one fewer of the first's (as many as make
    // up for it), the rest in turn from those on.
    struct At {
        int w, mb, nb, k0, k1, z;
    };
    auto walk = [&](int i, At &p) {
        const int n0 = g.of[0].tiles;
        int t = pair + i * pairs;
        p.w = 0;
        if (t >= n0) {
            if (MODE != kProducts)
                return false;
            p.w = 1;
            const int more = n0 % pairs; // pairs below it have one of the first product's more
            int j = i - (n0 / pairs + (pair < more ? 1 : 0));
            const int late = pairs - more;
            if (more && pair >= more) {
                if (j < g.extra) {
                    t = pair - more + j * late;
                    j = -1;
                } else {
                    j -= g.extra;
                }
            }
            if (j >= 0)
                t = (more ? g.extra * late : 0) + (pair >= more ? pair - more : pair + late) + j * pairs;
            if (t >= g.of[1].tiles)
                return false;
        }
        const Product &q = g.of[MODE == kProducts ? p.w : 0];
        p.z = q.by_split.of(t);
        int r = t - p.z * (int)q.by_split.d;
        const int gi = q.by_group.of(r);
        r -= gi * (int)q.by_group.d;
        const bool last = (gi + 1) * q.group > q.mt;
        p.nb = last ? q.by_last.of(r) : q.by_rows.of(r);
        p.mb = gi * q.group + r - p.nb * (int)(last ? q.by_last.d : q.by_rows.d);
        p.k0 = p.z * q.per;
        p.k1 = min(q.kb, p.k0 + q.per);
        return true;
    };

    if (warp == 0 && lane == 0) { // copies
        uint32_t step = 0;
        bool ok = true;
        At p;
        for (int i = 0; ok && walk(i, p); ++i) {
            const int m = p.mb * kTile + (int)rank * 128, n = p.nb * kTile + (int)rank * 128;
            const bool second = MODE == kProducts && p.w;
            const CUtensorMap *ta = second ? &maps1.a : &maps0.a, *tb = second ? &maps1.b : &maps0.b;
            const int b0 = g.of[second].b0;
            for (int k = p.k0; k < p.k1; ++k, ++step) {
                const uint32_t s = step % kStages, use = step / kStages;
                if (use > 0 && !mbar_wait(empty + s, (use - 1) & 1, status)) {
                    ok = false;
                    break;
                }
                uint8_t *a = smem + s * kStageBytes, *b = a + 16384;
                const uint32_t bar = leader_addr(full + s);
                if (rank == 0)
                    mbar_arrive_expect_tx(full + s, 2 * kStageBytes);
                if (second) {
                    const int ka = k < g.of[1].a_steps ? k : k - g.of[1].a_steps;
                    tma_load_pair(a, ta, m, 64 * ka, bar);
                    tma_load_pair(a + 8192, ta, m + 64, 64 * ka, bar);
                } else {
                    tma_load_pair(a, ta, 64 * k, m, bar);
                }
                if (MODE == kProducts) {
                    tma_load_pair(b, tb, n, b0 + 64 * k, bar);
                    tma_load_pair(b + 8192, tb, n + 64, b0 + 64 * k, bar);
                } else {
                    tma_load_pair(b, tb, 64 * k, b0 + n, bar);
                }
            }
        }
        // no arrival of the MMAs' commits is under way to this CTA when it leaves
        for (uint32_t s = 0; ok && s < kStages && s < step; ++s) {
            const uint32_t uses = (step - s + kStages - 1) / kStages;
            ok = mbar_wait(empty + s, (uses - 1) & 1, status);
        }
        // where a wait gave up: what both CTAs have under way lands before either leaves
        // (they leave together, and the bytes of both are counted on the leader's barriers)
        for (uint32_t j = step > kStages ? step - kStages : 0; !ok && rank == 0 && j < step; ++j)
            (void)mbar_wait(full + j % kStages, (j / kStages) & 1, status);
    } else if (warp == 1 && lane == 0 && rank == 0) { // products
        uint32_t step = 0, it = 0; // steps, and accumulators filled, so far
        bool ok = true;
        auto fill = [&](int k0, int k1, bool second) { // an accumulator takes steps k0 .. k1 - 1, from zero
            constexpr int kBMn = MODE == kProducts;
            const uint32_t idesc = second ? idesc_bf16(256, 256, 1, kBMn) : idesc_bf16(256, 256, 0, kBMn);
            // (a step of 16 lies 32 bytes on in rows that run along the contraction, 16 rows on in others)
            const uint32_t a_step = second ? 2048 : 32, b_step = kBMn ? 2048 : 32;
            const uint32_t a_lbo = second ? 8192 : 16, b_lbo = kBMn ? 8192 : 16;
            const uint32_t buf = it & 1, d = tm + buf * 256;
            if (it >= 2 && !mbar_wait(taken + buf, ((it >> 1) - 1) & 1, status))
                return false;
            tc_fence_after();
            for (int k = k0; k < k1; ++k, ++step) {
                const uint32_t s = step % kStages;
                if (!mbar_wait(full + s, (step / kStages) & 1, status))
                    return false;
                tc_fence_after();
                const uint32_t a = smem_u32(smem + s * kStageBytes), b = a + 16384;
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                    const uint64_t da = desc_sw128(a + st * a_step, a_lbo, 1024), db = desc_sw128(b + st * b_step, b_lbo, 1024);
                    mma_pair(d, da, db, idesc, k > k0 || st > 0);
                }
                commit_pair(empty + s);
            }
            commit_pair(ready + buf);
            ++it;
            return true;
        };
        At p;
        for (int i = 0; ok && walk(i, p); ++i) {
            for (int k = p.k0; ok && k < p.k1; k += g.chunk)
                ok = fill(k, min(k + g.chunk, p.k1), MODE == kProducts && p.w);
        }
        // every read of an accumulator has been told of
        for (uint32_t buf = 0; ok && buf < 2 && buf < it; ++buf)
            ok = mbar_wait(taken + buf, (((it - buf + 1) >> 1) - 1) & 1, status);
    } else if (warp >= 4) { // epilogue: lane = row
        const int quarter = warp & 3, part = (warp - 4) >> 2; // which 32 rows, which 64 columns
        uint8_t *out = smem + kOutOff + (warp - 4) * 4096;
        uint32_t it = 0; // accumulators read so far
        auto free_box = [&]() { // the staging box is free of the store before
            if (lane == 0)
                bulk_wait_read();
            __syncwarp();
        };
        auto put = [&](const CUtensorMap *to, int x, int y, bool add) { // it leaves
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (add)
                    tma_add(to, out, x, y);
                else
                    tma_store(to, out, x, y);
                bulk_commit();
            }
        };
        // the accumulator that is complete next, and word that it has been read
        auto next_acc = [&](uint32_t &acc) {
            if (!mbar_wait(ready + (it & 1), (it >> 1) & 1, status))
                return false;
            tc_fence_after();
            acc = tm + tmem_lane_base(warp) + (it & 1) * 256 + kCols * part;
            return true;
        };
        auto done_with_acc = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_at(leader_addr(taken + (it & 1)));
            ++it;
        };
        At p;
        for (int i = 0; walk(i, p); ++i) {
            const Product &q = g.of[MODE == kProducts ? p.w : 0];
            const int row0 = p.mb * kTile + (int)rank * 128 + 32 * quarter, row = row0 + lane;
            const int col0 = p.nb * kTile + kCols * part;
            const bool needed = row0 < q.N && col0 < q.V; // (else nothing of this warp's part is there)
            uint32_t acc = 0;
            if (MODE != kProducts) {
                // what the row brings (used once the logits are there: the loads are under way until then)
                int target = -1;
                float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
                if (needed && row < q.N) {
                    if (MODE == kLoss) {
                        target = token_at(targets, row, g.vocab);
                        target = target < g.vocab ? target : -1; // (past the vocabulary: none of the columns)
                    } else {
                        target = __ldcg(row_targets + row);
                        c = __ldcg(rows + row);
                    }
                }
                // its logits, from the bias on
                float z[kCols];
                const bool from_bias = bias && needed;
                if (from_bias) {
                    if (col0 + kCols <= q.V) {
#pragma unroll
                        for (int j = 0; j < kCols / 4; ++j) {
                            const float4 b = __ldcg(reinterpret_cast<const float4 *>(bias + col0) + j);
                            z[4 * j] = b.x;
                            z[4 * j + 1] = b.y;
                            z[4 * j + 2] = b.z;
                            z[4 * j + 3] = b.w;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < kCols; ++j)
                            z[j] = col0 + j < q.V ? __ldcg(bias + col0 + j) : 0.f;
                    }
                }
                bool ok = true;
                for (int k = p.k0; k < p.k1; k += g.chunk) {
                    ok = next_acc(acc);
                    if (!ok)
                        break;
                    if (needed) {
                        if (k == p.k0 && !from_bias) {
                            tmem_ld32(acc, z);
                            tmem_ld32(acc + 32, z + 32);
                        } else {
#pragma unroll
                            for (int i = 0; i < kCols; i += 16)
                                add_tmem(acc + i, z + i);
                        }
                    }
                    done_with_acc();
                }
                if (!ok)
                    break;
                if (!needed)
                    continue;
                if (col0 + kCols > q.V) { // nothing past the vocabulary
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        z[j] = col0 + j < q.V ? z[j] : -INFINITY;
                }
                const int tk = target < 0 ? -1 : target - q.b0 - col0; // the target's place among these (or not)
                if (MODE == kLoss) {
                    if (tk >= 0 && tk < kCols) {
                        float tz = 0.f;
#pragma unroll
                        for (int j = 0; j < kCols; ++j) { // (kept apart: the loss is log(1 + the others / it))
                            tz = j == tk ? z[j] : tz;
                            z[j] = j == tk ? -INFINITY : z[j];
                        }
                        g.target_z[row] = tz;
                    }
                    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int j = 0; j < kCols; j += 2)
                        m[(j >> 1) & 3] = fmaxf(m[(j >> 1) & 3], fmaxf(z[j], z[j + 1]));
                    const float ref = reference(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])));
                    float s[4] = {};
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        s[j & 3] += ex2(fmaf(z[j], kLog2e, -ref));
                    const float total = (s[0] + s[1]) + (s[2] + s[3]);
                    if (row < q.N)
                        g.part[(size_t)(col0 / kCols) * q.N + row] = make_float2(total == 0.f ? kNoRef : ref, total);
                } else {
                    const float ref = c.x, at_target = c.z, weight = c.w, weight_off = c.w * c.y;
                    const bool live = target >= 0;
                    free_box();
#pragma unroll
                    for (int j = 0; j < kCols; j += 8) {
                        float e[8];
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            e[x] = ex2(fmaf(z[j + x], kLog2e, -ref));
                        *reinterpret_cast<uint4 *>(out + lane * 128 + (((j >> 3) ^ (lane & 7)) << 4)) =
                            make_uint4(pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                                       pack_bf16x2(e[6], e[7]));
                        if (g.colsum)
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                z[j + x] = live ? (tk == j + x ? at_target * weight : e[x] * weight_off) : 0.f;
                    }
                    if (tk >= 0 && tk < kCols) // the target's entry
                        *reinterpret_cast<__nv_bfloat16 *>(out + lane * 128 + (((tk >> 3) ^ (lane & 7)) << 4) + 2 * (tk & 7)) =
                            __float2bfloat16_rn(at_target);
                    if (!live) // no gradient: zeros, whatever the logits are
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4 *>(out + lane * 128 + 16 * j) = make_uint4(0, 0, 0, 0);
                    put(&maps0.out, col0, row0, false);
                    if (g.colsum)
#pragma unroll
                        for (int c1 = 0; c1 < kCols; c1 += 32)
                            g.colsum[(size_t)(row0 / 32) * g.ldc + col0 + c1 + lane] = columns_sum(z + c1, lane);
                }
            } else {
                float v[kCols];
                bool ok = true;
                for (int k = p.k0; k < p.k1; k += g.chunk) {
                    ok = next_acc(acc);
                    if (!ok)
                        break;
                    if (needed) {
                        if (k == p.k0) {
                            tmem_ld32(acc, v);
                            tmem_ld32(acc + 32, v + 32);
                        } else {
#pragma unroll
                            for (int j = 0; j < kCols; j += 16)
                                add_tmem(acc + j, v + j);
                        }
                    }
                    done_with_acc();
                }
                if (!ok)
                    break;
                if (!needed)
                    continue;
                const CUtensorMap *to = p.w ? &maps1.out : &maps0.out;
                if (q.out == kWeighted) {
                    const bool there = row < q.N && __ldcg(row_targets + row) >= 0;
                    const float w = there ? __ldcg(rows + row).w : 0.f;
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        v[j] = there ? v[j] * w : 0.f;
                }
                free_box();
                if (q.out == kBf16 || q.out == kWeighted) {
#pragma unroll
                    for (int j = 0; j < kCols; j += 8) {
                        uint4 u;
                        u.x = pack_bf16x2(v[j], v[j + 1]);
                        u.y = pack_bf16x2(v[j + 2], v[j + 3]);
                        u.z = pack_bf16x2(v[j + 4], v[j + 5]);
                        u.w = pack_bf16x2(v[j + 6], v[j + 7]);
                        *reinterpret_cast<uint4 *>(out + lane * 128 + (((j >> 3) ^ (lane & 7)) << 4)) = u;
                    }
                    put(to, col0, row0, false);
                } else {
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) { // 32 columns of fp32 a box
                        if (c && col0 + c >= q.V)
                            break;
                        if (c)
                            free_box();
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4 *>(out + lane * 128 + (((j >> 2) ^ (lane & 7)) << 4)) =
                                make_float4(v[c + j], v[c + j + 1], v[c + j + 2], v[c + j + 3]);
                        put(to, col0 + c, row0 + p.z * q.rows_a_split, q.out == kAdd);
                    }
                }
            }
        }
        if (MODE != kLoss && lane == 0)
            bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync(); // nothing is under way between the CTAs
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tm), "r"(512) : "memory");
}

constexpr int kS = 256;

// What is left of a piece, by the CTA: dh's rows and dW's from the sums of the splits,
// added in order and rounded once (dh's times their weight, zeros without a gradient),
// and dbias from the sums of 32 tokens each, in order.
struct Rest {
    const float *part; // [splits][a_split]
    __nv_bfloat16 *out;
    int rows, splits, ctas;
    int64_t a_split;
};
struct RestArgs {
    Rest dh, dw; // (ctas 0: nothing to do)
    const float4 *row;
    const int *row_target;
    const float *colsum;
    float *dbias;
    int D, lg, V, blocks, ldc;
};

FW_DEV void join_rows(const Rest &q, const RestArgs &a, int cta, bool tokens) {
    const int n = cta * (kS >> a.lg) + (int)(threadIdx.x >> a.lg), lane = threadIdx.x & ((1 << a.lg) - 1);
    if (n >= q.rows)
        return;
    const bool live = !tokens || __ldcg(a.row_target + n) >= 0;
    const float w = tokens ? __ldcg(a.row + n).w : 1.f;
    for (int c = 8 * lane; c < a.D; c += 8 << a.lg) {
        float s[8] = {};
        if (live) {
            const float *p = q.part + (int64_t)n * a.D + c;
            int z = 0;
            for (; z < q.splits; z += 8) {
                float v[8][8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (z + u < q.splits)
                        load8(p + (z + u) * q.a_split, v[u]);
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (z + u < q.splits)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            s[e] += v[u][e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[e] = live ? s[e] * w : 0.f;
        store8(q.out + (size_t)n * a.D + c, s);
    }
}

__global__ void __launch_bounds__(kS) rest_kernel(RestArgs a) {
    __shared__ float red[kS / 32][33];
    griddep_launch_dependents();
    griddep_wait();
    a.dh.part = after_wait(a.dh.part);
    a.dw.part = after_wait(a.dw.part);
    a.row = after_wait(a.row);
    a.row_target = after_wait(a.row_target);
    a.colsum = after_wait(a.colsum);
    int cta = (int)blockIdx.x;
    if (cta < a.dh.ctas)
        return join_rows(a.dh, a, cta, true);
    cta -= a.dh.ctas;
    if (cta < a.dw.ctas)
        return join_rows(a.dw, a, cta, false);
    cta -= a.dw.ctas;
    const int i = threadIdx.x & 31, w = threadIdx.x >> 5, v = cta * 32 + i;
    float s = 0.f;
    for (int k = w; k < a.blocks; k += kS / 32 * 8) {
        float t[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            t[u] = k + u * (kS / 32) < a.blocks ? __ldcg(a.colsum + (size_t)(k + u * (kS / 32)) * a.ldc + v) : 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            s += t[u];
    }
    red[w][i] = s;
    __syncthreads();
    if (w == 0 && v < a.V) {
        s = 0.f;
#pragma unroll
        for (int k = 0; k < kS / 32; ++k)
            s += red[k][i];
        a.dbias[v] = s;
    }
}

// ------------------------------------------------------------------- plans
int tiles_of(int64_t n) { return (int)((n + kTile - 1) / kTile); }

// Splits of a contraction of kb steps for an output of `tiles`: where the
// tiles occupy no more than a quarter of the pairs, as many as fill them, of four
// steps at least.  (16 tiles, gradients of 2048 x 8000 at D 512: 52 us, not split 61; of
// 4096 x 32 000 at D 256: 186, 236.  Splits of few steps cost more in sums than they gain:
// 2048 x 2500 at D 512 37 us, not split 30; 1024 x 1000 at D 1024 30.5, 22.4.)
struct Splits {
    int n, per;
};
Splits splits_of(int64_t tiles, int kb) {
    int64_t n = tiles * 4 > kPairs ? 1 : std::min<int64_t>(kPairs / tiles, (kb + 3) / 4);
    n = std::max<int64_t>(1, n);
    const int per = (int)((kb + n - 1) / n);
    return {(kb + per - 1) / per, per};
}

// Whether w h goes into dW's product in two terms.
bool second_terms(int N, int V, int D) {
    return N <= kFewTokens || (V <= kTile && (int64_t)N * D <= kSecondValues);
}
struct Plan {
    int width;      // vocabulary entries of a piece (a multiple of 256)
    int ldg;        // row stride of G
    int pieces;
    int lo_rows;    // w h in two terms: the second ones from this row on (0: one term)
    Splits dh, dw;
    size_t row, row_target, G, wh, dh_part, dw_part, colsum, bytes; // offsets
};
Plan plan_of(int N, int V, int D) {
    Plan p;
    const int vt = tiles_of(V), kt = (D + kTile - 1) / kTile;
    const int64_t most = std::max<int64_t>(1, (int64_t)(kPieceBytes / ((size_t)2 * kTile * N)));
    const int64_t pieces = (vt + most - 1) / most;
    p.width = (int)((vt + pieces - 1) / pieces) * kTile;
    p.ldg = p.width;
    p.pieces = (V + p.width - 1) / p.width;
    p.dh = splits_of((int64_t)tiles_of(N) * kt, (std::min(p.width, V) + 63) / 64);
    const int kn = (N + 63) / 64;
    p.lo_rows = second_terms(N, V, D) ? 64 * kn : 0;
    p.dw = splits_of((int64_t)(p.width / kTile) * kt, kn);
    if (p.lo_rows)
        p.dw.per *= 2;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += up256(bytes);
        return o;
    };
    p.row = take(sizeof(float4) * (size_t)N);
    p.row_target = take(sizeof(int) * (size_t)N);
    p.G = take((size_t)2 * N * p.ldg);
    p.wh = take((size_t)2 * (p.lo_rows ? 2 * p.lo_rows : N) * D);
    // dh goes through sums in 32 bits where it has several parts (rows in whole tiles)
    p.dh_part = take(p.dh.n * p.pieces > 1 ? (size_t)4 * p.dh.n * tiles_of(N) * kTile * D : 0);
    p.dw_part = take(p.dw.n > 1 ? (size_t)4 * p.dw.n * p.width * D : 0);
    p.colsum = take((size_t)4 * ((N + 31) / 32) * p.width);
    p.bytes = at;
    return p;
}

// Pairs of CTAs that the device runs at once.
template <typename K> cudaError_t pairs_of(K *kern, int *out) {
    static std::atomic<int> known[64]; // by device; what it holds does not depend on who asks first
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const int have = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (have > 0) {
        *out = have;
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kT);
    cfg.dynamicSmemBytes = kSmem;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
    if (e != cudaSuccess)
        return e;
    n = std::max(1, n);
    if (dev < 64)
        known[dev].store(n, std::memory_order_relaxed);
    *out = n;
    return cudaSuccess;
}

// The tiles of a product of M x V by kb steps.
Product product(int M, int V, int kb, int per, int group) {
    Product q = {};
    q.mt = tiles_of(M);
    q.nt = tiles_of(V);
    q.kb = kb;
    q.per = per;
    q.splits = (kb + per - 1) / per;
    q.group = std::min(group, q.mt);
    q.by_split = Divisor(q.mt * q.nt);
    q.by_group = Divisor(q.group * q.nt);
    q.by_rows = Divisor(q.group);
    q.by_last = Divisor(q.mt % q.group ? q.mt % q.group : q.group);
    q.N = M;
    q.V = V;
    q.tiles = q.mt * q.nt * q.splits;
    return q;
}

template <Mode MODE> cudaError_t launch_gemm(const Maps &maps0, const Maps &maps1, GemmArgs g, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    auto kern = vocab_gemm_kernel<MODE>;
    cudaError_t e = allow_smem(kern, done);
    unsigned *status = nullptr;
    if (e == cudaSuccess)
        e = status_word(&status);
    int pairs = 0;
    if (e == cudaSuccess)
        e = pairs_of(kern, &pairs);
    if (e != cudaSuccess)
        return e;
    pairs = (int)std::min<int64_t>(pairs, (int64_t)g.of[0].tiles + g.of[1].tiles);
    const int more = g.of[0].tiles % pairs;
    if (MODE == kProducts && more && g.of[1].tiles) // (see walk)
        g.extra = std::min((g.of[0].per + g.of[1].per / 2) / g.of[1].per, g.of[1].tiles / (pairs - more));
    return launch_pdl(kern, dim3((unsigned)(2 * pairs)), dim3(kT), kSmem, st, maps0, maps1, g, status);
}

// Tile rows walked together in the products over tokens: their rows of A stay in L2 (32 MB of them).
int token_group(int N, int D) { return (int)std::max<int64_t>(8, std::min<int64_t>(tiles_of(N), (32 << 20) / ((int64_t)kTile * D * 2))); }


} // namespace

cudaError_t vocab::launch_join_bias(const float *colsum, float *dbias, int V, int blocks, int ldc, cudaStream_t st) {
    RestArgs r = {};
    r.colsum = colsum;
    r.dbias = dbias;
    r.V = V;
    r.blocks = blocks;
    r.ldc = ldc;
    return launch_pdl(rest_kernel, dim3((V + 31) / 32), dim3(kS), 0, st, r);
}

size_t vocab_loss_workspace_bytes(int N, int V, int D) {
    return up256(sizeof(float2) * (size_t)parts_of(N, V, D) * N) + up256(sizeof(float) * (size_t)N);
}

cudaError_t launch_vocab_loss(const void *h, const void *W, const float *bias, Tokens targets, float *loss, float *lse,
                              void *workspace, int N, int V, int D, int bf16, cudaStream_t st) {
    const int nparts = parts_of(N, V, D);
    float2 *part = static_cast<float2 *>(workspace);
    float *target_z = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + up256(sizeof(float2) * (size_t)nparts * N));
    cudaError_t e;
    if (few(N, D)) {
        e = launch_few(h, W, bias, targets, part, target_z, N, V, D, bf16, st);
    } else if (!bf16) {
        e = loss_products_f32(static_cast<const float *>(h), static_cast<const float *>(W), bias, targets, part, target_z, N,
                              V, D, st);
    } else {
        const int kb = (D + 63) / 64;
        GemmArgs g = {};
        g.vocab = V;
        g.bias = bias;
        g.targets = targets;
        g.part = part;
        g.target_z = target_z;
        g.of[0] = product(N, V, kb, kb, token_group(N, D));
        g.chunk = N <= kFewTokens ? kFewLogitSteps : kLogitSteps;
        Maps m;
        e = make_bf16_map(&m.a, h, N, D, D, 128);
        if (e == cudaSuccess)
            e = make_bf16_map(&m.b, W, V, D, D, 128);
        m.out = m.a; // (not read)
        if (e == cudaSuccess)
            e = launch_gemm<kLoss>(m, m, g, st);
    }
    return e != cudaSuccess ? e : launch_join_parts(part, target_z, targets, loss, lse, N, V, nparts, st);
}

size_t vocab_loss_backward_workspace_bytes(int N, int V, int D, int bf16) {
    return bf16 ? plan_of(N, V, D).bytes : backward_workspace_f32(N, V, D);
}

cudaError_t launch_vocab_loss_backward(const void *h, const void *W, const float *bias, Tokens targets,
                                       const float *loss, const float *lse, const float *dloss, void *dh, void *dW,
                                       float *dbias, void *workspace, int N, int V, int D, int bf16, cudaStream_t st) {
    if (!bf16)
        return backward_f32(static_cast<const float *>(h), static_cast<const float *>(W), bias, targets, loss, lse, dloss,
                            static_cast<float *>(dh), static_cast<float *>(dW), dbias, workspace, N, V, D, st);
    const Plan p = plan_of(N, V, D);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    __nv_bfloat16 *G = reinterpret_cast<__nv_bfloat16 *>(ws + p.G), *wh = reinterpret_cast<__nv_bfloat16 *>(ws + p.wh);
    float *dh_part = reinterpret_cast<float *>(ws + p.dh_part), *dw_part = reinterpret_cast<float *>(ws + p.dw_part);
    float *colsum = reinterpret_cast<float *>(ws + p.colsum);
    const int lg = group_log2(D), per_cta = kS >> lg, kd = (D + 63) / 64, kn = (N + 63) / 64;
    const int64_t dh_rows = (int64_t)tiles_of(N) * kTile;
    const bool dh_direct = p.dh.n * p.pieces == 1, dw_direct = p.dw.n == 1;
    float4 *row = reinterpret_cast<float4 *>(ws + p.row);
    int *row_target = reinterpret_cast<int *>(ws + p.row_target);
    // h and W along their width, G as it is written; G and W for dh, G and w h for dW
    Maps logits, to_dh, to_dw;
    cudaError_t e = make_bf16_map(&logits.a, h, N, D, D, 128);
    if (e == cudaSuccess) e = make_bf16_map(&logits.b, W, V, D, D, 128);
    if (e == cudaSuccess) e = make_bf16_map(&logits.out, G, N, p.ldg, p.ldg, 32);
    if (e == cudaSuccess) e = make_bf16_map(&to_dh.a, G, N, p.ldg, p.ldg, 128);
    if (e == cudaSuccess) e = make_bf16_map(&to_dh.b, W, V, D, D, 64);
    if (e == cudaSuccess && dh)
        e = dh_direct ? make_bf16_map(&to_dh.out, dh, N, D, D, 32)
                      : make_f32_sw128_map(&to_dh.out, dh_part, (int)(p.dh.n * dh_rows), D, D, 32);
    if (e == cudaSuccess) e = make_bf16_map(&to_dw.a, G, N, p.ldg, p.ldg, 64);
    if (e == cudaSuccess) e = make_bf16_map(&to_dw.b, wh, p.lo_rows ? 2 * p.lo_rows : N, D, D, 64);
    if (e == cudaSuccess && dW && !dw_direct)
        e = make_f32_sw128_map(&to_dw.out, dw_part, p.dw.n * p.width, D, D, 32);
    if (e == cudaSuccess)
        e = launch_rows(h, targets, loss, lse, dloss, row, row_target, dW ? wh : nullptr, p.lo_rows, true, N, V, D, st);
    for (int v0 = 0; e == cudaSuccess && v0 < V; v0 += p.width) {
        const int nv = std::min(p.width, V - v0);
        const bool last = v0 + p.width >= V;
        GemmArgs g = {};
        g.of[0] = product(N, nv, kd, kd, token_group(N, D));
        g.of[0].b0 = v0;
        g.chunk = N <= kFewTokens ? kFewLogitSteps : kLogitSteps;
        g.vocab = V;
        g.bias = bias ? bias + v0 : nullptr;
        g.row = row;
        g.row_target = row_target;
        g.colsum = dbias ? colsum : nullptr;
        g.ldc = p.width;
        e = launch_gemm<kGrad>(logits, logits, g, st);
        __nv_bfloat16 *dw_piece = dW ? static_cast<__nv_bfloat16 *>(dW) + (size_t)v0 * D : nullptr;
        if (e == cudaSuccess && (dh || dW)) {
            GemmArgs q = {};
            q.row = row;
            q.row_target = row_target;
            q.chunk = kSumSteps;
            q.of[1].per = 1;
            if (dh) {
                q.of[0] = product(N, D, (nv + 63) / 64, p.dh.per, 4);
                q.of[0].b0 = v0;
                q.of[0].out = dh_direct ? kWeighted : v0 ? kAdd : kF32;
                q.of[0].rows_a_split = (int)dh_rows;
            }
            if (dW) {
                q.of[1] = product(nv, D, p.lo_rows ? 2 * kn : kn, p.dw.per, 4);
                q.of[1].a_steps = kn;
                q.of[1].out = dw_direct ? kBf16 : kF32;
                q.of[1].rows_a_split = p.width;
                if (dw_direct)
                    e = make_bf16_map(&to_dw.out, dw_piece, nv, D, D, 32);
            }
            if (e == cudaSuccess)
                e = launch_gemm<kProducts>(to_dh, to_dw, q, st);
        }
        RestArgs r = {};
        if (dh && last && !dh_direct)
            r.dh = {dh_part, static_cast<__nv_bfloat16 *>(dh), N, p.dh.n, (N + per_cta - 1) / per_cta, dh_rows * D};
        if (dW && !dw_direct)
            r.dw = {dw_part, dw_piece, nv, p.dw.n, (nv + per_cta - 1) / per_cta, (int64_t)p.width * D};
        r.row = row;
        r.row_target = row_target;
        r.colsum = colsum;
        r.dbias = dbias ? dbias + v0 : nullptr;
        r.D = D;
        r.lg = lg;
        r.V = nv;
        r.blocks = (N + 31) / 32;
        r.ldc = p.width;
        const int ctas = r.dh.ctas + r.dw.ctas + (dbias ? (nv + 31) / 32 : 0);
        if (e == cudaSuccess && ctas)
            e = launch_pdl(rest_kernel, dim3(ctas), dim3(kS), 0, st, r);
    }
    return e;
}

} // namespace fw
