// kq_i8_tc.cu -- tensor-core int8 product with one scale per token and per output channel.
//
// sm_103a has no int8 tcgen05 MMA, so the integer sum is carried exactly on the f16 tensor pipe: codes of
// -128..127 are exact in f16, their products in fp32, and a sum of 1024 products stays within
// 1024 * 2^14 = 2^24, where fp32 still holds every integer.  So an accumulator in tensor memory runs over
// 1024 elements of K at most (a chunk) and is then added to int32 sums in the epilogue's registers.
//   * weights (int8 rows) reach shared memory by TMA; converter warps turn 128 rows x 128 codes into f16
//     and store them into tensor memory, where the MMA reads them as its A operand.
//   * activations come as an f16 panel (written once by a prologue), by TMA, as the B operand.
//   * outputs: weight rows = TMEM lanes, tokens = columns.
// Large products: a pair of CTAs (cta_group::2) computes 256 rows x 256 tokens; each CTA converts its own
// 128 rows and loads half of the tokens.  [14336 x 4096], 2048 tokens, bf16 out: 137 us in short bursts, 1.76
// PFLOP/s, 0.94 of what a plain bf16 product reaches so.  The accumulator's two 128-token halves are filled in turn,
// four units (of 128 K) each, so that one half's chunk is read out (1 us) while the other half computes (1.2 us; with
// two units each it waited 0.8 us a chunk).
// (Tiles of fewer tokens, to cover a batch with less, are left out: an MMA of 96 columns takes nearly as long as one
// of 128.  768 tokens took 69 us in three waves of 192s for 74 in 256s, but the choice made the 256s 5% slower.)
// Small products: one CTA, 128 rows x 32, 64 or 128 tokens, two accumulators taking turns chunk by
// chunk; up to 64 tokens are converted from int8 by the CTA itself, without a panel.
// Few tiles split K over a cluster; its CTAs exchange their int32 sums through distributed shared memory,
// which is exact in any order.
//
// Roles: EPI warps read accumulators (TMEM lane quarter = warp % 4), CONV warps convert weights, one warp
// loads weights, ACT warps load or convert activations, one issues MMAs (in the pair: the first CTA's only).
// Every wait is bounded; on expiry the CTA counts an error in the device flag and leaves in order.
#include <algorithm>
#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include "kq_i8_tc.cuh"
#include "kq_launch.cuh"

namespace kq {

using namespace sm100;

constexpr int I8_ROWS = 128;      // weight rows of a CTA's tile: TMEM lanes
constexpr int I8_KS = 64;         // K per activation tile (a 128-byte swizzled row of f16)
constexpr int I8_UNIT = 128;      // K per unit: a weight tile, two activation tiles, one TMEM stage of A
constexpr int I8_CHUNK = 8;       // units per chunk: 1024 elements, the longest exact fp32 accumulation
constexpr int I8_MAX_SPLIT = 8;  // CTAs that share a tile's K (portable cluster size)

template <int CG_, int NT_, int EPI_, int CONV_, int STAGES_, int WSTAGES_>
struct I8Cfg {
    static constexpr int CG = CG_;                // CTAs per tile
    static constexpr int NT = NT_;                // tokens per tile
    static constexpr int H = NT > 128 ? 2 : 1;    // halves of a tile's tokens, filled in turn
    static constexpr int NM = NT / H;             // N of one MMA
    static constexpr int NACC = 2;  // accumulators of NM columns
    static constexpr int EPI = EPI_, CONV = CONV_;
    static constexpr int COLS = NT / (EPI / 4);   // accumulator columns of an epilogue thread
    static constexpr int STAGES = STAGES_;        // units in flight (activation tiles and TMEM stages)
    static constexpr int WSTAGES = WSTAGES_;      // weight tiles in flight
    // Up to 64 tokens: no f16 panel; ACT warps turn int8 codes into the B tiles themselves
    static constexpr bool DIRECT = NT <= kI8DirectTokens;
    static constexpr int ACT = DIRECT ? NT / 8 : 1;
    static constexpr int GROUPS = CONV / 4;       // converters (and ACT warps) in groups that take units in turn
    static constexpr int ACT_G = DIRECT ? ACT / GROUPS : 1, ACT_TOK = NT / ACT_G;  // ACT warps of a unit, tokens of one
    static constexpr int BT = NT / CG * I8_KS * 2;  // activation tile bytes of one CTA (two tiles a unit)
    static constexpr int W_PROD = EPI + CONV, W_ACT = W_PROD + 1, W_MMA = W_ACT + ACT;
    static constexpr int THREADS = (W_MMA + 1) * 32;
    static constexpr uint32_t TM_A = NACC * NM;   // TMEM: accumulators, then A stages (64 columns each)
    static constexpr int W_OFF = STAGES * 2 * BT;
    static constexpr int WT = (I8_ROWS + (DIRECT ? NT : 0)) * I8_UNIT;  // a unit's codes: weight rows, then (direct) tokens
    static constexpr int BAR_OFF = W_OFF + WSTAGES * WT;
    static constexpr int RED_LD = I8_ROWS + 4;    // int32 per token of a parked split-K tile
    static constexpr int BARS = 2 * STAGES + 2 * WSTAGES + 5;
    static constexpr int DATA = BAR_OFF > NT * RED_LD * 4 ? BAR_OFF : NT * RED_LD * 4;
    static constexpr int TOTAL = ((DATA + 15) & ~15) + BARS * 8 + 16 + 1024;  // + slack to align the base
    static_assert(TOTAL <= 227 * 1024, "shared memory");
    static_assert(TM_A + STAGES * 64 <= 512, "TMEM");
    static_assert(EPI % 4 == 0 && (CONV == 4 || CONV == 8) && COLS % 8 == 0, "roles");
};
using I8Pair = I8Cfg<2, 256, 16, 4, 4, 4>;
using I8One128 = I8Cfg<1, 128, 8, 8, 4, 5>;
using I8One64 = I8Cfg<1, 64, 8, 8, 4, 6>;
using I8One32 = I8Cfg<1, 32, 4, 8, 4, 9>;

struct I8TcParams {
    const float *sx, *sw, *bias;
    void *y;
    int64_t ldy;
    int M, N, n_tiles, tiles;
    int units, units_per_split, nsplit;  // K in units of 128
    unsigned long long *err;
    bool after_prologue;  // the weights may be read before the kernel before this one has ended
    bool clear;           // the device flag is cleared here
    unsigned long long wait_ns;
    int idle;
};

// ---------------------------------------------------------------- cta_group forms
template <int CG>
__device__ __forceinline__ void cg_alloc(uint32_t *dst) {
    if (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(dst)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void cg_dealloc(uint32_t taddr) {
    if (CG == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(taddr) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
// Eight MMAs over the 128 K of a unit (B tiles of 64 K at b and b2); the first accumulates iff acc0.
template <int CG>
__device__ __forceinline__ void cg_mma8(uint32_t d, uint32_t a, uint64_t b, uint64_t b2, uint32_t idesc, uint32_t acc0) {
    if (CG == 1) {
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.u32 p, %17, 0;\n setp.eq.u32 q, %17, %17;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %9, %18, p;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [%2], %10, %18, q;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [%3], %11, %18, q;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [%4], %12, %18, q;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [%5], %13, %18, q;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [%6], %14, %18, q;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [%7], %15, %18, q;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], [%8], %16, %18, q;\n}"
            ::"r"(d),
            "r"(a), "r"(a + 8), "r"(a + 16), "r"(a + 24), "r"(a + 32), "r"(a + 40), "r"(a + 48), "r"(a + 56), "l"(b), "l"(b + 2),
            "l"(b + 4), "l"(b + 6), "l"(b2), "l"(b2 + 2), "l"(b2 + 4), "l"(b2 + 6), "r"(acc0), "r"(idesc)
            : "memory");
    } else {
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.u32 p, %17, 0;\n setp.eq.u32 q, %17, %17;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %9, %18, p;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], [%2], %10, %18, q;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], [%3], %11, %18, q;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], [%4], %12, %18, q;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], [%5], %13, %18, q;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], [%6], %14, %18, q;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], [%7], %15, %18, q;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], [%8], %16, %18, q;\n}"
            ::"r"(d),
            "r"(a), "r"(a + 8), "r"(a + 16), "r"(a + 24), "r"(a + 32), "r"(a + 40), "r"(a + 48), "r"(a + 56), "l"(b), "l"(b + 2),
            "l"(b + 4), "l"(b + 6), "l"(b2), "l"(b2 + 2), "l"(b2 + 4), "l"(b2 + 6), "r"(acc0), "r"(idesc)
            : "memory");
    }
}
// Arrive on `bar` (in both CTAs of a pair) when this thread's MMAs so far have completed.
template <int CG>
__device__ __forceinline__ void cg_commit(uint64_t *bar, uint16_t mask) {
    if (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"(mask)
            : "memory");
}
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// TMA load into this CTA whose bytes count on the barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const void *tmap, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(tmap), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
// Arrive at a barrier given by its cluster address.  Relaxed: what it announces went to (or was read from)
// tensor memory and is ordered by the tcgen05 fences around it.  A release at cluster scope in its place
// cost the converters 940 cycles a k-step.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A wait that a whole warp makes succeeds for all its lanes or for none, so that the warp stays together.
__device__ __forceinline__ bool all_lanes(bool ok) { return __all_sync(~0u, ok); }

template <typename C, typename TY>
__global__ void __launch_bounds__(C::THREADS, 1)
    i8_tc_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, I8TcParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *sB = sm, *sW = sm + C::W_OFF;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + ((C::DATA + 15) & ~15));
    // k_full/k_empty: one unit's activation tiles and converted weights; k_full and acc_empty are waited on
    // in the pair's first CTA only, and every arrival goes there
    uint64_t *k_full = bars, *k_empty = k_full + C::STAGES;
    uint64_t *w_full = k_empty + C::STAGES, *w_empty = w_full + C::WSTAGES;
    uint64_t *acc_full = w_empty + C::WSTAGES, *acc_empty = acc_full + 2, *mma_done = acc_empty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = cooperative_groups::this_cluster().block_rank();
    const int r = C::CG == 2 ? (int)(crank & 1) : 0;       // place in the pair
    const uint32_t lead = C::CG == 2 ? crank & ~1u : crank;  // the pair's first CTA
    const int z = blockIdx.z;                              // split-K rank
    const int u0 = z * P.units_per_split, nu = min(P.units, u0 + P.units_per_split) - u0;
    const int tile0 = blockIdx.x / C::CG, tstride = gridDim.x / C::CG;

    if (tid == 0) {
        for (int i = 0; i < C::STAGES; ++i) { mbar_init(&k_full[i], C::ACT_G + 4 * C::CG); mbar_init(&k_empty[i], 1); }
        for (int i = 0; i < C::WSTAGES; ++i) { mbar_init(&w_full[i], 1); mbar_init(&w_empty[i], 4 + (C::DIRECT ? C::ACT_G : 0)); }
        for (int i = 0; i < 2; ++i) { mbar_init(&acc_full[i], 1); mbar_init(&acc_empty[i], C::EPI / C::H * C::CG); }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == C::W_MMA) cg_alloc<C::CG>(tmem_holder);
    if (warp == C::W_PROD && lane == 0) prefetch_tmap(&tmW);
    if (warp == C::W_ACT && lane == 0) prefetch_tmap(&tmX);
    tc_fence_before();
    if (!P.after_prologue) grid_dependency_wait();
    __syncthreads();
    if (C::CG > 1) cooperative_groups::this_cluster().sync();  // the pair's barriers are ready
    tc_fence_after();
    // all 512 columns are this kernel's, so the allocation starts at column 0 of lane 0
    constexpr uint32_t tbase = 0;
    int acc[C::COLS];  // epilogue: this thread's sums, one weight row

    if (warp == C::W_PROD) {
        // ------------------------------------------------------------ weight tiles
        if (lane == 0) {
            bool ok = true;
            int g = 0, ahead = 0;
            if (C::DIRECT) {
                // the weights of the first units start before the codes, which the kernel before this one
                // may still be writing
                ahead = min(C::WSTAGES, nu);
                for (int u = 0; u < ahead; ++u) {
                    mbar_arrive_expect_tx(&w_full[u], C::WT);
                    tma_load_2d(sW + u * C::WT, &tmW, &w_full[u], (u0 + u) * I8_UNIT, (tile0 % P.n_tiles) * I8_ROWS);
                }
                grid_dependency_wait();
                grid_launch_dependents();
            }
            for (int tile = tile0; tile < P.tiles && ok; tile += tstride) {
                const int n0 = (tile % P.n_tiles) * (I8_ROWS * C::CG) + r * I8_ROWS;
                for (int u = 0; u < nu; ++u, ++g) {
                    const int s = g % C::WSTAGES, x = (u0 + u) * I8_UNIT;
                    if (g >= ahead) {
                        if (!(ok = mbar_wait_sleep(&w_empty[s], ((g / C::WSTAGES) & 1) ^ 1, abort_flag, P.wait_ns))) break;
                        mbar_arrive_expect_tx(&w_full[s], C::WT);
                        tma_load_2d(sW + s * C::WT, &tmW, &w_full[s], x, n0);
                    }
                    if (C::DIRECT) tma_load_2d(sW + s * C::WT + I8_ROWS * I8_UNIT, &tmX, &w_full[s], x, 0);
                }
            }
            // whoever gives up, the copies in flight land before this thread leaves (bounded): shared memory is used
            // again or left after that
            for (int i = 0; i < C::WSTAGES; ++i) {
                const int last = g - 1 - i;
                volatile int no_abort = 0;
                if (last >= 0) mbar_wait_sleep(&w_full[last % C::WSTAGES], (last / C::WSTAGES) & 1, &no_abort, 100000000ull);
            }
        }
    } else if (C::DIRECT && warp >= C::W_ACT && warp < C::W_MMA) {
        // ------------------------------------------------------------ activation tiles from int8 codes
        // Eight lanes take a token's 128 codes of a unit, four tokens a pass, and write them as f16 in the
        // 128-byte swizzle.  (Read from global memory here instead, under the weights' stream, a unit's codes
        // took 3000 cycles to come.)
        const int aw = warp - C::W_ACT, grp = aw / C::ACT_G;
        const int row0 = aw % C::ACT_G * C::ACT_TOK + (lane >> 3), c = lane & 7;
        constexpr int PASSES = C::ACT_TOK / 4;
        bool ok = true;
        int g = 0;
        for (int tile = tile0; tile < P.tiles && ok && P.idle != I8_IDLE_ACT; tile += tstride) {
            for (int u = 0; u < nu; ++u, ++g) {
                if (g % C::GROUPS != grp) continue;
                const int s = g % C::STAGES, ws = g % C::WSTAGES;
                if (!(ok = all_lanes(mbar_wait_sleep(&w_full[ws], (g / C::WSTAGES) & 1, abort_flag, P.wait_ns)))) break;
                const uint8_t *xt = sW + ws * C::WT + I8_ROWS * I8_UNIT;
                uint4 v[PASSES];
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int row = row0 + 4 * i;
                    v[i] = *reinterpret_cast<const uint4 *>(xt + row * I8_UNIT + ((c ^ (row & 7)) << 4));
                }
                if (!(ok = all_lanes(mbar_wait_sleep(&k_empty[s], ((g / C::STAGES) & 1) ^ 1, abort_flag, P.wait_ns)))) break;
                uint8_t *bt = sB + (2 * s + (c >> 2)) * C::BT;
#pragma unroll
                for (int i = 0; i < PASSES; ++i) {
                    const int row = row0 + 4 * i, pc = 2 * (c & 3);
                    uint4 a, b;
                    i8x4_to_f16(v[i].x, a.x, a.y);
                    i8x4_to_f16(v[i].y, a.z, a.w);
                    i8x4_to_f16(v[i].z, b.x, b.y);
                    i8x4_to_f16(v[i].w, b.z, b.w);
                    *reinterpret_cast<uint4 *>(bt + row * 128 + ((pc ^ (row & 7)) << 4)) = a;
                    *reinterpret_cast<uint4 *>(bt + row * 128 + (((pc + 1) ^ (row & 7)) << 4)) = b;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&k_full[s]);
                    mbar_arrive(&w_empty[ws]);
                }
            }
        }
    } else if (!C::DIRECT && warp == C::W_ACT) {
        // ------------------------------------------------------------ activation tiles from the panel
        if (lane == 0) {
            bool ok = true;
            int g = 0;
            grid_dependency_wait();  // the panel is the output of the kernel before this one
            grid_launch_dependents();
            for (int tile = tile0; tile < P.tiles && ok && P.idle != I8_IDLE_ACT; tile += tstride) {
                const int m0 = (tile / P.n_tiles) * C::NT + r * (C::NT / C::CG);
                for (int u = 0; u < nu; ++u, ++g) {
                    const int s = g % C::STAGES, ph = (g / C::STAGES) & 1;
                    if (!(ok = mbar_wait_sleep(&k_empty[s], ph ^ 1, abort_flag, P.wait_ns))) break;
                    const int x = (u0 + u) * I8_UNIT;
                    if (r == 0) mbar_arrive_expect_tx(&k_full[s], C::CG * 2 * C::BT);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint8_t *dst = sB + (2 * s + j) * C::BT;
                        if (C::CG == 1) tma_load_2d(dst, &tmX, &k_full[s], x + j * I8_KS, m0);
                        else tma_load_2d_pair(dst, &tmX, cluster_addr(&k_full[s], lead), x + j * I8_KS, m0);
                    }
                }
            }
            // as above: once the MMAs have read them the copies have landed; where somebody gave up, time alone bounds
            // them (their barrier may be the other CTA's, or wait for converters that have left), far more than they need
            for (int i = 0; i < C::STAGES && ok; ++i) {
                const int last = g - 1 - i;
                if (last >= 0) ok = mbar_wait_sleep(&k_empty[last % C::STAGES], (last / C::STAGES) & 1, abort_flag, P.wait_ns);
            }
            if (!ok) {
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 10000000ull) {}
            }
        }
    } else if (warp == C::W_MMA) {
        // ------------------------------------------------------------ MMAs
        // The whole warp walks the loop, so that the operands stay in uniform registers; one lane issues.
        if (r == 0) {
            const bool one = elect_one();
            constexpr uint32_t idesc = idesc_f16_f32(I8_ROWS * C::CG, C::NM);
            const uint64_t dB = smem_desc(smem_u32(sB), 1024, 2);
            const uint16_t mask = (uint16_t)(3u << lead);
            constexpr uint64_t half_rows = (uint64_t)(C::BT / C::H) >> 4;  // a half's rows in an activation tile
            bool ok = true;
            int s = 0, job = 0;  // stage, and accumulator fills so far
            uint32_t ph = 0;     // phase of stage s's barriers
            for (int tile = tile0; tile < P.tiles && ok && P.idle != I8_IDLE_MMA; tile += tstride) {
                for (int c0 = 0; c0 < nu && ok; c0 += I8_CHUNK, ++job) {
                    const int un = min(I8_CHUNK, nu - c0);
                    // all stages at a time: the first half's MMAs over them, then the second half's, which free
                    // them one by one
                    for (int u = 0; u < un && ok; u += C::STAGES) {
                        const int kn = min(C::STAGES, un - u);
                        for (int h = 0; h < C::H && ok; ++h) {
                            const int buf = C::H == 2 ? h : job % C::NACC;
                            const uint32_t use = C::H == 2 ? job : job / C::NACC;
                            if (u == 0) {
                                if (!(ok = all_lanes(mbar_wait_sleep(&acc_empty[buf], (use & 1) ^ 1, abort_flag, P.wait_ns)))) break;
                                tc_fence_after();
                            }
                            for (int k = 0; k < kn; ++k) {
                                const int sk = (s + k) % C::STAGES;
                                if (h == 0) {
                                    const uint32_t phk = s + k < C::STAGES ? ph : ph ^ 1;
                                    if (!(ok = all_lanes(mbar_wait_sleep(&k_full[sk], phk, abort_flag, P.wait_ns)))) break;
                                    tc_fence_after();
                                }
                                const uint64_t b = dB + (uint64_t)(sk * (2 * C::BT >> 4)) + h * half_rows;
                                if (one) {
                                    cg_mma8<C::CG>(tbase + buf * C::NM, tbase + C::TM_A + sk * 64, b, b + (C::BT >> 4), idesc, u + k);
                                    if (h == C::H - 1) cg_commit<C::CG>(&k_empty[sk], mask);
                                }
                                __syncwarp();
                            }
                            if (ok && one && u + C::STAGES >= un) cg_commit<C::CG>(&acc_full[buf], mask);
                        }
                        s += kn;
                        if (s >= C::STAGES) { s -= C::STAGES; ph ^= 1; }
                    }
                }
            }
            // every MMA issued has finished before tensor memory is freed
            if (one) cg_commit<C::CG>(mma_done, (uint16_t)(1u << lead));
            __syncwarp();
            volatile int no_abort = 0;
            mbar_wait(mma_done, 0, &no_abort, 100000000ull);
        }
    } else if (warp >= C::EPI) {
        // ------------------------------------------------------------ weight converters
        // A thread converts its row's 128 codes of a unit; all eight loads go out before the first conversion.
        // With eight warps, four take every other unit: a unit's barriers and latencies cost a warp more
        // than its conversions do.
        const int q = warp & 3, row = 32 * q + lane, grp = (warp - C::EPI) >> 2;
        const uint32_t ta = tbase + ((uint32_t)(32 * q) << 16) + C::TM_A;
        bool ok = true;
        int g = 0;  // units so far
        for (int tile = tile0; tile < P.tiles && ok; tile += tstride) {
            for (int u = 0; u < nu && ok; ++u, ++g) {
                if (g % C::GROUPS != grp) continue;
                const int ws = g % C::WSTAGES, s = g % C::STAGES;
                if (!(ok = all_lanes(mbar_wait_sleep(&w_full[ws], (g / C::WSTAGES) & 1, abort_flag, P.wait_ns)))) break;
                // 16-byte piece p of row `row` sits at piece p ^ (row & 7) (128-byte swizzle)
                const uint8_t *wr = sW + ws * C::WT + row * I8_UNIT;
                uint4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint4 *>(wr + ((i ^ (row & 7)) << 4));
                if (!(ok = all_lanes(mbar_wait_sleep(&k_empty[s], ((g / C::STAGES) & 1) ^ 1, abort_flag, P.wait_ns)))) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t o[32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        i8x4_to_f16(v[4 * j + i].x, o[8 * i], o[8 * i + 1]);
                        i8x4_to_f16(v[4 * j + i].y, o[8 * i + 2], o[8 * i + 3]);
                        i8x4_to_f16(v[4 * j + i].z, o[8 * i + 4], o[8 * i + 5]);
                        i8x4_to_f16(v[4 * j + i].w, o[8 * i + 6], o[8 * i + 7]);
                    }
                    tmem_st32(ta + s * 64 + j * 32, o);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (C::CG == 1) mbar_arrive(&k_full[s]);
                    else mbar_arrive_cluster(cluster_addr(&k_full[s], lead));
                    mbar_arrive(&w_empty[ws]);
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int q = warp & 3, col0 = (warp >> 2) * C::COLS, row = 32 * q + lane;
        const uint32_t lane_base = tbase + ((uint32_t)(32 * q) << 16);
        const int h = C::H == 2 ? col0 / C::NM : 0;
        // the token of column col0 (columns of a pair's half: 64 tokens of the first CTA, 64 of the second)
        const int tok0 = C::CG == 1 ? col0 : (col0 % C::NM) / (C::NM / 2) * (C::NT / 2) + h * (C::NM / 2) + col0 % (C::NM / 2);
        bool ok = true;
        int job = 0;
        grid_dependency_wait();  // scales may be the output of the kernel before this one
        // the direct form's flag: an error is counted two seconds later at the earliest
        if (P.clear && tid == 0 && blockIdx.x == 0 && z == 0) *P.err = 0ull;
        for (int tile = tile0; tile < P.tiles && ok; tile += tstride) {
            // this tile's scales, on their way while it is computed: lane l keeps the tokens l, l + 32
            const int n = (tile % P.n_tiles) * (I8_ROWS * C::CG) + r * I8_ROWS + row;
            const int m0 = (tile / P.n_tiles) * C::NT + tok0;
            float sx[(C::COLS + 31) / 32];
#pragma unroll
            for (int j = 0; j < (C::COLS + 31) / 32; ++j) sx[j] = m0 + lane + 32 * j < P.M ? P.sx[m0 + lane + 32 * j] : 0.0f;
            const bool mine = n < P.N;
            const float sw = mine ? P.sw[n] : 0.0f, b = P.bias && mine ? P.bias[n] : 0.0f;
            for (int c0 = 0; c0 < nu; c0 += I8_CHUNK, ++job) {
                const int buf = C::H == 2 ? h : job % C::NACC;
                const uint32_t use = C::H == 2 ? job : job / C::NACC;
                if (!(ok = all_lanes(mbar_wait_sleep(&acc_full[buf], use & 1, abort_flag, P.wait_ns)))) break;
                tc_fence_after();
                const uint32_t t = lane_base + (C::H == 2 ? col0 : buf * C::NM + col0);
#pragma unroll
                for (int c = 0; c < C::COLS; c += 8) {
                    float v[8];
                    tmem_ld8(t + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[c + i] = (c0 ? acc[c + i] : 0) + __float2int_rn(v[i]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (C::CG == 1) mbar_arrive(&acc_empty[buf]);
                    else mbar_arrive_cluster(cluster_addr(&acc_empty[buf], lead));
                }
            }
            if (!ok || P.nsplit > 1) break;  // a split tile (one a cluster) is summed below
            TY *y = static_cast<TY *>(P.y) + (int64_t)m0 * P.ldy + n;
#pragma unroll
            for (int i = 0; i < C::COLS; ++i) {
                float v = __fmul_rn(__fmul_rn((float)acc[i], __shfl_sync(~0u, sx[i / 32], i % 32)), sw);
                if (P.bias) v = __fadd_rn(v, b);
                if (mine && m0 + i < P.M) *y = from_f32<TY>(v);
                // one addition a token: left to itself the compiler multiplies 64 offsets out (3.8 us for 128
                // tokens against 1.2)
                y += P.ldy;
                asm volatile("" : "+l"(y));
            }
        }
    }

    __syncthreads();
    if (P.nsplit > 1) {
        // Split K: every CTA parks its int32 tile in its (now idle) shared memory, then sums a slice of
        // tokens over the cluster's splits and stores it.
        int *red = reinterpret_cast<int *>(sm);
        if (warp < C::EPI) {
            const int row = 32 * (warp & 3) + lane, col0 = (warp >> 2) * C::COLS;
#pragma unroll
            for (int i = 0; i < C::COLS; ++i) red[(col0 + i) * C::RED_LD + row] = acc[i];
        }
        // four rows a thread, the same in every round, and all splits' loads at once
        const int n = (tile0 % P.n_tiles) * (I8_ROWS * C::CG) + r * I8_ROWS + lane * 4;
        float sw[4], bias[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sw[j] = n + j < P.N ? P.sw[n + j] : 0.0f;
            bias[j] = P.bias && n + j < P.N ? P.bias[n + j] : 0.0f;
        }
        cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();
        grid_dependency_wait();
        const int per = (C::NT + P.nsplit - 1) / P.nsplit;
        const int c_end = min(C::NT, (z + 1) * per);
        const int m0 = (tile0 / P.n_tiles) * C::NT;
        const int *peer[I8_MAX_SPLIT];
#pragma unroll
        for (int k = 0; k < I8_MAX_SPLIT; ++k) peer[k] = cluster.map_shared_rank(red, min(k, P.nsplit - 1) * C::CG + r);
        for (int c = z * per + warp; c < c_end; c += C::THREADS / 32) {
            const int hh = c / C::NM, cm = c % C::NM;
            const int m = m0 + (C::CG == 1 ? c : cm / (C::NM / 2) * (C::NT / 2) + hh * (C::NM / 2) + cm % (C::NM / 2));
            if (m >= P.M) continue;
            const float sx = P.sx[m];
            int4 v[I8_MAX_SPLIT];
#pragma unroll
            for (int k = 0; k < I8_MAX_SPLIT; ++k)
                v[k] = k < P.nsplit ? *reinterpret_cast<const int4 *>(peer[k] + c * C::RED_LD + lane * 4) : make_int4(0, 0, 0, 0);
            int sum[4] = {};
#pragma unroll
            for (int k = 0; k < I8_MAX_SPLIT; ++k) {
                sum[0] += v[k].x; sum[1] += v[k].y; sum[2] += v[k].z; sum[3] += v[k].w;
            }
            TY *y = static_cast<TY *>(P.y) + (int64_t)m * P.ldy + n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f = __fmul_rn(__fmul_rn((float)sum[j], sx), sw[j]);
                if (P.bias) f = __fadd_rn(f, bias[j]);
                if (n + j < P.N) y[j] = from_f32<TY>(f);
            }
        }
    }
    if (tid == 0 && *abort_flag) {
        grid_dependency_wait();  // the panel's kernel clears the flag
        atomicAdd(P.err, 1ull);
    }
    tc_fence_before();
    // nobody still reads or signals another CTA's memory
    if (C::CG > 1 || P.nsplit > 1) cooperative_groups::this_cluster().sync();
    else __syncthreads();
    if (warp == C::W_MMA) {
        tc_fence_after();
        cg_dealloc<C::CG>(*tmem_holder);
    }
}

// ---------------------------------------------------------------- host
static PFN_cuTensorMapEncodeTiled_v12000 i8_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// Clusters of CG x 1 x splits CTAs of this form that the current device holds at once (clusters fill a GPC
// only in whole multiples of their size).  Looked up once a device and split.
template <typename C>
static int i8_resident(int splits) {
    static std::atomic<int> cache[64][I8_MAX_SPLIT + 1];
    const int fallback = 8 * (19 / (C::CG * splits));
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return fallback;
    }
    return looked_up(cache[dev][splits], [&] {
        auto kern = i8_tc_kernel<C, float>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(C::CG, 1, splits);
        cfg.blockDim = dim3(C::THREADS);
        cfg.dynamicSmemBytes = C::TOTAL;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = C::CG;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = splits;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::TOTAL) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            n = fallback;
        }
        return n;
    });
}

template <typename C, typename TY>
static kq_status i8_launch(const char *fn, const I8TcArgs &a, int splits, cudaStream_t st) {
    auto encode = i8_encoder();
    if (!encode) return fail(KQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", fn);
    CUtensorMap tmW, tmX;
    const cuuint32_t es[2] = {1, 1};
    {
        const cuuint64_t dims[2] = {(cuuint64_t)a.K, (cuuint64_t)a.N}, strides[1] = {(cuuint64_t)a.ldw};
        const cuuint32_t box[2] = {I8_UNIT, I8_ROWS};
        const CUresult e = encode(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(a.w), dims, strides, box, es,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (e != CUDA_SUCCESS) return fail(KQ_ERR_CUDA, "%s: tensor map of w failed (%d)", fn, (int)e);
    }
    if (C::DIRECT) {
        const cuuint64_t dims[2] = {(cuuint64_t)a.K, (cuuint64_t)a.M}, strides[1] = {(cuuint64_t)a.ldq};
        const cuuint32_t box[2] = {I8_UNIT, C::NT};
        const CUresult e = encode(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(a.q), dims, strides, box, es,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (e != CUDA_SUCCESS) return fail(KQ_ERR_CUDA, "%s: tensor map of q failed (%d)", fn, (int)e);
    } else {
        const cuuint64_t dims[2] = {(cuuint64_t)a.ldp, (cuuint64_t)a.M}, strides[1] = {(cuuint64_t)a.ldp * 2};
        const cuuint32_t box[2] = {I8_KS, C::NT / C::CG};
        const CUresult e = encode(&tmX, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half *>(a.panel), dims, strides, box,
                                  es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (e != CUDA_SUCCESS) return fail(KQ_ERR_CUDA, "%s: tensor map of the panel failed (%d)", fn, (int)e);
    }
    I8TcParams p{};
    p.sx = a.sx; p.sw = a.sw; p.bias = a.bias; p.y = a.y; p.ldy = a.ldy;
    p.M = (int)a.M; p.N = (int)a.N;
    p.n_tiles = (int)((a.N + I8_ROWS * C::CG - 1) / (I8_ROWS * C::CG));
    const int64_t tiles = (int64_t)p.n_tiles * ((a.M + C::NT - 1) / C::NT);
    if (tiles > 0x7fffffff / C::CG) return fail(KQ_ERR_INVALID_ARG, "%s: too many tiles", fn);
    p.tiles = (int)tiles;
    p.units = (int)((a.K + I8_UNIT - 1) / I8_UNIT);
    p.units_per_split = (p.units + splits - 1) / splits;
    p.nsplit = splits;
    p.err = a.err;
    p.after_prologue = a.after_prologue;
    p.clear = C::DIRECT && a.idle == I8_IDLE_NONE;
    p.wait_ns = a.wait_ns;
    p.idle = a.idle;
    auto kern = i8_tc_kernel<C, TY>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::TOTAL);
    if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    const int64_t groups = splits > 1 ? tiles : std::min<int64_t>(tiles, i8_resident<C>(1));
    e = launch_beside(kern, dim3((unsigned)(groups * C::CG), 1, (unsigned)splits), dim3(C::THREADS), C::TOTAL,
                      dim3(C::CG, 1, (unsigned)splits), st, tmW, tmX, p);
    if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    count_launch(R_I8);
    return KQ_OK;
}

// How a product is shared out: splits of K, and the time that the estimate below gives it (us): the CTAs of a
// wave walk `per` units at `unit` each, 4 us go to starting and ending, a split adds its reduction.
struct I8Plan {
    int splits;
    double t;
};

template <typename C>
static I8Plan i8_plan(int64_t M, int64_t N, int64_t units, double unit, double reduction) {
    I8Plan best = {1, 1e30};
    const int64_t tiles = (N + I8_ROWS * C::CG - 1) / (I8_ROWS * C::CG) * ((M + C::NT - 1) / C::NT);
    for (int s = 1; s <= I8_MAX_SPLIT / C::CG; ++s) {
        const int64_t per = (units + s - 1) / s;
        if (s > 1 && (per < 2 || per * (s - 1) >= units)) continue;
        const int64_t groups = i8_resident<C>(s), waves = (tiles + groups - 1) / groups;
        // (unsplit CTAs are persistent: they start and end once; clusters of a split do in every wave)
        const double t = s == 1 ? 4.0 + (double)(waves * per) * unit : (double)waves * (4.0 + (double)per * unit + reduction);
        if (t < best.t) best = {s, t};
    }
    return best;
}

I8Form i8_tc_form(int64_t M, int64_t N, int64_t K) {
    const int64_t units = (K + I8_UNIT - 1) / I8_UNIT;
    // (weights from memory, 16 tokens, [4096 x 4096]: split 9.1 us, unsplit 14.6; [4096 x 14336]: 16.9 and 42.7)
    if (M <= 32) return {1, 32, i8_plan<I8One32>(M, N, units, 0.43, 3.0).splits};
    if (M <= 64) return {1, 64, i8_plan<I8One64>(M, N, units, 0.43, 3.0).splits};
    const I8Plan one = i8_plan<I8One128>(M, N, units, 0.43, 3.5);
    if (M <= 128) return {1, 128, one.splits};
    // A pair does a unit of four times the work in 0.62 us, but its tiles are fewer and its reduction is
    // dearer.  [4096 x 4096]: 256 tokens 18.9 us by pairs, 16.3 by single CTAs, 512 tokens 23.3 and 20.5;
    // [14336 x 4096]: 384 tokens 49.5 and 45.8, 2048 tokens 155 and 186 (many in a row, under the power cap)
    const I8Plan pair = i8_plan<I8Pair>(M, N, units, 0.62, 6.0);
    if (pair.t + 3.0 <= one.t) return {2, 256, pair.splits};
    return {1, 128, one.splits};
}

kq_status i8_tc_product(const char *fn, const I8TcArgs &a, cudaStream_t st) {
    const I8Form f = i8_tc_form(a.M, a.N, a.K);
    return with_type(a.yt, [&](auto t) {
        using TY = decltype(t);
        switch (f.tokens) {
        case 32: return i8_launch<I8One32, TY>(fn, a, f.splits, st);
        case 64: return i8_launch<I8One64, TY>(fn, a, f.splits, st);
        case 128: return i8_launch<I8One128, TY>(fn, a, f.splits, st);
        default: return i8_launch<I8Pair, TY>(fn, a, f.splits, st);
        }
    });
}

}  // namespace kq
