// kq_attn_tc.cu -- attention over whole prompts on the tensor cores: heads of up to 128 elements, rows on 16-byte
// boundaries (the other rows take kq_attn_prompt.cu's form).
//
// Bound by the two products, 4 D flops a score, and their operands' shared-memory reads: 16384 tokens, 32 heads over 8 of
// 128, causal, 1468 us, 1.5 PFLOP/s; with nothing done between the products they take 1355.  A thread block takes two row tiles of
// one key head, 128 tokens of one query head each (two heads of the same tokens where the group is even), so that every
// key and value tile that is brought in serves 256 rows and one tile's products run while the other's weights
// are made:
//   S = Q K^T   128 x 128, fp32 in tensor memory, both operands in shared memory
//   P = 2^(scale (S - m)), one row a thread; written over S as the rows' type
//   O += P V    P from tensor memory, V in shared memory as it lies there ([token][d]: the transposed form of the operand)
// The sums stay relative to an old maximum until a row's grows by more than 2^8: then its warp scales O in place.
// Key tiles go from the last to the first, so the masked ones come first.
// Roles: warps 0-3 and 4-7 a row tile each, warp 8 issues the products, warp 9 brings tiles by TMA, warps 10 and 11 look through
// the values of masked tiles: a masked weight is 0, but 0 times an infinity is not, so values that are not finite
// are taken out of the tile, remembered bit by bit, and given back at the end to the rows that see them.
// The blocks, one an SM, take the pairs of row tiles from a line as they get through with them; the next pair's tiles come and
// its first products run while this one's results leave.  (A block a pair lost 6 us each to starting and ending.)
// Every wait is bounded; on expiry the block counts an error in the device flag and leaves in order.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <algorithm>
#include <math.h>

#include "kq_attn_prompt.cuh"
#include "kq_launch.cuh"

namespace kq {

using namespace sm100;

constexpr int PT = 128;             // rows of a tile, keys of a tile
constexpr int PT_THREADS = 384;
constexpr int PT_MASKED = 3;        // key tiles that some row of a block's (at most 256 tokens) sees only in part
constexpr unsigned long long kPtPairNs = 20000;  // far longer than a pair of key tiles takes (2 us)
constexpr float kPtSlack = 8.0f;    // in units of log 2
// Up to this |m * scale| weights are 2^(S scale - m scale), one fused operation each: m * scale, rounded, is off by less than
// a sixteenth.  Beyond it the rounding would make weights of any size, so S - m is formed first.
constexpr float kPtFused = 1048576.0f;

template <int DP_, int OW_>
struct PtCfg {
    static constexpr int DP = DP_;             // D rounded up to 64 or 128: what is loaded
    static constexpr int OW = OW_;             // D rounded up to 64, 96 or 128: columns of the sums
    static constexpr int CH = DP / 64;         // boxes of 64 elements
    static constexpr int BOX = PT * 128;       // bytes of one
    static constexpr int TILE = CH * BOX;
    static constexpr int STAGES = DP == 128 ? 4 : 8;
    static constexpr int KV_OFF = 2 * TILE;
    static constexpr int FIX_OFF = KV_OFF + STAGES * TILE;
    static constexpr int FIX_ROW = 2 * DP / 8;  // a key's bits: +infinities (and NaN), then -infinities (and NaN)
    static constexpr int BAR_OFF = FIX_OFF + 2 * PT_MASKED * PT * FIX_ROW;  // of two pairs in turn
    static constexpr int BARS = 4 + 2 * STAGES + 6 + 4 * PT_MASKED + 2 + 4 + 1;
    static constexpr int TOTAL = BAR_OFF + BARS * 8 + 24 + 2 * PT_MASKED * 2 * 4 + 1024;
    static_assert(TOTAL <= 227 * 1024, "shared memory");
    static constexpr uint32_t O_COL = 256;     // tensor memory: S (and P) of both tiles, then O of both
};

struct PtParams {
    PaParams p;
    int64_t pairs;        // for one key head
    int n_kv;
    unsigned long long wait_ns;
    int idle;
    bool wide;            // output rows on 32 bytes, and whole heads of them
    unsigned *next;       // pairs handed out beyond the blocks' first ones; NULL: there are no more
    const int *order;     // the pairs by their places on the line, or NULL: the last first
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
        "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, uint64_t *bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(tmap), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
__device__ __forceinline__ bool pt_elect() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ float pt_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <typename T> __device__ __forceinline__ uint32_t pt_pack(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pt_pack<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <> __device__ __forceinline__ uint32_t pt_pack<__half>(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// What a block works on.  Sequence b's pairs of row tiles start at floor(G * (floor(cu_q[b] / 128) + b) / 2) + b.
struct PtWork {
    PaTile t;
    int head[2], first[2];    // of the two row tiles: query head of the group, token
    int tiles[2], lowest[2];  // key tiles that it sees, and the keys that its first token sees
    int n, masked;            // key tiles of the block, and how many of them (the last ones) are masked for some row
};
__device__ __forceinline__ int of(const int (&v)[2], int q) { return q ? v[1] : v[0]; }  // (an index would put them in local memory)
__device__ __forceinline__ int64_t pt_start(const PaParams &P, int64_t b) { return ((pa_row(P.cu_q, b, P.Tq) / PT + b) * P.G >> 1) + b; }
// The pair's work, if there is such a pair; sequence b is the last that starts at or before it.
__device__ __forceinline__ bool pt_fill(const PaParams &P, int64_t b, int64_t pair, PtWork &w) {
    PaTile &t = w.t;
    t.q_row = pa_row(P.cu_q, b, P.Tq);
    t.k_row = pa_row(P.cu_k, b, P.Tk);
    const int64_t n_q = pa_row(P.cu_q, b + 1, P.Tq) - t.q_row, n_k = pa_row(P.cu_k, b + 1, P.Tk) - t.k_row, r = (pair - pt_start(P, b)) * 2;
    if (r >= (n_q + PT - 1) / PT * P.G) return false;
    t.n_q = (int)n_q;
    t.n_k = n_k > 0 ? (int)n_k : 0;
    w.n = 0;
    int lowest = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned tt = (unsigned)(r + i) / (unsigned)P.G;  // (row tiles of a call are below 2^31)
        w.head[i] = (int)(r + i - (int64_t)tt * P.G);
        w.first[i] = (int)(tt * PT);
        w.tiles[i] = w.lowest[i] = 0;
        if ((int64_t)tt * PT >= n_q) continue;
        w.lowest[i] = pa_limit(P, t, w.first[i]);
        w.tiles[i] = (pa_limit(P, t, min(w.first[i] + PT, t.n_q) - 1) + PT - 1) / PT;
        w.n = max(w.n, w.tiles[i]);
        lowest = min(lowest, w.lowest[i]);
    }
    w.masked = min(w.n - min(w.n, lowest / PT), PT_MASKED);
    return true;
}
// A warp finds it out (every role on its own).
__device__ __forceinline__ bool pt_work(const PaParams &P, int64_t pair, PtWork &w) {
    const int lane = threadIdx.x & 31;
    int64_t b = 0;
    for (int64_t n = P.B; n > 1;) {  // the sequence is one of n from b on
        const int64_t step = (n + 31) / 32, at = lane * step;
        const int k = __popc(__ballot_sync(~0u, at < n && pt_start(P, b + at) <= pair)) - 1;
        if (k < 0) return false;
        b += k * step;
        n = min(step, n - k * step);
    }
    return pt_start(P, b) <= pair && pt_fill(P, b, pair, w);
}

template <typename T, typename C>
__global__ void __launch_bounds__(PT_THREADS, 1)
    pt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              PtParams X) {
    extern __shared__ uint8_t pt_smem[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(pt_smem) + 1023) & ~(uintptr_t)1023);
    uint8_t *sKV = sm + C::KV_OFF, *fix = sm + C::FIX_OFF;
    uint64_t *q_full = reinterpret_cast<uint64_t *>(sm + C::BAR_OFF), *q_empty = q_full + 2, *kv_full = q_empty + 2, *kv_empty = kv_full + C::STAGES;
    uint64_t *s_full = kv_empty + C::STAGES, *p_full = s_full + 2, *o_full = p_full + 2;
    // masked tiles, [pair % 2][place]: its copies have been asked for; its values have been looked through; and of a pair: done with
    uint64_t *v_sent = o_full + 2, *v_ok = v_sent + 2 * PT_MASKED, *fix_free = v_ok + 2 * PT_MASKED, *turn_full = fix_free + 2,
             *turn_empty = turn_full + 2, *mma_done = turn_empty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(mma_done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    volatile unsigned *turns = reinterpret_cast<volatile unsigned *>(abort_flag + 1);  // [turn % 2]: a place on the line
    volatile int *fixed = abort_flag + 3;  // [pair % 2][place][half]: values that are not finite were taken out

    const PaParams &P = X.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_full[i], 1);
            mbar_init(&fix_free[i], 8);
            mbar_init(&turn_full[i], 1);
            mbar_init(&turn_empty[i], PT_THREADS / 32 - 1);
        }
        for (int i = 0; i < C::STAGES; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
        for (int i = 0; i < 2 * PT_MASKED; ++i) { mbar_init(&v_sent[i], 1); mbar_init(&v_ok[i], 2); }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 9 && lane == 0) { prefetch_tmap(&tmQ); prefetch_tmap(&tmK); prefetch_tmap(&tmV); }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_holder)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns are this kernel's, so the allocation starts at column 0 of lane 0
    grid_dependency_wait();
    grid_launch_dependents();
    if (!X.next && blockIdx.x == 0 && tid == 0) *P.err = 0ull;  // (an error is counted two seconds later at the earliest)

    // Every role walks the same pairs: f(w, key head), false to stop.  The warp that brings tiles asks for the next place on the
    // line and passes it on when it has sent for a pair's last tiles, which a role may wait for that is through with the pair
    // long before (what looks through the values; a row tile that is not there): the longer the pair, the longer.
    auto walk = [&](auto f) {
        unsigned long long limit = X.wait_ns;
        const unsigned items = (unsigned)(X.pairs * X.n_kv);
        unsigned ahead = blockIdx.x;
        for (unsigned r = 0;; ++r) {
            const int s = r & 1;
            unsigned i = 0;
            if (warp == 9) {
                bool ok = true;
                if (lane == 0) {
                    i = ahead;
                    ok = mbar_wait_sleep(&turn_empty[s], (r >> 1 & 1) ^ 1, abort_flag, X.wait_ns);
                    turns[s] = i;
                    mbar_arrive(&turn_full[s]);
                }
                i = __shfl_sync(~0u, i, 0);
                if (!__shfl_sync(~0u, (int)ok, 0)) return;
            } else {
                if (!__all_sync(~0u, mbar_wait_sleep(&turn_full[s], r >> 1 & 1, abort_flag, limit))) return;
                i = turns[s];
                __syncwarp();
                if (lane == 0) mbar_arrive(&turn_empty[s]);
            }
            if (i >= items) return;
            // the longest first: later tokens of a sequence see more keys
            const unsigned turn = i / (unsigned)X.n_kv;
            PtWork w;
            w.n = 0;
            if (pt_work(P, X.order ? X.order[turn] : X.pairs - 1 - turn, w) && !f(w, (int)(i - turn * X.n_kv))) return;
            limit = X.wait_ns + kPtPairNs * w.n;
            // (asked for when the pair's last tiles have been sent for, not before: a place taken early waits behind a long pair)
            if (warp == 9 && lane == 0) ahead = X.next ? gridDim.x + atomicAdd(X.next, 1u) : items;
        }
    };
    // The pairs with masked tiles so far; which barriers of theirs are this pair's, and their phase.
    int pairs_masked = 0;
    auto place = [&](int i) { return (pairs_masked & 1) * PT_MASKED + i; };
    uint32_t uses = 0;  // bit `place`: the phase of its barriers
    auto phase = [&](int i) { return uses >> place(i) & 1; };
    auto masked_done = [&](const PtWork &w) {
        for (int i = 0; i < w.masked; ++i) uses ^= 1u << place(i);
        if (w.masked) ++pairs_masked;
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 8) {
            // ------------------------------------------------------------ products
            const bool one = pt_elect();
            constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? (1u << 7) | (1u << 10) : 0u;
            const uint32_t id_s = idesc_f16_f32(PT, PT) | type | (P.negate ? 1u << 13 : 0u);
            constexpr uint32_t id_o = idesc_f16_f32(PT, C::OW) | type | (1u << 16);  // V: [token][d]
            const uint64_t dQ = smem_desc(smem_u32(sm), 1024, 2), dK = smem_desc(smem_u32(sKV), 1024, 2);
            // 64 elements of d a box, boxes BOX apart; eight tokens 1024 bytes apart
            const uint64_t dV = (dK & ~((uint64_t)0x3FFF << 16)) | (uint64_t)(C::BOX >> 4) << 16;
            bool ok = X.idle != 2;
            unsigned g = 0;                    // key and value tiles so far
            uint32_t q_phase[2] = {}, p_phase[2] = {};
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = ok && __all_sync(~0u, mbar_wait(bar, parity, abort_flag, X.wait_ns));
                return ok;
            };
            auto kv_wait = [&](unsigned t) { return wait(&kv_full[t % C::STAGES], t / C::STAGES & 1); };
            auto commit = [&](uint64_t *bar) {
                if (one) mma_commit(bar);
                __syncwarp();
            };
            walk([&](const PtWork &w, int) {
                // row tile q's scores of the pair's i-th key tile; after its last the queries may be overwritten
                auto qk = [&](int q, int i) {
                    const int s = (g + 2 * i) % C::STAGES;
                    if (one) {
#pragma unroll
                        for (int k = 0; k < C::DP / 16; ++k) {
                            if (k * 16 >= P.D) break;
                            const uint64_t off = (uint64_t)((k / 4) * (C::BOX >> 4) + (k % 4) * 2);
                            mma_f16(q * 128, dQ + q * (C::TILE >> 4) + off, dK + s * (C::TILE >> 4) + off, id_s, k > 0);
                        }
                        mma_commit(&s_full[q]);
                        if (i + 1 == w.n) mma_commit(&q_empty[q]);
                    }
                    __syncwarp();
                };
                auto queries = [&](int q) {
                    const uint32_t parity = q ? q_phase[1] : q_phase[0];
                    (q ? q_phase[1] : q_phase[0]) ^= 1;
                    return wait(&q_full[q], parity);
                };
                if (w.n && kv_wait(g)) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (ok && w.tiles[q] == w.n && queries(q)) {
                            tc_fence_after();
                            qk(q, 0);
                        }
                    if (ok) commit(&kv_empty[g % C::STAGES]);
                }
                for (int i = 0; i < w.n && ok; ++i) {
                    const unsigned tv = g + 2 * i + 1;
                    const int sv = tv % C::STAGES;
                    if (!kv_wait(tv)) break;
                    if (i < w.masked && !wait(&v_ok[place(i)], phase(i))) break;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int at = i - (w.n - w.tiles[q]);  // the row tile's own count
                        if (ok && at >= 0 && wait(&p_full[q], p_phase[q])) {
                            p_phase[q] ^= 1;
                            tc_fence_after();
                            if (one && !(q && X.idle == 4)) {
#pragma unroll
                                for (int k = 0; k < PT / 16; ++k)
                                    mma_f16_ts(C::O_COL + q * C::OW, q * 128 + k * 8, dV + (uint64_t)(sv * (C::TILE >> 4) + k * (2048 >> 4)),
                                               id_o, at > 0 || k > 0);
                                mma_commit(&o_full[q]);
                            }
                            __syncwarp();
                        }
                        if (ok && i + 1 < w.n && at + 1 >= 0 && kv_wait(tv + 1) && (at + 1 > 0 || queries(q))) {
                            tc_fence_after();
                            qk(q, i + 1);
                        }
                    }
                    if (!ok) break;
                    commit(&kv_empty[sv]);
                    if (i + 1 < w.n) commit(&kv_empty[(tv + 1) % C::STAGES]);
                }
                g += 2 * w.n;
                masked_done(w);
                return ok;
            });
            // every product issued has finished before tensor memory is freed
            commit(mma_done);
            volatile int no_abort = 0;
            mbar_wait(mma_done, 0, &no_abort, 100000000ull);
        } else if (warp == 9) {
            // ------------------------------------------------------------ tiles
            bool ok = true;
            unsigned g = 0, rows_sent[2] = {};
            if (X.idle != 1) walk([&](const PtWork &w, int kv_head) {
                if (lane == 0 && w.n) {
                    auto tile = [&](uint8_t *dst, const CUtensorMap *tm, uint64_t *bar, int head, int64_t row) {
                        mbar_arrive_expect_tx(bar, C::TILE);
#pragma unroll
                        for (int c = 0; c < C::CH; ++c) tma_load_3d(dst + c * C::BOX, tm, bar, c * 64, head, (int)row);
                    };
                    auto kv = [&](const CUtensorMap *tm, int j) {
                        const int s = g % C::STAGES;
                        if (!ok || !(ok = mbar_wait_sleep(&kv_empty[s], (g / C::STAGES & 1) ^ 1, abort_flag, X.wait_ns))) return;
                        tile(sKV + s * C::TILE, tm, &kv_full[s], kv_head, w.t.k_row + (int64_t)j * PT);
                        ++g;
                    };
                    auto rows = [&](int q) {
                        if (!ok || !of(w.tiles, q)) return;
                        unsigned &sent = q ? rows_sent[1] : rows_sent[0];
                        if (!(ok = mbar_wait_sleep(&q_empty[q], (sent & 1) ^ 1, abort_flag, X.wait_ns))) return;
                        tile(sm + q * C::TILE, &tmQ, &q_full[q], kv_head * P.G + of(w.head, q), w.t.q_row + of(w.first, q));
                        ++sent;
                    };
                    rows(0);
                    kv(&tmK, w.n - 1);
                    rows(1);
                    for (int i = 0; i < w.n; ++i) {
                        if (i) kv(&tmK, w.n - 1 - i);
                        kv(&tmV, w.n - 1 - i);
                        if (ok && i < w.masked) mbar_arrive(&v_sent[place(i)]);
                    }
                }
                masked_done(w);
                return (bool)__shfl_sync(~0u, ok, 0);
            });
            // the copies in flight land before this thread leaves (bounded)
            if (lane == 0) {
                volatile int no_abort = 0;
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (rows_sent[q]) mbar_wait_sleep(&q_full[q], (rows_sent[q] - 1) & 1, &no_abort, 100000000ull);
                for (unsigned i = 1; i <= C::STAGES; ++i)
                    if (g >= i) mbar_wait_sleep(&kv_full[(g - i) % C::STAGES], (g - i) / C::STAGES & 1, &no_abort, 100000000ull);
            }
        } else {
            // ------------------------------------------------------------ values of masked tiles
            constexpr uint32_t EXP = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
            const int half = warp - 10;  // tokens 64 * half on
            unsigned g = 0;
            walk([&](const PtWork &w, int) {
                bool ok = true;
                auto wait = [&](uint64_t *bar, uint32_t parity) {
                    return ok = ok && __all_sync(~0u, mbar_wait_sleep(bar, parity, abort_flag, X.wait_ns));
                };
                if (w.masked) wait(&fix_free[pairs_masked & 1], (pairs_masked >> 1 & 1) ^ 1);
                for (int i = 0; i < w.masked && ok; ++i) {
                    const unsigned tv = g + 2 * i + 1;
                    const int s = tv % C::STAGES;
                    // (only a tile that has been asked for has the phase that is waited for)
                    if (!wait(&v_sent[place(i)], phase(i)) || !wait(&kv_full[s], tv / C::STAGES & 1)) break;
                    uint8_t *v = sKV + s * C::TILE + half * (C::BOX / 2);
                    uint32_t top = 0;
#pragma unroll 8
                    for (int k = 0; k < C::CH * 16; ++k) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(v + (k / 16) * C::BOX + (k % 16) * 512 + lane * 16);
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
                    }
                    const bool found = __any_sync(~0u, (top & 0xffffu) >= EXP || (top >> 16) >= EXP);
                    if (found) {
                        // a lane takes eight elements of a token: out of the tile, into the bits
                        uint8_t *bits = fix + (place(i) * PT + half * 64) * C::FIX_ROW;
                        for (int k = lane; k < 64 * C::DP / 8; k += 32) {
                            const int r = k / (C::DP / 8), c = k % (C::DP / 8);
                            uint4 *at = reinterpret_cast<uint4 *>(v + (c / 8) * C::BOX + r * 128 + ((c % 8 ^ (r & 7)) << 4));
                            uint4 u = *at;
                            uint32_t plus = 0, minus = 0;
                            uint16_t *e = reinterpret_cast<uint16_t *>(&u);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const uint32_t x = e[j];
                                if ((x & 0x7fffu) < EXP) continue;
                                const bool nan = (x & 0x7fffu) > EXP;
                                if (nan || !(x >> 15)) plus |= 1u << j;
                                if (nan || x >> 15) minus |= 1u << j;
                                e[j] = 0;
                            }
                            *at = u;
                            bits[r * C::FIX_ROW + c] = (uint8_t)plus;
                            bits[r * C::FIX_ROW + C::DP / 8 + c] = (uint8_t)minus;
                        }
                        fence_proxy_async_smem();
                    }
                    if (lane == 0) fixed[place(i) * 2 + half] = found;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&v_ok[place(i)]);
                }
                g += 2 * w.n;
                masked_done(w);
                return ok;
            });
        }
    } else {
        // ------------------------------------------------------------ weights and results, one row a thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int q = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16, ts = lane_base + q * 128, to = lane_base + C::O_COL + q * C::OW;
        unsigned t = 0;  // this row tile's key tiles so far
        walk([&](const PtWork &w, int kv_head) {
            const int first = of(w.first, q), token = first + row, limit = first < w.t.n_q ? pa_limit(P, w.t, token) : 0, n = of(w.tiles, q);
            float m = -INFINITY, mc = 0.0f, l = 0.0f;  // the maximum, and times the scale (0 without keys); this row's sum
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = __all_sync(~0u, mbar_wait(bar, parity, abort_flag, X.wait_ns));
                tc_fence_after();
                return ok;
            };
            for (int i = 0; i < n; ++i, ++t) {
                const int j = n - 1 - i;
                if (!wait(&s_full[q], t & 1)) break;
                float s[PT];
#pragma unroll
                for (int c = 0; c < PT; c += 32) tmem_ld32(ts + c, s + c);
                tmem_wait_ld();
                if ((j + 1) * PT > of(w.lowest, q)) {
                    const int seen = limit - j * PT;
#pragma unroll
                    for (int c = 0; c < PT; ++c) s[c] = c < seen ? s[c] : -INFINITY;
                }
                float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int c = 4; c < PT; ++c) top[c & 3] = fmaxf(top[c & 3], s[c]);
                const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                float less = mc;
                if (__any_sync(~0u, (mx - m) * P.scale > kPtSlack || (fabsf(mc) > kPtFused && mx > -INFINITY))) {
                    const float f = mx > m ? pt_exp2((m - mx) * P.scale) : 1.0f;
                    if (mx > m) m = mx, less = mc = fmaxf(m * P.scale, kPaNone);
                    l *= f;
                    if (i > 0) {
                        if (!wait(&o_full[q], (t - 1) & 1)) break;
#pragma unroll 1
                        for (int c = 0; c < C::OW; c += 32) {
                            float o[32];
                            uint32_t r[32];
                            tmem_ld32(to + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(o[k] * f);
                            tmem_st32(to + c, r);
                        }
                    }
                    if (__any_sync(~0u, fabsf(mc) > kPtFused)) {
                        const bool far = fabsf(mc) > kPtFused;
                        const float at = far ? m : 0.0f;
                        if (far) less = 0.0f;
#pragma unroll
                        for (int c = 0; c < PT; c += 2) {
                            const float2 x = fma2(make_float2(s[c], s[c + 1]), make_float2(1.0f, 1.0f), make_float2(-at, -at));
                            s[c] = x.x, s[c + 1] = x.y;
                        }
                    }
                }
                const float2 sc = make_float2(P.scale, P.scale), off = make_float2(-less, -less);
                float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int c = 0; c < PT; c += 64) {
                    uint32_t r[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        float2 x = fma2(make_float2(s[c + 2 * k], s[c + 2 * k + 1]), sc, off);
                        x.x = pt_exp2(x.x);
                        x.y = pt_exp2(x.y);
                        sum[k & 1] = fma2(x, make_float2(1.0f, 1.0f), sum[k & 1]);
                        r[k] = pt_pack<T>(x.x, x.y);
                    }
                    tmem_st32(ts + c / 2, r);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[q]);
            }
            if (ok && n) wait(&o_full[q], (t - 1) & 1);
            for (int i = 0; i < w.masked && ok; ++i) wait(&v_ok[place(i)], phase(i));  // (the flags are in place)
            if (!ok) return false;
            uint32_t bits[C::FIX_ROW / 4] = {};
            bool any = false;
#pragma unroll 1
            for (int i = 0; i < w.masked * 2; ++i) {
                if (!fixed[place(0) * 2 + i]) continue;
                any = true;
                const int r0 = (i & 1) * 64, key0 = (w.n - 1 - (i >> 1)) * PT + r0;
#pragma unroll 1
                for (int r = 0; r < 64 && key0 + r < limit; ++r) {
                    const uint32_t *b = reinterpret_cast<const uint32_t *>(fix + (place(i >> 1) * PT + r0 + r) * C::FIX_ROW);
                    uint32_t one_sign = 0;
#pragma unroll
                    for (int k = 0; k < C::DP / 32; ++k) one_sign |= b[k] ^ b[C::DP / 32 + k];
                    // an infinite value whose score is -inf weighs 0: NaN, not infinity
                    bool none = false;
                    if (one_sign) {
                        const T *x = static_cast<const T *>(P.q) + (w.t.q_row + token) * P.ldq + (int64_t)(kv_head * P.G + of(w.head, q)) * P.D;
                        const T *k = static_cast<const T *>(P.k) + (w.t.k_row + key0 + r) * P.ldk + (int64_t)kv_head * P.D;
                        float dot = 0.0f;
                        for (int d = 0; d < P.D; ++d) dot += to_f32(x[d]) * to_f32(k[d]);
                        none = (P.negate ? -dot : dot) == -INFINITY;
                    }
#pragma unroll
                    for (int k = 0; k < C::DP / 32; ++k) {
                        const uint32_t plus = b[k], minus = b[C::DP / 32 + k];
                        bits[k] |= none ? plus | minus : plus;
                        bits[C::DP / 32 + k] |= none ? plus | minus : minus;
                    }
                }
            }
            __syncwarp();
            if (w.masked && lane == 0) mbar_arrive(&fix_free[pairs_masked & 1]);
            const bool live = first < w.t.n_q && token < w.t.n_q;
            const float inv = 1.0f / l;
            T *y = static_cast<T *>(P.y) + (w.t.q_row + token) * P.ldy + (int64_t)(kv_head * P.G + of(w.head, q)) * P.D;
            // (not unrolled: code that runs once a pair comes from memory)
#pragma unroll 1
            for (int c = 0; c < C::OW; c += 32) {
                float o[32];
                if (n) {
                    tmem_ld32(to + c, o);
                    tmem_wait_ld();
                }
                if (any) {
                    uint32_t plus = bits[0], minus = bits[C::DP / 32];
#pragma unroll
                    for (int k = 1; k < C::DP / 32; ++k)
                        if (c == 32 * k) plus = bits[k], minus = bits[C::DP / 32 + k];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (plus >> k & 1) o[k] += INFINITY;
                        if (minus >> k & 1) o[k] -= INFINITY;
                    }
                }
                uint32_t r[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) r[k] = limit ? pt_pack<T>(o[2 * k] * inv, o[2 * k + 1] * inv) : 0u;
                if (X.wide) {  // whole sectors
#pragma unroll
                    for (int k = 0; k < 16; k += 8)
                        if (live && c + 2 * k < P.D)
                            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(y + c + 2 * k), "r"(r[k]), "r"(r[k + 1]),
                                         "r"(r[k + 2]), "r"(r[k + 3]), "r"(r[k + 4]), "r"(r[k + 5]), "r"(r[k + 6]), "r"(r[k + 7])
                                         : "memory");
                } else {
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        if (live && c + 2 * k < P.D) *reinterpret_cast<uint4 *>(y + c + 2 * k) = make_uint4(r[k], r[k + 1], r[k + 2], r[k + 3]);
                }
            }
            masked_done(w);
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort_flag) atomicAdd(P.err, 1ull);  // (here: any role may have given up last)
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(*tmem_holder) : "memory");
    }
}

// Clears the device flag and the line's counter and, for several sequences, puts the pairs in order of their key tiles, most
// first (pairs of the same number in any order, which no result depends on): a long one that starts last is what all wait
// for (nine sequences, heads of 80: 40.3 us without).
constexpr int PT_BINS = 256;
__global__ void __launch_bounds__(1024) pt_order_kernel(PaParams P, int64_t pairs, unsigned *next, int *order) {
    __shared__ int bins[PT_BINS];
    grid_dependency_wait();
    grid_launch_dependents();
    if (threadIdx.x == 0) *P.err = 0ull, *next = 0u;
    if (!order) return;
    auto bin = [&](int64_t pair) {
        int64_t b = 0;
        for (int64_t n = P.B; n > 1;) {
            const int64_t half = n / 2;
            if (pt_start(P, b + half) <= pair) b += half, n -= half;
            else n = half;
        }
        PtWork w;
        return pt_start(P, b) <= pair && pt_fill(P, b, pair, w) ? PT_BINS - 1 - min(w.n, PT_BINS - 2) : PT_BINS - 1;
    };
    for (int i = threadIdx.x; i < PT_BINS; i += blockDim.x) bins[i] = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < pairs; i += blockDim.x) atomicAdd(&bins[bin(i)], 1);
    __syncthreads();
    if (threadIdx.x < 32) {  // where each bin begins
        constexpr int PER = PT_BINS / 32;
        int n[PER], sum = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) n[k] = bins[threadIdx.x * PER + k], sum += n[k];
        int upto = sum;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int o = __shfl_up_sync(~0u, upto, s);
            if ((int)threadIdx.x >= s) upto += o;
        }
        int at = upto - sum;
#pragma unroll
        for (int k = 0; k < PER; ++k) bins[threadIdx.x * PER + k] = at, at += n[k];
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < pairs; i += blockDim.x) order[atomicAdd(&bins[bin(i)], 1)] = (int)i;
}

// ---------------------------------------------------------------- host
static PFN_cuTensorMapEncodeTiled_v12000 pt_encoder() {
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

static int64_t pt_pairs(int64_t B, int64_t Tq, int64_t G) { return ((Tq / PT + B) * G >> 1) + B; }
size_t pa_tc_workspace(int64_t B, int64_t Tq, int64_t G) { return 256 + (size_t)(pt_pairs(B, Tq, G) * 4 + 255) / 256 * 256; }

int64_t pa_tc_units(int64_t B, int64_t Tq, int64_t n_q, int64_t n_kv) { return pt_pairs(B, Tq, n_q / n_kv) * n_kv; }

bool pa_aligned(const PaParams &P) {
    return P.D % 8 == 0 && aligned(P.q, 16) && aligned(P.k, 16) && aligned(P.v, 16) && aligned(P.y, 16) && P.ldq % 8 == 0 &&
           P.ldk % 8 == 0 && P.ldv % 8 == 0 && P.ldy % 8 == 0;
}
bool pa_takes_tc(const PaParams &P) { return P.D <= 128 && pa_aligned(P); }

template <typename T, typename C>
static kq_status pt_launch(const char *fn, PtParams X, cudaStream_t st) {
    auto encode = pt_encoder();
    if (!encode) return fail(KQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", fn);
    const PaParams &P = X.p;
    CUtensorMap tm[3];
    const struct { const void *p; int64_t ld, rows; int heads; } in[3] = {
        {P.q, P.ldq, P.Tq, P.n_q}, {P.k, P.ldk, P.Tk, X.n_kv}, {P.v, P.ldv, P.Tk, X.n_kv}};
    for (int i = 0; i < 3; ++i) {
        const cuuint64_t dims[3] = {(cuuint64_t)P.D, (cuuint64_t)in[i].heads, (cuuint64_t)in[i].rows};
        const cuuint64_t strides[2] = {(cuuint64_t)P.D * 2, (cuuint64_t)in[i].ld * 2};
        const cuuint32_t box[3] = {64, 1, PT}, es[3] = {1, 1, 1};
        const CUresult e = encode(&tm[i], std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                  3, const_cast<void *>(in[i].p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (e != CUDA_SUCCESS) return fail(KQ_ERR_CUDA, "%s: tensor map %d failed (%d)", fn, i, (int)e);
    }
    X.pairs = pt_pairs(P.B, P.Tq, P.G);
    auto kern = pt_kernel<T, C>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::TOTAL);
    const int64_t items = X.pairs * X.n_kv;
    constexpr int SMS = 152;
    X.next = items > SMS ? reinterpret_cast<unsigned *>(P.err + 1) : nullptr;
    int *order = X.next && P.B > 1 ? reinterpret_cast<int *>(P.err + 32) : nullptr;
    X.order = order;
    if (e == cudaSuccess && X.next) {
        e = launch_beside(pt_order_kernel, dim3(1), dim3(order ? 1024 : 32), 0, dim3(1), st, P, X.pairs, X.next, order);
        if (e == cudaSuccess) count_launch(R_ATTN);
    }
    if (e == cudaSuccess)
        e = launch_beside(kern, dim3((unsigned)std::min<int64_t>(items, SMS)), dim3(PT_THREADS), C::TOTAL, dim3(1), st, tm[0], tm[1], tm[2], X);
    if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    count_launch(R_ATTN);
    return KQ_OK;
}

kq_status pa_tc(const char *fn, kq_dtype xt, const PaParams &P, unsigned long long wait_ns, int idle, cudaStream_t st) {
    PtParams X{P, 0, P.n_q / P.G, wait_ns, idle, aligned(P.y, 32) && P.ldy % 16 == 0 && P.D % 16 == 0, nullptr, nullptr};
    auto go = [&](auto t) {
        using T = decltype(t);
        if (P.D <= 64) return pt_launch<T, PtCfg<64, 64>>(fn, X, st);
        return P.D <= 96 ? pt_launch<T, PtCfg<128, 96>>(fn, X, st) : pt_launch<T, PtCfg<128, 128>>(fn, X, st);
    };
    return xt == KQ_F16 ? go(__half{}) : go(__nv_bfloat16{});
}

}  // namespace kq
