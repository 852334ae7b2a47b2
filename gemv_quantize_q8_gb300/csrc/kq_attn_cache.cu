// kq_attn_cache.cu -- attention of a few query tokens over the paged 8-bit cache.
//
// For a query row q (one token and head) over the tokens j that it sees, with s_j = scale * ks * (q . K_j) for codes
// K, V and their blocks' scales ks, vs:
//   m = max s_j,  l = sum 2^(s_j - m),  y = (sum 2^(s_j - m) vs V_j) / l       (s in units of log 2)
// What is handed from warp to warp or block to block is m, l and y of a part: sums that are not divided yet may leave fp32.
// Bound by the cache's bytes: each is read once, by TMA, into a ring of the warp that needs it (2 or 4 KB a copy, two
// or three units under way; a warp waits for nobody else).  Two sequences of 131072 tokens, 32 heads over 8 of 128, 537 MB: 87.8
// us, 6.1 TB/s, of which the start, the parts and their join take 10; 64 users of up to 8192 tokens, 516 MB, 89.3; one user of
// 900 tokens 10.1, all of it latency.  (By 16-byte copies of every lane the loads alone took 136 us for the first.)
//
// The products run on m16n8k16 instructions.  Codes are exact in f16; a query row is brought to |q| < 2 by a power
// of two and split into two f16 (22 bits), as the weights 2^(s - m) vs are, held against the largest of their own row.
// With up to eight rows (the query heads of one key head) the second parts fill the tile's other eight rows, so they cost
// nothing; tiles of 16 rows take twice the instructions.  Which of its elements a lane holds is free where both operands agree, so it follows the loads:
//   keys:   lane 4n + c of an eight-token tile takes the 16-byte pieces 2c and 2c + 1 of token n; 4 bytes make the two
//           registers of one step.
//   values: lane 4n + c takes piece n of tokens 2c, 2c + 1, 2c + 8, 2c + 9: the tokens whose weights it holds, the
//           bytes of two tokens paired by permutes.
// With the copies' 128-byte swizzle neither has bank conflicts.
// A unit is 32 tokens, two halves of 16 with scales of their own (a page holds whole halves).  All units of all sequences
// and heads form one line, cut into equal shares, one a warp (an item's beginning counts as units, too): lengths may differ
// as they like.  A row whose units are shared by warps is put together in shared memory, one that is shared by thread
// blocks through the workspace and a second kernel, in a fixed order.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <type_traits>

#include "kq_i8_tc.cuh"
#include "kq_kv.cuh"
#include "kq_launch.cuh"

namespace kq {

constexpr int kAcUnit = 32;           // tokens
constexpr int kAcLeast = 1;           // units of a warp
// What an item's beginning (its queries are loaded and split) costs a warp, in units, where the line is cut into shares; 64
// users of up to 8192 tokens: 98.5 us without it, 91.0 with 1, 88.4 with 2 and 3.  Not for shares of fewer than two units
// with it: their borders then fall less evenly (16 users of up to 512 tokens 13.2 us without, 13.6 with it; 32 users,
// whose shares have two: 18.9 and 15.5).
constexpr int kAcStart = 2;
constexpr int kAcMaxBlocks = 152;     // one an SM
constexpr unsigned long long kAcWaitNs = 2000000000ull;  // limit of every wait
constexpr float kAcSlack = 8.0f;      // a weight may grow to 2^8 before the sums are brought to a new maximum
// Weights are held times this power of two: f16 keeps their low bits, with room for kAcSlack.
constexpr float kAcLift = 7.0f;
constexpr float kAcLeastRef = -119.0f;  // the least reference that they are held against: 2^(kAcLift + 119) is finite
constexpr float kAcNone = -3.402823466e38f;  // the maximum of no token: no finite score is below it

struct AcParams {
    KvCache c;
    const void *q;
    void *y;
    int64_t ldq, ldy;
    kq_dtype xt, yt;
    bool qvec, yvec;      // query rows on boundaries of four elements, output rows on 16 bytes
    int n_new, n_q, G;    // query tokens of a sequence, query heads, and those of a key head
    int rows, tiles;      // rows of a key head (n_new * G), and the row tiles that they take
    float scale;          // times log2 e
    unsigned long long *err;  // device flag, cleared by the call
    float *parts;             // [blocks][2] partial results
    int blocks, warps;    // of the first kernel's grid
    unsigned long long wait_ns;  // limit of every wait
    bool idle;            // test hook: nothing is fetched
};

// What a warp (or a block) hands over: m and l of its rows, then their weighted averages, in the order in which a
// warp's lanes hold them (32 lanes side by side, 16 bytes each: no bank conflicts).
template <int DP, int MT> constexpr int kAcPart = MT * (DP + 2);

// A place on the line of units.
struct AcItem {
    int64_t b;       // sequence
    int h, tile;     // key head, row tile
    int units;       // of this sequence
};

__device__ __forceinline__ int64_t ac_len(const AcParams &P, int64_t b) {
    const int64_t n = P.c.lens[b], most = P.c.ldt << P.c.lp;
    return n < 0 ? 0 : n > most ? most : n;  // (past the table's end: NaN, see ac_bad)
}
__device__ __forceinline__ bool ac_bad(const AcParams &P, int64_t b) { return P.c.lens[b] > P.c.ldt << P.c.lp; }
__device__ __forceinline__ int ac_units(const AcParams &P, int64_t b) { return (int)((ac_len(P, b) + kAcUnit - 1) / kAcUnit); }

// Quotients: 32 bits wherever they do.
__device__ __forceinline__ int64_t ac_div(int64_t a, int64_t b) {
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// The line of units cut into n shares (n is at most a few hundred): where share w begins.
struct AcShares {
    int64_t each;
    int rest, n;
    __device__ __forceinline__ AcShares(int64_t total, int n_) : each(ac_div(total, n_)), rest((int)(total - each * n_)), n(n_) {}
    __device__ __forceinline__ int64_t operator()(int w) const { return each * w + (unsigned)(rest * w) / (unsigned)n; }
};
// The blocks that share the line: each warp has kAcLeast units at least, if there are so many.
__device__ __forceinline__ int ac_blocks(const AcParams &P, int64_t total, int warps) {
    const int64_t n = ac_div(total, kAcLeast * warps);
    return n < 1 ? 1 : n < P.blocks ? (int)n : P.blocks;
}

// Where the sequences lie on the line: thread t of the block sums up `per` of them; units and places up to their end.
template <int THREADS>
struct AcLine {
    int64_t units[THREADS], places[THREADS], warps[THREADS / 32];
    int full[THREADS / 32];
};
// Its length.  Every item begins with `start` places without units.
struct AcTotal {
    int64_t units, places;
    int blocks, start;
};
// All threads of the block.
template <int THREADS>
__device__ __forceinline__ AcTotal ac_line(const AcParams &P, AcLine<THREADS> &line, int warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t per = (P.c.B + THREADS - 1) / THREADS, b0 = threadIdx.x * per;
    const int64_t items = (int64_t)P.c.n_kv * P.tiles;  // of a sequence
    int64_t n = 0;
    int full = 0;  // sequences with units
    for (int64_t b = b0; b < b0 + per && b < P.c.B; ++b) {
        const int units = ac_units(P, b);
        n += units;
        full += units > 0;
    }
    n *= items;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, n, s);
        const int f = __shfl_up_sync(~0u, full, s);
        if (lane >= s) n += o, full += f;
    }
    if (lane == 31) line.warps[warp] = n, line.full[warp] = full;
    __syncthreads();
    int64_t total = 0;
    int all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w == warp) n += total, full += all;
        total += line.warps[w];
        all += line.full[w];
    }
    AcTotal r;
    r.units = total;
    r.blocks = ac_blocks(P, total, warps);
    r.places = total + kAcStart * items * all;
    r.start = r.places >= 2ll * r.blocks * warps ? kAcStart : 0;
    if (!r.start) r.places = total;
    line.units[threadIdx.x] = n;
    line.places[threadIdx.x] = n + r.start * items * full;
    __syncthreads();
    return r;
}
// The item that place u (below the line's length) lies in, and its place in it; returns the units of the line before it.
template <int THREADS>
__device__ __forceinline__ int64_t ac_find(const AcParams &P, const AcLine<THREADS> &line, int start, int64_t u, AcItem &it, int &at) {
    int lo = 0;  // threads whose sequences end at or before u
#pragma unroll
    for (int s = THREADS / 2; s; s >>= 1)
        if (line.places[lo + s - 1] <= u) lo += s;
    int64_t before = 0;
    if (lo) before = line.units[lo - 1], u -= line.places[lo - 1];
    const int64_t per = (P.c.B + THREADS - 1) / THREADS;
    for (it.b = lo * per;; ++it.b) {
        it.units = ac_units(P, it.b);
        const int64_t items = it.units ? (int64_t)P.c.n_kv * P.tiles : 0, mine = items * (it.units + start);
        if (u < mine) break;
        u -= mine;
        before += items * it.units;
    }
    const int64_t i = ac_div(u, it.units + start);
    at = (int)(u - i * (it.units + start));
    it.h = (int)((uint32_t)i / (uint32_t)P.tiles);
    it.tile = (int)i - it.h * P.tiles;
    return before + i * it.units;
}
// The next item that has units (there is one).
__device__ __forceinline__ void ac_next(const AcParams &P, AcItem &it) {
    if (++it.tile < P.tiles) return;
    it.tile = 0;
    if (++it.h < P.c.n_kv) return;
    it.h = 0;
    do ++it.b;
    while (it.b < P.c.B - 1 && ac_units(P, it.b) == 0);
    it.units = ac_units(P, it.b);
}

// Four consecutive elements.
template <typename T, bool VEC>
__device__ __forceinline__ void ac_load4(const T *p, float (&v)[4]) {
    if constexpr (VEC) {
        const auto u = *reinterpret_cast<const typename VecOf<4 * (int)sizeof(T)>::type *>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = to_f32(reinterpret_cast<const T *>(&u)[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = to_f32(p[j]);
    }
}
__device__ __forceinline__ void ac_store(void *p, kq_dtype t, int64_t i, float v) {
    if (t == KQ_F32) static_cast<float *>(p)[i] = v;
    else if (t == KQ_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float ac_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^x for whole numbers -126 .. 127.
__device__ __forceinline__ float ac_pow2(float x) { return __uint_as_float((uint32_t)(127 + (int)x) << 23); }
// A whole number above log2 |x|, -126 below the normal numbers.
__device__ __forceinline__ float ac_size(float x) {
    return __uint_as_float(0x4b000000u | (__float_as_uint(x) >> 23 & 255u)) - (8388608.0f + 126.0f);
}
// 1/l of a sum of weights.  A part of an item's tokens may have none that a row sees: 0.  (All of them: 0 * infinity, which
// is NaN where a row sees tokens, all of scores below fp32, and is not written where it sees none.)
__device__ __forceinline__ float ac_inverse(float l, bool all) { return l == 0.0f && !all ? 0.0f : 1.0f / l; }
__device__ __forceinline__ void ac_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two values as f16, and what they leave as f16.
__device__ __forceinline__ void ac_split(float x, float y, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(x, y);
    const __half2 l = __floats2half2_rn(x - __low2float(h), y - __high2float(h));
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}
// Four codes each of two tokens as f16 pairs, one pair an element.
__device__ __forceinline__ void ac_pair(uint32_t x, uint32_t y, uint32_t (&o)[4]) {
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152, as i8x4_to_f16
    x ^= 0x80808080u;
    y ^= 0x80808080u;
    const uint32_t a = __byte_perm(x, y, 0x5140), b = __byte_perm(x, y, 0x7362);
    o[0] = __byte_perm(a, 0x64646464u, 0x4140);
    o[1] = __byte_perm(a, 0x64646464u, 0x4342);
    o[2] = __byte_perm(b, 0x64646464u, 0x4140);
    o[3] = __byte_perm(b, 0x64646464u, 0x4342);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&o[i]), bias);
        o[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Element (of D) that value j of a lane's row holds, in the half `e` (0, 1) of its accumulators: lane 4g + c owns
// the columns n = 2c + e of every eight-column tile j, and column n of tile j is this element.
template <int DP>
__device__ __forceinline__ int ac_element(int j, int n) {
    return DP == 64 ? n * 8 + j : (j / 16) * 128 + n * 16 + j % 16;
}

__device__ __forceinline__ void ac_copy(uint8_t *dst, const CUtensorMap *tm, uint64_t *bar, int d, int row, int page) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            sm100::smem_u32(dst)),
        "l"(tm), "r"(sm100::smem_u32(bar)), "r"(d), "r"(row), "r"(page)
        : "memory");
}

// A unit in a warp's ring: 32 rows of keys, then of values, in boxes of W bytes of a row as the copies write them
// (16-byte pieces swizzled: by row % 8 in rows of 128 bytes, by row / 2 % 4 in rows of 64).
template <int DP>
struct AcRing {
    static constexpr int W = DP < 128 ? DP : 128, BOXES = DP / W, BOX = kAcUnit * W, BYTES = 2 * BOXES * BOX;
    static constexpr int KP = DP / 64;               // 16-byte pieces of a key that a lane takes
    static constexpr int VWORDS = DP == 64 ? 2 : 4;  // 4-byte words of a value that a lane takes at once
    // Piece i of a lane's key (of eight-token tile t) begins at this element of the head.
    static __device__ __forceinline__ int key_element(int i) {
        const int c = threadIdx.x & 3;
        return DP == 64 ? c * 16 : (i >> 1) * 128 + (2 * c + (i & 1)) * 16;
    }
    // (volatile: the loads stay where they are written, well ahead of their use)
    static __device__ __forceinline__ void get_key(uint32_t stage, int t, int i, uint32_t (&v)[4]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        const uint32_t at = stage + (i >> 1) * BOX + (t * 8 + g) * W + ((DP == 64 ? c ^ (g >> 1) : (2 * c + (i & 1)) ^ g) << 4);
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at));
    }
    // Words 4i on of a lane's value of token 16h + 2c + (t & 1) + 8 (t >> 1).
    static __device__ __forceinline__ void get_value(uint32_t stage, int h, int t, int i, uint32_t (&v)[VWORDS]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, low = 2 * c + (t & 1), row = 16 * h + low + 8 * (t >> 1);
        const uint32_t at = stage + (BOXES + i) * BOX + row * W;
        if constexpr (DP == 64)
            asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(at + (((g >> 1) ^ c) << 4) + (g & 1) * 8));
        else
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(at + ((g ^ low) << 4)));
    }
};

// A warp's state for one item: DP is D rounded up to 64, 128 or 256; MT is 8 rows (parts of the split in the other
// eight) or 16.
template <int DP, int MT>
struct AcWarp {
    static constexpr int KS = DP / 16;   // steps of the first product
    static constexpr int NT = DP / 8;    // column tiles of the second
    static constexpr int KP = DP / 64;   // 16-byte pieces of a key that a lane loads
    static constexpr int VW = DP / 32;   // 4-byte words of a value that a lane loads
    uint32_t qh[KS][MT == 8 ? 2 : 4], ql[KS][MT == 8 ? 2 : 4];
    float o[NT][4];
    static constexpr int R = MT / 8;     // rows of a lane: g and, with 16, g + 8
    float m[R], l[R], factor[R];         // (factor: the power of two that the row was brought down by)
    int limit[R], sure;                  // tokens that a row sees, and that all rows see
    // A row's weights times their blocks' value scales are held against a power of two of its own, 2^ref, that is above
    // the largest of them so far and not far above: blocks that a row does not see, or weighs next to nothing, cost
    // the others no bits, however large their scales.  They are held times down * up = 2^(kAcLift - ref); down is at
    // most 1 and goes with the scale, up is at least 1 and comes last, so that nothing overflows on the way.
    float ref[R], down[R], up[R];

    __device__ __forceinline__ void begin(const AcParams &P, const AcItem &it) {
        const int g = (threadIdx.x & 31) >> 2;
        const int64_t len = ac_len(P, it.b);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = it.tile * MT + g + 8 * r;
            const bool live = row < P.rows;
            const int token = live ? row / P.G : 0, head = it.h * P.G + (live ? row - token * P.G : 0);
            const int64_t at = (it.b * P.n_new + token) * P.ldq + (int64_t)head * P.c.D;
            const int64_t sees = len - P.n_new + 1 + token;
            limit[r] = live && sees > 0 ? (int)sees : 0;
            float v[KS][4], amax = 0.0f;
            // (one branch a type around all loads: they are under way together)
            auto fill = [&](auto type, auto vec) {
                using T = decltype(type);
                const T *x = static_cast<const T *>(P.q) + at;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const int d = AcRing<DP>::key_element(s / 4) + (s % 4) * 4;
                    v[s][0] = v[s][1] = v[s][2] = v[s][3] = 0.0f;
                    if (live && d < P.c.D) ac_load4<T, decltype(vec)::value>(x + d, v[s]);
                }
            };
            auto typed = [&](auto vec) { P.xt == KQ_F32 ? fill(float{}, vec) : P.xt == KQ_F16 ? fill(__half{}, vec) : fill(__nv_bfloat16{}, vec); };
            if (P.qvec) typed(std::true_type{});
            else typed(std::false_type{});
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(v[s][i]));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            // the power of two at or below the largest (2^-126 for rows below the normal numbers, 1 for infinities)
            uint32_t e = __float_as_uint(amax) & 0x7f800000u;
            if (e == 0x7f800000u) e = 0x3f800000u;
            if (e == 0u) e = 0x00800000u;
            if (e > 0x7e800000u) e = 0x7e800000u;
            const float down = __uint_as_float(0x7f000000u - e);
            factor[r] = __uint_as_float(e);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                ac_split(v[s][0] * down, v[s][1] * down, qh[s][r * 2], ql[s][r * 2]);
                ac_split(v[s][2] * down, v[s][3] * down, qh[s][r * 2 + 1], ql[s][r * 2 + 1]);
            }
            m[r] = kAcNone;
            l[r] = 0.0f;
            refer(r, kAcLeastRef);
        }
        sure = (int)max(len - P.n_new + 1, (int64_t)0);  // (rows past the tile's end are not kept)
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    }

    __device__ __forceinline__ void refer(int r, float to) {
        ref[r] = to;
        down[r] = ac_pow2(fminf(kAcLift - to, 0.0f));
        up[r] = ac_pow2(fmaxf(kAcLift - to, 0.0f));
    }

    // A unit: tokens t0 .. t0 + 31, of which a row sees those below its limit.
    // scales: of keys and values, of its first and second half.
    __device__ __forceinline__ void unit(uint32_t stage, float4 scales, int t0, float scale) {
        using Ring = AcRing<DP>;
        const int c = threadIdx.x & 3;
        uint32_t k[KP][4][4];
        constexpr int AHEAD = KP < 2 ? KP : 2;  // (all four pieces of heads of 256 do not fit the registers)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t) Ring::get_key(stage, t, i, k[i][t]);
        float s[4][4] = {};
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            if (i + 1 >= AHEAD && i + 1 < KP)
#pragma unroll
                for (int t = 0; t < 4; ++t) Ring::get_key(stage, t, i + 1, k[i + 1][t]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    uint32_t b0, b1;
                    i8x4_to_f16(k[i][t][w], b0, b1);
                    const int st = i * 4 + w;
                    if constexpr (MT == 8) {
                        ac_mma(s[t], qh[st][0], ql[st][0], qh[st][1], ql[st][1], b0, b1);
                    } else {
                        ac_mma(s[t], qh[st][0], qh[st][2], qh[st][1], qh[st][3], b0, b1);
                        ac_mma(s[t], ql[st][0], ql[st][2], ql[st][1], ql[st][3], b0, b1);
                    }
                }
            }
        }
        uint32_t v[VW / Ring::VWORDS][2][4][Ring::VWORDS];
        auto values = [&](int i) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < 4; ++t) Ring::get_value(stage, h, t, i, v[i][h][t]);
        };
        values(0);
        // x[r][2t + e]: a row's logits for tokens 8t + 2c + e, in units of log 2
        float x[R][8], top[R][2];
        bool grows = false;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // the product first and the scale last, each rounded: the scale alone may be as large as fp32
            const float f[2] = {factor[r] * scales.x, factor[r] * scales.z};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float2 sum = MT == 8 ? make_float2(s[t][0] + s[t][2], s[t][1] + s[t][3]) : make_float2(s[t][2 * r], s[t][2 * r + 1]);
                const float2 v = mul2(mul2(sum, make_float2(f[t >> 1], f[t >> 1])), make_float2(scale, scale));
                x[r][2 * t] = v.x;
                x[r][2 * t + 1] = v.y;
            }
        }
        if (t0 > sure - kAcUnit) {  // not every row sees all of the unit
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (t0 + (i >> 1) * 8 + 2 * c + (i & 1) >= limit[r]) x[r][i] = -INFINITY;
        }
        float vs[2] = {scales.y, scales.w};
        const float size[2] = {ac_size(vs[0]), ac_size(vs[1])};
        // what the unit's halves would be held as: the largest weight, and the largest times its block's scale
        auto heights = [&](int r, float base, float &p, float &pv) {
            p = fmaxf(top[r][0], top[r][1]) - base;
            pv = fmaxf(top[r][0] - base + size[0], top[r][1] - base + size[1]);
        };
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                top[r][h] = fmaxf(fmaxf(x[r][4 * h], x[r][4 * h + 1]), fmaxf(x[r][4 * h + 2], x[r][4 * h + 3]));
            float p, pv;
            heights(r, m[r], p, pv);
            grows |= p > kAcSlack || pv > ref[r] + kAcSlack;
        }
        if (__any_sync(~0u, grows)) {
            // bring the sums of the rows that grow to a new maximum and a new reference
            float f[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top[r][h] = fmaxf(top[r][h], __shfl_xor_sync(~0u, top[r][h], 1));
                    top[r][h] = fmaxf(top[r][h], __shfl_xor_sync(~0u, top[r][h], 2));
                }
                f[r] = 1.0f;
                float p, pv;
                heights(r, m[r], p, pv);
                if (!(p > kAcSlack || pv > ref[r] + kAcSlack)) continue;
                const float mx = fmaxf(m[r], fmaxf(top[r][0], top[r][1])), by = m[r] - mx, was = ref[r];
                heights(r, mx, p, pv);
                refer(r, fmaxf(fmaxf(floorf(was + by), ceilf(pv)), kAcLeastRef));
                l[r] *= ac_exp2(by);
                f[r] = ac_exp2(by + (was - ref[r]));
                m[r] = mx;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o[j][0] *= f[0];
                o[j][1] *= f[0];
                o[j][2] *= f[R - 1];
                o[j][3] *= f[R - 1];
            }
        }
        const bool poison = !(fabsf(vs[0]) < INFINITY && fabsf(vs[1]) < INFINITY);
        if (poison) poisoned(x, vs);
        uint32_t ph[R][4], pl[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = ac_exp2(x[r][i] - m[r]);
            l[r] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
            const float by[2] = {vs[0] * down[r], vs[1] * down[r]};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float2 w = mul2(mul2(make_float2(p[2 * t], p[2 * t + 1]), make_float2(by[t >> 1], by[t >> 1])), make_float2(up[r], up[r]));
                ac_split(w.x, w.y, ph[r][t], pl[r][t]);
            }
        }
#pragma unroll
        for (int n = 0; n < VW / Ring::VWORDS; ++n) {
            if (n) values(n);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int w = 0; w < Ring::VWORDS; ++w) {
                    uint32_t a[4], b[4];
                    ac_pair(v[n][h][0][w], v[n][h][1][w], a);
                    ac_pair(v[n][h][2][w], v[n][h][3][w], b);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float (&acc)[4] = o[4 * (n * Ring::VWORDS + w) + i];
                        if constexpr (MT == 8) {
                            ac_mma(acc, ph[0][2 * h], pl[0][2 * h], ph[0][2 * h + 1], pl[0][2 * h + 1], a[i], b[i]);
                        } else {
                            ac_mma(acc, ph[0][2 * h], ph[1][2 * h], ph[0][2 * h + 1], ph[1][2 * h + 1], a[i], b[i]);
                            ac_mma(acc, pl[0][2 * h], pl[1][2 * h], pl[0][2 * h + 1], pl[1][2 * h + 1], a[i], b[i]);
                        }
                    }
                }
        }
    }
    // A block of values with an infinity: NaN for the rows that see it, for them alone.
    __device__ __forceinline__ void poisoned(const float (&x)[R][8], float (&vs)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (!(fabsf(vs[h]) < INFINITY)) {
                vs[h] = 0.0f;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (x[r][4 * h + i] > -INFINITY) l[r] = NAN;
            }
    }

    // The item's results so far: m, l, and D values a row, which are weighted averages already: sums relative to 2^m could
    // leave fp32 where the values do not.
    __device__ __forceinline__ void end(bool all) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[r] += __shfl_xor_sync(~0u, l[r], 1);
            l[r] += __shfl_xor_sync(~0u, l[r], 2);
        }
        float back[R];
#pragma unroll
        for (int r = 0; r < R; ++r) back[r] = ac_pow2(ref[r] - kAcLift);
        float inv[R];
#pragma unroll
        for (int r = 0; r < R; ++r) inv[r] = ac_inverse(l[r], all);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (MT == 8) {
                o[j][0] += o[j][2];
                o[j][1] += o[j][3];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = o[j][i] * inv[i / 2 * (R - 1)] * back[i / 2 * (R - 1)];
        }
    }
    // What a lane holds of a row lies in runs: f(r, d0, run) for the RUN elements from d0 on of its row r.
    static constexpr int RUN = DP == 64 ? 8 : 16;
    template <typename F>
    __device__ __forceinline__ void runs(int D, F f) {
        const int c = threadIdx.x & 3;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < NT; j += RUN)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d0 = ac_element<DP>(j, 2 * c + e);
                    float v[RUN];
#pragma unroll
                    for (int i = 0; i < RUN; ++i) v[i] = o[j + i][2 * r + e];
                    if (d0 < D) f(r, d0, v);
                }
    }
    __device__ __forceinline__ void put(float *part) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (c == 0) part[g + 8 * r] = m[r], part[MT + g + 8 * r] = l[r];
        float4 *dst = reinterpret_cast<float4 *>(part + 2 * MT) + lane;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < NT; j += 4)
#pragma unroll
                for (int e = 0; e < 2; ++e, dst += 32)
                    *dst = make_float4(o[j][2 * r + e], o[j + 1][2 * r + e], o[j + 2][2 * r + e], o[j + 3][2 * r + e]);
    }
};
// Row and first element of the four at place x of a part.
template <int DP>
__device__ __forceinline__ void ac_place(int x, int &row, int &d) {
    const int lane = x & 31, e = x >> 5 & 1, j = (x >> 6) % (DP / 32) * 4;
    row = (lane >> 2) + 8 * ((x >> 6) / (DP / 32));
    d = ac_element<DP>(j, 2 * (lane & 3) + e);
}

// A run of row `row` (of the item's tile) of the output; a token that sees nothing gives 0.
template <int N>
__device__ __forceinline__ void ac_write_run(const AcParams &P, const AcItem &it, int MT, int row, int d0, const float (&v)[N]) {
    const int i = it.tile * MT + row;
    if (i >= P.rows) return;
    const int token = i / P.G, head = it.h * P.G + i - token * P.G;
    const bool sees = ac_len(P, it.b) - P.n_new + token >= 0;
    const int64_t at = (it.b * P.n_new + token) * P.ldy + (int64_t)head * P.c.D + d0;
    float x[N];
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = sees ? v[j] : 0.0f;
    if (!P.yvec) {
#pragma unroll
        for (int j = 0; j < N; ++j) ac_store(P.y, P.yt, at + j, x[j]);
    } else if (P.yt == KQ_F32) {
        float4 *y = reinterpret_cast<float4 *>(static_cast<float *>(P.y) + at);
#pragma unroll
        for (int j = 0; j < N; j += 4) y[j / 4] = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    } else {
        uint2 *y = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(P.y) + at);
        uint32_t w[N / 2];
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const __half2 h = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
            w[k] = P.yt == KQ_F16 ? *reinterpret_cast<const uint32_t *>(&h) : *reinterpret_cast<const uint32_t *>(&b);
        }
        if constexpr (N % 8 == 0) {
#pragma unroll
            for (int k = 0; k < N / 2; k += 4) reinterpret_cast<uint4 *>(y)[k / 4] = make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
        } else {
            y[0] = make_uint2(w[0], w[1]);
        }
    }
}
__device__ __forceinline__ void ac_write4(const AcParams &P, const AcItem &it, int MT, int row, int d0, float4 v) {
    const float x[4] = {v.x, v.y, v.z, v.w};
    ac_write_run(P, it, MT, row, d0, x);
}

__device__ __forceinline__ void ac_copy4(float *dst, const float *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sm100::smem_u32(dst)), "l"(src) : "memory");
}

// The units of one consumer's share, brought by one lane of the fetching warp: codes by TMA, scales by small copies
// that arrive at the same barrier.  The numbers of the next unit's pages are asked for when a unit has been sent off.
template <int DP>
struct AcFetch {
    AcItem it;
    int at;        // next unit of the item
    int64_t left;  // units to fetch
    int page[2];   // the next unit's
    int64_t len;   // of the item's sequence
    bool bad;
    const int32_t *table;
    __device__ __forceinline__ void start(const AcParams &P) {
        len = ac_len(P, it.b);
        bad = ac_bad(P, it.b);
        table = P.c.table + it.b * P.c.ldt;
    }
    __device__ __forceinline__ bool valid(const AcParams &P, int number) const { return number >= 0 && number < P.c.n_pages && !bad; }
    __device__ __forceinline__ void look(const AcParams &P) {
        const int t0 = at * kAcUnit;
        page[0] = table[t0 >> P.c.lp];
        if (P.c.lp == 4) page[1] = t0 + 16 < len ? table[(t0 + 16) >> P.c.lp] : 0;  // (a page of 16 holds half a unit)
    }
    __device__ __forceinline__ void send(const AcParams &P, const CUtensorMap *tmK, const CUtensorMap *tmV, uint8_t *stage, float4 *scales,
                                         uint64_t *bar) {
        using Ring = AcRing<DP>;
        const int t0 = at * kAcUnit, row = (it.h << P.c.lp) + (t0 & ((1 << P.c.lp) - 1));
        const bool small = P.c.lp == 4;
        // a unit's second half may lie past the last page: weight 0, whatever is there
        const int parts = small && t0 + 16 < len ? 2 : 1;
        const int number[2] = {page[0], small ? page[1] : page[0]};
        const bool there[2] = {true, parts == 2 || !small}, ok[2] = {valid(P, number[0]), there[1] && valid(P, number[1])};
        float *sc = reinterpret_cast<float *>(scales);
        // (what is written without a copy comes before the arrival, which releases it)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (!ok[h]) sc[2 * h] = there[h] ? NAN : 0.0f, sc[2 * h + 1] = 0.0f;
        sm100::mbar_arrive_expect_tx(bar, small && parts == 1 ? Ring::BYTES / 2 : Ring::BYTES);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (h < parts) {
#pragma unroll
                for (int i = 0; i < Ring::BOXES; ++i) {
                    ac_copy(stage + i * Ring::BOX + h * 16 * Ring::W, tmK, bar, i * 128, row, ok[h] ? number[h] : 0);
                    ac_copy(stage + (Ring::BOXES + i) * Ring::BOX + h * 16 * Ring::W, tmV, bar, i * 128, row, ok[h] ? number[h] : 0);
                }
            }
            if (ok[h]) {
                const int64_t block = (int64_t)number[h] * P.c.n_kv + it.h;
                ac_copy4(sc + 2 * h, P.c.k_scale + block);
                ac_copy4(sc + 2 * h + 1, P.c.v_scale + block);
            }
        }
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(bar)) : "memory");
        if (--left == 0) return;
        if (++at == it.units) {
            const int64_t b = it.b;
            ac_next(P, it);
            at = 0;
            if (it.b != b) start(P);
        }
        look(P);
    }
};

template <int DP, int MT, int NW, int NS>
__global__ void __launch_bounds__(NW * 64, 1)
    ac_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, AcParams P) {
    using Ring = AcRing<DP>;
    extern __shared__ __align__(1024) uint8_t rings[];
    // the warps' rings, then a part each.  A warp shares at most its first and its last item with others: what it has of
    // the first goes to that part, what it has of the last into its ring, which is idle by then.
    __shared__ int64_t owner[NW][2];  // the item (its first unit on the line) of each, or -1
    __shared__ AcItem items[NW][2];
    __shared__ float4 scales[NW][NS];
    __shared__ uint64_t full[NW][NS], empty[NW][NS];
    __shared__ int aborted;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = P.c.D;
    constexpr int size = kAcPart<DP, MT>;
    uint8_t *ring = rings + warp * NS * Ring::BYTES;
    auto part = [&](int s) {
        return reinterpret_cast<float *>(rings + (s & 1 ? (s >> 1) * NS * Ring::BYTES : NW * NS * Ring::BYTES + (s >> 1) * size * 4));
    };
    static_assert(kAcPart<DP, MT> * 4 <= NS * Ring::BYTES, "a part fits a ring");
    __shared__ AcLine<NW * 64> line;
    if (warp < NW) {
        if (lane < NS) sm100::mbar_init(&full[warp][lane], 2), sm100::mbar_init(&empty[warp][lane], 1);
        if (lane < 2) owner[warp][lane] = -1;
    } else if (tid == NW * 32) {
        aborted = 0;
        sm100::prefetch_tmap(&tmK);
        sm100::prefetch_tmap(&tmV);
    }
    sm100::fence_mbar_init();
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    if (blockIdx.x == 0 && tid == 0) *P.err = 0ull;  // (an error is counted two seconds later at the earliest)
    const AcTotal total = ac_line(P, line, NW);
    // rows of sequences without tokens
    for (int64_t b = blockIdx.x; b < P.c.B; b += gridDim.x)
        if (P.c.lens[b] <= 0)
            for (int i = tid; i < P.n_new * P.n_q * D; i += NW * 64) {
                const int t = i / (P.n_q * D);
                ac_store(P.y, P.yt, (b * P.n_new + t) * P.ldy + i - t * (P.n_q * D), 0.0f);
            }
    if ((int)blockIdx.x >= total.blocks || !total.units) return;
    const AcShares shares(total.places, total.blocks);
    const int64_t first_place = shares(blockIdx.x), last_place = shares(blockIdx.x + 1);
    const AcShares mine(last_place - first_place, NW);
    const int mate = warp % NW;  // the first warps work on what the others bring
    // where the warp's units begin (lane 0) and end, and the block's: a lane each
    AcItem it;
    int at = 0;
    int64_t unit = total.units;
    {
        const int64_t place = lane & 2 ? (lane & 1 ? last_place : first_place) : first_place + mine(mate + (lane & 1));
        if (place < total.places) {
            unit = ac_find(P, line, total.start, place, it, at);
            at = max(at - total.start, 0);
            unit += at;
        }
    }
    const int64_t u1 = __shfl_sync(~0u, unit, 1);
    if (warp >= NW) {
        // ------------------------------------------------------------ one lane brings the units of one of the first warps
        // (one warp for all, its lanes in turns, could not keep up, nor could two lanes a warp)
        if (NW == 8) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (lane == 0) {
            AcFetch<DP> f{it, at, u1 - unit};
            if (f.left > 0) f.start(P), f.look(P);
            int stage = 0;
            uint32_t phase = 1;
            while (f.left > 0 && !P.idle) {
                bool free = sm100::mbar_test_wait(&empty[mate][stage], phase);
                if (!free) {  // (bounded: whoever waits too long tells the others)
                    const uint64_t since = sm100::globaltimer_ns();
                    for (int i = 0; !free; ++i) {
                        free = sm100::mbar_test_wait(&empty[mate][stage], phase);
                        if (!free && (i & 255) == 255 && (*(volatile int *)&aborted || sm100::globaltimer_ns() - since > P.wait_ns)) break;
                    }
                }
                if (!free) {
                    *(volatile int *)&aborted = 1;
                    break;
                }
                f.send(P, &tmK, &tmV, rings + (mate * NS + stage) * Ring::BYTES, &scales[mate][stage], &full[mate][stage]);
                if (++stage == NS) stage = 0, phase ^= 1;
            }
        }
        __syncwarp();
    } else {
        if (NW == 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int64_t u0 = __shfl_sync(~0u, unit, 0), first = __shfl_sync(~0u, unit, 2), last = __shfl_sync(~0u, unit, 3);
        it.b = __shfl_sync(~0u, it.b, 0);
        it.h = __shfl_sync(~0u, it.h, 0);
        it.tile = __shfl_sync(~0u, it.tile, 0);
        it.units = __shfl_sync(~0u, it.units, 0);
        at = __shfl_sync(~0u, at, 0);
        AcWarp<DP, MT> w;
        int stage = 0;
        uint32_t phase = 0;
        for (int64_t u = u0; u < u1;) {
            const int n = (int)min((int64_t)(it.units - at), u1 - u);
            const int64_t start = u - at;  // the item's first unit on the line
            w.begin(P, it);
            for (int i = 0; i < n; ++i) {
                // (a wait that runs out spoils the result, which the device flag tells)
                if (!sm100::mbar_wait(&full[warp][stage], phase, &aborted, P.wait_ns)) aborted = 1;
                w.unit(sm100::smem_u32(ring + stage * Ring::BYTES), scales[warp][stage], (at + i) * kAcUnit, P.scale);
                __syncwarp();
                if (lane == 0) sm100::mbar_arrive(&empty[warp][stage]);
                if (++stage == NS) stage = 0, phase ^= 1;
            }
            const bool all = at == 0 && n == it.units;
            w.end(all);
            if (all) {
                w.runs(D, [&](int r, int d0, const auto &v) { ac_write_run(P, it, MT, (lane >> 2) + 8 * r, d0, v); });
            } else {
                const int slot = u == u0 ? 0 : 1;
                __syncwarp();
                w.put(part(warp * 2 + slot));
                if (lane == 0) owner[warp][slot] = start, items[warp][slot] = it;
            }
            u += n;
            at = 0;
            if (u < u1) ac_next(P, it);
        }
        // the first warps meet: what they share is in place
        asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
        if (aborted) {
            // copies may be under way still: far more time than they need
            const uint64_t t0 = sm100::globaltimer_ns();
            while (sm100::globaltimer_ns() - t0 < 10000000ull) {}
            if (tid == 0) atomicAdd(P.err, 1ull);
        }
        // Items that several warps share, in the order of the line.  A lane goes over the parts for what it holds of its rows;
        // every two pieces of 16 bytes of it are a job, and the warps take jobs in turn.
        const int64_t mine_of = lane < 2 * NW ? owner[lane >> 1][lane & 1] : -1;
        constexpr int N = DP / 16, JOBS = N / 2 * (MT / 8);  // a lane's pieces in a row, an item's jobs
        int job = -warp;
        for (unsigned left = __ballot_sync(~0u, mine_of >= 0); left;) {
            const int lead = __ffs(left) - 1;
            const int64_t start = __shfl_sync(~0u, mine_of, lead);
            const unsigned group = __ballot_sync(~0u, mine_of == start);
            left &= ~group;
            const AcItem item = items[lead >> 1][lead & 1];
            const bool whole = start >= first && start + item.units <= last;
            float *out = P.parts + ((int64_t)blockIdx.x * 2 + (start < first ? 0 : 1)) * size;
#pragma unroll 1
            for (int n = 0; n < JOBS; ++n, ++job) {
                if (job % NW) continue;
                const int row = (lane >> 2) + n / (N / 2) * 8;
                float pm[2 * NW], m = kAcNone, l = 0.0f;
#pragma unroll
                for (int s = 0; s < 2 * NW; ++s) pm[s] = group >> s & 1 ? part(s)[row] : kAcNone;
#pragma unroll
                for (int s = 0; s < 2 * NW; ++s) m = fmaxf(m, pm[s]);
                float4 o[2] = {};
#pragma unroll
                for (int s = 0; s < 2 * NW; ++s) {
                    pm[s] = group >> s & 1 ? part(s)[MT + row] * ac_exp2(pm[s] - m) : 0.0f;
                    l += pm[s];
                }
                const float inv = ac_inverse(l, whole);
#pragma unroll
                for (int s = 0; s < 2 * NW; ++s)
                    if (group >> s & 1) {
                        const float f = pm[s] * inv;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float4 v = reinterpret_cast<const float4 *>(part(s) + 2 * MT)[(2 * n + k) * 32 + lane];
                            o[k].x += v.x * f;
                            o[k].y += v.y * f;
                            o[k].z += v.z * f;
                            o[k].w += v.w * f;
                        }
                    }
                if (!whole && n % (N / 2) == 0 && (lane & 3) == 0) out[row] = m, out[MT + row] = l;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int x = (2 * n + k) * 32 + lane;
                    int at_row, d;
                    ac_place<DP>(x, at_row, d);
                    if (!whole) reinterpret_cast<float4 *>(out + 2 * MT)[x] = o[k];
                    else if (d < D) ac_write4(P, item, MT, row, d, o[k]);
                }
            }
        }
    }
}

// Items that thread blocks share.  Block c takes the item that the c-th border between shares cuts, if no earlier
// border does: its parts are those of the shares that it reaches into, in their order.  Which those are follows from
// the lengths alone, which were there before the first kernel: it is found out while that one still runs.
template <int DP, int MT>
__global__ void __launch_bounds__(256) ac_join_kernel(AcParams P) {
    __shared__ AcLine<256> line;
    __shared__ float weight[kAcMaxBlocks][MT];
    const int c = blockIdx.x + 1, D = P.c.D;
    constexpr int size = kAcPart<DP, MT>;
    const AcTotal total = ac_line(P, line, P.warps);
    bool cut = c < total.blocks;
    const AcShares shares(total.places, total.blocks);
    AcItem it;
    int parts = 0;
    if (cut) {
        const int64_t border = shares(c);
        int in;
        ac_find(P, line, total.start, border, it, in);
        const int64_t begin = border - in + total.start, end = begin + it.units;  // of its units
        cut = border > begin && shares(c - 1) <= begin;  // (else the border cuts nothing, or an earlier one cuts the item)
        // the shares up to the one that the item ends in; none of them is empty
        for (parts = 2; c - 1 + parts < total.blocks && shares(c - 1 + parts) < end;) ++parts;
    }
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    if (!cut) return;
    auto part = [&](int s) { return P.parts + ((int64_t)(c - 1 + s) * 2 + (s == 0 ? 1 : 0)) * size; };
    // the first parts' sums are on their way while the weights are found
    constexpr int AHEAD = 8, PER = (MT * DP / 4 + 255) / 256;
    float4 ahead[AHEAD];
#pragma unroll
    for (int s = 0; s < AHEAD; ++s)
        if (s < parts) ahead[s] = __ldcg(reinterpret_cast<const float4 *>(part(s) + 2 * MT) + threadIdx.x % (MT * DP / 4));
    const int lane = threadIdx.x & 31;
    for (int row = threadIdx.x >> 5; row < MT; row += 8) {
        float top = kAcNone, l = 0.0f;
        for (int s = lane; s < parts; s += 32) top = fmaxf(top, weight[s][row] = part(s)[row]);
#pragma unroll
        for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
        for (int s = lane; s < parts; s += 32) {
            const float f = part(s)[MT + row] * ac_exp2(weight[s][row] - top);
            weight[s][row] = f;
            l += f;
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(~0u, l, x);
        const float inv = ac_inverse(l, true);
        for (int s = lane; s < parts; s += 32) weight[s][row] *= inv;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int x = threadIdx.x + k * 256;
        if (x >= MT * DP / 4) break;
        int row, d;
        ac_place<DP>(x, row, d);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        auto add = [&](float4 v, int s) {
            const float f = weight[s][row];
            o.x += v.x * f;
            o.y += v.y * f;
            o.z += v.z * f;
            o.w += v.w * f;
        };
#pragma unroll
        for (int s = 0; s < AHEAD; ++s)
            if (s < parts) add(k == 0 ? ahead[s] : __ldcg(reinterpret_cast<const float4 *>(part(s) + 2 * MT) + x), s);
#pragma unroll 4
        for (int s = AHEAD; s < parts; ++s) add(__ldcg(reinterpret_cast<const float4 *>(part(s) + 2 * MT) + x), s);
        if (d < D) ac_write4(P, it, MT, row, d, o);
    }
}

// ---------------------------------------------------------------- host
static int ac_width(int64_t D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
// Tiles of 16 rows fetch a unit half as often for the same instructions, but double what a warp begins, keeps and hands
// over; with heads of 256 that does not fit the registers.
static bool ac_may_be_wide(int64_t rows, int64_t D) { return rows > 8 && D <= 128; }
// They are taken where the tables have room for kAcWideFrom units a warp and more (the lengths are known on the device only; both
// kinds in one kernel, chosen there, cost the short calls 2.5 us).  24 rows of 128: 5 sequences of up to 5001 tokens 20.4 us
// with 16 rows, 15.5 with 8; 16 of up to 7500 (six units a warp) 23.1 and 22.3, of up to 20001 32.5 and 35.2; 64 of up to 8192
// with 8 key heads 241 and 249, and with 12 rows of each 134 and 170.  Heads of 256: 38.0 and 21.6, 100.0 and 72.4.
constexpr int kAcWideFrom = 6;
static int ac_row_tile(const AcParams &P) {
    if (!ac_may_be_wide(P.rows, P.c.D)) return 8;
    const double units = (double)P.c.B * P.c.ldt * (1 << P.c.lp) / kAcUnit * P.c.n_kv * ((P.rows + 15) / 16);
    return units >= (double)kAcWideFrom * kAcMaxBlocks * 8 ? 16 : 8;
}
static size_t ac_workspace(int64_t rows, int64_t D) {
    return 256 + (size_t)kAcMaxBlocks * 2 * (ac_may_be_wide(rows, D) ? 16 : 8) * (ac_width(D) + 2) * 4;
}

static PFN_cuTensorMapEncodeTiled_v12000 ac_encoder() {
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

template <int DP, int MT>
static kq_status launch_ac(const char *fn, AcParams P, cudaStream_t st) {
    // 8 KB a unit of 128 elements, two a warp: more under way only makes everything queue longer (64 users of up to
    // 8192 tokens: three 106 us, two 102).  4 KB with 64 elements: three 60.6, two 64.0, four 60.9.
    constexpr int NW = DP == 256 ? 4 : 8, NS = DP == 64 ? 3 : 2;
    using Ring = AcRing<DP>;
    const int smem = NW * (NS * Ring::BYTES + kAcPart<DP, MT> * 4);
    static_assert(NW * (NS * Ring::BYTES + kAcPart<DP, MT> * 4) <= 216 * 1024, "shared memory");
    auto encode = ac_encoder();
    if (!encode) return fail(KQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled unavailable", fn);
    CUtensorMap tm[2];
    for (int i = 0; i < 2; ++i) {
        // a page's heads and tokens are the rows of one plane
        const int64_t D = P.c.D, rows = (int64_t)P.c.n_kv << P.c.lp;
        const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)P.c.n_pages};
        const cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)(D * rows)};
        const cuuint32_t box[3] = {Ring::W, (cuuint32_t)(P.c.lp == 4 ? 16 : kAcUnit), 1}, es[3] = {1, 1, 1};
        const CUresult e = encode(&tm[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, i ? P.c.v : P.c.k, dims, strides, box, es,
                                  CU_TENSOR_MAP_INTERLEAVE_NONE, DP == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (e != CUDA_SUCCESS) return fail(KQ_ERR_CUDA, "%s: tensor map of the cache failed (%d)", fn, (int)e);
    }
    auto kern = ac_kernel<DP, MT, NW, NS>;
    P.warps = NW;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_beside(kern, dim3(P.blocks), dim3(NW * 64), smem, dim3(1), st, tm[0], tm[1], P);
    if (e == cudaSuccess) count_launch(R_ATTN);
    if (e == cudaSuccess) {
        e = launch_beside(ac_join_kernel<DP, MT>, dim3(P.blocks - 1), dim3(256), 0, dim3(1), st, P);
        if (e == cudaSuccess) count_launch(R_ATTN);
    }
    return e == cudaSuccess ? KQ_OK : fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
}

static bool ac_shape(int64_t B, int64_t n_new, int64_t n_q, int64_t n_kv, int64_t D) {
    return B > 0 && B <= (1 << 24) && n_new > 0 && n_new <= 65536 && n_kv > 0 && n_kv <= kKvMaxHeads && n_q > 0 && n_q <= 65536 &&
           n_new * n_q <= 65536 && n_q % n_kv == 0 && D > 0 && D <= kKvMaxD && D % 16 == 0;
}

static kq_status ac_call(const char *fn, kq_dtype xt, const void *q, int64_t ldq, int64_t B, int64_t n_new, int64_t n_q, int64_t n_kv,
                         int64_t D, float scale, const int8_t *k_cache, const int8_t *v_cache, const float *k_scale, const float *v_scale,
                         int64_t n_pages, int64_t page, const int32_t *table, int64_t ldt, const int32_t *lens, kq_dtype yt, void *y,
                         int64_t ldy, void *workspace, size_t ws_bytes, kq_stream_t stream, unsigned long long wait_ns, bool idle) {
    if (!is_value_type(xt) || !is_value_type(yt))
        return fail(KQ_ERR_UNSUPPORTED_DTYPE, "%s: %s type %s is not F32, F16 or BF16", fn, is_value_type(xt) ? "output" : "query",
                    dtype_name(is_value_type(xt) ? yt : xt));
    if (!q || !y) return fail(KQ_ERR_INVALID_ARG, "%s: null %s", fn, q ? "y" : "q");
    AcParams P{};
    kq_status s = kv_check(fn, k_cache, v_cache, k_scale, v_scale, n_pages, page, table, ldt, lens, B, n_kv, D, P.c);
    if (s != KQ_OK) return s;
    if (!ac_shape(B, n_new, n_q, n_kv, D))
        return fail(KQ_ERR_INVALID_ARG, "%s: need n_new > 0, n_q a multiple of n_kv and n_new*n_q up to 65536 (n_new=%lld n_q=%lld n_kv=%lld)",
                    fn, (long long)n_new, (long long)n_q, (long long)n_kv);
    if (ldq < n_q * D || ldy < n_q * D)
        return fail(KQ_ERR_INVALID_ARG, "%s: ldq=%lld or ldy=%lld is less than n_q*D", fn, (long long)ldq, (long long)ldy);
    if (!(fabsf(scale) <= 2.0e38f)) return fail(KQ_ERR_INVALID_ARG, "%s: scale must be finite, up to 2e38", fn);  // (times log2 e, too)
    if (!aligned(q, value_bytes(xt)) || !aligned(y, value_bytes(yt)))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    const size_t need = ac_workspace(n_new * (n_q / n_kv), D);
    if (!workspace || ws_bytes < need)
        return fail(KQ_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, workspace ? ws_bytes : (size_t)0, need);
    if (!aligned(workspace, 256)) return fail(KQ_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    P.q = q; P.y = y; P.ldq = ldq; P.ldy = ldy; P.xt = xt; P.yt = yt;
    P.qvec = aligned(q, 4 * value_bytes(xt)) && ldq % 4 == 0;
    P.yvec = aligned(y, 16) && ldy * (int64_t)value_bytes(yt) % 16 == 0;
    P.n_new = (int)n_new; P.n_q = (int)n_q; P.G = (int)(n_q / n_kv);
    P.rows = P.n_new * P.G;
    const int mt = ac_row_tile(P);
    P.tiles = (P.rows + mt - 1) / mt;
    P.scale = scale * 1.44269504f;
    P.err = static_cast<unsigned long long *>(workspace);
    P.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + 256);
    P.blocks = kAcMaxBlocks;
    P.wait_ns = wait_ns;
    P.idle = idle;
    const cudaStream_t st = (cudaStream_t)stream;
    if (D > 128) return launch_ac<256, 8>(fn, P, st);
    if (mt == 8) return D <= 64 ? launch_ac<64, 8>(fn, P, st) : launch_ac<128, 8>(fn, P, st);
    return D <= 64 ? launch_ac<64, 16>(fn, P, st) : launch_ac<128, 16>(fn, P, st);
}

}  // namespace kq

using namespace kq;

extern "C" {

size_t kq_attn_cache_i8_workspace_bytes(int64_t B, int64_t n_new, int64_t n_q, int64_t n_kv, int64_t D) {
    return ac_shape(B, n_new, n_q, n_kv, D) ? ac_workspace(n_new * (n_q / n_kv), D) : 0;
}

kq_status kq_attn_cache_i8(kq_dtype xt, const void *q, int64_t ldq, int64_t B, int64_t n_new, int64_t n_q, int64_t n_kv, int64_t D,
                           float scale, const int8_t *k_cache, const int8_t *v_cache, const float *k_scale, const float *v_scale,
                           int64_t n_pages, int64_t page, const int32_t *table, int64_t ldt, const int32_t *lens, kq_dtype yt, void *y,
                           int64_t ldy, void *workspace, size_t ws_bytes, kq_stream_t stream) {
    return ac_call("kq_attn_cache_i8", xt, q, ldq, B, n_new, n_q, n_kv, D, scale, k_cache, v_cache, k_scale, v_scale, n_pages, page, table,
                   ldt, lens, yt, y, ldy, workspace, ws_bytes, stream, kAcWaitNs, false);
}

kq_status kq_debug_attn_cache_wait_timeout(kq_dtype xt, const void *q, int64_t ldq, int64_t B, int64_t n_new, int64_t n_q, int64_t n_kv,
                                           int64_t D, float scale, const int8_t *k_cache, const int8_t *v_cache, const float *k_scale,
                                           const float *v_scale, int64_t n_pages, int64_t page, const int32_t *table, int64_t ldt,
                                           const int32_t *lens, kq_dtype yt, void *y, int64_t ldy, int64_t wait_limit_ns, void *workspace,
                                           size_t ws_bytes, kq_stream_t stream) {
    const char *fn = "kq_debug_attn_cache_wait_timeout";
    if (wait_limit_ns < 1000 || wait_limit_ns > 1000000000)
        return fail(KQ_ERR_INVALID_ARG, "%s: wait_limit_ns must be in [1e3, 1e9]", fn);
    return ac_call(fn, xt, q, ldq, B, n_new, n_q, n_kv, D, scale, k_cache, v_cache, k_scale, v_scale, n_pages, page, table, ldt, lens, yt, y,
                   ldy, workspace, ws_bytes, stream, (unsigned long long)wait_limit_ns, true);
}

}  // extern "C"
