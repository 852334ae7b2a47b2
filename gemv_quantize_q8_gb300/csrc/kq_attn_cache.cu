// kq_attn_cache.cu -- attention of a few query tokens over the paged 8-bit cache.
//
// For a query row q (one token and head) over the tokens j that it sees, with s_j = scale * ks * (q . K_j) for codes
// K, V and their blocks' scales ks, vs:
//   m = max s_j,  l = sum 2^(s_j - m),  y = (sum 2^(s_j - m) vs V_j) / l       (s in units of log 2)
// Bound by the cache's bytes: each is read once, by the warp that needs it, straight into the registers that
// feed its matrix instructions; nothing is staged.
//
// The products run on m16n8k16 instructions.  Codes are exact in f16; a query row is brought to |q| < 2 by a power
// of two and split into two f16 (22 bits), as the weights 2^(s - m) vs are.  With up to eight rows (the query heads of
// one key head) the second parts fill the tile's other eight rows, so they cost nothing; 9 to 16 rows take twice
// the instructions.  Which of its elements a lane holds is free where both operands agree, so it follows the loads:
//   keys:   lane 4n + c of an eight-token tile loads 16-byte pieces c, c + 4, .. of token n; 4 bytes make the two
//           registers of one step.
//   values: lane 4n + c loads 16 bytes at n * 16 of tokens 2c, 2c + 1, 2c + 8, 2c + 9: the tokens whose weights it
//           holds, the bytes of two tokens paired by permutes.
// A unit is 16 tokens (a page holds whole units).  All units of all sequences and heads form one line, cut into equal shares, one a
// warp: lengths may differ as they like.  A row whose units are shared by warps is put together in shared memory,
// one that is shared by thread blocks through the workspace and a second kernel, in a fixed order.
#include <algorithm>
#include <math.h>

#include "kq_i8_tc.cuh"
#include "kq_kv.cuh"
#include "kq_launch.cuh"

namespace kq {

constexpr int kAcUnit = 16;           // tokens
constexpr float kAcLift = 128.0f;     // weights are held times this: f16 keeps their low bits, with room for kAcSlack
constexpr float kAcSlack = 8.0f;      // a weight may grow to 2^8 before the sums are brought to a new maximum
constexpr float kAcNone = -3.0e38f;   // the maximum of no token

struct AcParams {
    KvCache c;
    const void *q;
    void *y;
    int64_t ldq, ldy;
    kq_dtype xt, yt;
    bool qvec;            // query rows on boundaries of four elements
    int n_new, n_q, G;    // query tokens of a sequence, query heads, and those of a key head
    int rows, tiles;      // rows of a key head (n_new * G), and the row tiles that they take
    float scale;          // times log2 e
    float *parts;         // [blocks][2] partial results
    int blocks;           // of the first kernel's grid
};

// What a warp (or a block) hands over: rows of m, l and D sums, relative to 2^m.
template <int MT> __host__ __device__ constexpr int ac_part_floats(int D) { return MT * (D + 2); }

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

// All threads of the block: the units of all sequences together (times heads and row tiles).
template <int THREADS>
__device__ __forceinline__ int64_t ac_total(const AcParams &P, int64_t *red) {
    int64_t n = 0;
    for (int64_t b = threadIdx.x; b < P.c.B; b += THREADS) n += ac_units(P, b);
#pragma unroll
    for (int s = 16; s; s >>= 1) n += __shfl_xor_sync(~0u, n, s);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) n += red[i];
    return n * P.c.n_kv * P.tiles;
}
// The share that worker w of n begins with.  (n is at most a few thousand, the line below 2^50.)
__device__ __forceinline__ int64_t ac_share(int64_t total, int w, int n) { return total / n * w + total % n * w / n; }

// The warp finds the item that unit u lies in, and its place in it.
__device__ __forceinline__ AcItem ac_find(const AcParams &P, int64_t u, int &at) {
    const int lane = threadIdx.x & 31;
    const int64_t per = (int64_t)P.c.n_kv * P.tiles;
    AcItem it;
    for (int64_t b0 = 0;; b0 += 32) {
        const int64_t b = b0 + lane;
        const int64_t mine = b < P.c.B ? ac_units(P, b) * per : 0;
        int64_t sum = mine;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int64_t o = __shfl_up_sync(~0u, sum, s);
            if (lane >= s) sum += o;
        }
        const unsigned past = __ballot_sync(~0u, sum > u);
        if (past || b0 + 32 >= P.c.B) {
            const int l = past ? __ffs(past) - 1 : 31;
            const int64_t rest = u - __shfl_sync(~0u, sum - mine, l);
            it.b = b0 + l;
            it.units = (int)(__shfl_sync(~0u, mine, l) / per);
            const int64_t i = rest / it.units;
            at = (int)(rest - i * it.units);
            it.h = (int)(i / P.tiles);
            it.tile = (int)(i - it.h * P.tiles);
            return it;
        }
        u -= __shfl_sync(~0u, sum, 31);
    }
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

__device__ __forceinline__ float ac_load(const void *p, kq_dtype t, int64_t i) {
    return t == KQ_F32 ? static_cast<const float *>(p)[i] : t == KQ_F16 ? __half2float(static_cast<const __half *>(p)[i])
                                                                        : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void ac_load4(const void *p, kq_dtype t, int64_t i, bool vec, float (&v)[4]) {
    if (!vec) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = ac_load(p, t, i + j);
    } else if (t == KQ_F32) {
        const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint16_t e = (uint16_t)((j < 2 ? u.x : u.y) >> (16 * (j & 1)));
            v[j] = t == KQ_F16 ? __half2float(__ushort_as_half(e)) : __uint_as_float((uint32_t)e << 16);
        }
    }
}
__device__ __forceinline__ void ac_store(void *p, kq_dtype t, int64_t i, float v) {
    if (t == KQ_F32) static_cast<float *>(p)[i] = v;
    else if (t == KQ_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void ac_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
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
    float m[R], l[R], factor[R];
    int limit[R];                        // tokens that a row sees
    float vref;                          // a power of two above the value scales so far

    __device__ __forceinline__ void begin(const AcParams &P, const AcItem &it) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
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
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int d = (s / 4) * 64 + c * 16 + (s % 4) * 4;
                v[s][0] = v[s][1] = v[s][2] = v[s][3] = 0.0f;
                if (live && d < P.c.D) ac_load4(P.q, P.xt, at + d, P.qvec, v[s]);
#pragma unroll
                for (int i = 0; i < 4; ++i) amax = fmaxf(amax, fabsf(v[s][i]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            // the power of two at or below the largest (1 for rows of zeros and of infinities)
            uint32_t e = __float_as_uint(amax) & 0x7f800000u;
            if (e == 0x7f800000u || e == 0u) e = 0x3f800000u;
            if (e > 0x7e800000u) e = 0x7e800000u;
            const float down = __uint_as_float(0x7f000000u - e);
            factor[r] = P.scale * __uint_as_float(e);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                ac_split(v[s][0] * down, v[s][1] * down, qh[s][r * 2], ql[s][r * 2]);
                ac_split(v[s][2] * down, v[s][3] * down, qh[s][r * 2 + 1], ql[s][r * 2 + 1]);
            }
            m[r] = kAcNone;
            l[r] = 0.0f;
        }
        vref = 0.0f;
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
    }

    __device__ __forceinline__ void load(const int8_t *kb, const int8_t *vb, int D, uint4 (&k)[2][KP], uint32_t (&v)[4][VW]) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const int d = i * 64 + c * 16;
                k[t][i] = make_uint4(0, 0, 0, 0);
                if (d < D) k[t][i] = __ldg(reinterpret_cast<const uint4 *>(kb + (t * 8 + g) * D + d));
            }
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int8_t *p = vb + (2 * c + (t & 1) + (t >> 1) * 8) * D;
            if constexpr (DP == 64) {
                uint2 u = make_uint2(0, 0);
                if (g * 8 < D) u = __ldg(reinterpret_cast<const uint2 *>(p + g * 8));
                v[t][0] = u.x; v[t][1] = u.y;
            } else {
#pragma unroll
                for (int i = 0; i < VW / 4; ++i) {
                    const int d = i * 128 + g * 16;
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (d < D) u = __ldg(reinterpret_cast<const uint4 *>(p + d));
                    v[t][4 * i] = u.x; v[t][4 * i + 1] = u.y; v[t][4 * i + 2] = u.z; v[t][4 * i + 3] = u.w;
                }
            }
        }
    }

    // A unit: tokens t0 .. t0 + 15, of which a row sees those below its limit.
    __device__ __forceinline__ void unit(const uint4 (&k)[2][KP], const uint32_t (&v)[4][VW], float ks, float vs, int t0) {
        const int c = threadIdx.x & 3;
        float s[2][4] = {};
#pragma unroll
        for (int i = 0; i < KP; ++i)
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t b0, b1;
                    const uint4 q = k[t][i];
                    i8x4_to_f16(w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w, b0, b1);
                    const int st = i * 4 + w;
                    if constexpr (MT == 8) {
                        ac_mma(s[t], qh[st][0], ql[st][0], qh[st][1], ql[st][1], b0, b1);
                    } else {
                        ac_mma(s[t], qh[st][0], qh[st][2], qh[st][1], qh[st][3], b0, b1);
                        ac_mma(s[t], ql[st][0], ql[st][2], ql[st][1], ql[st][3], b0, b1);
                    }
                }
        // x[r][0..3]: a row's logits for tokens 2c, 2c + 1, 2c + 8, 2c + 9
        float x[R][4];
        bool grows = false;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float raw = MT == 8 ? s[i >> 1][i & 1] + s[i >> 1][2 + (i & 1)] : s[i >> 1][2 * r + (i & 1)];
                const int token = t0 + 2 * c + (i & 1) + (i >> 1) * 8;
                x[r][i] = token < limit[r] ? raw * (factor[r] * ks) : -INFINITY;
                grows |= x[r][i] > m[r] + kAcSlack;
            }
        const bool wider = vs > vref && vs < INFINITY;
        if (__any_sync(~0u, grows || wider)) {
            // bring the sums to a new maximum and a new reference of the value scales
            float ref = vref;
            if (wider) {
                const uint32_t e = __float_as_uint(vs) & 0x7f800000u;
                ref = e < 0x00800000u ? 2.3509887e-38f : e >= 0x7f000000u ? vs : __uint_as_float(e + 0x00800000u);
            }
            const float fv = vref > 0.0f ? vref / ref : 0.0f;
            vref = ref;
            float f[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float top = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                top = fmaxf(top, m[r]);
                f[r] = exp2f(m[r] - top);
                l[r] *= f[r];
                m[r] = top;
                f[r] *= fv;
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o[j][0] *= f[0];
                o[j][1] *= f[0];
                o[j][2] *= f[R - 1];
                o[j][3] *= f[R - 1];
            }
        }
        float lift = vref > 0.0f ? vs / vref * kAcLift : 0.0f * vs;
        const bool poison = !(lift <= kAcLift);  // a block with an infinity: NaN for the rows that see it, for them alone
        if (poison) lift = 0.0f;
        uint32_t ph[R][2], pl[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[i] = exp2f(x[r][i] - m[r]);
                l[r] += poison && x[r][i] > -INFINITY ? NAN : p[i];
            }
            ac_split(p[0] * lift, p[1] * lift, ph[r][0], pl[r][0]);
            ac_split(p[2] * lift, p[3] * lift, ph[r][1], pl[r][1]);
        }
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            uint32_t a[4], b[4];
            ac_pair(v[0][w], v[1][w], a);
            ac_pair(v[2][w], v[3][w], b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (MT == 8) {
                    ac_mma(o[4 * w + i], ph[0][0], pl[0][0], ph[0][1], pl[0][1], a[i], b[i]);
                } else {
                    ac_mma(o[4 * w + i], ph[0][0], ph[1][0], ph[0][1], ph[1][1], a[i], b[i]);
                    ac_mma(o[4 * w + i], pl[0][0], pl[1][0], pl[0][1], pl[1][1], a[i], b[i]);
                }
            }
        }
    }

    // The item's sums so far: m, l, and D values a row that stand relative to 2^m.
    __device__ __forceinline__ void end() {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            l[r] += __shfl_xor_sync(~0u, l[r], 1);
            l[r] += __shfl_xor_sync(~0u, l[r], 2);
        }
        const float back = vref / kAcLift;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (MT == 8) {
                o[j][0] += o[j][2];
                o[j][1] += o[j][3];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[j][i] = o[j][i] * back;
        }
    }
    __device__ __forceinline__ void put(float *part, int D) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = g + 8 * r;
            if (c == 0) part[row] = m[r], part[MT + row] = l[r];
            float *dst = part + 2 * MT + row * D;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int d = ac_element<DP>(j, 2 * c + e);
                    if (d < D) dst[d] = o[j][2 * r + e];
                }
        }
    }
};

// Row `row` (of the item's tile) of the output, element d; a token that sees nothing gives 0.
__device__ __forceinline__ void ac_write(const AcParams &P, const AcItem &it, int MT, int row, int d, float o, float l) {
    const int i = it.tile * MT + row;
    if (i >= P.rows) return;
    const int token = i / P.G, head = it.h * P.G + i - token * P.G;
    const bool sees = ac_len(P, it.b) - P.n_new + token >= 0;
    ac_store(P.y, P.yt, (it.b * P.n_new + token) * P.ldy + (int64_t)head * P.c.D + d, sees ? o / l : 0.0f);
}

template <int DP, int MT, int NW>
__global__ void __launch_bounds__(NW * 32, 1) ac_kernel(AcParams P) {
    extern __shared__ float parts[];  // [NW][2] parts of items that warps share
    __shared__ int64_t red[NW];
    __shared__ int64_t owner[NW][2];  // the item (its first unit on the line) of each, or -1
    __shared__ AcItem items[NW][2];
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = P.c.D;
    const int size = ac_part_floats<MT>(D);
    const int64_t total = ac_total<NW * 32>(P, red);
    if (lane < 2) owner[warp][lane] = -1;
    // rows of sequences without tokens
    for (int64_t b = blockIdx.x; b < P.c.B; b += gridDim.x)
        if (P.c.lens[b] <= 0)
            for (int i = tid; i < P.n_new * P.n_q * D; i += NW * 32) {
                const int t = i / (P.n_q * D);
                ac_store(P.y, P.yt, (b * P.n_new + t) * P.ldy + i - t * (P.n_q * D), 0.0f);
            }
    const int64_t first = ac_share(total, blockIdx.x, P.blocks), last = ac_share(total, blockIdx.x + 1, P.blocks);
    if (first >= last) return;
    const int64_t u0 = first + ac_share(last - first, warp, NW), u1 = first + ac_share(last - first, warp + 1, NW);
    if (u0 < u1) {
        int at;
        AcItem it = ac_find(P, u0, at);
        AcWarp<DP, MT> w;
        uint4 k[2][AcWarp<DP, MT>::KP];
        uint32_t v[4][AcWarp<DP, MT>::VW];
        for (int64_t u = u0; u < u1;) {
            const int n = (int)min((int64_t)(it.units - at), u1 - u);
            const int64_t start = u - at;  // the item's first unit on the line
            w.begin(P, it);
            const bool bad = ac_bad(P, it.b);
            const int32_t *table = P.c.table + it.b * P.c.ldt;
            for (int i = 0; i < n; ++i) {
                const int t0 = (at + i) * kAcUnit;
                int64_t page = table[t0 >> P.c.lp];
                const bool ok = page >= 0 && page < P.c.n_pages && !bad;
                if (!ok) page = 0;
                const int64_t block = page * P.c.n_kv + it.h;
                const int64_t off = ((block << P.c.lp) + (t0 & ((1 << P.c.lp) - 1))) * D;
                w.load(P.c.k + off, P.c.v + off, D, k, v);
                const float ks = ok ? P.c.k_scale[block] : NAN, vs = P.c.v_scale[block];
                w.unit(k, v, ks, vs, t0);
            }
            w.end();
            if (at == 0 && n == it.units) {
                const int g = lane >> 2, c = lane & 3;
#pragma unroll
                for (int r = 0; r < MT / 8; ++r)
#pragma unroll
                    for (int j = 0; j < DP / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = ac_element<DP>(j, 2 * c + e);
                            if (d < D) ac_write(P, it, MT, g + 8 * r, d, w.o[j][2 * r + e], w.l[r]);
                        }
            } else {
                const int slot = u == u0 ? 0 : 1;
                w.put(parts + (warp * 2 + slot) * size, D);
                if (lane == 0) owner[warp][slot] = start, items[warp][slot] = it;
            }
            u += n;
            at = 0;
            if (u < u1) ac_next(P, it);
        }
    }
    __syncthreads();
    // items that several warps share, in the order of the line
    for (int i = 0; i < 2 * NW;) {
        const int64_t start = owner[i >> 1][i & 1];
        if (start < 0) { ++i; continue; }
        int j = i + 1;
        while (j < 2 * NW && (owner[j >> 1][j & 1] == start || owner[j >> 1][j & 1] < 0)) ++j;
        const AcItem it = items[i >> 1][i & 1];
        const bool whole = start >= first && start + it.units <= last;
        float *out = P.parts + ((int64_t)blockIdx.x * 2 + (start < first ? 0 : 1)) * size;
        for (int e = tid; e < MT * D; e += NW * 32) {
            const int row = e / D, d = e - row * D;
            float m = kAcNone, l = 0.0f, o = 0.0f;
            for (int s = i; s < j; ++s)
                if (owner[s >> 1][s & 1] >= 0) m = fmaxf(m, parts[s * size + row]);
            for (int s = i; s < j; ++s)
                if (owner[s >> 1][s & 1] >= 0) {
                    const float f = exp2f(parts[s * size + row] - m);
                    l += parts[s * size + MT + row] * f;
                    o += parts[s * size + 2 * MT + e] * f;
                }
            if (whole) {
                ac_write(P, it, MT, row, d, o, l);
            } else {
                out[2 * MT + e] = o;
                if (d == 0) out[row] = m, out[MT + row] = l;
            }
        }
        i = j;
    }
}

// Items that thread blocks share.  Block c takes the item that the c-th border between shares cuts, if no earlier
// border does: its parts are those of the shares that it reaches into, in their order.
template <int MT>
__global__ void __launch_bounds__(256) ac_join_kernel(AcParams P) {
    __shared__ int64_t red[8];
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int c = blockIdx.x + 1, D = P.c.D;
    const int size = ac_part_floats<MT>(D);
    const int64_t total = ac_total<256>(P, red);
    const int64_t border = ac_share(total, c, P.blocks), before = ac_share(total, c - 1, P.blocks);
    if (border >= total || border == 0 || before == border) return;
    int at;
    const AcItem it = ac_find(P, border, at);
    const int64_t start = border - at, end = start + it.units;
    if (at == 0 || before > start) return;  // the border cuts nothing, or an earlier one cuts the item
    // the shares up to the one that the item ends in (empty shares, between equal borders, have no part)
    int last = c;
    while (last + 1 < P.blocks && ac_share(total, last + 1, P.blocks) < end) ++last;
    for (int e = threadIdx.x; e < MT * D; e += 256) {
        const int row = e / D, d = e - row * D;
        float m = kAcNone, l = 0.0f, o = 0.0f;
        auto part = [&](int s) { return P.parts + ((int64_t)s * 2 + (s == c - 1 ? 1 : 0)) * size; };
        for (int s = c - 1; s <= last; ++s)
            if (ac_share(total, s, P.blocks) < ac_share(total, s + 1, P.blocks)) m = fmaxf(m, part(s)[row]);
        for (int s = c - 1; s <= last; ++s)
            if (ac_share(total, s, P.blocks) < ac_share(total, s + 1, P.blocks)) {
                const float f = exp2f(part(s)[row] - m);
                l += part(s)[MT + row] * f;
                o += part(s)[2 * MT + e] * f;
            }
        ac_write(P, it, MT, row, d, o, l);
    }
}

// ---------------------------------------------------------------- host
constexpr int kAcMaxBlocks = 152;
static int ac_row_tile(int64_t rows) { return rows <= 8 ? 8 : 16; }
static size_t ac_workspace(int64_t rows, int64_t D) {
    const int mt = ac_row_tile(rows);
    return (size_t)kAcMaxBlocks * 2 * mt * (D + 2) * 4;
}

template <int DP, int MT>
static kq_status launch_ac(const char *fn, const AcParams &P, cudaStream_t st) {
    constexpr int NW = DP * MT >= 4096 ? 4 : 8;  // a part is up to 16 KB, two a warp
    const int smem = NW * 2 * ac_part_floats<MT>(P.c.D) * 4;
    auto kern = ac_kernel<DP, MT, NW>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = launch_beside(kern, dim3(P.blocks), dim3(NW * 32), smem, dim3(1), st, P);
    if (e == cudaSuccess) count_launch(R_ATTN);
    if (e == cudaSuccess && P.blocks > 1) {
        e = launch_beside(ac_join_kernel<MT>, dim3(P.blocks - 1), dim3(256), 0, dim3(1), st, P);
        if (e == cudaSuccess) count_launch(R_ATTN);
    }
    return e == cudaSuccess ? KQ_OK : fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
}

static bool ac_shape(int64_t B, int64_t n_new, int64_t n_q, int64_t n_kv, int64_t D) {
    return B > 0 && B <= (1 << 24) && n_new > 0 && n_new <= 65536 && n_kv > 0 && n_kv <= kKvMaxHeads && n_q > 0 && n_q <= 65536 &&
           n_new * n_q <= 65536 && n_q % n_kv == 0 && D > 0 && D <= kKvMaxD && D % 16 == 0;
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
    const char *fn = "kq_attn_cache_i8";
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
    if (!(fabsf(scale) <= 3.0e38f)) return fail(KQ_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (!aligned(q, value_bytes(xt)) || !aligned(y, value_bytes(yt)))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    const size_t need = ac_workspace(n_new * (n_q / n_kv), D);
    if (!workspace || ws_bytes < need)
        return fail(KQ_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, workspace ? ws_bytes : (size_t)0, need);
    if (!aligned(workspace, 256)) return fail(KQ_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    P.q = q; P.y = y; P.ldq = ldq; P.ldy = ldy; P.xt = xt; P.yt = yt;
    P.qvec = aligned(q, 4 * value_bytes(xt)) && ldq % 4 == 0;
    P.n_new = (int)n_new; P.n_q = (int)n_q; P.G = (int)(n_q / n_kv);
    P.rows = P.n_new * P.G;
    const int mt = ac_row_tile(P.rows);
    P.tiles = (P.rows + mt - 1) / mt;
    P.scale = scale * 1.44269504f;
    P.parts = static_cast<float *>(workspace);
    P.blocks = kAcMaxBlocks;
    const cudaStream_t st = (cudaStream_t)stream;
    if (mt == 8) return D <= 64 ? launch_ac<64, 8>(fn, P, st) : D <= 128 ? launch_ac<128, 8>(fn, P, st) : launch_ac<256, 8>(fn, P, st);
    return D <= 64 ? launch_ac<64, 16>(fn, P, st) : D <= 128 ? launch_ac<128, 16>(fn, P, st) : launch_ac<256, 16>(fn, P, st);
}

}  // extern "C"
