// kq_kv.cu -- new keys (rotated on the way) and values into the paged 8-bit cache, and cached rows back.
//
// A block of the cache (a page and head) has one scale, so its largest magnitude has to be known before its
// first code is written, and when a later token raises it the codes that are there follow:
//   s' = max(s, max |x| / 127),   q' = rint(q * (s / s')) for the old tokens,   q = rint(x * (1 / s')) for the new.
// A group of threads (256, or a warp where the sequences have few rows) takes one block of the cache that the call
// touches and keeps its new rows in registers between the maximum and the codes: 8192 elements of 256 threads (64 tokens
// of 128), 1024 of a warp.  Those are read once; what a block has beyond them (pages of 128 tokens of 128) is read and
// rotated for the maximum and again for the codes.  Every code is written once.  Which blocks those are follows from cu and
// lens on the device: a run of n tokens touches at most floor(n / page) + 2 pages, and at most n; so sequence b's share of
// the grid starts at floor(cu[b] / page) + 2b, or at cu[b], whichever makes the smaller grid.
// 8192 tokens, 8 heads of 128, fp32: append 22 us (84 MB, 12.4 at the memory's rate), bound by a block's chain of waits (where
// it is, positions, rows, maximum); reading them back as bf16 11 us (one after the other 34).  One token each of 64 users: 8.9
// us both.
// The maximum, every product and sum are rounded one by one, so that codes and scales are the same bits whatever
// the grid or the vector width.
#include <type_traits>

#include "kq_kv.cuh"
#include "kq_launch.cuh"

namespace kq {

constexpr int kKvThreads = 256;
// threads of a block of the cache (8192 tokens, 8 heads of 128: 34.0 us with the read, 43 with 128 that hold twice as much)
constexpr int kKvGroup = 256;
constexpr int kKvHeld = 4;  // vector pairs of a thread that stay in registers: 64 tokens of 128

struct KvRows {
    void *k, *v;  // [T][ldk], [T][ldv]
    int64_t ldk, ldv;
    const int32_t *cu;  // [B + 1] or NULL
    int64_t T;
    bool by_row;        // sequence b's share of the grid starts at cu[b]
};
struct KvTurn {
    const int32_t *pos;
    const float *cos_tab, *sin_tab;
    int64_t n_pos;
    int rot;
};

__device__ __forceinline__ int64_t kv_start(const KvRows &r, const KvCache &c, int64_t row, int64_t b) {
    return r.by_row ? row : (row >> c.lp) + 2 * b;
}

// A thread block's part of the cache: tokens [lo, hi) of a page from row `row` on.
struct KvPart {
    int64_t page, row;
    int lo, hi;  // none: lo = hi
};
// All threads of the block call it; false where there is nothing to do.  (One thread finds it out for all: the block's
// instructions count.)
__device__ __forceinline__ KvPart kv_find(const KvCache &c, const KvRows &r, int64_t unit, int64_t b);
__device__ __forceinline__ bool kv_part(const KvCache &c, const KvRows &r, int64_t unit, KvPart &p) {
    __shared__ KvPart shared;
    // the last sequence whose share starts at or before the unit; shares start in rising order
    int64_t b = 0;
    for (int64_t n = c.B; b >= 0;) {  // it is one of n from b on
        const int64_t step = (n + kKvThreads - 1) / kKvThreads, at = threadIdx.x * step;
        const int k = __syncthreads_count(at < n && kv_start(r, c, kv_row(r.cu, b + at, c.B, r.T), b + at) <= unit) - 1;
        b = k < 0 ? -1 : b + k * step;
        if (step == 1) break;
        n = min(step, n - k * step);
    }
    if (threadIdx.x == 0) shared = kv_find(c, r, unit, b);
    __syncthreads();
    p = shared;
    return p.lo < p.hi;
}
__device__ __forceinline__ KvPart kv_find(const KvCache &c, const KvRows &r, int64_t unit, int64_t b) {
    KvPart p = {0, 0, 0, 0};
    if (b < 0) return p;
    const int64_t r0 = kv_row(r.cu, b, c.B, r.T), r1 = kv_row(r.cu, b + 1, c.B, r.T), len = c.lens[b], n = r1 - r0;
    const int64_t first = len - n, begin = first > 0 ? first : 0;  // positions of the rows; those before 0 have no place
    const int64_t i = (begin >> c.lp) + (unit - kv_start(r, c, r0, b));
    const int64_t lo = max(begin, i << c.lp), hi = min(len, (i + 1) << c.lp);
    if (n <= 0 || lo >= hi || i >= c.ldt) return p;
    p.page = c.table[b * c.ldt + i];
    if (p.page < 0 || p.page >= c.n_pages) return p;
    p.row = r0 + (lo - first);
    p.lo = (int)(lo - (i << c.lp));
    p.hi = (int)(hi - (i << c.lp));
    return p;
}
// The threads of a group meet.
template <int G>
__device__ __forceinline__ void kv_sync() {
    if (G > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / G), "n"(G) : "memory");
    else __syncwarp();
}

// W elements as fp32; the address is aligned to all of them.
template <int W, typename T>
__device__ __forceinline__ void kv_load(const T *p, float (&v)[W]) {
    if constexpr (W == 1) {
        v[0] = to_f32(*p);
    } else {
        using Vec = typename VecOf<W * (int)sizeof(T)>::type;
        const Vec u = __ldcs(reinterpret_cast<const Vec *>(p));
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = to_f32(reinterpret_cast<const T *>(&u)[i]);
    }
}

// A code (|x * inv| is at most 127 and a few units of rounding, or NaN, which gives 0).
__device__ __forceinline__ int kv_code(float x, float inv) {
    const float v = __fmul_rn(x, inv);
    return isnan(v) ? 0 : __float2int_rn(v);
}
// The same without NaN, in the lowest byte: 1.5 * 2^23 leaves the nearest even whole number in the last bits.  (Conversions
// go at a quarter of this rate.)
__device__ __forceinline__ uint32_t kv_byte(float x, float inv) { return __float_as_uint(__fadd_rn(__fmul_rn(x, inv), 12582912.0f)); }
__device__ __forceinline__ uint32_t kv_join(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ float kv_max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ uint32_t kv_pack(int a, int b, int c, int d) {
    return (a & 255) | (b & 255) << 8 | (c & 255) << 16 | (uint32_t)d << 24;
}

// Vector pair j of a row covers [lo, lo + W) and [hi, hi + W): first the rotated pairs (both partners in one
// thread), then the rest of the head.  W is 4, or 1 where rows or halves do not lie on four elements.
// G: threads of a group.
template <typename TX, bool PAIRS, int W, int G>
__global__ void __launch_bounds__(kKvThreads, 3) kv_append_kernel(KvCache c, KvRows r, KvTurn turn) {
    __shared__ float red[kKvThreads / 32];
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int tid = threadIdx.x % G, which_head = blockIdx.y * (kKvThreads / G) + threadIdx.x / G;
    KvPart p;
    if (!kv_part(c, r, blockIdx.x, p) || which_head >= 2 * c.n_kv) return;
    const int which = which_head >= c.n_kv, head = which_head - (which ? c.n_kv : 0);
    const int64_t block = p.page * c.n_kv + head;
    float *scale = (which ? c.v_scale : c.k_scale) + block;
    int8_t *codes = (which ? c.v : c.k) + (block << c.lp) * c.D;
    const int64_t ld = which ? r.ldv : r.ldk;
    const TX *x = static_cast<const TX *>(which ? r.v : r.k) + p.row * ld + head * c.D;
    const float was = p.lo ? *scale : 0.0f;  // a page's first token starts it anew
    const int rot = which ? 0 : turn.rot, half = rot / 2, turned = half / W, np = c.D / (2 * W), items = (p.hi - p.lo) * np;

    // this thread's items are tid, tid + G, ..: token t and pair j of it, stepped without divisions
    const int t0 = (unsigned)tid / (unsigned)np, j0 = tid - t0 * np, dt = G / np, dj = G - dt * np;
    struct Place {
        int t, j, left;
    };
    auto first = [&](int skip) {
        const int i = tid + skip * G;
        if (!skip) return Place{t0, j0, items - i};
        if (items <= skip * G) return Place{0, 0, 0};
        const int t = (unsigned)i / (unsigned)np;
        return Place{t, i - t * np, items - i};
    };
    auto next = [&](Place &a) {
        a.t += dt;
        a.j += dj;
        if (a.j >= np) a.j -= np, ++a.t;
        a.left -= G;
    };
    auto low = [&](const Place &a) { return PAIRS || a.j >= turned ? 2 * W * a.j : W * a.j; };
    auto high = [&](const Place &a, int lo) { return PAIRS || a.j >= turned ? lo + W : lo + half; };
    // an item's position; -1: it has no angle (NaN, whose code is 0).  Items that are not rotated need none.
    auto position = [&](const Place &a) {
        const int at = a.j < turned ? turn.pos[p.row + a.t] : 0;
        return at < turn.n_pos ? at : -1;
    };
    auto load = [&](const Place &a, float (&u)[W], float (&w)[W]) {
        const TX *row = x + a.t * ld;
        const int lo = low(a);
        kv_load<W>(row + lo, u);
        kv_load<W>(row + high(a, lo), w);
    };
    struct Angle {
        float c[W], s[W];
    };
    auto angle = [&](const Place &a, int at, Angle &g) {
#pragma unroll
        for (int i = 0; i < W; ++i) g.c[i] = g.s[i] = nanf("");
        if (a.j < turned && at >= 0) {
            const int64_t i = (int64_t)at * half + a.j * W;
            kv_load<W>(turn.cos_tab + i, g.c);
            kv_load<W>(turn.sin_tab + i, g.s);
        }
    };
    auto rotate = [&](const Place &place, const Angle &g, float (&u)[W], float (&w)[W]) {
        if (place.j >= turned) return;
        auto pair = [&](float &a, float &b, float cv, float sv) {
            const float a0 = a, b0 = b;
            a = __fsub_rn(__fmul_rn(a0, cv), __fmul_rn(b0, sv));
            b = __fadd_rn(__fmul_rn(b0, cv), __fmul_rn(a0, sv));
        };
        if constexpr (PAIRS && W == 4) {
            pair(u[0], u[1], g.c[0], g.s[0]);
            pair(u[2], u[3], g.c[1], g.s[1]);
            pair(w[0], w[1], g.c[2], g.s[2]);
            pair(w[2], w[3], g.c[3], g.s[3]);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) pair(u[i], w[i], g.c[i], g.s[i]);
        }
    };
    auto turned_item = [&](const Place &a, float (&v)[W], float (&z)[W]) {
        Angle g;
        load(a, v, z);
        angle(a, position(a), g);
        rotate(a, g, v, z);
    };
    // all positions, then rows and angles of four items at once: one by one the angles' loads took as long as all the rest
    float u[kKvHeld][W], w[kKvHeld][W];
    {
        int at[kKvHeld];
        Place a = first(0);
#pragma unroll
        for (int k = 0; k < kKvHeld; ++k, next(a))
            if (a.left > 0) at[k] = position(a);
        a = first(0);
#pragma unroll
        for (int k0 = 0; k0 < kKvHeld; k0 += 4) {
            Angle g[4];
            Place four = a;
#pragma unroll
            for (int k = k0; k < k0 + 4; ++k, next(a)) {
                if (a.left > 0) {
                    load(a, u[k], w[k]);
                    angle(a, at[k], g[k - k0]);
                } else {
#pragma unroll
                    for (int i = 0; i < W; ++i) u[k][i] = w[k][i] = 0.0f;
                }
            }
#pragma unroll
            for (int k = k0; k < k0 + 4; ++k, next(four))
                if (four.left > 0) rotate(four, g[k - k0], u[k], w[k]);
        }
    }
    // the largest magnitude; NaN wins here (one instruction an element either way), and is looked after when it did
    auto largest = [&](auto max2) {
        float amax = 0.0f;
#pragma unroll
        for (int k = 0; k < kKvHeld; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) amax = max2(max2(amax, fabsf(u[k][i])), fabsf(w[k][i]));
        for (Place a = first(kKvHeld); a.left > 0; next(a)) {
            float v[W], z[W];
            turned_item(a, v, z);
#pragma unroll
            for (int i = 0; i < W; ++i) amax = max2(max2(amax, fabsf(v[i])), fabsf(z[i]));
        }
#pragma unroll
        for (int s = 16; s; s >>= 1) amax = max2(amax, __shfl_xor_sync(~0u, amax, s));
        kv_sync<G>();  // (all have read the old scale, too, before the new one is written)
        if (G > 32) {
            const int w0 = threadIdx.x / G * (G / 32);
            if ((tid & 31) == 0) red[w0 + (tid >> 5)] = amax;
            kv_sync<G>();
            amax = red[w0];
#pragma unroll
            for (int i = 1; i < G / 32; ++i) amax = max2(amax, red[w0 + i]);
        }
        return amax;
    };
    float amax = largest([](float a, float b) { return kv_max_nan(a, b); });
    const bool nans = isnan(amax);
    if (nans) amax = largest([](float a, float b) { return fmaxf(a, b); });

    const float now = fmaxf(was, __fdiv_rn(amax, 127.0f));
    if (tid == 0) *scale = now;
    if (now > was && was > 0.0f) {
        const float f = __fdiv_rn(was, now);
        uint32_t *old = reinterpret_cast<uint32_t *>(codes);
#pragma unroll 4
        for (int i = tid; i < p.lo * c.D / 4; i += G) {
            const uint32_t q = old[i];
            auto again = [&](int shift) { return kv_byte((float)(int8_t)(q >> shift), f); };
            old[i] = kv_join(again(0), again(8), again(16), again(24));
        }
    }
    float inv = __fdiv_rn(1.0f, now);
    if (isinf(inv)) inv = 0.0f;  // a block of zeros, or below 2^-128
    auto store = [&](const Place &a, const float (&v)[W], const float (&z)[W], bool careful) {
        const int lo = low(a);
        int8_t *row = codes + (p.lo + a.t) * c.D;
        if constexpr (W == 4) {
            auto word = [&](const float (&f)[W]) {
                return careful ? kv_pack(kv_code(f[0], inv), kv_code(f[1], inv), kv_code(f[2], inv), kv_code(f[3], inv))
                               : kv_join(kv_byte(f[0], inv), kv_byte(f[1], inv), kv_byte(f[2], inv), kv_byte(f[3], inv));
            };
            *reinterpret_cast<uint32_t *>(row + lo) = word(v);
            *reinterpret_cast<uint32_t *>(row + high(a, lo)) = word(z);
        } else {
            row[lo] = (int8_t)kv_code(v[0], inv);
            row[high(a, lo)] = (int8_t)kv_code(z[0], inv);
        }
    };
    auto finish = [&](bool careful) {
        Place a = first(0);
#pragma unroll
        for (int k = 0; k < kKvHeld; ++k, next(a))
            if (a.left > 0) store(a, u[k], w[k], careful);
        for (a = first(kKvHeld); a.left > 0; next(a)) {
            float v[W], z[W];
            turned_item(a, v, z);
            store(a, v, z, careful);
        }
    };
    if (nans || isinf(now)) finish(true);  // (an infinity times 1/infinity is NaN, too)
    else finish(false);
}

// As many codes at a time as make 16 bytes of the rows' type.  VEC: rows that 16-byte stores fit.
template <typename TY, bool VEC, int G>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(KvCache c, KvRows r) {
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int tid = threadIdx.x % G, which_head = blockIdx.y * (kKvThreads / G) + threadIdx.x / G;
    KvPart p;
    if (!kv_part(c, r, blockIdx.x, p) || which_head >= 2 * c.n_kv) return;
    const int which = which_head >= c.n_kv, head = which_head - (which ? c.n_kv : 0);
    const int64_t block = p.page * c.n_kv + head;
    const float scale = (which ? c.v_scale : c.k_scale)[block];
    const int8_t *codes = (which ? c.v : c.k) + ((block << c.lp) + p.lo) * c.D;
    const int64_t ld = which ? r.ldv : r.ldk;
    TY *y = static_cast<TY *>(which ? r.v : r.k) + p.row * ld + head * c.D;
    constexpr int N = kVec<TY>;
    using Codes = typename VecOf<N>::type;
    const int pieces = c.D / N, items = (p.hi - p.lo) * pieces, dt = G / pieces, dj = G - dt * pieces;
    int t = (unsigned)tid / (unsigned)pieces, j = tid - t * pieces;
#pragma unroll 4
    for (int i = tid; i < items; i += G) {
        const Codes q = *reinterpret_cast<const Codes *>(codes + i * N);
        TY *dst = y + t * ld + j * N;
        t += dt;
        j += dj;
        if (j >= pieces) j -= pieces, ++t;
        uint4 u;
        TY *v = reinterpret_cast<TY *>(&u);
#pragma unroll
        for (int x = 0; x < N; ++x) {
            // the byte with its sign bit turned under the exponent of 2^23 is 2^23 + 128 + code
            const uint32_t word = reinterpret_cast<const uint32_t *>(&q)[x / 4] ^ 0x80808080u;
            const float code = __uint_as_float(__byte_perm(word, 0x4b000000u, 0x7440 | x % 4)) - 8388736.0f;
            v[x] = from_f32<TY>(__fmul_rn(code, scale));
        }
        if (VEC) {
            *reinterpret_cast<uint4 *>(dst) = u;
        } else {
#pragma unroll
            for (int x = 0; x < N; ++x) dst[x] = v[x];
        }
    }
}

// ---------------------------------------------------------------- host
kq_status kv_check(const char *fn, const int8_t *k_cache, const int8_t *v_cache, const float *k_scale, const float *v_scale,
                   int64_t n_pages, int64_t page, const int32_t *table, int64_t ldt, const int32_t *lens, int64_t B,
                   int64_t n_kv, int64_t D, KvCache &c) {
    if (!k_cache || !v_cache || !k_scale || !v_scale) return fail(KQ_ERR_INVALID_ARG, "%s: null cache or scales", fn);
    if (!table || !lens) return fail(KQ_ERR_INVALID_ARG, "%s: null %s", fn, table ? "lens" : "table");
    if (B <= 0 || B > (1 << 24) || n_kv <= 0 || n_kv > kKvMaxHeads || D <= 0 || D > kKvMaxD || D % 16)
        return fail(KQ_ERR_INVALID_ARG, "%s: need 1 to 2^24 sequences, 1 to %d key heads and D a multiple of 16 up to %d (B=%lld n_kv=%lld D=%lld)",
                    fn, kKvMaxHeads, kKvMaxD, (long long)B, (long long)n_kv, (long long)D);
    if (page < 16 || page > kKvMaxPage || (page & (page - 1)))
        return fail(KQ_ERR_INVALID_ARG, "%s: page=%lld is not a power of two in 16..%d", fn, (long long)page, kKvMaxPage);
    if (n_pages <= 0 || n_pages > 0x7fffffff || ldt <= 0 || ldt > 0x7fffffff)
        return fail(KQ_ERR_INVALID_ARG, "%s: need n_pages and ldt in 1..2^31-1 (n_pages=%lld ldt=%lld)", fn, (long long)n_pages, (long long)ldt);
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(table, 4) || !aligned(lens, 4))
        return fail(KQ_ERR_ALIGNMENT, "%s: the caches must be 16-byte aligned, scales, table and lens to their elements", fn);
    c.k = const_cast<int8_t *>(k_cache);
    c.v = const_cast<int8_t *>(v_cache);
    c.k_scale = const_cast<float *>(k_scale);
    c.v_scale = const_cast<float *>(v_scale);
    c.table = table;
    c.lens = lens;
    c.n_pages = n_pages;
    c.ldt = ldt;
    c.B = B;
    c.n_kv = (int)n_kv;
    c.D = (int)D;
    for (c.lp = 4; (1 << c.lp) < page; ++c.lp) {}
    return KQ_OK;
}

// Threads of a group: a warp for sequences of four rows or fewer on average.
static int kv_group(const KvCache &c, int64_t T) { return T <= 4 * c.B ? 32 : kKvGroup; }

// The packed rows of a call, and the grid over the blocks of the cache that they can touch.
static kq_status kv_check_rows(const char *fn, kq_dtype t, const void *k, int64_t ldk, const void *v, int64_t ldv, const int32_t *cu,
                               int64_t T, const KvCache &c, KvRows &r, dim3 &grid) {
    if (!is_value_type(t)) return fail(KQ_ERR_UNSUPPORTED_DTYPE, "%s: row type %s is not F32, F16 or BF16", fn, dtype_name(t));
    if (!k || !v) return fail(KQ_ERR_INVALID_ARG, "%s: null rows", fn);
    const int64_t width = (int64_t)c.n_kv * c.D;
    if (T <= 0 || T > 0x7fffffff || (!cu && T % c.B))
        return fail(KQ_ERR_INVALID_ARG, "%s: need T > 0, and a multiple of B where cu is NULL (T=%lld)", fn, (long long)T);
    if (ldk < width || ldv < width)
        return fail(KQ_ERR_INVALID_ARG, "%s: ldk=%lld or ldv=%lld is less than n_kv*D", fn, (long long)ldk, (long long)ldv);
    const size_t e = value_bytes(t);
    if (!aligned(k, e) || !aligned(v, e) || !aligned(cu, 4))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    const bool by_row = T <= (T >> c.lp) + 2 * c.B;
    const int64_t units = by_row ? T : (T >> c.lp) + 2 * c.B;
    if (units > 0x7fffffff) return fail(KQ_ERR_INVALID_ARG, "%s: T=%lld is too large", fn, (long long)T);
    r = {const_cast<void *>(k), const_cast<void *>(v), ldk, ldv, cu, T, by_row};
    grid = dim3((unsigned)units, (unsigned)((2 * c.n_kv * kv_group(c, T) + kKvThreads - 1) / kKvThreads));
    return KQ_OK;
}

template <typename TX>
static cudaError_t launch_append(const KvCache &c, const KvRows &r, const KvTurn &t, bool pairs, bool vec, dim3 grid, cudaStream_t st) {
    auto go = [&](auto group) {
        constexpr int G = decltype(group)::value;
        auto kern = vec ? (pairs ? kv_append_kernel<TX, true, 4, G> : kv_append_kernel<TX, false, 4, G>)
                        : (pairs ? kv_append_kernel<TX, true, 1, G> : kv_append_kernel<TX, false, 1, G>);
        return launch_beside(kern, grid, dim3(kKvThreads), 0, dim3(1), st, c, r, t);
    };
    return kv_group(c, r.T) == 32 ? go(std::integral_constant<int, 32>{}) : go(std::integral_constant<int, kKvGroup>{});
}
template <typename TY>
static cudaError_t launch_read(const KvCache &c, const KvRows &r, bool vec, dim3 grid, cudaStream_t st) {
    auto go = [&](auto group) {
        constexpr int G = decltype(group)::value;
        return launch_beside(vec ? kv_read_kernel<TY, true, G> : kv_read_kernel<TY, false, G>, grid, dim3(kKvThreads), 0, dim3(1), st, c, r);
    };
    return kv_group(c, r.T) == 32 ? go(std::integral_constant<int, 32>{}) : go(std::integral_constant<int, kKvGroup>{});
}

}  // namespace kq

using namespace kq;

extern "C" {

kq_status kq_kv_append_i8(kq_dtype xt, const void *k, int64_t ldk, const void *v, int64_t ldv, const int32_t *cu,
                          const int32_t *lens, int64_t B, int64_t T, int64_t n_kv, int64_t D, const int32_t *positions,
                          const float *cos_tab, const float *sin_tab, int64_t n_pos, int64_t rot, int pairs, int8_t *k_cache,
                          int8_t *v_cache, float *k_scale, float *v_scale, int64_t n_pages, int64_t page, const int32_t *table,
                          int64_t ldt, kq_stream_t stream) {
    const char *fn = "kq_kv_append_i8";
    KvCache c;
    KvRows r;
    dim3 grid;
    kq_status s = kv_check(fn, k_cache, v_cache, k_scale, v_scale, n_pages, page, table, ldt, lens, B, n_kv, D, c);
    if (s == KQ_OK) s = kv_check_rows(fn, xt, k, ldk, v, ldv, cu, T, c, r, grid);
    if (s != KQ_OK) return s;
    if (rot < 0 || rot > D || rot % 2) return fail(KQ_ERR_INVALID_ARG, "%s: rot=%lld is not even in 0..D", fn, (long long)rot);
    if (pairs != 0 && pairs != 1) return fail(KQ_ERR_INVALID_ARG, "%s: pairs=%d is not 0 or 1", fn, pairs);
    if (rot && (!positions || !cos_tab || !sin_tab || n_pos <= 0))
        return fail(KQ_ERR_INVALID_ARG, "%s: a rotation needs positions, cos_tab, sin_tab and n_pos > 0", fn);
    if (!rot) positions = nullptr, cos_tab = sin_tab = nullptr;
    if (!aligned(positions, 4) || !aligned(cos_tab, 4) || !aligned(sin_tab, 4))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    // four elements at once: rows, halves and the tables' rows on boundaries of four
    const size_t four = 4 * value_bytes(xt);
    const bool vec = aligned(k, four) && aligned(v, four) && ldk % 4 == 0 && ldv % 4 == 0 && (rot / 2) % 4 == 0 && aligned(cos_tab, 16) &&
                     aligned(sin_tab, 16);
    return with_type(xt, [&](auto t) {
        const cudaError_t e = launch_append<decltype(t)>(c, r, {positions, cos_tab, sin_tab, n_pos, (int)rot}, pairs != 0, vec, grid,
                                                         (cudaStream_t)stream);
        if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
        count_launch(R_KV);
        return KQ_OK;
    });
}

kq_status kq_kv_read_i8(const int8_t *k_cache, const int8_t *v_cache, const float *k_scale, const float *v_scale, int64_t n_pages,
                        int64_t page, const int32_t *table, int64_t ldt, const int32_t *cu, const int32_t *lens, int64_t B, int64_t T,
                        int64_t n_kv, int64_t D, kq_dtype yt, void *k_out, int64_t ldk, void *v_out, int64_t ldv, kq_stream_t stream) {
    const char *fn = "kq_kv_read_i8";
    KvCache c;
    KvRows r;
    dim3 grid;
    kq_status s = kv_check(fn, k_cache, v_cache, k_scale, v_scale, n_pages, page, table, ldt, lens, B, n_kv, D, c);
    if (s == KQ_OK) s = kv_check_rows(fn, yt, k_out, ldk, v_out, ldv, cu, T, c, r, grid);
    if (s != KQ_OK) return s;
    const int64_t e16 = 16 / (int64_t)value_bytes(yt);
    const bool vec = aligned(k_out, 16) && aligned(v_out, 16) && ldk % e16 == 0 && ldv % e16 == 0;
    return with_type(yt, [&](auto t) {
        const cudaError_t e = launch_read<decltype(t)>(c, r, vec, grid, (cudaStream_t)stream);
        if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
        count_launch(R_KV);
        return KQ_OK;
    });
}

}  // extern "C"
