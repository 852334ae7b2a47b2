// kq_qk_rope.cu -- per-head RMS norm of queries and keys with the position rotation in the same pass.
//
// Bound by bytes: every element is read once and written once, 4 + 2 bytes for fp32 rows into bf16; 8192
// tokens of 40 heads of 128 take 37 us, 6.9 TB/s.  LANES lanes (8, 16 or 32) own a head, its elements in
// registers between the read and the write, so nothing is staged and a head's sum of squares is a butterfly
// over its lanes.  The layout follows the rotation:
//   halves (a = v[i], b = v[i + rot/2]): a lane's vectors lie in pairs, one below rot/2 and its partner
//   above, so both members of every rotated pair are the lane's own; the rest of the head (rot .. D) is
//   spread over the lanes behind them;
//   neighbours (a = v[2i], b = v[2i+1]): any vector of four holds whole pairs.
// Either way a lane rotates alone, and its angles are consecutive in the tables (one vector each).
#include <algorithm>
#include <math.h>

#include "kq_launch.cuh"
#include "kq_value.cuh"

namespace kq {

struct QkParams {
    const void *x[2];     // queries, keys
    void *y[2];
    int64_t ldx[2], ldy[2];
    const float *gamma[2];
    int64_t M;
    int heads[2], D, rot;
    int64_t n_pos;
    float eps;
    const int32_t *pos;
    const float *cos_tab, *sin_tab;
    // the vector form: 1/D, and the division by a token's groups as (u * magic) >> shift
    float inv_d;
    uint32_t magic;
    int shift;
};

constexpr int kQkMaxD = 1024;
constexpr int kQkThreads = 256;

// N consecutive elements as fp32; the address is aligned to all of them, or to 16 bytes.
template <typename T, int N>
__device__ __forceinline__ void load_n(const T *p, float (&v)[N]) {
    constexpr int W = N * sizeof(T) < 16 ? N : 16 / (int)sizeof(T);
    using Vec = typename VecOf<W * (int)sizeof(T)>::type;
#pragma unroll
    for (int i = 0; i < N; i += W) {
        const Vec u = *reinterpret_cast<const Vec *>(p + i);
#pragma unroll
        for (int j = 0; j < W; ++j) v[i + j] = to_f32(reinterpret_cast<const T *>(&u)[j]);
    }
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T *p, const float (&v)[N]) {
    constexpr int W = N * sizeof(T) < 16 ? N : 16 / (int)sizeof(T);
    using Vec = typename VecOf<W * (int)sizeof(T)>::type;
#pragma unroll
    for (int i = 0; i < N; i += W) {
        Vec u;
#pragma unroll
        for (int j = 0; j < W; ++j) reinterpret_cast<T *>(&u)[j] = from_f32<T>(v[i + j]);
        *reinterpret_cast<Vec *>(p + i) = u;
    }
}

// Four consecutive elements in two packed pairs (the arithmetic below is two operations an instruction: the
// scalar form of this kernel was bound by its instructions, 51 us where the bytes take 38).
struct Four {
    float2 lo, hi;
};
__device__ __forceinline__ Four mul(Four a, Four b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ Four fma(Four a, Four b, Four c) { return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)}; }
__device__ __forceinline__ Four all(float v) { return {make_float2(v, v), make_float2(v, v)}; }
// v where the mask is all ones, 0 where it is 0.
__device__ __forceinline__ Four masked(Four v, uint32_t mask) {
    auto m = [mask](float f) { return __uint_as_float(__float_as_uint(f) & mask); };
    return {make_float2(m(v.lo.x), m(v.lo.y)), make_float2(m(v.hi.x), m(v.hi.y))};
}
template <typename T>
__device__ __forceinline__ Four load4(const T *p) {
    float v[4];
    load_n<T, 4>(p, v);
    return {make_float2(v[0], v[1]), make_float2(v[2], v[3])};
}
template <typename T>
__device__ __forceinline__ void store4(T *p, Four f) {
    const float v[4] = {f.lo.x, f.lo.y, f.hi.x, f.hi.y};
    store_n<T, 4>(p, v);
}

// R rounds of LANES vector pairs: pair j (j = lane + LANES*round) of a head covers elements [lo, lo + 4) and
// [hi, hi + 4).  Pairs 0 .. rot/8 - 1 are rotated: lo = 4j, hi = lo + rot/2 (halves) or lo = 8j, hi = lo + 4
// (neighbours); the following pairs cover rot .. D.
// The lanes take G heads of their token (queries or keys, not both): angles and gamma are read once for them.
// PART: rot < D.  Lanes past the rotated part go through the rotation's arithmetic too, by an angle of 0 (c = 1, s = 0),
// but with 0 for their partners: an infinity or NaN times s = 0 would be a NaN.  (8192 tokens, 40 heads of 128, half of
// them rotated, fp32 to bf16: 40.0 us with the masks, 38.5 with a branch a head, 37.1 with neither; bf16: 31.1, 32.3
// and 30.2; heads of 80 in f16: 13.6, 14.4 and 13.5.  So whole heads have a form without.)
template <typename TX, typename TY, bool PAIRS, bool PART, int R, int LANES, int G>
__global__ void __launch_bounds__(kQkThreads) qk_kernel(QkParams P) {
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const unsigned gq = (P.heads[0] + G - 1) / G, per_token = gq + (P.heads[1] + G - 1) / G;
    const unsigned unit = blockIdx.x * (kQkThreads / LANES) + threadIdx.x / LANES;  // below 2^31
    const int lane = threadIdx.x % LANES;
    const unsigned token = (unsigned)((unit * (uint64_t)P.magic) >> P.shift);       // unit / per_token
    const bool live = token < (unsigned)P.M;
    const int64_t t = live ? token : 0;
    const unsigned gg = live ? unit - token * per_token : 0;
    const int which = gg >= gq, h0 = (which ? gg - gq : gg) * G, n = live ? min(G, P.heads[which] - h0) : 0;
    const TX *x = static_cast<const TX *>(P.x[which]) + t * P.ldx[which] + (int64_t)h0 * P.D;
    TY *y = static_cast<TY *>(P.y[which]) + t * P.ldy[which] + (int64_t)h0 * P.D;
    const float *gamma = P.gamma[which];
    const int half = P.rot / 2, np = P.D / 8, rotated = half / 4;
    const int64_t p = P.rot && live ? P.pos[t] : 0;
    const bool known = !P.rot || (p >= 0 && p < P.n_pos);
    int lo[R], hi[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int j = lane + LANES * r;
        lo[r] = PAIRS || j >= rotated ? 8 * j : 4 * j;  // (rest: 8*rotated = rot)
        hi[r] = PAIRS || j >= rotated ? lo[r] + 4 : lo[r] + half;
    }
    Four a[G][R], b[G][R];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool mine = g < n && lane + LANES * r < np;
            a[g][r] = mine ? load4(x + g * P.D + lo[r]) : all(0.0f);
            b[g][r] = mine ? load4(x + g * P.D + hi[r]) : all(0.0f);
        }
    Four c[R], s[R], ga[R], gb[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int j = lane + LANES * r;
        const bool turned = n && known && j < rotated, normed = gamma && j < np;
        c[r] = turned ? load4(P.cos_tab + p * half + j * 4) : all(1.0f);
        s[r] = turned ? load4(P.sin_tab + p * half + j * 4) : all(0.0f);
        ga[r] = normed ? load4(gamma + lo[r]) : all(1.0f);
        gb[r] = normed ? load4(gamma + hi[r]) : all(1.0f);
        if (!known) ga[r] = gb[r] = all(nanf(""));
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
        Four sq = all(0.0f);
#pragma unroll
        for (int r = 0; r < R; ++r) sq = fma(a[g][r], a[g][r], fma(b[g][r], b[g][r], sq));
        float ss = (sq.lo.x + sq.lo.y) + (sq.hi.x + sq.hi.y);
        // (every lane of the warp takes part, whichever tensor its heads are of)
#pragma unroll
        for (int d = LANES / 2; d; d >>= 1) ss += __shfl_xor_sync(~0u, ss, d);
        const Four rs = all(gamma ? rsqrtf(fmaf(ss, P.inv_d, P.eps)) : 1.0f);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            Four u = mul(mul(a[g][r], rs), ga[r]), w = mul(mul(b[g][r], rs), gb[r]);
            const uint32_t partners = !PART || lane + LANES * r < rotated ? ~0u : 0u;
            Four u0, w0;  // the elements' own shares, then their partners'
            if (PAIRS) {  // angles: c.lo for the pairs of u, c.hi for those of w
                auto twice = [](float2 v) { return Four{make_float2(v.x, v.x), make_float2(v.y, v.y)}; };
                auto signs = [](float2 v) { return Four{make_float2(-v.x, v.x), make_float2(-v.y, v.y)}; };
                auto swap = [](Four v) { return Four{make_float2(v.lo.y, v.lo.x), make_float2(v.hi.y, v.hi.x)}; };
                u0 = mul(u, twice(c[r].lo));
                w0 = mul(w, twice(c[r].hi));
                if (PART) u = masked(u, partners), w = masked(w, partners);
                u0 = fma(swap(u), signs(s[r].lo), u0);
                w0 = fma(swap(w), signs(s[r].hi), w0);
            } else {
                const Four minus = {make_float2(-s[r].lo.x, -s[r].lo.y), make_float2(-s[r].hi.x, -s[r].hi.y)};
                u0 = mul(u, c[r]);
                w0 = mul(w, c[r]);
                if (PART) u = masked(u, partners), w = masked(w, partners);
                u0 = fma(w, minus, u0);
                w0 = fma(u, s[r], w0);
            }
            if (g < n && lane + LANES * r < np) {
                store4(y + g * P.D + lo[r], u0);
                store4(y + g * P.D + hi[r], w0);
            }
        }
    }
}

// Heads that no vector form fits (odd widths, unaligned rows, over 512 elements): one warp a head, partners
// met through shared memory.  Bound by its instructions, a few for every single element: 8192 tokens of 40 heads of 128
// from rows at odd addresses, fp32 to bf16, 139 us (37 in the vector form); heads of 100 217 us; 2048 tokens of 18
// heads of 1024 90 us.
template <typename TX, typename TY>
__global__ void __launch_bounds__(128) qk_any_kernel(QkParams P, bool pairs) {
    __shared__ float buf[4][kQkMaxD];
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned nh = P.heads[0] + P.heads[1], unit = blockIdx.x * 4 + warp;
    if (unit >= (unsigned)P.M * nh) return;
    const int64_t t = unit / nh;
    const int hh = (int)(unit % nh), which = hh >= P.heads[0], h = which ? hh - P.heads[0] : hh;
    const TX *x = static_cast<const TX *>(P.x[which]) + t * P.ldx[which] + (int64_t)h * P.D;
    TY *y = static_cast<TY *>(P.y[which]) + t * P.ldy[which] + (int64_t)h * P.D;
    const float *gamma = P.gamma[which];
    float *b = buf[warp], ss = 0.0f;
    for (int i = lane; i < P.D; i += 32) {
        const float v = to_f32(x[i]);
        b[i] = v;
        ss += v * v;
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) ss += __shfl_xor_sync(~0u, ss, s);
    if (gamma) {
        const float r = 1.0f / sqrtf(ss / (float)P.D + P.eps);
        for (int i = lane; i < P.D; i += 32) b[i] = b[i] * r * gamma[i];
    }
    __syncwarp();
    const int64_t p = P.rot ? P.pos[t] : 0;
    const bool known = !P.rot || (p >= 0 && p < P.n_pos);
    const int half = P.rot / 2;
    for (int i = lane; i < P.D; i += 32) {
        float v = b[i];
        if (i < P.rot && known) {
            const int j = pairs ? i >> 1 : (i < half ? i : i - half);
            const bool second = pairs ? i & 1 : i >= half;
            const float c = P.cos_tab[p * half + j], s = P.sin_tab[p * half + j];
            const float other = b[pairs ? i ^ 1 : (second ? i - half : i + half)];
            v = second ? v * c + other * s : v * c - other * s;
        }
        y[i] = from_f32<TY>(known ? v : nanf(""));
    }
}

template <typename TX, typename TY>
static cudaError_t launch_qk(const QkParams &P, bool pairs, bool aligned4, cudaStream_t st) {
    const int64_t units = P.M * (P.heads[0] + P.heads[1]);
    // vectors of four elements (16 bytes of fp32, 8 of 16-bit types) wherever they tile the halves and the rest
    const bool vec = aligned4 && P.D % 8 == 0 && (P.rot / 2) % 4 == 0 && P.D <= 512;
    if (!vec) {
        return launch_beside(qk_any_kernel<TX, TY>, dim3((unsigned)((units + 3) / 4)), dim3(128), 0, dim3(1), st, P, pairs);
    }
    auto go = [&](auto pr, auto rounds, auto lanes, auto heads) {
        constexpr int R = decltype(rounds)::value, L = decltype(lanes)::value, G = decltype(heads)::value;
        const int64_t groups = P.M * ((P.heads[0] + G - 1) / G + (P.heads[1] + G - 1) / G);
        const int64_t blocks = (groups * L + kQkThreads - 1) / kQkThreads;
        QkParams q = P;
        // exact for u below 2^31: 2^(31+l)/d rounded up, 2^(l-1) < d <= 2^l
        const uint64_t d = groups / P.M;
        int l = 0;
        while ((1ull << l) < d) ++l;
        q.shift = 31 + l;
        q.magic = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
        q.inv_d = 1.0f / (float)P.D;
        auto kern = P.rot < P.D ? qk_kernel<TX, TY, decltype(pr)::value, true, R, L, G> : qk_kernel<TX, TY, decltype(pr)::value, false, R, L, G>;
        return launch_beside(kern, dim3((unsigned)blocks), dim3(kQkThreads), 0, dim3(1), st, q);
    };
    auto heads = [&](auto pr, auto rounds, auto lanes) {
        // four heads a lane group once that still fills every SM's threads (152 * 2048): 8192 tokens of 40
        // heads of 128, fp32 to bf16, 37.2 us (6.9 TB/s) against 40.1 with two and 42.8 with eight
        if (units * decltype(lanes)::value / 4 >= 152 * 2048) return go(pr, rounds, lanes, std::integral_constant<int, 4>{});
        return go(pr, rounds, lanes, std::integral_constant<int, 1>{});
    };
    auto form = [&](auto pr) {
        // a lane for each of a head's D/8 vector pairs (two from 256 elements on)
        if (P.D <= 64) return heads(pr, std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
        if (P.D <= 128) return heads(pr, std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
        if (P.D <= 256) return heads(pr, std::integral_constant<int, 1>{}, std::integral_constant<int, 32>{});
        return heads(pr, std::integral_constant<int, 2>{}, std::integral_constant<int, 32>{});
    };
    return pairs ? form(std::true_type{}) : form(std::false_type{});
}

}  // namespace kq

using namespace kq;

extern "C" kq_status kq_qk_norm_rope(kq_dtype xt, const void *q, int64_t ldq, const void *k, int64_t ldk, int64_t M,
                                     int64_t n_q, int64_t n_k, int64_t D, const float *q_gamma, const float *k_gamma,
                                     float eps, const int32_t *positions, const float *cos_tab, const float *sin_tab,
                                     int64_t n_pos, int64_t rot, int pairs, kq_dtype yt, void *q_out, int64_t ldqo,
                                     void *k_out, int64_t ldko, kq_stream_t stream) {
    const char *fn = "kq_qk_norm_rope";
    if (!is_value_type(xt) || !is_value_type(yt))
        return fail(KQ_ERR_UNSUPPORTED_DTYPE, "%s: %s type %s is not F32, F16 or BF16", fn, is_value_type(xt) ? "output" : "input",
                    dtype_name(is_value_type(xt) ? yt : xt));
    if (M <= 0 || n_q < 0 || n_k < 0 || n_q + n_k <= 0 || n_q > 65536 || n_k > 65536)
        return fail(KQ_ERR_INVALID_ARG, "%s: need M > 0 and 1 to 65536 heads (M=%lld n_q=%lld n_k=%lld)", fn, (long long)M,
                    (long long)n_q, (long long)n_k);
    if (D < 2 || D > kQkMaxD || D % 2 || rot < 0 || rot > D || rot % 2)
        return fail(KQ_ERR_INVALID_ARG, "%s: need D even in 2..%d and rot even in 0..D (D=%lld rot=%lld)", fn, kQkMaxD,
                    (long long)D, (long long)rot);
    if (pairs != 0 && pairs != 1) return fail(KQ_ERR_INVALID_ARG, "%s: pairs=%d is not 0 or 1", fn, pairs);
    if (!(eps >= 0.0f) || isinf(eps)) return fail(KQ_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    if ((n_q && (!q || !q_out)) || (n_k && (!k || !k_out))) return fail(KQ_ERR_INVALID_ARG, "%s: null rows", fn);
    if (n_q && (ldq < n_q * D || ldqo < n_q * D))
        return fail(KQ_ERR_INVALID_ARG, "%s: ldq=%lld or ldqo=%lld is less than n_q*D", fn, (long long)ldq, (long long)ldqo);
    if (n_k && (ldk < n_k * D || ldko < n_k * D))
        return fail(KQ_ERR_INVALID_ARG, "%s: ldk=%lld or ldko=%lld is less than n_k*D", fn, (long long)ldk, (long long)ldko);
    if (rot && (!positions || !cos_tab || !sin_tab || n_pos <= 0))
        return fail(KQ_ERR_INVALID_ARG, "%s: a rotation needs positions, cos_tab, sin_tab and n_pos > 0", fn);
    // what the call does not use is not looked at
    if (!n_q) q = q_out = nullptr, q_gamma = nullptr, ldq = ldqo = 0;
    if (!n_k) k = k_out = nullptr, k_gamma = nullptr, ldk = ldko = 0;
    if (!rot) positions = nullptr, cos_tab = sin_tab = nullptr;
    const size_t xb = value_bytes(xt), yb = value_bytes(yt);
    if (!aligned(q, xb) || !aligned(q_out, yb) || !aligned(k, xb) || !aligned(k_out, yb) || !aligned(q_gamma, 4) ||
        !aligned(k_gamma, 4) || !aligned(positions, 4) || !aligned(cos_tab, 4) || !aligned(sin_tab, 4))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    QkParams P{};
    P.x[0] = q; P.x[1] = k; P.y[0] = q_out; P.y[1] = k_out;
    P.ldx[0] = ldq; P.ldx[1] = ldk; P.ldy[0] = ldqo; P.ldy[1] = ldko;
    P.gamma[0] = q_gamma; P.gamma[1] = k_gamma;
    P.M = M; P.heads[0] = (int)n_q; P.heads[1] = (int)n_k; P.D = (int)D; P.rot = (int)rot;
    P.n_pos = n_pos; P.eps = eps; P.pos = positions; P.cos_tab = cos_tab; P.sin_tab = sin_tab;
    if (M > 0x7fffffff || M * (n_q + n_k) > 0x7fffffff)
        return fail(KQ_ERR_INVALID_ARG, "%s: M=%lld is too large", fn, (long long)M);
    // every head's first element on a boundary of four elements, and the tables' rows on 16 bytes
    const bool al = aligned(cos_tab, 16) && aligned(sin_tab, 16) && aligned(q_gamma, 16) && aligned(k_gamma, 16) &&
                    aligned(q, 4 * xb) && aligned(k, 4 * xb) && aligned(q_out, 4 * yb) && aligned(k_out, 4 * yb) &&
                    ldq % 4 == 0 && ldk % 4 == 0 && ldqo % 4 == 0 && ldko % 4 == 0;
    return with_type(xt, [&](auto tx) {
        return with_type(yt, [&](auto ty) {
            const cudaError_t e = launch_qk<decltype(tx), decltype(ty)>(P, pairs != 0, al, (cudaStream_t)stream);
            if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
            count_launch(R_QK);
            return KQ_OK;
        });
    });
}
