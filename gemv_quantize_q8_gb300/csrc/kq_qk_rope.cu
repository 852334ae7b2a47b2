// kq_qk_rope.cu -- per-head RMS norm of queries and keys with the position rotation in the same pass.
#include <algorithm>
#include <math.h>

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
};

constexpr int kQkMaxD = 1024;

// One warp per (token, head).  A head's elements meet their partners through shared memory.
template <typename TX, typename TY, bool PAIRS>
__global__ void __launch_bounds__(128) qk_kernel(QkParams P) {
    __shared__ float buf[4][kQkMaxD];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nh = P.heads[0] + P.heads[1];
    const int64_t unit = (int64_t)blockIdx.x * 4 + warp;
    if (unit >= P.M * nh) return;
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
            const int j = PAIRS ? i >> 1 : (i < half ? i : i - half);
            const bool second = PAIRS ? i & 1 : i >= half;
            const float c = P.cos_tab[p * half + j], s = P.sin_tab[p * half + j];
            const float other = b[PAIRS ? i ^ 1 : (second ? i - half : i + half)];
            v = second ? v * c + other * s : v * c - other * s;
        }
        y[i] = from_f32<TY>(known ? v : nanf(""));
    }
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
    const size_t xb = value_bytes(xt), yb = value_bytes(yt);
    if ((n_q && (!aligned(q, xb) || !aligned(q_out, yb))) || (n_k && (!aligned(k, xb) || !aligned(k_out, yb))) ||
        (q_gamma && !aligned(q_gamma, 4)) || (k_gamma && !aligned(k_gamma, 4)) ||
        (rot && (!aligned(positions, 4) || !aligned(cos_tab, 4) || !aligned(sin_tab, 4))))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    QkParams P{};
    P.x[0] = q; P.x[1] = k; P.y[0] = q_out; P.y[1] = k_out;
    P.ldx[0] = ldq; P.ldx[1] = ldk; P.ldy[0] = ldqo; P.ldy[1] = ldko;
    P.gamma[0] = q_gamma; P.gamma[1] = k_gamma;
    P.M = M; P.heads[0] = (int)n_q; P.heads[1] = (int)n_k; P.D = (int)D; P.rot = (int)rot;
    P.n_pos = n_pos; P.eps = eps; P.pos = positions; P.cos_tab = cos_tab; P.sin_tab = sin_tab;
    const int64_t blocks = (M * (n_q + n_k) + 3) / 4;
    if (M > 0x7fffffff || blocks > 0x7fffffff) return fail(KQ_ERR_INVALID_ARG, "%s: M=%lld is too large", fn, (long long)M);
    return with_type(xt, [&](auto tx) {
        return with_type(yt, [&](auto ty) {
            using TX = decltype(tx);
            using TY = decltype(ty);
            if (pairs) qk_kernel<TX, TY, true><<<(unsigned)blocks, 128, 0, (cudaStream_t)stream>>>(P);
            else qk_kernel<TX, TY, false><<<(unsigned)blocks, 128, 0, (cudaStream_t)stream>>>(P);
            kq_status s = check_launch(fn);
            if (s == KQ_OK) count_launch(R_QK);
            return s;
        });
    });
}
