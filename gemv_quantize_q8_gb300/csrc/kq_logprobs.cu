// kq_logprobs.cu -- log probabilities of given tokens, with the entropy and the top alternatives of a row.
#include <math.h>

#include "kq_value.cuh"

namespace kq {

constexpr int kLpThreads = 256;
constexpr int kLpMaxTop = 32;

// The order of the alternatives as one unsigned number: larger logits first, then lower ids.  NaN ranks
// with -inf, -0 with +0.
__device__ __forceinline__ uint64_t lp_key(float x, int id) {
    if (isnan(x)) x = -INFINITY;
    uint32_t b = __float_as_uint(x + 0.0f);
    b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return ((uint64_t)b << 32) | (uint32_t)~id;
}

template <typename V, typename F>
__device__ V lp_block(V v, V *red, F f) {
#pragma unroll
    for (int s = 16; s; s >>= 1) v = f(v, __shfl_xor_sync(~0u, v, s));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kLpThreads / 32; ++i) v = f(v, red[i]);
    return v;
}

// One block per row.
template <typename T>
__global__ void __launch_bounds__(kLpThreads)
    lp_kernel(const T *__restrict__ x, int64_t ldx, int V, const int32_t *__restrict__ targets, int n_targets,
              float *__restrict__ logprob, float *__restrict__ entropy, int top_k, int32_t *__restrict__ top_ids,
              float *__restrict__ top_logprob) {
    __shared__ uint64_t red[kLpThreads / 32];
    const int64_t row = blockIdx.x;
    const T *xr = x + row * ldx;
    auto add = [](float a, float b) { return a + b; };
    auto larger = [](uint64_t a, uint64_t b) { return a > b ? a : b; };
    float m = -INFINITY, bad = 0.0f;
    for (int i = threadIdx.x; i < V; i += kLpThreads) {
        const float v = to_f32(xr[i]);
        m = fmaxf(m, v);
        if (isnan(v) || v == INFINITY) bad = 1.0f;
    }
    m = lp_block(m, reinterpret_cast<float *>(red), [](float a, float b) { return fmaxf(a, b); });
    bad = lp_block(bad, reinterpret_cast<float *>(red), add);
    float S = 0.0f, U = 0.0f;
    for (int i = threadIdx.x; i < V && m > -INFINITY; i += kLpThreads) {
        const float d = to_f32(xr[i]) - m, e = expf(d);
        S += e;
        if (e > 0.0f) U += e * d;
    }
    S = lp_block(S, reinterpret_cast<float *>(red), add);
    U = lp_block(U, reinterpret_cast<float *>(red), add);
    const bool empty = m == -INFINITY;
    const float logS = logf(S);
    auto lp_of = [&](float v) { return bad > 0.0f ? NAN : empty ? -INFINITY : (v - m) - logS; };
    if (threadIdx.x == 0 && entropy) entropy[row] = bad > 0.0f ? NAN : empty ? 0.0f : logS - U / S;
    for (int j = threadIdx.x; j < n_targets; j += kLpThreads) {
        const int t = targets[row * n_targets + j];
        logprob[row * n_targets + j] = t < 0 ? 0.0f : t >= V ? NAN : lp_of(to_f32(xr[t]));
    }
    uint64_t last = ~0ull;
    for (int j = 0; j < top_k; ++j) {
        uint64_t best = 0;
        for (int i = threadIdx.x; i < V; i += kLpThreads) {
            const uint64_t key = lp_key(to_f32(xr[i]), i);
            if (key < last && key > best) best = key;
        }
        last = lp_block(best, red, larger);
        if (threadIdx.x == 0) {
            const int id = (int)~(uint32_t)last;
            top_ids[row * top_k + j] = id;
            top_logprob[row * top_k + j] = lp_of(to_f32(xr[id]));
        }
    }
}

}  // namespace kq

using namespace kq;

extern "C" kq_status kq_logprobs(kq_dtype xt, const void *logits, int64_t ldx, int64_t M, int64_t V,
                                 const int32_t *targets, int64_t n_targets, float *logprob, float *entropy,
                                 int64_t top_k, int32_t *top_ids, float *top_logprob, kq_stream_t stream) {
    const char *fn = "kq_logprobs";
    if (!is_value_type(xt))
        return fail(KQ_ERR_UNSUPPORTED_DTYPE, "%s: logits type %s is not F32, F16 or BF16", fn, dtype_name(xt));
    if (!logits) return fail(KQ_ERR_INVALID_ARG, "%s: null logits", fn);
    if (M <= 0 || M > 0x7fffffff || V <= 0 || V > (1 << 30) || ldx < V)
        return fail(KQ_ERR_INVALID_ARG, "%s: need M > 0, 0 < V <= 2^30 and ldx >= V (M=%lld V=%lld ldx=%lld)", fn,
                    (long long)M, (long long)V, (long long)ldx);
    if (n_targets < 0 || n_targets > V || (n_targets && (!targets || !logprob)))
        return fail(KQ_ERR_INVALID_ARG, "%s: n_targets=%lld needs targets and logprob, and is 0..V", fn, (long long)n_targets);
    if (top_k < 0 || top_k > kLpMaxTop || top_k > V || (top_k && (!top_ids || !top_logprob)))
        return fail(KQ_ERR_INVALID_ARG, "%s: top_k=%lld needs top_ids and top_logprob, and is 0..min(%d, V)", fn,
                    (long long)top_k, kLpMaxTop);
    if (!aligned(logits, value_bytes(xt)) || (n_targets && (!aligned(targets, 4) || !aligned(logprob, 4))) ||
        (entropy && !aligned(entropy, 4)) || (top_k && (!aligned(top_ids, 4) || !aligned(top_logprob, 4))))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    return with_type(xt, [&](auto t) {
        using T = decltype(t);
        lp_kernel<T><<<(unsigned)M, kLpThreads, 0, (cudaStream_t)stream>>>(
            static_cast<const T *>(logits), ldx, (int)V, targets, (int)n_targets, logprob, entropy, (int)top_k, top_ids,
            top_logprob);
        kq_status s = check_launch(fn);
        if (s == KQ_OK) count_launch(R_LOGPROBS);
        return s;
    });
}
