// kq_i8.cu -- int8 products with one scale per token and one per output channel, and their quantizer.
//
// y[m][n] = ((float)(sum_k q[m][k]*w[n][k]) * sx[m]) * sw[n] (+ bias[n]); the sum is exact in int32, so the
// order in which a kernel adds it up is free and every kernel gives the same bits.  Up to eight tokens take
// kq_i8_gemv.cu (bound by the weights' bytes), more the tensor cores (kq_i8_tc.cu).
#include "kq_i8_gemv.cuh"
#include "kq_i8_quant.cuh"
#include "kq_i8_tc.cuh"
#include "kq_launch.cuh"

namespace kq {

// ---------------------------------------------------------------- quantizer
constexpr int kI8QuantThreads = 256;

// One block per row: the row's largest magnitude, then its codes, as int8 or (the tensor-core product's
// panel) as f16; the row's end is filled with zeros up to `fill`.  Clears the device flag where given one.
template <typename T, typename TQ>
__global__ void __launch_bounds__(kI8QuantThreads)
    i8_quant_kernel(const T *__restrict__ x, int64_t ldx, int K, TQ *__restrict__ q, int64_t ldq, int fill,
                    float *__restrict__ scale, unsigned long long *__restrict__ err) {
    __shared__ float red[kI8QuantThreads / 32];
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int64_t m = blockIdx.x;
    if (err && m == 0 && threadIdx.x == 0) *err = 0ull;
    const T *xr = x + m * ldx;
    float amax = i8_amax(xr, K, threadIdx.x, kI8QuantThreads);
#pragma unroll
    for (int s = 16; s; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, s));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int w = 1; w < kI8QuantThreads / 32; ++w) amax = fmaxf(amax, red[w]);
    const I8Scale s = i8_scale(amax);
    if (threadIdx.x == 0) scale[m] = s.scale;
    i8_codes(xr, K, fill, s.inv, q + m * ldq, threadIdx.x, kI8QuantThreads);
}

// The tensor-core product's panel from int8 rows: f16 codes, zeros from K to ldp.  One thread a 16-code piece.
__global__ void __launch_bounds__(256)
    i8_panel_kernel(const int8_t *__restrict__ q, int64_t ldq, int64_t M, int K, __half *__restrict__ panel, int64_t ldp,
                    unsigned long long *__restrict__ err) {
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, pieces = ldp / 16;
    if (i == 0) *err = 0ull;
    if (i >= M * pieces) return;
    const int64_t m = i / pieces;
    const int k = (int)(i % pieces) * 16;
    uint4 v = make_uint4(0, 0, 0, 0), o[2];
    if (k < K) v = *reinterpret_cast<const uint4 *>(q + m * ldq + k);  // rows are 16-byte pieces up to ldq
    if (k + 16 > K && k < K) {  // the last piece's bytes past K are not codes
        int8_t *c = reinterpret_cast<int8_t *>(&v);
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (k + j >= K) c[j] = 0;
    }
    i8x4_to_f16(v.x, o[0].x, o[0].y);
    i8x4_to_f16(v.y, o[0].z, o[0].w);
    i8x4_to_f16(v.z, o[1].x, o[1].y);
    i8x4_to_f16(v.w, o[1].z, o[1].w);
    uint4 *dst = reinterpret_cast<uint4 *>(panel + m * ldp + k);
    dst[0] = o[0];
    dst[1] = o[1];
}

// ---------------------------------------------------------------- host
constexpr int64_t kI8MaxK = 131071;  // 2^14 * K below 2^31: any sum of K products of two int8 fits 32 bits
constexpr int64_t kI8MaxDim = 0x7fffff00;

static int64_t up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

// The workspace: device flag, the dynamic form's scales, and its codes (up to kI8DirectTokens) or the f16 panel.
struct I8Workspace {
    size_t scale, codes, total;
    int64_t ld;
};
static I8Workspace i8_workspace(int64_t M, int64_t K) {
    I8Workspace l;
    l.scale = 256;
    l.codes = l.scale + (size_t)up(M * 4, 256);
    l.ld = up(K, M > kI8DirectTokens ? 64 : 16);
    l.total = l.codes + (size_t)up(M * l.ld * (M > kI8DirectTokens ? 2 : 1), 256);
    return l;
}

static kq_status i8_launched(const char *fn, cudaError_t e) {
    if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    count_launch(R_I8);
    return KQ_OK;
}

template <typename TQ>
static kq_status i8_quant(const char *fn, kq_dtype xt, const void *x, int64_t M, int64_t K, int64_t ldx, TQ *q, int64_t ldq,
                          int64_t fill, float *scale, unsigned long long *err, cudaStream_t st) {
    return with_type(xt, [&](auto t) {
        using T = decltype(t);
        const cudaError_t e = launch_beside(i8_quant_kernel<T, TQ>, dim3((unsigned)M), dim3(kI8QuantThreads), 0, dim3(1), st,
                                            static_cast<const T *>(x), ldx, (int)K, q, ldq, (int)fill, scale, err);
        return i8_launched(fn, e);
    });
}

static kq_status i8_check_rows(const char *fn, kq_dtype xt, const void *x, int64_t M, int64_t K, int64_t ldx) {
    if (!is_value_type(xt))
        return fail(KQ_ERR_UNSUPPORTED_DTYPE, "%s: x type %s is not F32, F16 or BF16", fn, dtype_name(xt));
    if (!x) return fail(KQ_ERR_INVALID_ARG, "%s: null x", fn);
    if (M <= 0 || M > kI8MaxDim || K <= 0 || K > kI8MaxK || ldx < K)
        return fail(KQ_ERR_INVALID_ARG, "%s: need M > 0, 0 < K <= %lld and ldx >= K (M=%lld K=%lld ldx=%lld)", fn,
                    (long long)kI8MaxK, (long long)M, (long long)K, (long long)ldx);
    if (!aligned(x, value_bytes(xt))) return fail(KQ_ERR_ALIGNMENT, "%s: x must be aligned to its elements", fn);
    return KQ_OK;
}

static kq_status i8_check_codes(const char *fn, const char *name, const void *p, int64_t K, int64_t ld) {
    if (!p) return fail(KQ_ERR_INVALID_ARG, "%s: null %s", fn, name);
    if (ld < K) return fail(KQ_ERR_INVALID_ARG, "%s: ld%s=%lld is less than K=%lld", fn, name, (long long)ld, (long long)K);
    if (!aligned(p, 16) || ld % 16)
        return fail(KQ_ERR_ALIGNMENT, "%s: %s must be 16-byte aligned and ld%s a multiple of 16", fn, name, name);
    return KQ_OK;
}

static kq_status i8_check_product(const char *fn, const int8_t *w, int64_t ldw, const float *sw, const float *bias,
                                  int64_t M, int64_t N, int64_t K, kq_dtype yt, const void *y, int64_t ldy,
                                  const void *ws, size_t ws_bytes) {
    if (!is_value_type(yt))
        return fail(KQ_ERR_UNSUPPORTED_DTYPE, "%s: y type %s is not F32, F16 or BF16", fn, dtype_name(yt));
    if (!sw || !y) return fail(KQ_ERR_INVALID_ARG, "%s: null %s", fn, sw ? "y" : "sw");
    if (M <= 0 || M > kI8MaxDim || N <= 0 || N > kI8MaxDim || K <= 0 || K > kI8MaxK || ldy < N)
        return fail(KQ_ERR_INVALID_ARG, "%s: need M, N > 0, 0 < K <= %lld and ldy >= N (M=%lld N=%lld K=%lld ldy=%lld)",
                    fn, (long long)kI8MaxK, (long long)M, (long long)N, (long long)K, (long long)ldy);
    kq_status s = i8_check_codes(fn, "w", w, K, ldw);
    if (s != KQ_OK) return s;
    if (!aligned(sw, 4) || (bias && !aligned(bias, 4)) || !aligned(y, value_bytes(yt)))
        return fail(KQ_ERR_ALIGNMENT, "%s: sw, bias and y must be aligned to their elements", fn);
    const size_t need = i8_workspace(M, K).total;
    if (!ws || ws_bytes < need)
        return fail(KQ_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, ws ? ws_bytes : (size_t)0, need);
    if (!aligned(ws, 256)) return fail(KQ_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    return KQ_OK;
}

// kq_gemm_i8, its checks among it; idle: a role of the tensor-core kernel that does nothing, its waits limited to wait_ns.
static kq_status i8_gemm(const char *fn, const int8_t *q, int64_t ldq, const float *sx, const int8_t *w, int64_t ldw,
                         const float *sw, const float *bias, int64_t M, int64_t N, int64_t K, kq_dtype yt, void *y,
                         int64_t ldy, void *workspace, size_t ws_bytes, cudaStream_t st, I8Idle idle = I8_IDLE_NONE,
                         unsigned long long wait_ns = kI8WaitNs) {
    kq_status s = i8_check_product(fn, w, ldw, sw, bias, M, N, K, yt, y, ldy, workspace, ws_bytes);
    if (s == KQ_OK) s = i8_check_codes(fn, "q", q, K, ldq);
    if (s != KQ_OK) return s;
    if (!sx) return fail(KQ_ERR_INVALID_ARG, "%s: null sx", fn);
    if (!aligned(sx, 4)) return fail(KQ_ERR_ALIGNMENT, "%s: sx must be 4-byte aligned", fn);
    unsigned long long *err = static_cast<unsigned long long *>(workspace);
    if (idle != I8_IDLE_NONE) {
        if (M <= kI8FewTokens) return fail(KQ_ERR_INVALID_ARG, "%s: M=%lld does not take the tensor-core path", fn, (long long)M);
        const cudaError_t e = cudaMemsetAsync(err, 0, sizeof *err, st);
        if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
    }
    if (M <= kI8FewTokens) return i8_gemv(fn, {q, ldq, sx, w, ldw, sw, bias, M, N, K, yt, y, ldy, err, false}, st);
    if (M <= kI8DirectTokens)
        return i8_tc_product(fn, {q, ldq, nullptr, 0, sx, w, ldw, sw, bias, M, N, K, yt, y, ldy, err, false, wait_ns, idle}, st);
    const I8Workspace l = i8_workspace(M, K);
    __half *panel = reinterpret_cast<__half *>(static_cast<uint8_t *>(workspace) + l.codes);
    const int64_t blocks = (M * (l.ld / 16) + 255) / 256;
    if (blocks > 0x7fffffff) return fail(KQ_ERR_INVALID_ARG, "%s: M=%lld is too large", fn, (long long)M);
    s = i8_launched(fn, launch_beside(i8_panel_kernel, dim3((unsigned)blocks), dim3(256), 0, dim3(1), st, q, ldq, M, (int)K, panel,
                                      l.ld, err));
    if (s != KQ_OK) return s;
    return i8_tc_product(fn, {nullptr, 0, panel, l.ld, sx, w, ldw, sw, bias, M, N, K, yt, y, ldy, err, true, wait_ns, idle}, st);
}

}  // namespace kq

using namespace kq;

extern "C" {

kq_status kq_quantize_i8(kq_dtype xt, const void *x, int64_t M, int64_t K, int64_t ldx, int8_t *q, int64_t ldq,
                         float *scale, kq_stream_t stream) {
    const char *fn = "kq_quantize_i8";
    kq_status s = i8_check_rows(fn, xt, x, M, K, ldx);
    if (s == KQ_OK) s = i8_check_codes(fn, "q", q, K, ldq);
    if (s != KQ_OK) return s;
    if (!scale) return fail(KQ_ERR_INVALID_ARG, "%s: null scale", fn);
    if (!aligned(scale, 4)) return fail(KQ_ERR_ALIGNMENT, "%s: scale must be 4-byte aligned", fn);
    return i8_quant(fn, xt, x, M, K, ldx, q, ldq, up(K, 16), scale, nullptr, (cudaStream_t)stream);
}

size_t kq_gemm_i8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || M > kI8MaxDim || N <= 0 || N > kI8MaxDim || K <= 0 || K > kI8MaxK) return 0;
    return i8_workspace(M, K).total;
}

kq_status kq_gemm_i8(const int8_t *q, int64_t ldq, const float *sx, const int8_t *w, int64_t ldw, const float *sw,
                     const float *bias, int64_t M, int64_t N, int64_t K, kq_dtype yt, void *y, int64_t ldy,
                     void *workspace, size_t ws_bytes, kq_stream_t stream) {
    return i8_gemm("kq_gemm_i8", q, ldq, sx, w, ldw, sw, bias, M, N, K, yt, y, ldy, workspace, ws_bytes, (cudaStream_t)stream);
}

kq_status kq_debug_i8_wait_timeout(const int8_t *q, int64_t ldq, const float *sx, const int8_t *w, int64_t ldw, const float *sw,
                                   int64_t M, int64_t N, int64_t K, float *y, int64_t ldy, int idle, int64_t wait_limit_ns,
                                   void *workspace, size_t ws_bytes, kq_stream_t stream) {
    const char *fn = "kq_debug_i8_wait_timeout";
    if (idle != I8_IDLE_ACT && idle != I8_IDLE_MMA) return fail(KQ_ERR_INVALID_ARG, "%s: idle=%d is not 1 or 2", fn, idle);
    if (wait_limit_ns < 1000 || wait_limit_ns > 1000000000)
        return fail(KQ_ERR_INVALID_ARG, "%s: wait_limit_ns must be in [1e3, 1e9]", fn);
    return i8_gemm(fn, q, ldq, sx, w, ldw, sw, nullptr, M, N, K, KQ_F32, y, ldy, workspace, ws_bytes, (cudaStream_t)stream,
                   static_cast<I8Idle>(idle), (unsigned long long)wait_limit_ns);
}

kq_status kq_debug_i8_form(int64_t M, int64_t N, int64_t K, int *ctas, int *tokens, int *splits) {
    const char *fn = "kq_debug_i8_form";
    if (!kq_gemm_i8_workspace_bytes(M, N, K) || !ctas || !tokens || !splits)
        return fail(KQ_ERR_INVALID_ARG, "%s: a shape that kq_gemm_i8 refuses (M=%lld N=%lld K=%lld) or a null pointer", fn, (long long)M,
                    (long long)N, (long long)K);
    const I8Form f = M <= kI8FewTokens ? I8Form{0, 0, 0} : i8_tc_form(M, N, K);
    *ctas = f.ctas;
    *tokens = f.tokens;
    *splits = f.splits;
    return KQ_OK;
}

kq_status kq_gemm_i8_dyn(kq_dtype xt, const void *x, int64_t ldx, const int8_t *w, int64_t ldw, const float *sw,
                         const float *bias, int64_t M, int64_t N, int64_t K, kq_dtype yt, void *y, int64_t ldy,
                         void *workspace, size_t ws_bytes, kq_stream_t stream) {
    const char *fn = "kq_gemm_i8_dyn";
    kq_status s = i8_check_rows(fn, xt, x, M, K, ldx);
    if (s == KQ_OK) s = i8_check_product(fn, w, ldw, sw, bias, M, N, K, yt, y, ldy, workspace, ws_bytes);
    if (s != KQ_OK) return s;
    const cudaStream_t st = (cudaStream_t)stream;
    const I8Workspace l = i8_workspace(M, K);
    uint8_t *b = static_cast<uint8_t *>(workspace);
    float *sx = reinterpret_cast<float *>(b + l.scale);
    unsigned long long *err = static_cast<unsigned long long *>(workspace);
    if (i8_gemv_quantizes(M, K))
        return i8_gemv_rows(fn, xt, {x, ldx, nullptr, w, ldw, sw, bias, M, N, K, yt, y, ldy, err, false}, st);
    if (M <= kI8DirectTokens) {
        int8_t *q = reinterpret_cast<int8_t *>(b + l.codes);
        s = i8_quant(fn, xt, x, M, K, ldx, q, l.ld, l.ld, sx, static_cast<unsigned long long *>(nullptr), st);
        if (s != KQ_OK) return s;
        if (M > kI8FewTokens)
            return i8_tc_product(fn, {q, l.ld, nullptr, 0, sx, w, ldw, sw, bias, M, N, K, yt, y, ldy, err, true}, st);
        return i8_gemv(fn, {q, l.ld, sx, w, ldw, sw, bias, M, N, K, yt, y, ldy, err, true}, st);
    }
    __half *panel = reinterpret_cast<__half *>(b + l.codes);
    s = i8_quant(fn, xt, x, M, K, ldx, panel, l.ld, l.ld, sx, err, st);
    return s != KQ_OK ? s : i8_tc_product(fn, {nullptr, 0, panel, l.ld, sx, w, ldw, sw, bias, M, N, K, yt, y, ldy, err, true}, st);
}

}  // extern "C"
