// kq_i8_quant.cuh -- the arithmetic of the per-token int8 quantizer, shared by its kernels (internal).
#pragma once
#include "kq_value.cuh"

namespace kq {

// A row's scale and the factor of its codes from its largest magnitude.  127/amax overflows below 3.74e-37:
// such a row is the zero row.
struct I8Scale {
    float scale, inv;
};
__device__ __forceinline__ I8Scale i8_scale(float amax) {
    const float inv = __fdiv_rn(127.0f, amax);
    if (isinf(inv)) return {0.0f, 0.0f};
    return {__fdiv_rn(amax, 127.0f), inv};
}
__device__ __forceinline__ int i8_code(float x, float inv) {
    const float v = __fmul_rn(x, inv);
    return isnan(v) ? 0 : __float2int_rn(v);
}

// This thread's part of a row's largest magnitude (thread tid of n; 16-byte loads where the row allows them).
template <typename T>
__device__ __forceinline__ float i8_amax(const T *x, int K, int tid, int n) {
    constexpr int VEC = kVec<T>;
    float a = 0.0f;
    const int nv = (reinterpret_cast<uintptr_t>(x) & 15) == 0 ? K / VEC : 0;
    for (int i = tid; i < nv; i += n) {
        float v[VEC];
        unpack16<T>(reinterpret_cast<const uint4 *>(x)[i], v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a = fmaxf(a, fabsf(v[j]));
    }
    for (int i = nv * VEC + tid; i < K; i += n) a = fmaxf(a, fabsf(to_f32(x[i])));
    return a;
}

__device__ __forceinline__ int8_t i8_as(int c, int8_t) { return (int8_t)c; }
__device__ __forceinline__ __half i8_as(int c, __half) { return __int2half_rn(c); }

// This thread's part of a row's codes, as int8 or f16 (exact), zeros from K to `fill`; q is 16-byte aligned.
template <typename T, typename TQ>
__device__ __forceinline__ void i8_codes(const T *x, int K, int fill, float inv, TQ *q, int tid, int n) {
    constexpr int VEC = kVec<T>;
    using Vec = typename VecOf<VEC * (int)sizeof(TQ)>::type;
    const int nv = (reinterpret_cast<uintptr_t>(x) & 15) == 0 ? K / VEC : 0;
    for (int i = tid; i < nv; i += n) {
        float v[VEC];
        unpack16<T>(reinterpret_cast<const uint4 *>(x)[i], v);
        Vec o;
#pragma unroll
        for (int j = 0; j < VEC; ++j) reinterpret_cast<TQ *>(&o)[j] = i8_as(i8_code(v[j], inv), TQ{});
        reinterpret_cast<Vec *>(q)[i] = o;
    }
    for (int i = nv * VEC + tid; i < fill; i += n) q[i] = i8_as(i < K ? i8_code(to_f32(x[i]), inv) : 0, TQ{});
}

}  // namespace kq
