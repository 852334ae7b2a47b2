// kq_value.cuh -- plain rows of fp32, f16 or bf16 elements: loads to fp32 and stores rounded to the type.
#pragma once
#include <cuda_bf16.h>

#include "kq_internal.cuh"

namespace kq {

inline bool is_value_type(kq_dtype t) { return t == KQ_F32 || t == KQ_F16 || t == KQ_BF16; }
inline size_t value_bytes(kq_dtype t) { return t == KQ_F32 ? 4 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)), "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}

// Elements of a 16-byte vector, and their values.
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);
template <typename T>
__device__ __forceinline__ void unpack16(uint4 u, float (&v)[kVec<T>]) {
    const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) v[i] = to_f32(e[i]);
}

// The type that moves 4, 8 or 16 bytes at once.
template <int BYTES> struct VecOf;
template <> struct VecOf<4> { using type = uint32_t; };
template <> struct VecOf<8> { using type = uint2; };
template <> struct VecOf<16> { using type = uint4; };

// Calls f with a value of the C++ type of t (t is one of the three).
template <typename F>
inline kq_status with_type(kq_dtype t, F f) {
    return t == KQ_F32 ? f(float{}) : t == KQ_F16 ? f(__half{}) : f(__nv_bfloat16{});
}

}  // namespace kq
