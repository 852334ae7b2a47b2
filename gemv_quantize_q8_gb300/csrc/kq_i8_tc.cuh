// kq_i8_tc.cuh -- tensor-core (tcgen05) int8 product with scales per token and channel (internal).
#pragma once
#include "kq_value.cuh"

namespace kq {

// Wall-time limit of every wait of the pipeline: past it the CTA counts an error in the device flag, lets its copies and
// MMAs in flight end, and leaves.
constexpr unsigned long long kI8WaitNs = 2000000000ull;
// Test hook: a role that does nothing, so that what waits for it runs into the limit.
enum I8Idle { I8_IDLE_NONE = 0, I8_IDLE_ACT = 1, I8_IDLE_MMA = 2 };

// Tokens up to which the kernel takes int8 codes as they are; more come as an f16 panel.
constexpr int kI8DirectTokens = 64;

// Four codes to four f16.  A byte under a 0x64 high byte is the f16 1024 + byte, so with the sign bit
// flipped it is 1152 + c, and one subtraction gives c exactly.
__device__ __forceinline__ void i8x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
}

struct I8TcArgs {
    const int8_t *q;      // M <= kI8DirectTokens: codes [M][ldq], ldq a multiple of 16
    int64_t ldq;
    const __half *panel;  // M above that: codes as f16 [M][ldp], ldp a multiple of 64, zeros from K to ldp
    int64_t ldp;
    const float *sx;      // [M]
    const int8_t *w;      // [N][ldw]
    int64_t ldw;
    const float *sw, *bias;
    int64_t M, N, K;
    kq_dtype yt;
    void *y;
    int64_t ldy;
    unsigned long long *err;  // device flag: cleared here (int8 codes) or by the panel's kernel
    bool after_prologue;      // the kernel just before is the quantizer or the panel's: the weights may be read before its end
    unsigned long long wait_ns = kI8WaitNs;
    I8Idle idle = I8_IDLE_NONE;  // other than none: the flag has been cleared before
};
// The form that a product takes: CTAs that share a tile's rows, tokens of a tile, CTAs that share its K.
struct I8Form {
    int ctas, tokens, splits;
};
I8Form i8_tc_form(int64_t M, int64_t N, int64_t K);
kq_status i8_tc_product(const char *fn, const I8TcArgs &a, cudaStream_t st);

}  // namespace kq
