// kq_i8_tc.cuh -- tensor-core (tcgen05) int8 product with scales per token and channel (internal).
#pragma once
#include "kq_value.cuh"

namespace kq {

// Tokens up to which the kernel takes int8 codes as they are; more come as an f16 panel.
constexpr int kI8DirectTokens = 64;

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
    bool after_prologue;      // the kernel just before is this library's own (quantizer or panel): start beside it
};
kq_status i8_tc_product(const char *fn, const I8TcArgs &a, cudaStream_t st);

}  // namespace kq
