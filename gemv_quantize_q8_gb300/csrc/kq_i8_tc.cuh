// kq_i8_tc.cuh -- tensor-core (tcgen05) int8 product with scales per token and channel (internal).
#pragma once
#include "kq_value.cuh"

namespace kq {

// One product over an f16 panel of activation codes (exact: |code| <= 128).
struct I8TcArgs {
    const __half *panel;  // [M][ldp] codes as f16, ldp a multiple of 64, zeros from K to ldp
    int64_t ldp;
    const float *sx;      // [M]
    const int8_t *w;      // [N][ldw]
    int64_t ldw;
    const float *sw, *bias;
    int64_t M, N, K;
    kq_dtype yt;
    void *y;
    int64_t ldy;
    unsigned long long *err;  // device flag, cleared by the kernel before this one
};
kq_status i8_tc_product(const char *fn, const I8TcArgs &a, cudaStream_t st);

}  // namespace kq
