// kq_i8_gemv.cuh -- int8 product of a few tokens: the weights streamed once through dp4a (internal).
#pragma once
#include "kq_value.cuh"

namespace kq {

constexpr int kI8FewTokens = 8;

struct I8GemvArgs {
    const int8_t *q;  // [M][ldq]
    int64_t ldq;
    const float *sx;
    const int8_t *w;  // [N][ldw]
    int64_t ldw;
    const float *sw, *bias;
    int64_t M, N, K;  // M <= kI8FewTokens
    kq_dtype yt;
    void *y;
    int64_t ldy;
    unsigned long long *err;  // device flag, cleared here
    bool after_quant;         // q and sx are written by the kernel just before: start beside it
};
kq_status i8_gemv(const char *fn, const I8GemvArgs &a, cudaStream_t st);

}  // namespace kq
