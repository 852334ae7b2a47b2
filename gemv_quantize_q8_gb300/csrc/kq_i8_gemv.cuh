// kq_i8_gemv.cuh -- int8 product of a few tokens: the weights streamed once through dp4a (internal).
#pragma once
#include "kq_value.cuh"

namespace kq {

constexpr int kI8FewTokens = 8;

struct I8GemvArgs {
    const void *rows;  // codes [M][ldq], or (i8_gemv_rows) rows of another type
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
    bool after_quant;         // the kernel just before is the quantizer: the weights may be read before its end
};
kq_status i8_gemv(const char *fn, const I8GemvArgs &a, cudaStream_t st);
// The same from rows of type xt, quantised by the product's own blocks (sx unused): where the rows are so
// short that every block can do it again (16384 elements, some 1 us, against a launch).
bool i8_gemv_quantizes(int64_t M, int64_t K);
kq_status i8_gemv_rows(const char *fn, kq_dtype xt, const I8GemvArgs &a, cudaStream_t st);

}  // namespace kq
