// kq_kv.cuh -- the paged 8-bit cache of keys and values (internal).
//
// A page holds `page` consecutive tokens of one sequence; keys and values are int8 [n_pages][n_kv][page][D] with
// one fp32 scale for each page and head, [n_pages][n_kv]: the block that a page and head make is contiguous, so
// whatever reads or writes it moves whole rows of D bytes, D a multiple of 16.
#pragma once
#include "kq_value.cuh"

namespace kq {

constexpr int kKvMaxD = 256, kKvMaxPage = 256, kKvMaxHeads = 1024;

struct KvCache {
    int8_t *k, *v;
    float *k_scale, *v_scale;
    const int32_t *table;  // [B][ldt] page numbers
    const int32_t *lens;   // [B] tokens in the cache, a call's new ones among them
    int64_t n_pages, ldt, B;
    int n_kv, D, lp;       // heads; elements; log2 of a page's tokens
};

// Checks the cache's arguments and fills c.
kq_status kv_check(const char *fn, const int8_t *k_cache, const int8_t *v_cache, const float *k_scale, const float *v_scale,
                   int64_t n_pages, int64_t page, const int32_t *table, int64_t ldt, const int32_t *lens, int64_t B,
                   int64_t n_kv, int64_t D, KvCache &c);

// Rows of sequence b in a packed batch of T rows: from cu[b] to cu[b+1], or T/B each where cu is NULL.
__device__ __forceinline__ int64_t kv_row(const int32_t *cu, int64_t b, int64_t B, int64_t T) {
    if (!cu) return b * (T / B);
    const int64_t r = cu[b];
    return r < 0 ? 0 : r > T ? T : r;
}

}  // namespace kq
