// kq_attn_prompt.cuh -- attention over whole prompts: what its kernels share (internal).
#pragma once
#include "kq_value.cuh"

namespace kq {

struct PaParams {
    const void *q, *k, *v;
    void *y;
    int64_t ldq, ldk, ldv, ldy;
    const int32_t *cu_q, *cu_k;  // [B + 1]
    int64_t B, Tq, Tk;
    int n_q, G, D;               // query heads, those of a key head, elements
    float scale;                 // its magnitude times log2 e, above 0
    bool negate;                 // it is negative: the scores' signs turn
    bool causal;
    unsigned long long *err;     // device flag, cleared by the call
};

// Running maxima are those of the scores as the products give them (their signs turned where the scale is negative), and
// weights are 2^((s - m) * scale): at any scale a row's largest weight is then 1, and nothing but s itself can leave fp32.
constexpr float kPaNone = -3.402823466e38f;  // the maximum of no key: no finite score is below it

// Some tokens of one sequence: `first` on of its n_q, with its n_k keys.
struct PaTile {
    int64_t q_row, k_row;
    int n_q, n_k, first;
};

__device__ __forceinline__ int64_t pa_row(const int32_t *cu, int64_t b, int64_t T) {
    const int64_t r = cu[b];
    return r < 0 ? 0 : r > T ? T : r;
}
// Tile `unit` of `size` tokens: sequence b's tiles start at floor(cu_q[b] / size) + b, which leaves room for them all.
// All threads of the block call it; false where there is no such tile.
template <int THREADS>
__device__ __forceinline__ bool pa_tile(const PaParams &P, int64_t unit, int size, PaTile &t) {
    int64_t b = 0;
    for (int64_t n = P.B;;) {  // the sequence is one of n from b on
        const int64_t step = (n + THREADS - 1) / THREADS, at = threadIdx.x * step;
        const int k = __syncthreads_count(at < n && pa_row(P.cu_q, b + at, P.Tq) / size + b + at <= unit) - 1;
        if (k < 0) return false;
        b += k * step;
        if (step == 1) break;
        n = min(step, n - k * step);
    }
    t.q_row = pa_row(P.cu_q, b, P.Tq);
    t.k_row = pa_row(P.cu_k, b, P.Tk);
    const int64_t first = (unit - t.q_row / size - b) * size;
    const int64_t n_q = pa_row(P.cu_q, b + 1, P.Tq) - t.q_row, n_k = pa_row(P.cu_k, b + 1, P.Tk) - t.k_row;
    if (first >= n_q) return false;
    t.n_q = (int)n_q;
    t.n_k = n_k > 0 ? (int)n_k : 0;
    t.first = (int)first;
    return true;
}
// The keys that token i of the sequence sees: those below this (the last token sees them all where causal).
__device__ __forceinline__ int pa_limit(const PaParams &P, const PaTile &t, int i) {
    if (i >= t.n_q) return 0;
    if (!P.causal) return t.n_k;
    const int n = t.n_k - t.n_q + 1 + i;
    return n > 0 ? n : 0;
}

// The tensor-core form (kq_attn_tc.cu): which rows it takes, and the launch.  wait_ns limits every wait of its pipeline;
// idle names a role that does nothing (test hook: 1 what brings tiles, 2 what issues the products, 4 the second row
// tile's second ones alone, others none).
constexpr unsigned long long kPtWaitNs = 2000000000ull;
bool pa_aligned(const PaParams &P);  // all rows on 16 bytes
bool pa_takes_tc(const PaParams &P);
size_t pa_tc_workspace(int64_t B, int64_t Tq, int64_t G);
// Either form numbers its units in 32 bits: pairs of row tiles times key heads here, row tiles times heads in the other.
constexpr int64_t kPaMaxUnits = 0x7fffffff;
int64_t pa_tc_units(int64_t B, int64_t Tq, int64_t n_q, int64_t n_kv);
kq_status pa_tc(const char *fn, kq_dtype xt, const PaParams &P, unsigned long long wait_ns, int idle, cudaStream_t st);

}  // namespace kq
