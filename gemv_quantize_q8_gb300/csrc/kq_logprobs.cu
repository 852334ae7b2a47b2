// kq_logprobs.cu -- log probabilities of given tokens, with the entropy and the top alternatives of a row,
// in one pass over the logits.
//
// Bound by the logits' bytes.  Every thread keeps a running maximum m and, relative to it,
//   S = sum 2^d,  T = sum 2^d * d,   d = max((x - m) * log2 e, -200)
// over batches of 16 elements: a batch's own maximum is taken first, and only when it is above m are S and T
// brought to the new one:  S' = f S,  T' = f (T + delta S),  delta = (m - m') log2 e,  f = 2^delta.  Threads,
// and the CTAs of a cluster that share a row when there are few rows, are joined the same way.  Then
//   log Z = m + ln S,   entropy = ln S - (T / S) ln 2.
// (The bound -200 stands for -inf: 2^-200 is 0 in fp32, and 0 * -200 is, unlike 0 * -inf, 0.)
//
// Alternatives: a thread also keeps its largest logit.  The k-th largest of 32 such maxima (eight threads
// each) is reached by k elements at least, and by few more (31 expected for k = 20, 130 for 32); so when the row has been read, only the threads whose
// maximum reaches it name the batches to look through again: those that reached the same bound of the first
// round (a bit each).  What is found there goes to a buffer in shared memory; should it
// overflow (a sorted row, a row of equals), its k-th best becomes the bound and they look again.  Order and
// ties are one 64-bit number: the logit in order-preserving bits, then the inverted id.  Masked tokens (-inf)
// and NaN are never candidates; a row with fewer than k others takes the first of them at the end.
#include <cooperative_groups.h>
#include <math.h>

#include "kq_launch.cuh"
#include "kq_value.cuh"

namespace kq {

constexpr int kLpThreads = 256;
constexpr int kLpMaxTop = 32;
constexpr int kLpBatch = 16;                        // elements whose maximum a thread takes at once
constexpr int kLpVecs = 4;                          // 16-byte vectors of a thread in a round: 64 bytes under way
constexpr int kLpMaxParts = 8;                      // CTAs that share a row (portable cluster size)
constexpr int kLpCap = 2048;                        // candidates that the buffer holds
constexpr int kLpFew = 256;                         // candidates that are ranked without a filter
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kLowest = -3.4028234663852886e38f;

// NaN ranks with -inf, -0 with +0.
__device__ __forceinline__ uint64_t lp_key(float x, int id) {
    if (isnan(x)) x = -INFINITY;
    uint32_t b = __float_as_uint(x + 0.0f);
    b = (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return ((uint64_t)b << 32) | (uint32_t)~id;
}
__device__ __forceinline__ int lp_key_id(uint64_t k) { return (int)~(uint32_t)k; }
__device__ __forceinline__ float lp_key_value(uint64_t k) {
    const uint32_t b = (uint32_t)(k >> 32);
    return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}

struct LpStats {
    float m, S, T, bad;  // bad != 0: a NaN was seen
};
__device__ __forceinline__ void lp_raise(LpStats &s, float m) {
    const float delta = fmaxf((s.m - m) * kLog2e, -200.0f), f = exp2_fast(delta);
    s.T = f * (s.T + delta * s.S);
    s.S *= f;
    s.m = m;
}
__device__ __forceinline__ LpStats lp_join(LpStats a, LpStats b) {
    const float m = fmaxf(a.m, b.m);
    if (a.m < m) lp_raise(a, m);
    if (b.m < m) lp_raise(b, m);
    return {m, a.S + b.S, a.T + b.T, a.bad + b.bad};
}

struct LpShared {
    LpStats warp[kLpThreads / 32], row;
    __align__(16) float part[32];
    uint64_t best[kLpMaxTop];
    int count, items;
};

// The k best of the buffer's n candidates to sh.best, best first (0 where there are fewer).  All threads.
__device__ __noinline__ void lp_cut(uint64_t *buf, int n, int k, LpShared &sh) {
    const int tid = threadIdx.x;
    __syncthreads();
    if (n > kLpFew) {
        // drop those below the k-th largest of 32 maxima over disjoint parts: k of them reach it
        uint64_t top = 0;
        for (int i = tid; i < n; i += kLpThreads) top = buf[i] > top ? buf[i] : top;
#pragma unroll
        for (int s = 1; s < 8; s *= 2) {
            const uint64_t o = __shfl_xor_sync(~0u, top, s);
            top = o > top ? o : top;
        }
        if ((tid & 7) == 0) sh.best[tid >> 3] = top;
        if (tid == 0) sh.count = 0;
        __syncthreads();
        const uint64_t mine = sh.best[tid & 31];
        int rank = 0;
        for (int i = 0; i < 32; ++i) {
            const uint64_t o = __shfl_sync(~0u, mine, i);
            rank += o > mine || (o == mine && i < (tid & 31));
        }
        const uint64_t least = __shfl_sync(~0u, mine, __ffs(__ballot_sync(~0u, rank == k - 1)) - 1);
        // in place: what a piece of the buffer keeps fits where that piece and those before it were
        for (int i0 = 0; i0 < n; i0 += kLpThreads) {
            const uint64_t key = i0 + tid < n ? buf[i0 + tid] : 0;
            const bool stays = key && key >= least;
            __syncthreads();
            const unsigned votes = __ballot_sync(~0u, stays);
            int at = 0;
            if ((tid & 31) == 0 && votes) at = atomicAdd(&sh.count, __popc(votes));
            at = __shfl_sync(~0u, at, 0) + __popc(votes & ((1u << (tid & 31)) - 1u));
            if (stays) buf[at] = key;
        }
        __syncthreads();
        n = sh.count;
    }
    if (tid < kLpMaxTop) sh.best[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kLpThreads) {
        const uint64_t key = buf[i];
        int rank = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank += buf[j] > key;
        if (rank < k) sh.best[rank] = key;
    }
    __syncthreads();
}

struct LpParams {
    const void *x;
    int64_t ldx;
    int V;
    const int32_t *targets;
    int n_targets;
    float *logprob, *entropy;
    int top_k;
    int32_t *top_ids;
    float *top_logprob;
    int64_t row0;
};

// The k-th largest of 32 maxima of the block's values, eight threads each.  All threads.
__device__ __forceinline__ float lp_kth(float v, int k, LpShared &sh) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int s = 1; s < 8; s *= 2) v = fmaxf(v, __shfl_xor_sync(~0u, v, s));
    __syncthreads();
    if ((threadIdx.x & 7) == 0) sh.part[threadIdx.x >> 3] = v;
    __syncthreads();
    v = sh.part[lane];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const float4 o = *reinterpret_cast<const float4 *>(sh.part + i);
        rank += (o.x > v || (o.x == v && i < lane)) + (o.y > v || (o.y == v && i + 1 < lane)) +
                (o.z > v || (o.z == v && i + 2 < lane)) + (o.w > v || (o.w == v && i + 3 < lane));
    }
    return __shfl_sync(~0u, v, __ffs(__ballot_sync(~0u, rank == k - 1)) - 1);
}

// One cluster (gridDim.x CTAs, one or more) a row; blockIdx.y the row.  DEPTH rounds of loads are under way: one
// where four or five CTAs share an SM, more where there are too few CTAs for that (300 rows of 32000 fp32, five
// alternatives: 12.1 us with one, 11.1 with three; 167 rows of 49999 f16, eight alternatives: 17.0 and 15.1).
template <typename T, bool TOP, int DEPTH>
__global__ void __launch_bounds__(kLpThreads, DEPTH == 1 ? (TOP ? 4 : 5) : DEPTH == 2 ? 3 : 2) lp_kernel(LpParams P) {
    constexpr int VEC = kVec<T>, NV = kLpVecs, NB = kLpBatch / VEC;  // NB: vectors of a batch
    extern __shared__ uint64_t buf[];  // TOP: kLpCap candidates, then the list of batches
    uint16_t *list = reinterpret_cast<uint16_t *>(buf + kLpCap);
    __shared__ LpShared sh;
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, part = blockIdx.x, parts = gridDim.x;
    const int64_t row = P.row0 + blockIdx.y;
    const T *x = static_cast<const T *>(P.x) + row * P.ldx;
    const int V = P.V, k = P.top_k;
    const float none = -INFINITY;
    // vectors from the first 16-byte boundary on; the few elements before and after them go separately
    const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T));
    const int nvec = (V - head) / VEC, rest = V - nvec * VEC;
    const int v0 = (int)((int64_t)nvec * part / parts), v1 = (int)((int64_t)nvec * (part + 1) / parts);

    LpStats st = {kLowest, 0.0f, 0.0f, 0.0f};
    float2 S2 = make_float2(0.0f, 0.0f), T2 = S2;
    // The statistics of a batch; returns its maximum (-inf for nothing but NaN and -inf).
    auto count_in = [&](const float (&v)[kLpBatch]) {
        float top = max_nan(v[0], v[1], v[1]);
#pragma unroll
        for (int i = 2; i < kLpBatch; i += 2) top = max_nan(top, v[i], v[i + 1]);
        if (!(top <= st.m)) {
            if (isnan(top)) {
                st.bad = 1.0f;
                top = none;
#pragma unroll
                for (int i = 0; i < kLpBatch; ++i) top = fmaxf(top, v[i]);
            }
            if (top > st.m) {
                st.S = S2.x + S2.y;
                st.T = T2.x + T2.y;
                lp_raise(st, top);
                S2 = make_float2(st.S, 0.0f);
                T2 = make_float2(st.T, 0.0f);
            }
        }
        const float2 minus = make_float2(-st.m, -st.m), l2e = make_float2(kLog2e, kLog2e);
#pragma unroll
        for (int i = 0; i < kLpBatch; i += 2) {
            float2 d = mul2(add2(make_float2(v[i], v[i + 1]), minus), l2e);
            d.x = fmaxf(d.x, -200.0f);
            d.y = fmaxf(d.y, -200.0f);
            const float2 e = make_float2(exp2_fast(d.x), exp2_fast(d.y));
            S2 = add2(S2, e);
            T2 = fma2(e, d, T2);
        }
        return top;
    };

    const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
    uint4 next[DEPTH][NV];
    auto fetch = [&](int d, int u0, int v) {  // vectors u0 .. u0 + NB - 1 of the round at v
#pragma unroll
        for (int u = u0; u < u0 + NB; ++u)
            if (v + u * kLpThreads < v1) next[d][u] = TOP ? __ldg(xv + v + u * kLpThreads) : __ldcs(xv + v + u * kLpThreads);
    };
    const int rounds = (v1 - v0 + NV * kLpThreads - 1) / (NV * kLpThreads);
    int shift = 0;  // rounds of one bit of `worth`
    while ((rounds - 1) >> shift >= 32) ++shift;
    float largest = none, bound = none;
    uint32_t worth = 0;  // rounds (in groups) in which this thread's batch reached the bound
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
#pragma unroll
        for (int u0 = 0; u0 < NV; u0 += NB) fetch(d, u0, v0 + tid + d * NV * kLpThreads);
    for (int j0 = 0; j0 < rounds; j0 += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const int j = j0 + d, at = v0 + tid + j * NV * kLpThreads;
            if (j >= rounds) break;
            float top = none;
#pragma unroll
            for (int u0 = 0; u0 < NV; u0 += NB) {
                float v[kLpBatch];
#pragma unroll
                for (int u = 0; u < NB; ++u) {
                    float f[VEC];
                    unpack16<T>(next[d][u0 + u], f);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[u * VEC + i] = f[i];
                }
                if (j + 1 == rounds) {  // the last round may be short
#pragma unroll
                    for (int i = 0; i < kLpBatch; ++i)
                        if (at + (u0 + i / VEC) * kLpThreads >= v1) v[i] = none;
                }
                fetch(d, u0, at + DEPTH * NV * kLpThreads);
                top = fmaxf(top, count_in(v));
            }
            if (TOP) {
                largest = fmaxf(largest, top);
                if (top >= bound) worth |= 1u << (j >> shift);
                if (j == 0 && rounds > 1) bound = lp_kth(largest, k, sh);
            }
        }
    }
    const int odd_id = part == 0 && tid < rest ? (tid < head ? tid : nvec * VEC + tid) : -1;
    float odd = none;  // elements before the first vector and after the last: one a thread
    if (part == 0 && rest) {
        float v[kLpBatch];
#pragma unroll
        for (int i = 0; i < kLpBatch; ++i) v[i] = none;
        if (odd_id >= 0) v[0] = odd = to_f32(x[odd_id]);
        largest = fmaxf(largest, count_in(v));
    }
    if (TOP) {
        float least_value = fmaxf(lp_kth(largest, k, sh), kLowest);  // never -inf
        uint64_t least = lp_key(least_value, -1);                    // the lowest key of that value
        for (;;) {
            if (tid == 0) sh.count = sh.items = 0;
            __syncthreads();
            auto put = [&](float v, int id) {
                if (!(v >= least_value)) return;
                const uint64_t key = lp_key(v, id);
                if (key < least) return;
                const int at = atomicAdd(&sh.count, 1);
                if (at < kLpCap) buf[at] = key;
            };
            // The batches to look through go on a list, so that all threads share their loads (by the thread that
            // found them, one after the other, they took longer than the row: 295 us for 157 + 42).
            if (largest >= least_value) {
                int at = atomicAdd(&sh.items, __popc(worth));
                for (uint32_t w = worth; w; w &= w - 1) list[at++] = (uint16_t)(tid * 32 + __ffs(w) - 1);
            }
            __syncthreads();
            const int vectors = sh.items * NV;
            for (int i = tid; i < vectors; i += kLpThreads) {
                const int item = list[i / NV], bit = item & 31;
                for (int j = bit << shift; j < min(rounds, (bit + 1) << shift); ++j) {
                    const int at = v0 + (item >> 5) + (j * NV + i % NV) * kLpThreads;
                    if (at >= v1 || *reinterpret_cast<volatile int *>(&sh.count) > kLpCap) break;
                    float f[VEC];
                    unpack16<T>(__ldg(xv + at), f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) put(f[e], head + at * VEC + e);
                }
            }
            if (odd_id >= 0) put(odd, odd_id);
            __syncthreads();
            const int n = sh.count;
            lp_cut(buf, min(n, kLpCap), k, sh);
            if (n <= kLpCap) break;
            least = sh.best[k - 1];
            least_value = lp_key_value(least);
            __syncthreads();
        }
    }

    // the threads' statistics, then (several CTAs a row) the cluster's, and its candidates
    st.S = S2.x + S2.y;
    st.T = T2.x + T2.y;
#pragma unroll
    for (int s = 16; s; s >>= 1)
        st = lp_join(st, {__shfl_xor_sync(~0u, st.m, s), __shfl_xor_sync(~0u, st.S, s), __shfl_xor_sync(~0u, st.T, s),
                          __shfl_xor_sync(~0u, st.bad, s)});
    if (lane == 0) sh.warp[tid >> 5] = st;
    __syncthreads();
    st = sh.warp[lane % (kLpThreads / 32)];
#pragma unroll
    for (int s = kLpThreads / 64; s; s >>= 1)
        st = lp_join(st, {__shfl_xor_sync(~0u, st.m, s), __shfl_xor_sync(~0u, st.S, s), __shfl_xor_sync(~0u, st.T, s),
                          __shfl_xor_sync(~0u, st.bad, s)});
    if (parts > 1) {
        namespace cg = cooperative_groups;
        cg::cluster_group cluster = cg::this_cluster();
        if (tid == 0) sh.row = st;
        cluster.sync();
        if (part == 0) {
            for (int i = 1; i < parts; ++i) st = lp_join(st, cluster.map_shared_rank(&sh, i)->row);
            if (TOP && tid < parts * k) buf[tid] = cluster.map_shared_rank(&sh, tid / k)->best[tid % k];  // at most 8 * 32
        }
        cluster.sync();
        if (part) return;
        if (TOP) {
            // an element's place in the merged lists: what precedes it in each (their empty ends are zeros)
            const uint64_t key = tid < parts * k ? buf[tid] : 0;
            int lo[kLpMaxParts] = {}, place = 0;  // the searches go side by side: their loads overlap
#pragma unroll
            for (int step = 32; step; step >>= 1)
#pragma unroll
                for (int i = 0; i < kLpMaxParts; ++i)
                    if (i < parts && lo[i] + step <= k && buf[i * k + lo[i] + step - 1] > key) lo[i] += step;
#pragma unroll
            for (int i = 0; i < kLpMaxParts; ++i) place += lo[i];
            if (tid < kLpMaxTop) sh.best[tid] = 0;
            __syncthreads();
            if (key && place < k) sh.best[place] = key;
            __syncthreads();
        }
    }

    const bool bad = st.bad != 0.0f || st.m == INFINITY, empty = st.S == 0.0f;
    const float logS = logf(st.S);
    auto lp_of = [&](float v) { return bad ? NAN : empty ? -INFINITY : (v - st.m) - logS; };
    if (tid == 0 && P.entropy) P.entropy[row] = bad ? NAN : empty ? 0.0f : logS - st.T / st.S * kLn2;
    for (int j = tid; j < P.n_targets; j += kLpThreads) {
        const int t = P.targets[row * P.n_targets + j];
        P.logprob[row * P.n_targets + j] = t < 0 ? 0.0f : t >= V ? NAN : lp_of(to_f32(x[t]));
    }
    // from here on the list is warp 0's alone (it has 32 entries at most)
    if (TOP && tid < 32) {
        int n = __popc(__ballot_sync(~0u, sh.best[lane] != 0));
        // fewer than k tokens are neither masked nor NaN: the first of those fill up, in the order of their ids
        for (int i = 0; i < V && n < k; i += 32) {
            const float v = i + lane < V ? to_f32(x[i + lane]) : 0.0f;
            const bool low = isnan(v) || v == none;
            const unsigned votes = __ballot_sync(~0u, low);
            const int at = n + __popc(votes & ((1u << lane) - 1u));
            if (low && at < k) sh.best[at] = lp_key(none, i + lane);
            n += __popc(votes);
        }
        __syncwarp();
        if (lane < k) {
            const uint64_t key = sh.best[lane];
            P.top_ids[row * k + lane] = lp_key_id(key);
            P.top_logprob[row * k + lane] = lp_of(lp_key_value(key));
        }
    }
}

template <typename T, bool TOP, int DEPTH>
static kq_status launch_lp(const char *fn, LpParams P, int64_t M, int parts, cudaStream_t st) {
    constexpr int smem = TOP ? kLpCap * 8 + kLpThreads * 32 * 2 : 0;
    auto kern = lp_kernel<T, TOP, DEPTH>;
    cudaError_t e = smem ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
    for (int64_t r = 0; e == cudaSuccess && r < M; r += 65535) {  // the grid's second dimension ends there
        P.row0 = r;
        e = launch_beside(kern, dim3((unsigned)parts, (unsigned)(M - r < 65535 ? M - r : 65535)), dim3(kLpThreads), smem,
                          dim3((unsigned)parts), st, P);
        if (e == cudaSuccess) count_launch(R_LOGPROBS);
    }
    return e == cudaSuccess ? KQ_OK : fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
}

template <typename T, bool TOP>
static kq_status share_rows(const char *fn, const LpParams &P, int64_t M, cudaStream_t st) {
    // CTAs that share a row: doubled up to two and a half an SM, while each has a whole round of its own (rows from
    // memory, 64 of 131072 bf16, 20 alternatives: four a row 13.4 us, eight 16.1, two 13.7; 167 of 49999 f16: two
    // 15.1, four 19.5, but one 11.8)
    int parts = 1;
    while (parts < kLpMaxParts && M * parts * 2 <= 380 && P.V >= parts * 2 * kLpThreads * kLpVecs * kVec<T>) parts *= 2;
    // as many CTAs an SM as it takes to hold them all, not more: they then spread over the SMs (64 rows as above:
    // 13.4 us with two an SM, 15.9 where a third would fit)
    if (M * parts <= 152 * 2) return launch_lp<T, TOP, 3>(fn, P, M, parts, st);
    if (M * parts <= 152 * 3) return launch_lp<T, TOP, 2>(fn, P, M, parts, st);
    return launch_lp<T, TOP, 1>(fn, P, M, parts, st);
}

}  // namespace kq

using namespace kq;

extern "C" kq_status kq_logprobs(kq_dtype xt, const void *logits, int64_t ldx, int64_t M, int64_t V,
                                 const int32_t *targets, int64_t n_targets, float *logprob, float *entropy,
                                 int64_t top_k, int32_t *top_ids, float *top_logprob, kq_stream_t stream) {
    const char *fn = "kq_logprobs";
    if (!is_value_type(xt))
        return fail(KQ_ERR_UNSUPPORTED_DTYPE, "%s: logits type %s is not F32, F16 or BF16", fn, dtype_name(xt));
    if (!logits) return fail(KQ_ERR_INVALID_ARG, "%s: null logits", fn);
    if (M <= 0 || M > 0x7fffffff || V <= 0 || V > (1 << 30) || ldx < V)
        return fail(KQ_ERR_INVALID_ARG, "%s: need M > 0, 0 < V <= 2^30 and ldx >= V (M=%lld V=%lld ldx=%lld)", fn,
                    (long long)M, (long long)V, (long long)ldx);
    if (n_targets < 0 || n_targets > V || (n_targets && (!targets || !logprob)))
        return fail(KQ_ERR_INVALID_ARG, "%s: n_targets=%lld needs targets and logprob, and is 0..V", fn, (long long)n_targets);
    if (top_k < 0 || top_k > kLpMaxTop || top_k > V || (top_k && (!top_ids || !top_logprob)))
        return fail(KQ_ERR_INVALID_ARG, "%s: top_k=%lld needs top_ids and top_logprob, and is 0..min(%d, V)", fn,
                    (long long)top_k, kLpMaxTop);
    if (!aligned(logits, value_bytes(xt)) || (n_targets && (!aligned(targets, 4) || !aligned(logprob, 4))) ||
        (entropy && !aligned(entropy, 4)) || (top_k && (!aligned(top_ids, 4) || !aligned(top_logprob, 4))))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    const LpParams P{logits, ldx, (int)V, targets, (int)n_targets, logprob, entropy, (int)top_k, top_ids, top_logprob, 0};
    return with_type(xt, [&](auto t) {
        using T = decltype(t);
        return top_k ? share_rows<T, true>(fn, P, M, (cudaStream_t)stream) : share_rows<T, false>(fn, P, M, (cudaStream_t)stream);
    });
}
