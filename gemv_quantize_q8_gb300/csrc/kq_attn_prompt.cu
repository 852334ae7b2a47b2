// kq_attn_prompt.cu -- attention over whole prompts: packed sequences, grouped heads, causal or not.
//
//   y_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = 2^(scale * log2 e * (s_ij - m_i)),   s_ij = q_i . k_j
// over the keys that token i sees, with a running maximum m_i and fp32 sums; weights are rounded to the rows' type for
// the second product (their errors are independent and average out over the keys; the sum below the line is
// of the unrounded ones).
//
// The form for any head width up to 256 and rows at any address: a thread block takes 64 tokens of one head, 16 a
// warp, and goes over the keys in tiles of 32, on m16n8k16 instructions.  Rows on 16 bytes (heads of over 128; the narrower ones
// take kq_attn_tc.cu's form) come by 16-byte copies, the next tile while this one's products run, and both products take
// their operands by ldmatrix: 4096 tokens, 32 heads over 8 of 256, causal, 1045 us, 0.26 PFLOP/s, bound by the instructions' rate
// and their operands' loads.  Other rows are staged element by element: 7.3 ms (16384 tokens of 128: 22.0 ms for 1468 us).
// A masked weight is 0, but 0 times an infinity is not: rows of values past the sequence's end are
// taken as zeros, and a tile that some row sees only in part and that holds an infinity or NaN is added up one key at
// a time, leaving out what is masked.
#include <math.h>

#include "kq_attn_prompt.cuh"
#include "kq_launch.cuh"

namespace kq {

constexpr int kPaRows = 64, kPaKeys = 32, kPaPad = 8;

__device__ __forceinline__ void pa_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void pa_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pa_pair(float x, float y) {
    T v[2] = {from_f32<T>(x), from_f32<T>(y)};
    return *reinterpret_cast<uint32_t *>(v);
}
__device__ __forceinline__ uint32_t pa_word(const void *p) { return *static_cast<const uint32_t *>(p); }

// Four 8 x 8 tiles of 16-bit elements; lane i gives row i % 8 of tile i / 8.
template <bool TRANS>
__device__ __forceinline__ void pa_matrices(const void *row, uint32_t (&r)[4]) {
    const uint32_t at = sm100::smem_u32(row);
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// 16 bytes, or 16 zeros where `in` is false.
__device__ __forceinline__ void pa_copy(void *dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
}

template <int DP, bool VEC>
constexpr int pa_smem() {
    return (kPaRows * (DP + kPaPad) + (VEC ? 4 * kPaKeys * (DP + kPaPad) : kPaKeys * (DP + kPaPad) + DP * (kPaKeys + kPaPad))) * 2;
}

// DP: the head's width rounded up to 64, 128 or 256.  VEC: rows on 16 bytes; then the next tile's keys and values are
// copied while this one's products run, and values stay as they lie (ldmatrix transposes them).
template <typename T, int DP, bool VEC>
__global__ void __launch_bounds__(128) pa_kernel(PaParams P) {
    extern __shared__ uint4 pa_sm[];
    constexpr int LD = DP + kPaPad, LV = kPaKeys + kPaPad;
    T *sq = reinterpret_cast<T *>(pa_sm), *sk = sq + kPaRows * LD, *sv = sk + kPaKeys * LD;  // values transposed: [d][key], unless VEC
    sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3, D = P.D;
    if (P.err && blockIdx.x == 0 && tid == 0) *P.err = 0ull;
    PaTile t;
    // heads side by side (their keys meet in the L2), the last tokens, which see the most, first: 1033 us for 1190
    const unsigned unit = blockIdx.x / (unsigned)P.n_q;
    const int head = (int)(blockIdx.x - unit * (unsigned)P.n_q);
    if (!pa_tile<128>(P, gridDim.x / (unsigned)P.n_q - 1 - unit, kPaRows, t)) return;
    const T *q = static_cast<const T *>(P.q) + (t.q_row + t.first) * P.ldq + (int64_t)head * D;
    const T *k = static_cast<const T *>(P.k) + t.k_row * P.ldk + (int64_t)(head / P.G) * D;
    const T *v = static_cast<const T *>(P.v) + t.k_row * P.ldv + (int64_t)(head / P.G) * D;
    const int rows = min(kPaRows, t.n_q - t.first);
    const T zero = from_f32<T>(0.0f);
    // (VEC) the tile from key j0 on into one of two buffers
    constexpr int TILE = 2 * kPaKeys * LD, PIECES = DP / 8;
    auto stage = [&](int j0, int buffer) {
        for (int i = tid; i < kPaKeys * PIECES; i += 128) {
            const int r = i / PIECES, d = i % PIECES * 8;
            const bool in = j0 + r < t.n_k && d < D;
            T *to = sk + buffer * TILE + r * LD + d;
            pa_copy(to, in ? k + (j0 + r) * P.ldk + d : k, in);
            pa_copy(to + kPaKeys * LD, in ? v + (j0 + r) * P.ldv + d : v, in);
        }
    };
    if constexpr (VEC) {
        for (int i = tid; i < kPaRows * PIECES; i += 128) {
            const int r = i / PIECES, d = i % PIECES * 8;
            const bool in = r < rows && d < D;
            pa_copy(sq + r * LD + d, in ? q + r * P.ldq + d : q, in);
        }
    } else {
        for (int i = tid; i < kPaRows * DP; i += 128) {
            const int r = i / DP, d = i % DP;
            sq[r * LD + d] = r < rows && d < D ? q[r * P.ldq + d] : zero;
        }
    }
    // row r of this lane (0, 1): token first + 16 * warp + g + 8r, which sees the keys below its limit
    int limit[2];
    float m[2] = {kPaNone, kPaNone}, l[2] = {}, o[DP / 8][4] = {};
#pragma unroll
    for (int r = 0; r < 2; ++r) limit[r] = pa_limit(P, t, t.first + 16 * warp + g + 8 * r);
    const int lowest = pa_limit(P, t, t.first), highest = pa_limit(P, t, t.first + rows - 1);
    if (VEC && highest > 0) stage(0, 0);
    if (VEC) asm volatile("cp.async.commit_group;" ::: "memory");
    for (int j0 = 0; j0 < highest; j0 += kPaKeys) {
        __syncthreads();
        bool odd = false;
        if constexpr (VEC) {
            const int buffer = j0 / kPaKeys & 1;
            sk = sq + kPaRows * LD;
            if (j0 + kPaKeys < highest) stage(j0 + kPaKeys, buffer ^ 1);
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory");
            sk += buffer * TILE;
            sv = sk + kPaKeys * LD;
            if (j0 + kPaKeys > lowest)  // (each thread looks at what it has copied)
                for (int i = tid; i < kPaKeys * PIECES; i += 128) {
                    const T *at = sv + i / PIECES * LD + i % PIECES * 8;
#pragma unroll
                    for (int x = 0; x < 8; ++x) odd |= !(fabsf(to_f32(at[x])) < INFINITY);
                }
        } else {
            for (int i = tid; i < kPaKeys * DP; i += 128) {
                const int r = i / DP, d = i % DP;
                const bool in = j0 + r < t.n_k && d < D;
                const T kv = in ? k[(j0 + r) * P.ldk + d] : zero, vv = in ? v[(j0 + r) * P.ldv + d] : zero;
                sk[r * LD + d] = kv;
                sv[d * LV + r] = vv;
                odd |= !(fabsf(to_f32(vv)) < INFINITY);
            }
        }
        // (part of the tile masked for some row, and not finite)
        odd = __syncthreads_or(odd && j0 + kPaKeys > lowest);
        float s[kPaKeys / 8][4] = {};
#pragma unroll
        for (int x = 0; x < DP / 16; ++x) {
            if constexpr (VEC) {
                uint32_t af[4], b[4];
                pa_matrices<false>(sq + (16 * warp + (lane & 15)) * LD + 16 * x + (lane >> 4) * 8, af);
#pragma unroll
                for (int n = 0; n < kPaKeys / 8; n += 2) {
                    pa_matrices<false>(sk + (8 * (n + (lane >> 4)) + (lane & 7)) * LD + 16 * x + (lane >> 3 & 1) * 8, b);
                    pa_mma(s[n], af, b[0], b[1], T{});
                    pa_mma(s[n + 1], af, b[2], b[3], T{});
                }
            } else {
                const T *a = sq + (16 * warp + g) * LD + 16 * x + 2 * c;
                const uint32_t af[4] = {pa_word(a), pa_word(a + 8 * LD), pa_word(a + 8), pa_word(a + 8 * LD + 8)};
#pragma unroll
                for (int n = 0; n < kPaKeys / 8; ++n) {
                    const T *b = sk + (8 * n + g) * LD + 16 * x + 2 * c;
                    pa_mma(s[n], af, pa_word(b), pa_word(b + 8), T{});
                }
            }
        }
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float top = m[r];
#pragma unroll
            for (int n = 0; n < kPaKeys / 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[n][2 * r + e];
                    x = j0 + 8 * n + 2 * c + e < limit[r] ? (P.negate ? -x : x) : -INFINITY;
                    top = fmaxf(top, x);
                }
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            f[r] = exp2f((m[r] - top) * P.scale);
            m[r] = top;
            l[r] *= f[r];
#pragma unroll
            for (int n = 0; n < kPaKeys / 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[n][2 * r + e];
                    x = exp2f((x - top) * P.scale);
                    l[r] += x;
                }
        }
#pragma unroll
        for (int j = 0; j < DP / 8; ++j) {
            o[j][0] *= f[0]; o[j][1] *= f[0]; o[j][2] *= f[1]; o[j][3] *= f[1];
        }
        if (!odd) {
#pragma unroll
            for (int x = 0; x < kPaKeys / 16; ++x) {
                const uint32_t af[4] = {pa_pair<T>(s[2 * x][0], s[2 * x][1]), pa_pair<T>(s[2 * x][2], s[2 * x][3]),
                                        pa_pair<T>(s[2 * x + 1][0], s[2 * x + 1][1]), pa_pair<T>(s[2 * x + 1][2], s[2 * x + 1][3])};
                if constexpr (VEC) {
#pragma unroll
                    for (int j = 0; j < DP / 8; j += 2) {
                        uint32_t b[4];
                        pa_matrices<true>(sv + (16 * x + (lane & 15)) * LD + 8 * (j + (lane >> 4)), b);
                        pa_mma(o[j], af, b[0], b[1], T{});
                        pa_mma(o[j + 1], af, b[2], b[3], T{});
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < DP / 8; ++j) {
                        const T *b = sv + (8 * j + g) * LV + 16 * x + 2 * c;
                        pa_mma(o[j], af, pa_word(b), pa_word(b + 8), T{});
                    }
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < kPaKeys / 8; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    for (int cc = 0; cc < 4; ++cc) {
                        const int key = 8 * n + 2 * cc + e;
                        const float p0 = __shfl_sync(~0u, s[n][e], (lane & ~3) | cc), p1 = __shfl_sync(~0u, s[n][2 + e], (lane & ~3) | cc);
#pragma unroll
                        for (int j = 0; j < DP / 8; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float x = to_f32(VEC ? sv[key * LD + 8 * j + 2 * c + i] : sv[(8 * j + 2 * c + i) * LV + key]);
                                if (j0 + key < limit[0]) o[j][i] += to_f32(from_f32<T>(p0)) * x;
                                if (j0 + key < limit[1]) o[j][2 + i] += to_f32(from_f32<T>(p1)) * x;
                            }
                    }
        }
    }
    if (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");  // (queries of rows that see nothing)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(~0u, l[r], 1);
        l[r] += __shfl_xor_sync(~0u, l[r], 2);
        const int row = 16 * warp + g + 8 * r;
        if (row >= rows) continue;
        T *y = static_cast<T *>(P.y) + (t.q_row + t.first + row) * P.ldy + (int64_t)head * D;
#pragma unroll
        for (int j = 0; j < DP / 8; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d = 8 * j + 2 * c + e;
                if (d < D) y[d] = from_f32<T>(limit[r] ? o[j][2 * r + e] / l[r] : 0.0f);
            }
    }
}

static int64_t pa_units(int64_t B, int64_t Tq, int64_t n_q) { return (Tq / kPaRows + B) * n_q; }

template <typename T, int DP, bool VEC>
static kq_status launch_pa(const char *fn, const PaParams &P, cudaStream_t st) {
    auto kern = pa_kernel<T, DP, VEC>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, pa_smem<DP, VEC>());
    if (e == cudaSuccess) e = launch_beside(kern, dim3((unsigned)pa_units(P.B, P.Tq, P.n_q)), dim3(128), pa_smem<DP, VEC>(), dim3(1), st, P);
    if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    count_launch(R_ATTN);
    return KQ_OK;
}

constexpr int64_t kPaMaxTokens = 0x7fffff00;
static bool pa_shape(int64_t B, int64_t Tq, int64_t n_q, int64_t n_kv, int64_t D) {
    return B > 0 && B <= (1 << 24) && Tq > 0 && Tq <= kPaMaxTokens && n_kv > 0 && n_kv <= 65535 && n_q > 0 && n_q <= 65535 &&
           n_q % n_kv == 0 && D > 0 && D <= 256 && D % 8 == 0;
}

static kq_status pa_call(const char *fn, kq_dtype xt, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                         const int32_t *cu_q, const int32_t *cu_k, int64_t B, int64_t Tq, int64_t Tk, int64_t n_q, int64_t n_kv,
                         int64_t D, float scale, int causal, void *y, int64_t ldy, void *workspace, size_t ws_bytes, kq_stream_t stream,
                         int idle = -1, unsigned long long wait_ns = kPtWaitNs) {
    if (xt != KQ_F16 && xt != KQ_BF16) return fail(KQ_ERR_UNSUPPORTED_DTYPE, "%s: row type %s is not F16 or BF16", fn, dtype_name(xt));
    if (!q || !k || !v || !y) return fail(KQ_ERR_INVALID_ARG, "%s: null rows", fn);
    if (!cu_q || !cu_k) return fail(KQ_ERR_INVALID_ARG, "%s: null %s", fn, cu_q ? "cu_k" : "cu_q");
    if (!pa_shape(B, Tq, n_q, n_kv, D) || Tk <= 0 || Tk > kPaMaxTokens)
        return fail(KQ_ERR_INVALID_ARG,
                    "%s: need B, Tq, Tk > 0, up to 65535 query heads, a multiple of the key heads, and D a multiple of 8 up to 256 "
                    "(B=%lld Tq=%lld Tk=%lld n_q=%lld n_kv=%lld D=%lld)",
                    fn, (long long)B, (long long)Tq, (long long)Tk, (long long)n_q, (long long)n_kv, (long long)D);
    if (ldq < n_q * D || ldy < n_q * D || ldk < n_kv * D || ldv < n_kv * D)
        return fail(KQ_ERR_INVALID_ARG, "%s: a row stride is less than its heads (ldq=%lld ldk=%lld ldv=%lld ldy=%lld)", fn, (long long)ldq,
                    (long long)ldk, (long long)ldv, (long long)ldy);
    if (causal != 0 && causal != 1) return fail(KQ_ERR_INVALID_ARG, "%s: causal=%d is not 0 or 1", fn, causal);
    if (!(fabsf(scale) <= 2.0e38f)) return fail(KQ_ERR_INVALID_ARG, "%s: scale must be finite, up to 2e38", fn);  // (times log2 e, too)
    if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(y, 2) || !aligned(cu_q, 4) || !aligned(cu_k, 4))
        return fail(KQ_ERR_ALIGNMENT, "%s: a pointer is not aligned to its elements", fn);
    // (a scale of 0 weighs all keys alike, as the smallest one does, which keeps -inf times it -inf)
    const float magnitude = fmaxf(fabsf(scale * 1.44269504f), 1.4e-45f);
    const PaParams P{q, k, v, y, ldq, ldk, ldv, ldy, cu_q, cu_k, B, Tq, Tk, (int)n_q, (int)(n_q / n_kv), (int)D,
                     magnitude, scale < 0.0f, causal != 0, static_cast<unsigned long long *>(workspace)};
    const bool tc = pa_takes_tc(P);
    if ((tc ? pa_tc_units(B, Tq, n_q, n_kv) : pa_units(B, Tq, n_q)) > kPaMaxUnits)
        return fail(KQ_ERR_INVALID_ARG, "%s: too many row tiles", fn);
    const size_t need = pa_tc_workspace(B, Tq, n_q / n_kv);
    if (!workspace || ws_bytes < need)
        return fail(KQ_ERR_WORKSPACE, "%s: workspace %zu bytes, need %zu", fn, workspace ? ws_bytes : (size_t)0, need);
    if (!aligned(workspace, 256)) return fail(KQ_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    const cudaStream_t st = (cudaStream_t)stream;
    if (tc) return pa_tc(fn, xt, P, wait_ns, idle, st);
    if (idle >= 0) return fail(KQ_ERR_INVALID_ARG, "%s: these rows do not take the tensor-core path", fn);
    auto go = [&](auto t) {
        using T = decltype(t);
        if (D <= 128) return D <= 64 ? launch_pa<T, 64, false>(fn, P, st) : launch_pa<T, 128, false>(fn, P, st);
        return pa_aligned(P) ? launch_pa<T, 256, true>(fn, P, st) : launch_pa<T, 256, false>(fn, P, st);
    };
    return xt == KQ_F16 ? go(__half{}) : go(__nv_bfloat16{});
}

}  // namespace kq

using namespace kq;

extern "C" {

size_t kq_attn_prompt_workspace_bytes(int64_t B, int64_t Tq, int64_t n_q, int64_t n_kv, int64_t D) {
    if (!pa_shape(B, Tq, n_q, n_kv, D)) return 0;
    // (which form a call takes follows from its addresses as well: 0 where neither would do)
    const bool tc = D <= 128 && pa_tc_units(B, Tq, n_q, n_kv) <= kPaMaxUnits;
    return tc || pa_units(B, Tq, n_q) <= kPaMaxUnits ? pa_tc_workspace(B, Tq, n_q / n_kv) : 0;
}

kq_status kq_attn_prompt(kq_dtype xt, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                         const int32_t *cu_q, const int32_t *cu_k, int64_t B, int64_t Tq, int64_t Tk, int64_t n_q, int64_t n_kv,
                         int64_t D, float scale, int causal, void *y, int64_t ldy, void *workspace, size_t ws_bytes,
                         kq_stream_t stream) {
    return pa_call("kq_attn_prompt", xt, q, ldq, k, ldk, v, ldv, cu_q, cu_k, B, Tq, Tk, n_q, n_kv, D, scale, causal, y, ldy, workspace,
                   ws_bytes, stream);
}

kq_status kq_debug_attn_prompt_wait_timeout(kq_dtype xt, const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                                            const int32_t *cu_q, const int32_t *cu_k, int64_t B, int64_t Tq, int64_t Tk, int64_t n_q,
                                            int64_t n_kv, int64_t D, float scale, int causal, void *y, int64_t ldy, int idle,
                                            int64_t wait_limit_ns, void *workspace, size_t ws_bytes, kq_stream_t stream) {
    const char *fn = "kq_debug_attn_prompt_wait_timeout";
    if (idle < 0 || idle == 3 || idle > 4) return fail(KQ_ERR_INVALID_ARG, "%s: idle=%d is not 0, 1, 2 or 4", fn, idle);
    if (wait_limit_ns < 1000 || wait_limit_ns > 1000000000)
        return fail(KQ_ERR_INVALID_ARG, "%s: wait_limit_ns must be in [1e3, 1e9]", fn);
    return pa_call(fn, xt, q, ldq, k, ldk, v, ldv, cu_q, cu_k, B, Tq, Tk, n_q, n_kv, D, scale, causal, y, ldy, workspace, ws_bytes, stream,
                   idle, (unsigned long long)wait_limit_ns);
}

}  // extern "C"
