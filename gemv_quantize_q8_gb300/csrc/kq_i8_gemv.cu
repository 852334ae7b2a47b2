// kq_i8_gemv.cu -- int8 product of up to eight tokens: every weight is read once, by one lane, and dotted
// (dp4a, exact int32) against all tokens.
//
// Bound by the weights' bytes.  A warp takes ROWS weight rows; its lanes take consecutive 16-byte pieces of
// them, the next pieces always on their way while the current ones are dotted.  The 1, 2, 4 or 8 warps of a
// group share the rows' pieces and add their sums through shared memory (whole numbers: exact in any order).
// Blocks stay and walk the row groups, so that a group's first pieces are on their way while the group before
// it is summed up and stored.  The tokens' codes are small and shared by every warp: they come through L1.
// Back to back, from memory (weights rotating over three times the L2; the same weights again, from the L2, in
// brackets): one token of [14336 x 4096] 10.6 us, 5.6 TB/s (6.5); five tokens of [4096 x 14336] 13.0 us (11.2).
//
// TX other than void: the tokens come as rows of that type and every block quantises them itself, into shared
// memory, while its first weights are on their way: one fp32 token of [9728 x 2560] 7.0 us (4.5), behind a quantizer
// of its own 7.2 (5.7); of [2560 x 9728] 8.2 (6.0) and 8.6 (7.9).
#include <type_traits>

#include "kq_i8_gemv.cuh"
#include "kq_i8_quant.cuh"
#include "kq_launch.cuh"

namespace kq {

constexpr int GV_WARPS = 8;

// A weight piece of 16 codes, not kept in L1: nothing reads it again.
__device__ __forceinline__ uint4 load_stream(const int8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
// Codes from `valid` on cleared: they lie past the row's end.
__device__ __forceinline__ uint32_t keep_bytes(uint32_t v, int valid) {
    return valid >= 4 ? v : valid <= 0 ? 0u : v & ((1u << (8 * valid)) - 1u);
}
__device__ __forceinline__ uint4 keep_codes(uint4 v, int valid) {
    return make_uint4(keep_bytes(v.x, valid), keep_bytes(v.y, valid - 4), keep_bytes(v.z, valid - 8), keep_bytes(v.w, valid - 12));
}

// Weight rows of a warp and blocks of an SM, by tokens: what a warp's pieces under way and its ROWS*M sums
// need in registers against how many warps there are to wait for memory.  [14336 x 4096], from memory (from the L2 in
// brackets): one token 10.6 us (6.5) with 2 rows and 4 blocks, 10.8 (6.3) with 4 and 2 ([4096 x 4096]: 4.4 and 4.7);
// three tokens 11.6 (7.8) with 4 and 2, 11.8 (8.6) with 2 and 4, 10.9 (7.4) with 2 and 3; eight tokens 14.0 (12.5)
// with 2 and 2, 16.9 (15.0) with 4 and 2, 16.1 (13.4) with 2 and 3.  Blocks that quantise are as good few where the
// weights come from memory, better from the L2 ([9728 x 2560], one fp32 token: 7.0 (4.5) with 4 and 2, 7.0 (4.9) with
// 2 and 4).
template <int M, typename TX> constexpr int kGemvRows = M == 3 || M == 4 || !std::is_void<TX>::value ? 4 : 2;
template <int M, typename TX> constexpr int kGemvPerSm = M <= 2 && std::is_void<TX>::value ? 4 : 2;

template <int M, int ROWS, typename TY, typename TX>
__global__ void __launch_bounds__(GV_WARPS * 32, kGemvPerSm<M, TX>)
    i8_gemv_kernel(const void *__restrict__ rows, int64_t ldq, const float *__restrict__ sx, const int8_t *__restrict__ w,
                   int64_t ldw, const float *__restrict__ sw, const float *__restrict__ bias, int N, int K, int split, int tasks,
                   TY *__restrict__ y, int64_t ldy, unsigned long long *__restrict__ err, bool weights_first) {
    constexpr bool QUANT = !std::is_void<TX>::value;
    constexpr int U = ROWS == 1 ? 4 : 2;  // pieces of a row in one batch
    extern __shared__ uint4 codes[];      // QUANT: [M][K rounded up to 16]
    __shared__ int part_sum[GV_WARPS][ROWS * M];
    __shared__ float part_max[GV_WARPS][M];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / split, part = warp % split, groups = GV_WARPS / split;
    const int pieces = (K + 15) >> 4, step = 32 * split, p0 = part * 32 + lane;
    const int8_t *wr[ROWS];
    auto rows_of = [&](int task) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) wr[r] = w + min(((int64_t)task * groups + group) * ROWS + r, (int64_t)N - 1) * ldw;
    };
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 cur[U][ROWS], nxt[U][ROWS];
    auto load = [&](uint4 (&v)[U][ROWS], int p) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) v[u][r] = p + u * step < pieces ? load_stream(wr[r] + (int64_t)(p + u * step) * 16) : none;
    };
    int task = blockIdx.x;
    rows_of(task);
    // behind the quantizer, which has waited for all that came before it, the weights need no wait
    if (!weights_first) sm100::grid_dependency_wait();
    load(cur, p0);
    if (weights_first) sm100::grid_dependency_wait();
    sm100::grid_launch_dependents();
    if (blockIdx.x == 0 && threadIdx.x == 0) *err = 0ull;
    const int8_t *q = static_cast<const int8_t *>(rows);
    float scale[M];
    if constexpr (QUANT) {
        const TX *x = static_cast<const TX *>(rows);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float a = i8_amax(x + m * ldq, K, threadIdx.x, GV_WARPS * 32);
#pragma unroll
            for (int s = 16; s; s >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, s));
            if (lane == 0) part_max[warp][m] = a;
        }
        __syncthreads();
        int8_t *c = reinterpret_cast<int8_t *>(codes);
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float a = part_max[0][m];
#pragma unroll
            for (int i = 1; i < GV_WARPS; ++i) a = fmaxf(a, part_max[i][m]);
            const I8Scale s = i8_scale(a);
            scale[m] = s.scale;
            i8_codes(x + m * ldq, K, pieces * 16, s.inv, c + m * pieces * 16, threadIdx.x, GV_WARPS * 32);
        }
        __syncthreads();
    }
    for (; task < tasks; task += gridDim.x) {
        int acc[ROWS][M] = {};
        for (int b = 0; b < pieces; b += U * step) {  // (b: the same for every lane)
            const int p = p0 + b;
            if (b + U * step < pieces) {
                load(nxt, p + U * step);
            } else if (task + (int)gridDim.x < tasks) {
                rows_of(task + gridDim.x);
                load(nxt, p0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pu = p + u * step;
                if (pu == pieces - 1 && (K & 15)) {
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) cur[u][r] = keep_codes(cur[u][r], K & 15);
                }
                const int64_t off = (int64_t)min(pu, pieces - 1) * 16;  // past the end the weights are zeros
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const uint4 x = QUANT ? codes[m * pieces + (off >> 4)] : *reinterpret_cast<const uint4 *>(q + m * ldq + off);
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        int a = acc[r][m];
                        a = dp4a((int)cur[u][r].x, (int)x.x, a);
                        a = dp4a((int)cur[u][r].y, (int)x.y, a);
                        a = dp4a((int)cur[u][r].z, (int)x.z, a);
                        acc[r][m] = dp4a((int)cur[u][r].w, (int)x.w, a);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int r = 0; r < ROWS; ++r) cur[u][r] = nxt[u][r];
        }
        // lane r*M + m ends with the warp's sum of row r, token m
        int mine = 0;
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int s = __reduce_add_sync(~0u, acc[r][m]);
                if (lane == r * M + m) mine = s;
            }
        if (split > 1) {
            if (lane < ROWS * M) part_sum[warp][lane] = mine;
            __syncthreads();
            mine = 0;
            for (int s = 0; s < split && !part && lane < ROWS * M; ++s) mine += part_sum[warp + s][lane];
            __syncthreads();
        }
        const int64_t n = ((int64_t)task * groups + group) * ROWS + lane / M;
        const int m = lane % M;
        if (!part && lane < ROWS * M && n < N) {
            float s = 0.0f;
            if constexpr (QUANT) {
#pragma unroll
                for (int i = 0; i < M; ++i)
                    if (i == m) s = scale[i];
            } else {
                s = sx[m];
            }
            float v = __fmul_rn(__fmul_rn((float)mine, s), sw[n]);
            if (bias) v = __fadd_rn(v, bias[n]);
            y[m * ldy + n] = from_f32<TY>(v);
        }
    }
}

// A launch's split of a group's pieces, its tasks (of 8/split groups) and its time in batches of a warp: every
// block walks its tasks, each so many batches and, for its sums and stores, about half a batch more.
struct GemvPlan {
    int split;
    int64_t tasks, blocks;
    double t;
};
static GemvPlan gemv_plan(int64_t N, int64_t K, int rows, int per_sm) {
    const int64_t groups = (N + rows - 1) / rows, pieces = (K + 15) / 16, batch = rows == 1 ? 4 * 32 : 2 * 32;
    GemvPlan best{};
    for (int s = 1; s <= GV_WARPS; s *= 2) {
        const int64_t tasks = (groups + GV_WARPS / s - 1) / (GV_WARPS / s), blocks = tasks < 152 * per_sm ? tasks : 152 * per_sm;
        const double t = (double)((tasks + blocks - 1) / blocks) * ((double)((pieces + batch * s - 1) / (batch * s)) + 0.5);
        if (s == 1 || t < best.t) best = {s, tasks, blocks, t};
    }
    return best;
}

template <int M, int ROWS, typename TY, typename TX>
static kq_status launch_rows(const char *fn, const I8GemvArgs &a, const GemvPlan &p, cudaStream_t st) {
    const size_t smem = std::is_void<TX>::value ? 0 : (size_t)M * ((a.K + 15) / 16) * 16;  // 17 KB at most
    const cudaError_t e = launch_beside(i8_gemv_kernel<M, ROWS, TY, TX>, dim3((unsigned)p.blocks), dim3(GV_WARPS * 32), smem,
                                        dim3(1), st, a.rows, a.ldq, a.sx, a.w, a.ldw, a.sw, a.bias, (int)a.N, (int)a.K, p.split,
                                        (int)p.tasks, static_cast<TY *>(a.y), a.ldy, a.err, a.after_quant);
    if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    count_launch(R_I8);
    return KQ_OK;
}

template <int M, typename TY, typename TX>
static kq_status launch_tokens(const char *fn, const I8GemvArgs &a, cudaStream_t st) {
    // Single rows a warp where more would leave most SMs without a task (a batch has the same bytes either way).
    constexpr int R = kGemvRows<M, TX>, S = kGemvPerSm<M, TX>;
    const GemvPlan some = gemv_plan(a.N, a.K, R, S), one = gemv_plan(a.N, a.K, 1, S);
    if (some.blocks < 152 && one.blocks > some.blocks) return launch_rows<M, 1, TY, TX>(fn, a, one, st);
    return launch_rows<M, R, TY, TX>(fn, a, some, st);
}

template <typename TY>
static kq_status launch_codes(const char *fn, const I8GemvArgs &a, cudaStream_t st) {
    switch (a.M) {
    case 1: return launch_tokens<1, TY, void>(fn, a, st);
    case 2: return launch_tokens<2, TY, void>(fn, a, st);
    case 3: return launch_tokens<3, TY, void>(fn, a, st);
    case 4: return launch_tokens<4, TY, void>(fn, a, st);
    case 5: return launch_tokens<5, TY, void>(fn, a, st);
    case 6: return launch_tokens<6, TY, void>(fn, a, st);
    case 7: return launch_tokens<7, TY, void>(fn, a, st);
    default: return launch_tokens<8, TY, void>(fn, a, st);
    }
}

kq_status i8_gemv(const char *fn, const I8GemvArgs &a, cudaStream_t st) {
    return with_type(a.yt, [&](auto t) { return launch_codes<decltype(t)>(fn, a, st); });
}

bool i8_gemv_quantizes(int64_t M, int64_t K) { return M <= 2 && M * K <= 16384; }

kq_status i8_gemv_rows(const char *fn, kq_dtype xt, const I8GemvArgs &a, cudaStream_t st) {
    return with_type(a.yt, [&](auto t) {
        using TY = decltype(t);
        return with_type(xt, [&](auto x) {
            using TX = decltype(x);
            return a.M == 1 ? launch_tokens<1, TY, TX>(fn, a, st) : launch_tokens<2, TY, TX>(fn, a, st);
        });
    });
}

}  // namespace kq
