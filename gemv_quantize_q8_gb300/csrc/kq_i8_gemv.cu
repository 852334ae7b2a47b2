// kq_i8_gemv.cu -- int8 product of up to eight tokens: every weight is read once, by one lane, and dotted
// (dp4a, exact int32) against all tokens.
//
// Bound by the weights' bytes.  A warp takes ROWS weight rows; its lanes take consecutive 16-byte pieces of
// them, the next pieces always on their way while the current ones are dotted.  When there are few rows,
// the 1, 2, 4 or 8 warps of a group share the rows' pieces and add their sums through shared memory (whole
// numbers: exact in any order).  The tokens' codes are small and shared by every warp: they come through L1.
#include "kq_i8_gemv.cuh"
#include "kq_sm100.cuh"

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

template <int M, int ROWS, typename TY>
__global__ void __launch_bounds__(GV_WARPS * 32)
    i8_gemv_kernel(const int8_t *__restrict__ q, int64_t ldq, const float *__restrict__ sx, const int8_t *__restrict__ w,
                   int64_t ldw, const float *__restrict__ sw, const float *__restrict__ bias, int N, int K, int split,
                   TY *__restrict__ y, int64_t ldy, unsigned long long *__restrict__ err) {
    constexpr int U = ROWS == 1 ? 4 : 2;  // pieces of a row in one batch
    __shared__ int part_sum[GV_WARPS][ROWS * M];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / split, part = warp % split;
    const int64_t n0 = ((int64_t)blockIdx.x * (GV_WARPS / split) + group) * ROWS;
    const int pieces = (K + 15) >> 4, step = 32 * split;
    const int8_t *wr[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) wr[r] = w + min(n0 + r, (int64_t)N - 1) * ldw;
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 cur[U][ROWS], nxt[U][ROWS];
    auto load = [&](uint4 (&v)[U][ROWS], int p) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) v[u][r] = p + u * step < pieces ? load_stream(wr[r] + (int64_t)(p + u * step) * 16) : none;
    };
    int p = part * 32 + lane;
    load(cur, p);
    sm100::grid_dependency_wait();  // the codes may be the output of the kernel before this one; the weights are not
    if (blockIdx.x == 0 && threadIdx.x == 0) *err = 0ull;
    int acc[ROWS][M] = {};
    for (; p < pieces; p += U * step) {
        load(nxt, p + U * step);
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
                const uint4 x = *reinterpret_cast<const uint4 *>(q + m * ldq + off);
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
        if (part || lane >= ROWS * M) return;
        mine = 0;
        for (int s = 0; s < split; ++s) mine += part_sum[warp + s][lane];
    }
    const int64_t n = n0 + lane / M;
    const int m = lane % M;
    if (lane >= ROWS * M || n >= N) return;
    float v = __fmul_rn(__fmul_rn((float)mine, sx[m]), sw[n]);
    if (bias) v = __fadd_rn(v, bias[n]);
    y[m * ldy + n] = from_f32<TY>(v);
}

template <int M, int ROWS, typename TY>
static kq_status launch_rows(const char *fn, const I8GemvArgs &a, int split, cudaStream_t st) {
    const int per_block = GV_WARPS / split * ROWS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + per_block - 1) / per_block));
    cfg.blockDim = dim3(GV_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.after_quant ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, i8_gemv_kernel<M, ROWS, TY>, a.q, a.ldq, a.sx, a.w, a.ldw, a.sw, a.bias,
                                             (int)a.N, (int)a.K, split, static_cast<TY *>(a.y), a.ldy, a.err);
    if (e != cudaSuccess) return fail(KQ_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    count_launch(R_I8);
    return KQ_OK;
}

template <int M, typename TY>
static kq_status launch_tokens(const char *fn, const I8GemvArgs &a, cudaStream_t st) {
    // Warps that share a row group: enough to give every SM 16 warps (152 * 16), while each still has a
    // piece for every lane.  A product too narrow for that even so takes single rows.
    constexpr int64_t want = 152 * 16;
    int split = 1;
    while (split < GV_WARPS && (a.N + 3) / 4 * split < want && a.K >= 512 * 2 * split) split *= 2;
    if ((a.N + 3) / 4 * split * 2 <= want) return launch_rows<M, 1, TY>(fn, a, split, st);
    return launch_rows<M, 4, TY>(fn, a, split, st);
}

kq_status i8_gemv(const char *fn, const I8GemvArgs &a, cudaStream_t st) {
    return with_type(a.yt, [&](auto t) {
        using TY = decltype(t);
        switch (a.M) {
        case 1: return launch_tokens<1, TY>(fn, a, st);
        case 2: return launch_tokens<2, TY>(fn, a, st);
        case 3: return launch_tokens<3, TY>(fn, a, st);
        case 4: return launch_tokens<4, TY>(fn, a, st);
        case 5: return launch_tokens<5, TY>(fn, a, st);
        case 6: return launch_tokens<6, TY>(fn, a, st);
        case 7: return launch_tokens<7, TY>(fn, a, st);
        default: return launch_tokens<8, TY>(fn, a, st);
        }
    });
}

}  // namespace kq
