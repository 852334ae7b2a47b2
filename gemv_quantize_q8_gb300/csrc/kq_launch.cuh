// kq_launch.cuh -- launches that may start beside the end of the kernel before them (internal).
//
// A kernel launched here waits (grid_dependency_wait()) before it touches global memory, so that it sees all that
// came before it on its stream; what overlaps is its launch and set-up.  After that wait, not before, it lets the
// next grid launch (grid_launch_dependents).
// One thing may be read before the wait: weights, their scales and the bias, and only where the launch directly
// before is the same call's own prologue (quantizer or panel) from here.  That prologue writes none of them and
// triggers after its own wait, so the product starts when everything before the prologue has completed, a kernel
// that wrote the weights among it.  (kq_gemv reads its weights before its wait behind any kernel, which must not
// be the one that wrote them; behind a kernel from here, what came before that one has completed.)
// Back to back, [9728 x 2560] with one int8 token: 5.4 us a call for 5.5 without, its weights coming from memory;
// 3.4 for 3.7 where they stay in the L2.  ([14336 x 4096]: 10.6 for 10.2, and 6.5 for 7.2.)
#pragma once
#include "kq_internal.cuh"
#include "kq_sm100.cuh"

namespace kq {

template <typename... Params, typename... Args>
inline cudaError_t launch_beside(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, dim3 cluster, cudaStream_t st,
                                 Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster.x;
    attr[1].val.clusterDim.y = cluster.y;
    attr[1].val.clusterDim.z = cluster.z;
    cfg.attrs = attr;
    cfg.numAttrs = cluster.x * cluster.y * cluster.z > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, Params(args)...);
}

}  // namespace kq
