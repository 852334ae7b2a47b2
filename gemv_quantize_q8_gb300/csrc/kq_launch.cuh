// kq_launch.cuh -- launches that may start beside the end of the kernel before them (internal).
//
// A kernel launched here calls grid_dependency_wait() before it touches global memory, so it sees all that
// came before it on its stream; what overlaps is its launch and set-up.  After that wait, not before, it lets
// the next grid launch (grid_launch_dependents): a grid that starts beside it thus starts after everything
// earlier has completed, also one that reads its weights before it waits (kq_gemv, and the products here
// behind their quantizer).
// (Back to back, [9728 x 2560] with one int8 token: 4.4 us a call without, 3.6 so.)
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
