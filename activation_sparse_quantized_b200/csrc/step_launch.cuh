// step_launch.cuh -- launch helper of the step kernels (norm.cu, cache.cu,
// tree_attn.cu): programmatic dependent launch, as every kernel of the
// library, and optionally a thread-block cluster.
#pragma once

#include <cuda_runtime.h>

namespace sgq {

namespace {

template <typename Kern, typename... Args>
cudaError_t launch_step(Kern kern, dim3 grid, int block, size_t smem, int cluster,
                        cudaStream_t stream, const Args &...args)
{
    if (smem > 48 * 1024) {
        cudaError_t err = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (err != cudaSuccess)
            return err;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

} // namespace

} // namespace sgq
