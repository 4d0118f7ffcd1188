// step_launch.cuh -- launch helper of the step kernels (norm.cu, cache.cu,
// tree_attn.cu): programmatic dependent launch, as every kernel of the
// library, and optionally a thread-block cluster.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

namespace sgq {

namespace {

// Lets a kernel have `smem` bytes of dynamic shared memory on the current
// device; asked once per device (a bit of `done` each, devices from 64 on every
// time).
template <typename Kern>
cudaError_t allow_smem(Kern kern, size_t smem, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit)
        return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <typename Kern, typename... Args>
cudaError_t launch_step(Kern kern, dim3 grid, int block, size_t smem, int cluster,
                        cudaStream_t stream, const Args &...args)
{
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
