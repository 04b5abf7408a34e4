// pdl.cuh -- programmatic dependent launch: a kernel of a chain starts (its
// launch latency and set-up) while the kernel before it in the stream still
// runs.  Every kernel launched this way calls grid_wait(): it returns once the
// kernel before has completed and its writes are visible, and as that kernel
// waited in turn, so has everything earlier in the stream.  grid_go() lets the
// next kernel's CTAs be placed as soon as all of this kernel's have called it.
//
// Before its wait a kernel touches global memory in two places only:
// k_head_combine reads the tokens' targets, anchors and rows of X and W, and
// k_head_gemm<DW> behind DX reads G and its lists and writes dW.  Both rest on
// this: the kernel before calls grid_go() after its own wait, so when the one
// behind it starts, everything before that kernel is complete.  What is touched
// early is nothing that the kernel before writes (nor, for dW, reads), and it is
// read past L1 (__ldcg, TMA), which may hold lines of an earlier call.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"

namespace pmoe {

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Sets attribute A of kernel K, once on each device (attributes are a device's
// own); a failure is not kept, the next call tries again.
template <auto K, cudaFuncAttribute A>
bool set_attribute(int value)
{
    static std::atomic<uint64_t> done{0};   // a bit per device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(K, A, value) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Launches kernel K, which calls grid_wait(), in clusters of `cluster` CTAs
template <auto K, class... A>
bool launch_chained(unsigned grid, unsigned block, size_t smem, unsigned cluster, cudaStream_t st, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, K, args...) != cudaSuccess) return false;
    note_launch();
    return true;
}

}  // namespace pmoe
