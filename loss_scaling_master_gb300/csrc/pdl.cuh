// pdl.cuh - programmatic dependent launch: a kernel of the chain may be
// scheduled while the kernel before it in the stream drains, so its launch
// and CTA ramp-up overlap that tail instead of following it.
//
// Contract of every kernel launched with launch_pdl: it calls pdl_wait()
// before its first global-memory access.  griddepcontrol.wait returns once
// every prerequisite grid has completed and its memory operations are
// visible, so data dependencies (read-after-write and write-after-read) are
// exactly those of plain stream order.  pdl_trigger() after the wait lets the
// next kernel of the stream be scheduled as soon as every CTA of this one has
// started; it never lets that kernel read before this one completes, because
// it waits in turn.  The wait is the hardware's own dependency mechanism, not
// a spin loop.  Where the stream holds no kernel before it, or the previous
// kernel never triggers, the wait returns when plain stream order would have
// started the kernel.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

namespace amp {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" :::); }

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t s, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// KB of shared memory that the small kernels want an SM's memory divided for.  An SM is
// emptied before it is divided anew, so kernels that follow one another overlap only with
// one division (2047 x 1111 fp32 dropout, forward and backward with its bias, 16.7 us as the
// driver chooses, 12.6 so; bias and GELU after a linear layer, 4096 x 8192, 102 and 90 us).
// All of it would leave too little for loads on the way (16384 x 5120 dropout 84 instead of
// 75 us), and for kernels with most on the way this is too much already (kAnyShared, as the
// driver chooses: token log probabilities 4096 x 128256 forward 158 us, with 64 KB 179).
// Column sums whose rows come ahead through shared memory need more for four CTAs an SM,
// and ask for it (bias_grad.cu, dropout.cu): 16384 x 5120 dropout's gradient 57.8 us, with
// 64 KB 74.4; the change between the two divisions is 1.6 us of dropout of 1024 x 768 with
// its gradients (6.8 us).
constexpr int kSmallShared = 64, kAnyShared = -1;

// The same in clusters of `cluster` CTAs along x.
template <auto Kernel, int SharedKB, typename... Args>
cudaError_t launch_pdl_cluster(int device, dim3 grid, dim3 block, int cluster, cudaStream_t s, Args &&...args) {
    static std::atomic<uint64_t> ready{0};  // one bit a device
    const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
    if (SharedKB >= 0 && (ready.load(std::memory_order_relaxed) & bit) == 0) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(Kernel),
                                                   cudaFuncAttributePreferredSharedMemoryCarveout,
                                                   SharedKB * 100 / 228);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, Kernel, std::forward<Args>(args)...);
}

}  // namespace amp
