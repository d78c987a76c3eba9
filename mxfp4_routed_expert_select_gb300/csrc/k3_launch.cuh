// k3_launch.cuh -- host-side launch helper shared by the kernels' launchers.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

namespace k3 {

void note_weight_writes(cudaStream_t s) noexcept;
bool weights_settled(cudaStream_t s) noexcept;

// Launches kernel<<<grid, block, smem, s>>>(args...), in clusters of `cluster` CTAs,
// as a programmatic dependent of the previous kernel on s where that is wanted and
// the driver takes it (the kernel then overlaps its prologue, and the weight loads it
// issues before griddep_wait, with that kernel's tail), else as a plain launch.
template <typename... KArgs, typename... Args>
static cudaError_t launch_dependent(bool wanted, int cluster, void (*kernel)(KArgs...), dim3 grid, dim3 block,
                                    size_t smem, cudaStream_t s, const Args &...args)
{
    static std::atomic<int> refused{0};
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        n++;
    }
    const bool dependent = wanted && !refused.load(std::memory_order_relaxed);
    if (dependent) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        n++;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = (unsigned)n;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess && dependent) {
        cudaGetLastError();
        cfg.numAttrs--;
        e = cudaLaunchKernelEx(&cfg, kernel, args...);
        if (e == cudaSuccess) refused.store(1, std::memory_order_relaxed);  // the attribute it was
    }
    return e;
}

// For kernels that touch nothing before griddep_wait.
template <typename... KArgs, typename... Args>
static cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              const Args &...args)
{
    return launch_dependent(true, 1, kernel, grid, block, smem, s, args...);
}
// For kernels that load weights before griddep_wait.
template <typename... KArgs, typename... Args>
static cudaError_t launch_pdl_weights(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                      const Args &...args)
{
    const bool settled = weights_settled(s);
    const cudaError_t e = launch_dependent(settled, 1, kernel, grid, block, smem, s, args...);
    if (e != cudaSuccess && !settled) note_weight_writes(s);  // nothing has waited for them
    return e;
}

}  // namespace k3
