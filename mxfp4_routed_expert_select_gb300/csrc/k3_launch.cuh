// k3_launch.cuh -- host-side launch helper shared by the kernels' launchers.
#pragma once
#include <cuda_runtime.h>

#include <atomic>

namespace k3 {

bool weights_settled(cudaStream_t s) noexcept;

// Launches kernel<<<grid, block, smem, s>>>(args...) as a programmatic
// dependent of the previous kernel on s where that is wanted and the driver takes
// it (the kernel then overlaps its prologue, and the weight loads it issues before
// griddep_wait, with that kernel's tail), else as a plain launch.
template <typename... KArgs, typename... Args>
static cudaError_t launch_dependent(bool wanted, void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                    cudaStream_t s, Args... args)
{
    static std::atomic<int> refused{0};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = wanted && !refused.load(std::memory_order_relaxed) ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess && cfg.numAttrs == 1) {
        cudaGetLastError();
        refused.store(1, std::memory_order_relaxed);
        cfg.numAttrs = 0;
        e = cudaLaunchKernelEx(&cfg, kernel, args...);
    }
    return e;
}

// For kernels that touch nothing before griddep_wait.
template <typename... KArgs, typename... Args>
static cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              Args... args)
{
    return launch_dependent(true, kernel, grid, block, smem, s, args...);
}
// For kernels that load weights before griddep_wait.
template <typename... KArgs, typename... Args>
static cudaError_t launch_pdl_weights(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                                      Args... args)
{
    return launch_dependent(weights_settled(s), kernel, grid, block, smem, s, args...);
}

}  // namespace k3
