// launch.cuh -- kernel launches chained to the stream's previous kernel.
#pragma once

#include <cuda_runtime.h>

namespace w4a16 {

// The kernel's CTAs may be scheduled while the previous kernel on the stream
// drains (pdl_launch_dependents in every CTA of that one lets them).
//
// Before its own pdl_wait a kernel touches only memory that was complete when it was
// let start: what kernel n - 2 and those before it wrote, and only where every CTA of
// kernel n - 1 waits before it lets kernel n start; the first kernel of a call waits
// before it touches anything.  Two kernels let the next one start before they wait
// (lora_sum_kernel, wgrad_sum_kernel): what follows them may rely on kernel n - 3 and
// those before it.  Who reads early, and what:
//   dispatch_copy_kernel   X                      (n - 1: sort_rank_kernel)
//   lora_down_kernel       X, prefetched          (n - 1: sort_rank_kernel)
//   lora_sum_kernel        the sort               (n - 1: lora_down_kernel)
//   lora_up_kernel         the sort, base, the weights; in the gradient also the planes
//                          of g, and dX is written (n - 1: lora_sum_kernel, in the
//                          gradient lora_wgrad_kernel)
//   lora_wgrad_kernel      the sort               (n - 1: lora_sum_kernel)
//   wgrad_sum_kernel       the sort               (n - 1: lora_up_kernel)
// Every kernel waits at some point, in CTAs enough to end after the one before it.
// cluster > 1: clusters of that many CTAs along x.
template <typename... Params, typename... Args>
cudaError_t launch_chained(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int cluster,
                           cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

}  // namespace w4a16
