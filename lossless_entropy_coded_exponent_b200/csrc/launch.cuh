// launch.cuh -- launches as programmatic dependents, and a kernel's dynamic shared memory.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dfx {
namespace {

// waits until the kernels before this one in the stream have completed and their writes are visible
__device__ __forceinline__ void wait_prior_grid() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// The dynamic shared-memory limit of a kernel is raised once per device (needed above
// 48 KiB).
template <class F>
cudaError_t allow_smem(F* kernel, size_t bytes, bool* done) {
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

// Launch with programmatic stream serialisation: the kernel may start while the work before it
// in the stream finishes, and calls wait_prior_grid before it touches memory that work uses.
// launch_clusters: in clusters of `ctas` CTAs.
template <class Kern, class... Arg>
cudaError_t launch_clusters(Kern* kernel, int grid, unsigned ctas, int threads, size_t smem, cudaStream_t s,
                            const Arg&... arg) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {ctas, 1, 1};
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, arg...);
}
template <class Kern, class... Arg>
cudaError_t launch_programmatic(Kern* kernel, int grid, int threads, size_t smem, cudaStream_t s, const Arg&... arg) {
    return launch_clusters(kernel, grid, 1, threads, smem, s, arg...);
}

}  // namespace
}  // namespace dfx
