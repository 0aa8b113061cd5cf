// pc_launch.cuh -- launches of a call's kernels one behind the other.
#pragma once

#include <cuda_runtime.h>

namespace pcn {

// A kernel launched `behind` may start while the last blocks of the one before it on the
// stream run, and waits for that one's end, and its writes, in after_previous(), which
// comes before anything else it does with global memory.  The one before allows it with
// let_next_start() (or by ending).  So the start of a kernel costs its few microseconds
// under the end of the one before.  Every kernel of such a chain has both; the first
// of a call is launched as usual.
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// `cluster`: blocks of a thread block cluster.
template <class... P, class... A>
cudaError_t launch_clusters(bool behind, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                            cudaStream_t st, int cluster, A &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (behind) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = unsigned(cluster);
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (e != cudaSuccess) cudaGetLastError();  // (it is returned, not left for others to find)
    return e;
}
template <class... P, class... A>
cudaError_t launch(bool behind, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem,
                   cudaStream_t st, A &&...args) {
    return launch_clusters(behind, kernel, grid, block, smem, st, 1, static_cast<A &&>(args)...);
}

}  // namespace pcn
