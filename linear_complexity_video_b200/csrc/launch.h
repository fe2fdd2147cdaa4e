// Launches with programmatic stream serialisation: the kernel's CTAs may be placed, and set
// up their barriers and TMEM, while the last CTAs of the grid ahead still run. Each of them
// calls tc::stream_wait() before its first access to global memory, so what a stream's
// user sees is plain stream order. The 8-bit products use it (their set-up is the longest);
// the row kernels between them only let them in early (tc::stream_release). Launched so
// themselves they lose more than they gain: norm, product, quantisation, product at 300,
// 4,096 and 8,192 tokens, 2,560 -> 2,560, in a graph take 25.3, 74.1 and 118.6 us in plain
// order, 22.2, 70.6 and 114.8 with the products launched so, 22.2, 74.9 and 123.5 with all.
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace mate {

// `cluster` CTAs per cluster; 0: as the kernel declares
template <typename... Params, typename... Args>
cudaError_t launch_in_stream(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s,
                             Args &&...args)
{
    cudaLaunchAttribute attrs[2];
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace mate
