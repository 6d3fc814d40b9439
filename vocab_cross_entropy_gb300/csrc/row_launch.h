// Host side of the row-streaming kernels: launches with a cluster dimension, and the shared
// argument checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "vce.h"
#include "vce_host.h"

namespace vce {
namespace rs {

// blocks in clusters of `cluster` along x.
template <typename Kern, typename Args>
cudaError_t launch_clusters(Kern kern, int64_t blocks, int cluster, int threads, int smem, cudaStream_t s,
                            const Args& args) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args);
}

// Whether a [T, V] matrix of es-byte elements and another (same T and V) share any byte of their
// extents (T >= 1).
inline bool overlap(const void* a, int64_t T, int64_t V, int64_t ld_a, size_t es_a, const void* b, int64_t ld_b,
                    size_t es_b) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + ((T - 1) * ld_b + V) * es_b && b0 < a0 + ((T - 1) * ld_a + V) * es_a;
}

// temperature is usable: finite, > 0, and so is its reciprocal (times log2 e)
inline bool temperature_ok(float t) {
    return std::isfinite(t) && t > 0.f && std::isfinite(1.4426950408889634f / t) && 1.f / t > 0.f;
}

}  // namespace rs
}  // namespace vce
