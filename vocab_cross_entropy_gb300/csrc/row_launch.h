// Host side of the row-streaming kernels: launches with a cluster dimension, and the shared
// argument checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cmath>

#include "vce.h"
#include "vce_host.h"

namespace vce {
namespace rs {

constexpr int kMaxSmem = 232448;   // shared memory of a block, at most

// Launches `blocks` blocks of kKernel in clusters of `cluster` along x.  A kernel that needs more than
// 48 KB of shared memory (and has none of its own) is allowed all of an SM's once per device (the attribute costs a launch about 2 us on the host); a
// launch that fails is tried once more with the attribute set again, since a device reset drops it.
// early: the kernel may start before the stream's previous one has ended (programmatic dependent
// launch); it waits for that one itself (wait_previous) before it reads what that writes.
template <auto kKernel, typename Args>
cudaError_t launch_clusters(int64_t blocks, int cluster, int threads, int smem, cudaStream_t s, const Args& args,
                            bool early = false) {
    static std::atomic<uint64_t> allowed{0};   // bit d: device d (kMaxDevices = 64)
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess) return e;
    const uint64_t bit = d >= 0 && d < kMaxDevices ? 1ull << d : 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (early) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = (unsigned)cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = (unsigned)n;
    const bool known = smem <= 49152 || (allowed.load(std::memory_order_acquire) & bit) != 0;
    for (int tries = known ? 0 : 1; tries < 2; ++tries) {
        if (tries && smem > 49152) {
            e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
            if (e != cudaSuccess) return e;
            allowed.fetch_or(bit, std::memory_order_release);
        }
        e = cudaLaunchKernelEx(&cfg, kKernel, args);
        if (e == cudaSuccess) return e;
        if (!tries) (void)cudaGetLastError();
    }
    return e;
}

// Clusters of `cluster` blocks of kKernel (one block an SM) that run at once, asked for once per device
// and cluster size; 0 if it cannot be told.
template <auto kKernel>
int resident_clusters(int cluster, int threads, int smem, int sms) {
    if (cluster == 1) return sms;
    static std::atomic<int> known[kMaxDevices][5];
    int d = 0, log2 = 0;
    if (cudaGetDevice(&d) != cudaSuccess || d < 0 || d >= kMaxDevices) return 0;
    while ((1 << log2) < cluster) ++log2;
    int n = known[d][log2].load(std::memory_order_acquire);
    if (n) return n;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(sms / cluster * cluster));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        return 0;
    }
    known[d][log2].store(n, std::memory_order_release);
    return n;
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
