// A matrix to e4m3 with a power of two for each block of 1 x 128 or 128 x 128 elements.
//
// The scale is the least 2^k with max |x| <= 448 * 2^k: with max |x| = f 2^e, 1 <= f < 2, and 448 = 1.75 * 2^8,
// k = e - 8 or, for f > 1.75, e - 7.  Multiplying by 2^-k is exact, so q carries the one rounding to e4m3.
//
// Bound by memory: a block's elements wait in registers between its largest magnitude and its conversion, so x is
// read once.  128256 x 4096 bf16 in blocks of 128 x 128: 236 us, 6.7 TB/s (0.99 of the measured copy); in blocks of
// 1 x 128: 242 us.  Rows that are not whole 16-byte vectors go element by element (602 us at that size, measured
// before the vectors).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "row_launch.h"
#include "vce_check.cuh"
#include "vce_device.cuh"
#include "vce_fp8.h"
#include "vce_host.h"

namespace vce {
namespace fp8 {

struct QuantArgs {
    const void* x;
    int64_t R, D, ld;
    uint8_t* q;
    float* scales;
    int64_t nd;                  // blocks of 128 columns
};

// Two floats to e4m3 (the first in the low byte), to nearest even.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The block's scale and its reciprocal from its largest magnitude.
__device__ __forceinline__ float scale_of(float amax, float& inv) {
    if (!(amax < kInf)) return inv = __int_as_float(0x7FC00000);
    if (amax == 0.f) return inv = 1.f;
    const uint32_t b = __float_as_uint(amax);
    int k = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u);
    k = max(k, -126);                                // subnormal magnitudes too
    inv = __int_as_float((127 - k) << 23);
    return __int_as_float((k + 127) << 23);
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

constexpr int kThreads = 256;

// A vector of 16 bytes of x: G elements, G bytes of q.
template <typename S>
__device__ __forceinline__ void store_q(uint8_t* q, const uint4& x, float inv) {
    constexpr int G = Elt<S>::kGroup;
    float v[G];
    Elt<S>::unpack(x, v);
    uint32_t w[G / 4];
#pragma unroll
    for (int i = 0; i < G / 4; ++i)
        w[i] = to_e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) | to_e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
    if constexpr (G == 8) *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(q) = w[0];
}

template <typename S>
__device__ __forceinline__ float amax_of(const uint4& x, float m) {
    constexpr int G = Elt<S>::kGroup;
    float v[G];
    Elt<S>::unpack(x, v);
#pragma unroll
    for (int i = 0; i < G; ++i) m = max_nan(m, fabsf(v[i]));
    return m;
}

// Blocks of 1 x 128, rows of whole aligned vectors: 128 / G lanes a block, four of them in flight a lane.
constexpr int kRowUnits = 4;
template <typename S>
__global__ void __launch_bounds__(kThreads) k_quantize_rows(const __grid_constant__ QuantArgs a) {
    constexpr int G = Elt<S>::kGroup, L = 128 / G;
    const uint32_t nd = (uint32_t)a.nd, blocks = (uint32_t)(a.R * a.nd);
    const uint32_t first = (blockIdx.x * (kThreads / 32) + threadIdx.x / 32) * (kRowUnits * (32 / L)) + threadIdx.x % 32 / L;
    const int lane = threadIdx.x % L;
    uint4 x[kRowUnits];
    int64_t row[kRowUnits];
    int col[kRowUnits];
#pragma unroll
    for (int u = 0; u < kRowUnits; ++u) {
        const uint32_t b = first + u * (32 / L), r = b / nd;
        row[u] = r;
        col[u] = (int)(b - r * nd) * 128 + lane * G;
        x[u] = make_uint4(0, 0, 0, 0);
        if (b < blocks && col[u] < a.D) x[u] = ld_stream16(static_cast<const S*>(a.x) + row[u] * a.ld + col[u]);
    }
#pragma unroll
    for (int u = 0; u < kRowUnits; ++u) {
        float m = amax_of<S>(x[u], 0.f);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        float inv;
        const float scale = scale_of(m, inv);
        const uint32_t b = first + u * (32 / L);
        if (b >= blocks) continue;
        if (lane == 0) a.scales[b] = scale;
        if (col[u] < a.D) store_q<S>(a.q + row[u] * a.D + col[u], x[u], inv);
    }
}

// Blocks of 128 x 128, rows of whole aligned vectors: a thread block each, which holds them in registers.
template <typename S>
__global__ void __launch_bounds__(kThreads) k_quantize_tiles(const __grid_constant__ QuantArgs a) {
    constexpr int G = Elt<S>::kGroup, L = 128 / G, U = 128 * L / kThreads;   // vectors of a row, of a thread
    __shared__ float part[kThreads / 32];
    const uint32_t rb = blockIdx.x / (uint32_t)a.nd, cb = blockIdx.x - rb * (uint32_t)a.nd;
    const int col = (int)cb * 128 + threadIdx.x % L * G;
    const int64_t r0 = (int64_t)rb * 128 + threadIdx.x / L;
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * (kThreads / L);
        x[u] = make_uint4(0, 0, 0, 0);
        if (r < a.R && col < a.D) x[u] = ld_stream16(static_cast<const S*>(a.x) + r * a.ld + col);
    }
    float m = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) m = amax_of<S>(x[u], m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max_nan(m, part[w]);
    float inv;
    const float scale = scale_of(m, inv);
    if (threadIdx.x == 0) a.scales[blockIdx.x] = scale;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t r = r0 + u * (kThreads / L);
        if (r < a.R && col < a.D) store_q<S>(a.q + r * a.D + col, x[u], inv);
    }
}

// Any layout, element by element: a block of the matrix a thread block.
template <typename S, int kRows>
__global__ void __launch_bounds__(kThreads) k_quantize_any(const __grid_constant__ QuantArgs a) {
    __shared__ float part[kThreads / 32];
    const int64_t nb = blockIdx.x, rb = nb / a.nd, cb = nb - rb * a.nd;
    const int64_t r0 = rb * kRows, c0 = cb * 128;
    const int rows = (int)min((int64_t)kRows, a.R - r0), cols = (int)min((int64_t)128, a.D - c0);
    const S* x = static_cast<const S*>(a.x) + r0 * a.ld + c0;
    float m = 0.f;
    for (int i = threadIdx.x; i < rows * 128; i += kThreads)
        if (i % 128 < cols) m = max_nan(m, fabsf(Elt<S>::load1(x + (int64_t)(i / 128) * a.ld + i % 128)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0.f;
    for (int w = 0; w < kThreads / 32; ++w) m = max_nan(m, part[w]);
    float inv;
    const float scale = scale_of(m, inv);
    if (threadIdx.x == 0) a.scales[nb] = scale;
    for (int i = threadIdx.x; i < rows * 128; i += kThreads)
        if (i % 128 < cols)
            a.q[(r0 + i / 128) * a.D + c0 + i % 128] =
                (uint8_t)to_e4m3x2(Elt<S>::load1(x + (int64_t)(i / 128) * a.ld + i % 128) * inv, 0.f);
}

template <typename S>
cudaError_t run_quantize(const QuantArgs& a, int block_rows, int64_t blocks, cudaStream_t s) {
    constexpr int G = Elt<S>::kGroup;
    const bool vectors = aligned(a.x, 16) && a.ld % G == 0 && a.D % G == 0 && aligned(a.q, G);
    if (block_rows == 1) {
        constexpr int kPer = kThreads / 32 * kRowUnits * (32 * G / 128);   // matrix blocks of a thread block
        if (vectors) return rs::launch_clusters<k_quantize_rows<S>>((blocks + kPer - 1) / kPer, 1, kThreads, 0, s, a);
        return rs::launch_clusters<k_quantize_any<S, 1>>(blocks, 1, kThreads, 0, s, a);
    }
    if (vectors) return rs::launch_clusters<k_quantize_tiles<S>>(blocks, 1, kThreads, 0, s, a);
    return rs::launch_clusters<k_quantize_any<S, 128>>(blocks, 1, kThreads, 0, s, a);
}

}  // namespace fp8
}  // namespace vce

using namespace vce;

extern "C" int vce_quantize_fp8(const void* x, vce_dtype dt, int64_t R, int64_t D, int64_t ld, int block_rows, void* q,
                                float* scales, vce_stream_t s) {
    if (dt != VCE_F32 && dt != VCE_BF16) return VCE_ERR_DTYPE;
    if (R < 0 || R > (int64_t)1 << 27 || D < 1 || D > (int64_t)1 << 24) return VCE_ERR_SHAPE;
    if (block_rows != 1 && block_rows != VCE_FP8_BLOCK) return VCE_ERR_ARG;
    if (ld < D) return VCE_ERR_LD;
    const size_t es = dt == VCE_BF16 ? 2 : 4;
    if (!fits_bytes(R, ld, es)) return VCE_ERR_SHAPE;
    const int64_t nd = (D + 127) / 128, blocks = (R + block_rows - 1) / block_rows * nd;
    if (blocks >= (int64_t)1 << 31) return VCE_ERR_SHAPE;
    if (R == 0) return VCE_OK;
    if (!x || !q || !scales) return VCE_ERR_NULL;
    if (!aligned(x, es) || !aligned(scales, 4)) return VCE_ERR_ALIGN;
    // blocks read x while others write (and some read it twice)
    const int64_t nx = ((R - 1) * ld + D) * (int64_t)es;
    if (overlap_bytes(x, nx, q, R * D) || overlap_bytes(x, nx, scales, blocks * 4) ||
        overlap_bytes(q, R * D, scales, blocks * 4))
        return VCE_ERR_ARG;
    int rc = require_sm100();
    if (rc) return rc;
    const fp8::QuantArgs a{x, R, D, ld, static_cast<uint8_t*>(q), scales, nd};
    const cudaError_t e = dt == VCE_BF16 ? fp8::run_quantize<uint16_t>(a, block_rows, blocks, s)
                                         : fp8::run_quantize<float>(a, block_rows, blocks, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}
