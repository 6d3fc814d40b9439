// Logits of a head in e4m3 with block scales.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "row_launch.h"
#include "vce_device.cuh"
#include "vce_check.cuh"
#include "vce_fp8.h"
#include "vce_host.h"

namespace vce {
namespace fp8 {

struct LinearArgs {
    const uint8_t* x;
    const float* xs;
    const uint8_t* w;
    const float* ws;
    int64_t T, D, V;
    int nd;
    void* out;
    int64_t ld;
};

__device__ __forceinline__ float from_e4m3(uint8_t v) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
    float f;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
    return f;
}

constexpr int kTile = 32;

// A 32 x 32 tile of the logits a block, a quarter of a block of 128 columns at a time.
template <typename O>
__global__ void __launch_bounds__(256) k_linear(const __grid_constant__ LinearArgs a) {
    __shared__ float xt[kTile][33], wt[kTile][33];
    const int64_t nv = (a.V + kTile - 1) / kTile;
    const int64_t t0 = blockIdx.x / nv * kTile, v0 = blockIdx.x % nv * kTile;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
    float acc[4] = {}, part[4] = {};
    for (int64_t k0 = 0; k0 < a.D; k0 += 32) {
        for (int i = 0; i < 4; ++i) {
            const int r = ty + 8 * i;
            const int64_t k = k0 + tx;
            xt[r][tx] = t0 + r < a.T && k < a.D ? from_e4m3(a.x[(t0 + r) * a.D + k]) : 0.f;
            wt[r][tx] = v0 + r < a.V && k < a.D ? from_e4m3(a.w[(v0 + r) * a.D + k]) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < 32; ++k)
            for (int i = 0; i < 4; ++i) part[i] = fmaf(xt[ty + 8 * i][k], wt[tx][k], part[i]);
        __syncthreads();
        if ((k0 + 32) % 128 == 0 || k0 + 32 >= a.D) {
            const int64_t b = k0 / 128;
            for (int i = 0; i < 4; ++i) {
                const int64_t t = t0 + ty + 8 * i, v = v0 + tx;
                if (t < a.T && v < a.V) acc[i] = fmaf(part[i], a.xs[t * a.nd + b] * a.ws[v / 128 * a.nd + b], acc[i]);
                part[i] = 0.f;
            }
        }
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t t = t0 + ty + 8 * i, v = v0 + tx;
        if (t < a.T && v < a.V) Elt<O>::store1(static_cast<O*>(a.out) + t * a.ld + v, acc[i]);
    }
}

}  // namespace fp8
}  // namespace vce

using namespace vce;

extern "C" int vce_linear_fp8(const void* x, const float* x_scales, const void* w, const float* w_scales, int64_t T,
                              int64_t D, int64_t V, void* out, vce_dtype out_dt, int64_t ld, vce_stream_t s) {
    if (out_dt != VCE_F32 && out_dt != VCE_BF16) return VCE_ERR_DTYPE;
    if (T < 0 || T > (int64_t)1 << 24 || V < 1 || V > (int64_t)1 << 24 || D < 16 || D > 65536 || D % 16) return VCE_ERR_SHAPE;
    if (ld < V) return VCE_ERR_LD;
    const size_t es = out_dt == VCE_BF16 ? 2 : 4;
    if (!fits_bytes(T, ld, es)) return VCE_ERR_SHAPE;
    if (T == 0) return VCE_OK;
    if (!x || !x_scales || !w || !w_scales || !out) return VCE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(out, es))
        return VCE_ERR_ALIGN;
    int rc = require_sm100();
    if (rc) return rc;
    const fp8::LinearArgs a{static_cast<const uint8_t*>(x), x_scales, static_cast<const uint8_t*>(w), w_scales, T, D, V,
                            (int)((D + 127) / 128), out, ld};
    const int64_t blocks = (T + 31) / 32 * ((V + 31) / 32);
    const cudaError_t e = out_dt == VCE_BF16 ? rs::launch_clusters<fp8::k_linear<uint16_t>>(blocks, 1, 256, 0, s, a)
                                             : rs::launch_clusters<fp8::k_linear<float>>(blocks, 1, 256, 0, s, a);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}
