// Arguments and host checks shared by the post-training losses' translation units.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "row_launch.h"
#include "vce_policy.h"

namespace vce {
namespace lp {

enum Mode { kLogprobs = 0, kPolicy = 1, kPreference = 2 };

// Of the row kernels.  row_stats per row, after the forward:
//   kLogprobs    (m, f, log p_t, H)            H NaN where it was not asked for
//   kPolicy      (m, c0, c1, gt)               for an upstream gradient of 1
//   kPreference  (m, f, log p_t, its low part), then (m, c0, pair (an int's bits), gt) from k_pairs
// and (+inf, -code, 0, 0) for a row without a gradient: code 0, or the row's error; (+inf, 0, 0, 1) for one
// of nothing but masks.
struct Args {
    const void* logits;
    int64_t T, V, ld;
    const int64_t* ids;
    int64_t ignore_index;
    int mode;
    float k2, k2_lo, inv_tau;    // log2(e) / temperature as k2 + k2_lo, 1 / temperature
    float* logprobs;
    float* entropy;              // or null
    float4* row_stats;
    // kPolicy
    const float *old, *adv, *ref, *weights;
    float lo, hi, dual, kl, ent; // 1 - clip_low, 1 + clip_high
    float* loss_rows;
    int red;
    // kPreference: rows outside [offsets[0], offsets[2 P]) are left out
    const int64_t* offsets;
    int64_t P;
    // kPolicy in one pass
    const float* go;
    const float* inv_n;          // MEAN
    void* grad;
    int64_t ld_g;
    int cluster, per;            // blocks of a row, vectors of a block
    uint64_t wait_ns;            // bound of every wait
    int withhold;                // n > 0 (test hook): in a cluster's block n - 1 the gradient waits in vain
};

// Of the gradient from saved statistics.
struct GradArgs {
    const void* logits;
    int64_t T, V, ld;
    const int64_t* ids;
    int mode;
    float k2, inv_tau;
    const float4* row_stats;
    const float* go;             // kPolicy, kPreference
    int go_each;                 // one for each row (pair), else one
    int64_t P;                   // kPreference: pairs
    float scale;                 // on go
    const float *ga, *gb;        // kLogprobs
    void* grad;
    int64_t ld_g;
    int parts, nbuf;
    uint64_t wait_ns;
    int withhold;                // 1 (test hook): a row's last block waits for its last stage in vain
};

// Whether a cluster's shared memory holds a row, which the one pass needs.
bool one_pass_holds(vce_dtype dt, int64_t V);
cudaError_t launch_one_pass(vce_dtype dt, vce_dtype gdt, Args& a, cudaStream_t s);
cudaError_t launch_grad(vce_dtype dt, vce_dtype gdt, GradArgs& a, cudaStream_t s);

// log2(e) / tau, and what is left of it.
inline float k2_of(float tau) { return (float)(1.4426950408889634 / (double)tau); }
inline float k2_rest(float tau) { return (float)(1.4426950408889634 / (double)tau - (double)k2_of(tau)); }

inline int check_shape(vce_dtype dt, int64_t T, int64_t V, int64_t ld, float tau) {
    if (dt != VCE_F32 && dt != VCE_BF16) return VCE_ERR_DTYPE;
    if (T < 0 || T > VCE_MAX_POLICY_T || V < 1 || V > VCE_MAX_POLICY_V) return VCE_ERR_SHAPE;
    if (!rs::temperature_ok(tau)) return VCE_ERR_ARG;
    if (ld < V) return VCE_ERR_LD;
    if (!fits_bytes(T, ld, dt == VCE_BF16 ? 2 : 4)) return VCE_ERR_SHAPE;
    return VCE_OK;
}

inline int check_grad(vce_dtype dt, const void* logits, int64_t T, int64_t V, int64_t ld, const void* grad,
                      vce_dtype gdt, int64_t ld_g) {
    if (gdt != VCE_F32 && gdt != VCE_BF16) return VCE_ERR_DTYPE;
    if (ld_g < V) return VCE_ERR_LD;
    const size_t es = dt == VCE_BF16 ? 2 : 4, gs = gdt == VCE_BF16 ? 2 : 4;
    if (!fits_bytes(T, ld_g, gs)) return VCE_ERR_SHAPE;
    if (T == 0) return VCE_OK;
    if (!logits || !grad) return VCE_ERR_NULL;
    if (!aligned(logits, es) || !aligned(grad, gs)) return VCE_ERR_ALIGN;
    if (rs::overlap(logits, T, V, ld, es, grad, ld_g, gs)) return VCE_ERR_ARG;
    return VCE_OK;
}

}  // namespace lp
}  // namespace vce
