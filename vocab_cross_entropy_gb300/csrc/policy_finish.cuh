// What comes of a row's sums: its log-probability, entropy and policy loss, and the statistics that are saved.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "logprob_rows.cuh"
#include "policy_rows.h"

namespace vce {
namespace lp {

// What a row's finish reads besides its sums.
struct RowIn {
    float zt, old, adv, ref, w;
};
template <typename S>
__device__ __forceinline__ RowIn row_in(const Args& a, int64_t row, int token) {
    RowIn in{Elt<S>::load1(static_cast<const S*>(a.logits) + row * a.ld + token), 0.f, 0.f, 0.f, 1.f};
    if (a.mode == kPolicy) {
        if (a.old) in.old = a.old[row];
        in.adv = a.adv[row];
        if (a.kl != 0.f) in.ref = a.ref[row];
        if (a.weights) in.w = a.weights[row];
    }
    return in;
}

// e^d - 1 - d >= 0 for |d| < 1/2 by its power series (to d^9 / 9!, 2e-9 relative at 0.5).
__device__ __forceinline__ float exp_minus_line(float d) {
    float c = 1.f / 362880.f;
    c = fmaf(c, d, 1.f / 40320.f);
    c = fmaf(c, d, 1.f / 5040.f);
    c = fmaf(c, d, 1.f / 720.f);
    c = fmaf(c, d, 1.f / 120.f);
    c = fmaf(c, d, 1.f / 24.f);
    c = fmaf(c, d, 1.f / 6.f);
    c = fmaf(c, d, 0.5f);
    return d * d * c;
}

// What a row that is left out (code 0), or one with an error, returns.
__device__ __forceinline__ void write_none(const Args& a, int64_t row, int code) {
    const float v = code ? nan_f() : 0.f;
    a.logprobs[row] = v;
    if (a.entropy) a.entropy[row] = v;
    if (a.mode == kPolicy) a.loss_rows[row] = v;
    a.row_stats[row] = make_float4(kInf, -(float)code, 0.f, 0.f);
}

// The row's statistics as they are saved, and for the policy loss its value; scale is on the gradient.
__device__ __forceinline__ float4 row_result(const Args& a, const Row& r, const RowIn& in, float scale, float& loss) {
    float4 st = make_float4(r.m, r.f, r.lp, a.mode == kPreference ? r.lp_lo : a.entropy ? r.ent : nan_f());
    if (a.mode == kPolicy) {
        const float A = in.adv;
        const float ratio = a.old ? expf((r.lp - in.old) + r.lp_lo) : 1.f;
        const float gain = ratio * A, clipped = fminf(fmaxf(ratio, a.lo), a.hi) * A;
        bool open = gain <= clipped;                 // the minimum is the unclipped one
        float got = open ? gain : clipped;
        if (a.dual > 0.f && A < 0.f && got < a.dual * A) {
            got = a.dual * A;
            open = false;
        }
        float da = open ? -gain : 0.f;
        if (A == 0.f) got = da = 0.f;
        if (ratio != ratio || A != A || r.lp != r.lp) got = da = nan_f();
        loss = -got;
        if (a.kl != 0.f) {
            // e^d - 1 - d from e^d - 1 where that keeps its digits, else by its power series
            const float d = (in.ref - r.lp) - r.lp_lo, e = expm1f(d);
            loss += a.kl * (fabsf(d) < 0.5f ? exp_minus_line(d) : e - d);
            da -= a.kl * e;
        }
        if (a.ent != 0.f) loss -= a.ent * r.ent;
        loss *= in.w;
        const float w = in.w * scale;
        const Coefs c = coefs_of(r.f, r.lnf, r.pt, r.pnt, r.lp, r.ent, w * da, -w * a.ent, a.inv_tau);
        st = make_float4(r.m, c.c0, c.c1, c.gt);
    }
    if (r.dead) st = make_float4(kInf, 0.f, 0.f, 1.f);
    return st;
}

__device__ __forceinline__ void write_result(const Args& a, int64_t row, const Row& r, float4 st, float loss) {
    a.logprobs[row] = r.lp;
    if (a.entropy) a.entropy[row] = r.ent;
    if (a.mode == kPolicy) a.loss_rows[row] = loss;
    a.row_stats[row] = st;
}

}  // namespace lp
}  // namespace vce
