// Writing gradients 2^y (c0 + c1 y), y = z k2 - bias, of a row's streamed stages (logprob_rows.cuh).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "logprob_rows.cuh"
#include "row_stream.cuh"

namespace vce {
namespace lp {

using rs::Slice;

// One value (+0.0 for a row without a gradient) over the slice's columns, by NT threads.
template <typename S, typename O>
__device__ __forceinline__ void fill_grads(const rs::Row& r, const Slice& s, O* grow, bool vec, int tid, int NT,
                                           float value = 0.f) {
    constexpr int G = Elt<S>::kGroup;
    float same[G];
#pragma unroll
    for (int k = 0; k < G; ++k) same[k] = value;
    for (int v = s.v0 + tid; v < s.v0 + s.n; v += NT) {
        const int64_t c0 = (int64_t)v * G - r.shift;
        if (vec && v >= r.iv0 && v < r.iv1) {
            GroupStore<O, G>::run(grow + c0, same);
        } else {
            for (int k = 0; k < G; ++k)
                if (c0 + k >= 0 && c0 + k < r.V) Elt<O>::store1(grow + c0 + k, value);
        }
    }
}

// Whether the row's whole vectors of columns are aligned in the gradient too.
template <typename S, typename O>
__device__ __forceinline__ bool grads_aligned(const rs::Row& r, const O* grow) {
    constexpr int G = Elt<S>::kGroup;
    return (reinterpret_cast<uintptr_t>(grow - r.shift) % (GroupStore<O, G>::kAlign)) == 0;
}

// +0.0 over a thread's U vectors of stage j of the slice.
template <typename S, typename O, int U, int NT>
__device__ __forceinline__ void write_zeros(const rs::Row& r, const Slice& s, int j, int tid, O* grow, bool vec) {
    Slice part{s.v0 + j * U * NT, min(s.n - j * U * NT, U * NT), 1};
    fill_grads<S, O>(r, part, grow, vec, tid, NT);
}

// The gradient of a thread's U vectors of stage j of the slice; the token's column takes c.gt.
// kEnt: c.c1 is not 0.  A mask's exponent of -inf is held at -200, as in the sums.
template <typename S, typename O, int U, int NT, bool kEnt>
__device__ __forceinline__ void write_grads(const uint4 (&x)[U], const rs::Row& r, const Slice& s, int j, int tid,
                                            O* grow, bool vec, const Coefs& c, float bias, float k2, int target) {
    constexpr int G = Elt<S>::kGroup;
    constexpr int B = U * NT;                        // vectors of a stage
    const int v0 = s.v0 + j * B + tid;
    const bool inside = vec && s.v0 + j * B >= r.iv0 && s.v0 + (j + 1) * B <= min(s.v0 + s.n, r.iv1);
    const int tv = target >= 0 ? (target + r.shift) / G - v0 : -1;   // the token's vector, from this thread's first
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        if (!inside && v >= s.v0 + s.n) continue;
        float g[G];
        Elt<S>::unpack(x[u], g);
#pragma unroll
        for (int k = 0; k < G; k += 2) {
            float a0, a1;
            ffma2(g[k], g[k + 1], k2, -bias, a0, a1);
            const float e0 = ex2(a0), e1 = ex2(a1);
            if (kEnt) {
                float f0, f1;
                ffma2(fmaxf(a0, -200.f), fmaxf(a1, -200.f), c.c1, c.c0, f0, f1);
                g[k] = e0 * f0;
                g[k + 1] = e1 * f1;
            } else {
                fmul2(e0, e1, c.c0, g[k], g[k + 1]);
            }
        }
        const int64_t c0 = (int64_t)v * G - r.shift;
        if (inside || (vec && v >= r.iv0 && v < r.iv1)) {
            GroupStore<O, G>::run(grow + c0, g);
        } else {
#pragma unroll
            for (int k = 0; k < G; ++k)
                if (c0 + k >= 0 && c0 + k < r.V) Elt<O>::store1(grow + c0 + k, g[k]);
        }
    }
    // over what this thread has just written there
    if (tv >= 0 && tv < B && tv % NT == 0 && v0 + tv < s.v0 + s.n) Elt<O>::store1(grow + target, c.gt);
}

}  // namespace lp
}  // namespace vce
