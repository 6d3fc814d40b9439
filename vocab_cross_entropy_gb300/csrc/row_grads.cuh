// Writing the gradients 2^y (c0 + c1 y), y = z k2 - bias, of a row's vectors (logprob_rows.cuh).  The token's entry
// is the caller's to write over them.
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

// The gradients of a vector's G logits, in their place.  kEnt: c.c1 is not 0.  A mask's exponent of -inf is
// held at -200 there, as in the sums.
template <int G, bool kEnt>
__device__ __forceinline__ void grads_of(float (&g)[G], const Coefs& c, float bias, float k2) {
#pragma unroll
    for (int k = 0; k < G; k += 2) {
        float a0, a1;
        ffma2(g[k], g[k + 1], k2, -bias, a0, a1);
        const float e0 = ex2(a0), e1 = ex2(a1);
        if (kEnt) {
            float f0, f1;
            ffma2(fmaxf(a0, -200.f), fmaxf(a1, -200.f), c.c1, c.c0, f0, f1);
            fmul2v(e0, e1, f0, f1, g[k], g[k + 1]);
        } else {
            fmul2(e0, e1, c.c0, g[k], g[k + 1]);
        }
    }
}

// A vector of the row from its first column c0 on (before the row's start where it is partial), element by
// element: partial vectors, gradients that are not aligned as the logits are, and rows with a large bias, whose
// products with k2 are rounded first, as they were in the sums.
template <typename S, typename O>
__device__ __noinline__ void write_single(uint4 x, int64_t c0, int64_t V, O* grow, Coefs c, float bias, float k2) {
    constexpr int G = Elt<S>::kGroup;
    float g[G];
    Elt<S>::unpack(x, g);
    if (beyond(bias)) {
#pragma unroll
        for (int k = 0; k < G; ++k) g[k] *= k2;
        k2 = 1.f;
    }
    grads_of<G, true>(g, c, bias, k2);
#pragma unroll
    for (int k = 0; k < G; ++k)
        if (c0 + k >= 0 && c0 + k < V) Elt<O>::store1(grow + c0 + k, g[k]);
}

// The gradients of U vectors of a thread, vector v0 + u * NT of the row each, the slice's end at v1.  fast: all of
// them lie wholly in the row and the slice, and are aligned in the gradient too.  vec, fast: not with a large bias.
template <typename S, typename O, int U, int NT, bool kEnt>
__device__ __forceinline__ void write_grads(const uint4 (&x)[U], const rs::Row& r, int v0, int v1, bool fast, O* grow,
                                            bool vec, const Coefs& c, float bias, float k2) {
    constexpr int G = Elt<S>::kGroup;
    if (fast) {
        O* p = grow + ((int64_t)v0 * G - r.shift);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float g[G];
            Elt<S>::unpack(x[u], g);
            grads_of<G, kEnt>(g, c, bias, k2);
            GroupStore<O, G>::run(p + u * NT * G, g);
        }
        return;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = v0 + u * NT;
        if (v >= v1) continue;
        const int64_t c0 = (int64_t)v * G - r.shift;
        if (vec && v >= r.iv0 && v < r.iv1) {
            float g[G];
            Elt<S>::unpack(x[u], g);
            grads_of<G, kEnt>(g, c, bias, k2);
            GroupStore<O, G>::run(grow + c0, g);
        } else {
            write_single<S, O>(x[u], c0, r.V, grow, c, bias, k2);
        }
    }
}

}  // namespace lp
}  // namespace vce
