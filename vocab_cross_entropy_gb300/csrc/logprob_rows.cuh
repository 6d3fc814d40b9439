// A row's log-probability of one column, its entropy, and their gradient: the arithmetic shared by the
// post-training losses' kernels (policy_forward.cu, policy_grad.cu).
//
// Mathematics.  With k2 = log2(e) / temperature and "rest" the columns but the token's, one read of
// the row gives (m, s, w): s = sum 2^(z k2 - m), w = sum 2^(z k2 - m) (z k2 - m) over the rest.  Then
//   u = L' - x_t = ln 2 (m - z_t k2 + log2 s),   log p_t = -softplus(u),   1 - p_t = sigmoid(u)
//   H' = ln 2 (log2 s - w / s)                   the entropy of the rest among itself
//   H = p_t softplus(u) + (1 - p_t) (softplus(-u) + H')
// the chain rule of entropy: a sum of terms >= 0, so neither a confident row nor a flat one cancels.
// For a loss with derivatives a = dl/dlog p_t and b = dl/dH, p_j = f 2^(z_j k2 - m) with
// f = (1 - p_t) / s, and log p_j = ln 2 (z_j k2 - m) + ln f:
//   dl/dz_j = 2^y (c0 + c1 y), y = z_j k2 - m,   c0 = f (-a - b (ln f + H)) / T,  c1 = -b f ln 2 / T
//   dl/dz_t = (a (1 - p_t) - b p_t (log p_t + H)) / T
// The exponents are taken from m, not from the log-sum-exp: m is some z_j k2 (or a thread's first
// maximum), exact, where a log-sum-exp of size 16 would be rounded by 5e-7 of every p_j.  Where |m| is 2^31 or more
// the products z k2 are rounded first, in the sums and the gradient alike: logits of that size (masks such as -1e10
// in a row of nothing larger) count as equal where the products round to the same number.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "row_stream.cuh"
#include "vce_device.cuh"

namespace vce {
namespace lp {

using rs::beyond;
using rs::count_of;
using rs::kLarge;
using rs::kLn2;
constexpr float kLn2Lo = -1.90465431e-9f;            // ln 2 = kLn2 + kLn2Lo

// The factor 2^d, d < 0, that brings a thread's, a warp's or a block's sums to another's reference.  All of a sum is
// multiplied by it, up to three times a row, and the hardware's base-2 exponential is low by 4.4e-8 on the mean, which
// is added: the mean errors of log p_t over fp32 rows of 4000, 32000 and 128256 columns are 7.2e-8, 9.4e-8 and 1.3e-7
// without it.  What a row's own terms are off by is not known beforehand: 1 to 5e-8 is left, 7e-8 with clusters of eight.
__device__ __forceinline__ float factor(float d) {
    const float e = ex2(d);
    return fmaf(e, 4.4e-8f, e);
}

__device__ __forceinline__ float nan_f() { return __int_as_float(0x7FC00000); }

// ---- (reference, sum, sum of products): s = sum 2^y, y = z k2 - m, and by kind w = nothing, sum 2^y z (for the
// mean logit) or sum 2^y y (for the entropy) ---------------------------------------------------------------

enum Kind { kSum = 0, kMean = 1, kEntropy = 2 };

struct Sums {
    float m, s, w;
};

// log2(e) / temperature as hi + lo.  The exponents take hi alone, which is off by up to 2^-25 of itself: the
// logarithm of a sum is then off by ln 2 lo E[z], 5e-8 at E[z] = 4, alike for all rows, which a sum over a
// sequence's rows would add up.  E[z] comes out of w, and what is known to be missing is added.  (Adding z lo to
// the exponents does nothing: they are rounded by more than that.)
struct Scale {
    float hi, lo;
};

// (s, w) to the reference M >= m.
template <int kKind>
__device__ __forceinline__ void rescale(Sums& x, float M) {
    const float d = x.m - M;
    const float e = (x.m == M) ? 1.f : factor(d);
    if (kKind == kEntropy) x.w = e == 0.f ? 0.f : e * (x.m == M ? x.w : fmaf(d, x.s, x.w));
    if (kKind == kMean) x.w *= e;
    x.s *= e;
    x.m = M;
}

// Merges each kSpan lanes' sums, in all of them.
template <int kKind, int kSpan = 32>
__device__ __forceinline__ void warp_merge(Sums& x) {
    float M = x.m;
#pragma unroll
    for (int off = kSpan / 2; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
    rescale<kKind>(x, M);
#pragma unroll
    for (int off = kSpan / 2; off > 0; off >>= 1) {
        x.s += __shfl_xor_sync(0xFFFFFFFFu, x.s, off);
        if (kKind != kSum) x.w += __shfl_xor_sync(0xFFFFFFFFu, x.w, off);
    }
}

// (d0, d1) = (a0 * b0 + c0, a1 * b1 + c1) in one packed instruction.
__device__ __forceinline__ void ffma2v(float a0, float a1, float b0, float b1, float c0, float c1, float& d0, float& d1) {
    asm("{\n\t.reg .b64 pa, pb, pc, pd;\n\t"
        "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\tmov.b64 pc, {%6, %7};\n\t"
        "fma.rn.f32x2 pd, pa, pb, pc;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}

// (d0, d1) = (a0 * b0, a1 * b1) in one packed instruction.
__device__ __forceinline__ void fmul2v(float a0, float a1, float b0, float b1, float& d0, float& d1) {
    asm("{\n\t.reg .b64 pa, pb, pd;\n\t"
        "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "mul.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// Adds a vector's terms against the reference m: even and odd values apart, two to an instruction, since the
// issue slots are what these kernels run short of.  For the entropy an exponent of -inf (a mask) is held at -200,
// whose power of two is 0; for the mean a mask makes w NaN, and push takes the reference's logit for the batch's mean
// instead.  A NaN stays one (in s).
template <int G, int kKind>
__device__ __forceinline__ void add_sums(const float (&v)[G], float k2, float m, float& s0, float& s1, float& w0,
                                         float& w1) {
#pragma unroll
    for (int i = 0; i < G; i += 2) {
        float a0, a1;
        ffma2(v[i], v[i + 1], k2, -m, a0, a1);
        const float e0 = ex2(a0), e1 = ex2(a1);
        rs::fadd2(s0, s1, e0, e1, s0, s1);
        if (kKind == kEntropy) ffma2v(e0, e1, fmaxf(a0, -200.f), fmaxf(a1, -200.f), w0, w1, w0, w1);
        if (kKind == kMean) ffma2v(e0, e1, v[i], v[i + 1], w0, w1, w0, w1);
    }
}

// s and w of a thread's vectors against the reference m.
template <int G, int U, int kKind>
__device__ __forceinline__ void sums_of(const float (&v)[U][G], float k2, float m, float& s, float& w) {
    float s0[U], s1[U], w0[U], w1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        s0[u] = s1[u] = w0[u] = w1[u] = 0.f;
        add_sums<G, kKind>(v[u], k2, m, s0[u], s1[u], w0[u], w1[u]);
    }
#pragma unroll
    for (int d = 1; d < U; d *= 2)
#pragma unroll
        for (int u = 0; u + d < U; u += 2 * d) {
            rs::fadd2(s0[u], s1[u], s0[u + d], s1[u + d], s0[u], s1[u]);
            if (kKind != kSum) rs::fadd2(w0[u], w1[u], w0[u + d], w1[u + d], w0[u], w1[u]);
        }
    s = s0[0] + s1[0];
    w = w0[0] + w1[0];
}

// A batch of a thread's vectors.
template <int G, int U>
struct Batch {
    float v[U][G];
};

template <int G, int U, int kKind>
__device__ __forceinline__ void add(Sums& x, float s, float w, float k2) {
    x.s += s;
    if (kKind == kMean && !(fabsf(w) < kInf)) w = s * (x.m / k2);
    if (kKind != kSum) x.w += w;
}

// A batch whose reference moves, or is large: then it is the row's largest rounded product so far, and the sum counts
// the logits whose products round to it (any other is 2^7 or more below).  The exponent of a mask of -1e10 with its
// own rounded product for a reference would be up to 2^9 in size.
template <int G, int U, int kKind>
__device__ __forceinline__ Sums push_moving(const Batch<G, U>& b, Sums x, float k2) {
    const float top = rs::max_of<G>(b.v) * k2;
    if (!(top <= x.m)) rescale<kKind>(x, top);       // (a NaN: s is one then)
    if (beyond(x.m)) {
        x.s += count_of(b.v, k2, x.m);
        return x;
    }
    float s, w;
    sums_of<G, U, kKind>(b.v, k2, x.m, s, w);
    add<G, U, kKind>(x, s, w, k2);
    return x;
}

// The same by a call: in the loop of the sums its code costs the one pass 2.4% (16384 x 128256).
template <int G, int U, int kKind>
__device__ __noinline__ Sums call_moving(Batch<G, U> b, Sums x, float k2) {
    return push_moving<G, U, kKind>(b, x, k2);
}

// Adds a thread's vectors of a stage; the reference moves only when a term would pass 2^32, or where it is large.
template <int G, int U, int kKind, bool kCall = true>
__device__ __forceinline__ void push(const float (&v)[U][G], Sums& x, float k2) {
    bool moving = false;
    if (!(fabsf(x.m) < kLarge)) {
        const float top = rs::max_of<G>(v) * k2;
        if (x.m == -kInf && top == -kInf) return;
        moving = x.m != -kInf || beyond(top);
        if (!moving) x.m = top;
    }
    if (!moving) {
        float s, w;
        sums_of<G, U, kKind>(v, k2, x.m, s, w);
        moving = !(s < 4294967296.f);
        if (!moving) add<G, U, kKind>(x, s, w, k2);
    }
    if (moving) {
        Batch<G, U> b;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < G; ++k) b.v[u][k] = v[u][k];
        x = kCall ? call_moving<G, U, kKind>(b, x, k2) : push_moving<G, U, kKind>(b, x, k2);
    }
}

// ---- a row's scalars ---------------------------------------------------------------------------------

// What a row's sums and its token's logit say.  dead: nothing but masks (everything NaN, no gradient).
struct Row {
    float m, f, lp, lp_lo, ent;   // lp + lp_lo: log p_t to about twice the digits
    float pt, pnt, lnf;           // p_t, 1 - p_t, ln f
    bool dead;
};

// c - a b as hi + lo.
__device__ __forceinline__ float minus_product(float c, float a, float b, float& lo) {
    const float p = a * b, pe = fmaf(a, b, -p);
    const float hi = c - p, t = hi - c;
    lo = ((c - (hi - t)) + (-p - t)) - pe;           // Knuth's TwoSum of c and -p
    return hi;
}

// The logarithm of a normal s > 0 as an integer's worth of ln 2 and the logarithm of a number near 1.
__device__ __forceinline__ float split_log(float s, float& near) {
    const int e = (__float_as_int(s) - 0x3F3504F3) >> 23;    // s = 2^e r, r in [sqrt 1/2, sqrt 2)
    near = logf(__int_as_float(__float_as_int(s) - (e << 23)));
    return (float)e;
}

template <int kKind>
__device__ __forceinline__ Row finish(const Sums& x, float zt, Scale k) {
    const float k2 = k.hi;
    Row r;
    r.dead = false;
    r.lp_lo = 0.f;
    const bool rest = x.s > 0.f, tok = zt * k2 > -kInf;
    if (!(x.s >= 0.f && x.s < kInf && zt * k2 < kInf)) {   // a NaN or +inf somewhere
        r.m = 0.f;
        r.f = r.lp = r.ent = r.pt = r.pnt = r.lnf = nan_f();
        return r;
    }
    if (!rest) {                                     // p_t = 1, or nothing at all
        r.dead = !tok;
        r.m = r.f = r.pnt = 0.f;
        r.pt = 1.f;
        r.lnf = -kInf;
        r.lp = r.ent = tok ? 0.f : nan_f();
        return r;
    }
    float near;
    const float e = split_log(x.s, near);
    // what the scale's low part leaves out
    const float ratio = kKind == kSum ? 0.f : x.w / x.s;
    const float mean = kKind == kMean ? ratio : (ratio + x.m) / k2;
    const float hrest = kKind == kEntropy ? fmaxf(0.f, fmaf(e - ratio, kLn2, near)) : 0.f;   // (of either side as much)
    const bool large = beyond(x.m);                  // then the scale's low part is lost
    if (kKind != kSum && !large && fabsf(mean) < kInf) near += kLn2 * k.lo * mean;
    r.m = x.m;
    const float lns = fmaf(e, kLn2, near);
    if (!tok) {
        r.f = 1.f / x.s;
        r.pt = 0.f;
        r.pnt = 1.f;
        r.lnf = -lns;
        r.lp = -kInf;
        r.ent = hrest;
        return r;
    }
    float lo;
    float gap = minus_product(x.m, zt, k2, lo);
    if (kKind != kSum) lo -= zt * k.lo;              // as the sum's side: one alone is off by the logits' common offset
    if (large) gap = __fsub_rn(x.m, __fmul_rn(zt, k2)), lo = 0.f;   // as the terms of the sum
    const float g = gap + e, t = g - gap;            // TwoSum of gap and e
    lo += (gap - (g - t)) + (e - t);
    float u = g * kLn2;
    float ul = fmaf(g, kLn2, -u) + fmaf(g, kLn2Lo, fmaf(lo, kLn2, near));
    if (!(fabsf(u) < kInf)) ul = 0.f;
    const float v = u + ul;
    ul = fabsf(u) < kInf ? ul - (v - u) : 0.f;
    u = v;
    // softplus of u + ul, and of its negative
    const float E = expf(-fabsf(u)), l = log1pf(E), d = 1.f / (1.f + E);
    const float pnt = u >= 0.f ? d : E * d, pt = u >= 0.f ? E * d : d;
    const float sp = u >= 0.f ? u + l : l, spn = u >= 0.f ? l : l - u;
    r.lp = -sp;
    r.lp_lo = u >= 0.f && u < kInf ? -((u - (sp - l)) + (l - (sp - (sp - l))) + ul * pnt) : -ul * pnt;
    if (u < 0.f) {
        const float a = r.lp + r.lp_lo;
        r.lp_lo -= a - r.lp;
        r.lp = a;
    }
    r.ent = (pt > 0.f ? pt * sp : 0.f) + (pnt > 0.f ? pnt * (spn + hrest) : 0.f);
    r.f = pnt / x.s;
    r.pt = pt;
    r.pnt = pnt;
    r.lnf = -spn - lns;
    return r;
}

// The gradient's coefficients (see above), lnf being ln f.
struct Coefs {
    float c0, c1, gt;
};
__device__ __forceinline__ Coefs coefs_of(float f, float lnf, float pt, float pnt, float lp, float ent, float a, float b,
                                          float inv_tau) {
    Coefs c;
    c.gt = inv_tau * (a * pnt - (b != 0.f && pt > 0.f ? b * pt * (lp + ent) : 0.f));
    c.c0 = c.c1 = 0.f;
    if (f != 0.f) {
        c.c0 = inv_tau * f * (b != 0.f ? -a - b * (lnf + ent) : -a);
        c.c1 = b != 0.f ? -inv_tau * f * b * kLn2 : 0.f;
    }
    if (f != f || lp != lp) c.c0 = c.gt = nan_f();
    return c;
}
// From what is saved of a row.
__device__ __forceinline__ Coefs coefs(float f, float lp, float ent, float a, float b, float inv_tau) {
    return coefs_of(f, b != 0.f ? logf(f) : 0.f, expf(lp), -expm1f(lp), lp, ent, a, b, inv_tau);
}

}  // namespace lp
}  // namespace vce
