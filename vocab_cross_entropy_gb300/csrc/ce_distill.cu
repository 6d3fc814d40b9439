// Distillation loss against a teacher's top K logits, its gradient, and both in one pass.
//
// Mathematics (one row, scale s = 1 / temperature; "top" the K columns of the teacher's entries,
// "tail" the other columns).  With log-sum-exps Lq, R of the teacher's top and tail, and Lr, L' of
// the student's (L' summed without the top columns, as the cross-entropy's forward leaves out its
// target), the masses are logistic functions of two numbers,
//     Q = sigma(a), q_T = sigma(-a), a = Lq - R;    P = sigma(b), p_T = sigma(-b), b = Lr - L',
// and with qh_k = e^{s t_k - Lq}, r_k = e^{s z_k - Lr}, phi(x) = e^x - 1 - x >= 0:
//     KL = Q phi(log P/Q) + q_T phi(log p_T/q_T) + Q sum_k qh_k phi(log r_k/qh_k)
// (the linear terms add up to 0, since p and q sum to 1), a sum of terms >= 0: nothing cancels
// when the student matches its teacher, nor when one column holds all the mass.  The gradient of
// tau^2 KL is tau (p - q):
//     tail:  tau (p_T - q_T) e^{s z_j - L'}        top:  tau [Q (r_k - qh_k) + (q_T - p_T) r_k]
// with p_T - q_T a difference of logistic functions taken as a product (sigmoid_diff).
//
// Kernels.
//   k_distill_ring     forward, and loss and gradient in one pass: persistent, warps with roles, the
//                      columns streamed through a shared-memory ring (described where it stands)
//   k_distill_long     one pass over rows that a cluster's shared memory does not hold
//   k_distill_bwd      the gradient alone, from the saved statistics
//   k_distill_reduce   the losses' sum in a fixed order, the rows' weights, the status word
//   k_distill_count    N, before a one-pass call with MEAN
// Nothing is shared between launches.
//
// What bounds them, bf16 with 64 entries a row: the forward reads the logits once (4096 x 128256: 160 us,
// 6.6 TB/s, 0.97 of the measured copy), one pass also writes the gradient (16384 x 128256: 1424 us, 5.9
// TB/s, 0.87; a row's exponentials are taken twice, 17 warp instructions for 32 columns where the
// copy's time leaves 24), the backward runs at the copy's speed (4096 x 128256: 307 us).  Short rows cost
// the consumer warps about 1 us beside their columns: 4096 rows of 32000 take 78 us forward (3.4 TB/s)
// and 134 us in one pass (3.9 TB/s).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ce_fold.cuh"
#include "row_launch.h"
#include "row_stream.cuh"
#include "vce_logits.h"

namespace vce {
namespace distill {

using namespace rs;

constexpr int kProducerWarp = kConsumerWarps, kTopWarp = kConsumerWarps + 1;
constexpr int kThreads = kConsumers + 64;
constexpr int kPerLane = VCE_MAX_TOPK / 32;   // entries per lane of the top warp

struct Args {
    const void* logits;
    int64_t T, V, ld;
    const int64_t* ids;
    const void* tvals;
    const float* tail;
    int K, tbf16;
    float tau, scale, k2;        // temperature, 1 / temperature, log2(e) / temperature
    const int64_t* labels;
    int64_t ignore_index;
    int red;
    const float* go;             // kGrad
    const float* inv_n;          // kGrad, MEAN
    float* loss_rows;
    float4* row_stats;
    float* top_grads;            // forward alone
    void* grad;                  // kGrad
    int64_t ld_g;
    int cluster;
    int nbuf, max_stages;        // k_distill_long
    uint64_t wait_ns;            // bound of every wait
    int withhold;                // n > 0 (test hook): in a cluster's block n - 1 the gradient waits in vain
};

// Of a row's entries: the largest logits z, t of the student and the teacher, the sums of e^{s (z - max)}
// and e^{s (t - max)} (0: no mass, NaN stays), and sum qh phi(log r/qh).
struct Top {
    float zmax, zsum, tmax, tsum, kl;
    float wt, q, inv_z;          // wt = q_T / Q (see Finish), Q = 1 / (1 + wt), 1 / zsum
};

struct alignas(16) Ctl {
    float4 slot[kMaxCluster];    // (max, sum-exp, error code, -) of the cluster's blocks
    Barriers bar;
    float red_m[kConsumerWarps], red_s[kConsumerWarps];
    Top top;                     // of the entries
    int code;                    // error found among the entries
    int skip;                    // the row is ignored
};

struct alignas(8) Entry {        // of each teacher entry
    float r, diff;               // r_k, r_k - qh_k
    int col;                     // column, -1: none
    int pad;
};

__host__ __device__ constexpr int smem_bytes(int nbuf, int max_stages, int K) {
    return nbuf * kStageBytes + max_stages * kConsumers * 4 + (K * (int)sizeof(Entry) + 15) / 16 * 16 +
           (int)sizeof(Ctl);
}

// ---- scalar functions --------------------------------------------------------------------------

__device__ __forceinline__ float sigmoid(float x) {
    const float e = expf(-fabsf(x));
    return (x >= 0.f ? 1.f : e) / (1.f + e);
}

// sigma(u) - sigma(v), without cancellation: for u > v, sigma(u) sigma(-v) (1 - e^{v-u}).
__device__ __forceinline__ float sigmoid_diff(float u, float v) {
    if (u == v) return 0.f;
    const float hi = fmaxf(u, v), lo = fminf(u, v);
    const float d = sigmoid(hi) * sigmoid(-lo) * -expm1f(lo - hi);
    return u > v ? d : -d;
}

// q phi(x), phi(x) = e^x - 1 - x, where p = q e^x: the power series of phi near 0 (to x^9 / 9!,
// 2e-9 relative at 0.5), else e^x - 1 - x, which loses at most two bits there.  Everything comes from
// x, not from p: an error common to all x_k (a log-sum-exp's) then leaves the sum of the terms as it
// is to first order, since both sides sum to 1.
__device__ __forceinline__ float q_phi(float q, float p, float x) {
    if (!(q > 0.f)) return p;
    if (fabsf(x) < 0.5f) {
        float c = 1.f / 362880.f;
        c = fmaf(c, x, 1.f / 40320.f);
        c = fmaf(c, x, 1.f / 5040.f);
        c = fmaf(c, x, 1.f / 720.f);
        c = fmaf(c, x, 1.f / 120.f);
        c = fmaf(c, x, 1.f / 24.f);
        c = fmaf(c, x, 1.f / 6.f);
        c = fmaf(c, x, 0.5f);
        return q * (x * x * c);
    }
    return x < 80.f ? q * (expm1f(x) - x) : (p - q) - q * x;   // e^x would overflow
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// ---- gradient entries ---------------------------------------------------------------------------

// Writes the gradient coef 2^(z k2 - bias) of a thread's U vectors of a stage (zero: +0.0 whatever
// they hold).  vec: the row's gradient vectors are aligned for GroupStore.
template <typename S, typename O, int U, int NT>
__device__ __forceinline__ void write_grads(const uint4 (&x)[U], const Row& r, const Slice& s, int j, int tid,
                                            O* grow, bool vec, float coef, float k2, float bias, bool zero = false) {
    constexpr int G = Elt<S>::kGroup;
    constexpr int B = U * NT;                        // vectors of a stage
    const int v0 = s.v0 + j * B + tid;
    const bool inside = vec && s.v0 + j * B >= r.iv0 && s.v0 + (j + 1) * B <= min(s.v0 + s.n, r.iv1);
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
            fmul2(ex2(a0), ex2(a1), coef, g[k], g[k + 1]);
        }
        if (zero) {
#pragma unroll
            for (int k = 0; k < G; ++k) g[k] = 0.f;
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
}

// One value (+0.0 for a row without a gradient) over the slice's columns, by NT threads.
template <typename S, typename O>
__device__ __forceinline__ void fill_grads(const Row& r, const Slice& s, O* grow, bool vec, int tid, int NT,
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

template <typename S, typename O>
__device__ __forceinline__ bool grads_aligned(const Row& r, const O* grow) {
    constexpr int G = Elt<S>::kGroup;
    return (reinterpret_cast<uintptr_t>(grow - r.shift) % (GroupStore<O, G>::kAlign)) == 0;
}

// ---- a row's scalars -------------------------------------------------------------------------------

// c - a b as hi + lo: the rounding of a result of size 8 is what is lost most of in its exponential.
__device__ __forceinline__ float minus_product(float c, float a, float b, float& lo) {
    const float p = a * b, pe = fmaf(a, b, -p);
    const float hi = c - p, t = hi - c;
    lo = ((c - (hi - t)) + (-p - t)) - pe;           // Knuth's TwoSum of c and -p
    return hi;
}

// All arithmetic on the K entries, by one warp (lane + 32 i: entry k; col -1: none, z, t -inf there):
// each entry's (r_k, r_k - qh_k), and the scalars of Top.
__device__ __forceinline__ Top top_arithmetic(const Args& a, int K, int lane, const int (&col)[kPerLane],
                                               float (&z)[kPerLane], const float (&t)[kPerLane], Entry* entry,
                                               float R) {
    float zm = -kInf, tm = -kInf;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        if (z[i] * a.k2 <= -kLarge) z[i] = -kInf;   // masks, as in the tail's pairs
        zm = fmaxf(zm, z[i]);
        tm = fmaxf(tm, t[i]);
    }
    zm = warp_max(zm);
    tm = warp_max(tm);
    float rs_ = 0.f, qs = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        if (32 * i >= K) break;
        if (z[i] != -kInf) rs_ += exp2f((z[i] - zm) * a.k2);   // as the tail's terms; NaN and +inf: NaN
        if (col[i] >= 0 && t[i] != -kInf) qs += expf((t[i] - tm) * a.scale);   // NaN: the row is refused
    }
    rs_ = warp_sum(rs_);
    qs = warp_sum(qs);
    const float ln = logf(rs_) - logf(qs), inv_r = 1.f / rs_, inv_q = 1.f / qs;
    float kl = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int k = lane + 32 * i;
        if (32 * i >= K) break;
        if (k >= K) continue;
        float rk = 0.f, diff = 0.f;
        if (col[i] >= 0) {
            float qk = 0.f, y = -kInf;
            if (z[i] > -kInf) rk = exp2f((z[i] - zm) * a.k2) * inv_r;
            if (t[i] > -kInf) qk = expf((t[i] - tm) * a.scale) * inv_q;
            if (z[i] > -kInf && t[i] > -kInf) {
                // log(r_k / qh_k): differences of logits first, which are exact or nearly so
                y = ((z[i] - zm) - (t[i] - tm)) * a.scale - ln;
                diff = y < 0.5f ? qk * expm1f(y) : rk - qk;
            } else {
                diff = rk - qk;
            }
            kl += q_phi(qk, rk, y);
        }
        entry[k] = Entry{rk, diff, col[i], 0};
    }
    kl = warp_sum(kl);
    float lo;
    const float hi = minus_product(R, tm, a.scale, lo);
    const float wt = expf(hi) * (fabsf(lo) < 1.f ? 1.f + lo : 1.f) * inv_q;   // lo: NaN where hi is infinite
    return Top{zm, rs_, tm, qs, kl, wt, 1.f / (1.f + wt), inv_r};
}

// What the gradient needs of a row's masses, in few dependent steps (consumers wait for it), and what
// the loss needs besides.  The masses of the student and the teacher enter as the ratios
// ws = p_T / P = e^-b and wt = q_T / Q = e^-at: a logarithm of size 8 is rounded by 5e-7, which is all
// the loss's error where the masses are nearly alike, a ratio by 6e-8 of itself.
struct Finish {
    float lt, bias, d, q;        // L', L' log2(e), p_T - q_T, Q
    float ws, wt;
    int code;                    // the row's error
    bool ratios;                 // ws and wt are within range: else the logarithms at and b are used
    bool dead;                   // no gradient (an error, or a student row of masks only)
    float at, b;
};

// From the tail's pair (M, S0), the entries' scalars and the teacher's tail R.
__device__ __forceinline__ Finish finish_row(const Args& a, float M, float S0, const Top& t, float R, int code) {
    Finish f;
    f.code = code;
    // no finite teacher mass (comparisons that a NaN fails)
    if (!code && !((t.tsum > 0.f || R > -kInf) && t.tsum < kInf && R < kInf)) f.code = VCE_ERR_TEACHER;
    const bool has_tail = S0 > 0.f, has_top = t.zmax > -kInf;
    bool lost = false;                               // a NaN or +inf among the student's logits: NaN throughout
    float lo;
    const float gap = minus_product(M, t.zmax, a.k2, lo);
    // expf for this one factor, not the base-2 exponential: that one's error has a mean of 5e-8, which the
    // sums of both sides share
    const float x = gap * kLn2;
    lo = fmaf(gap, kLn2, -x) + fmaf(gap, -1.90465431e-9f, lo * kLn2);   // ln 2 = kLn2 - 1.90465431e-9
    f.ws = S0 * t.inv_z * expf(x) * (fabsf(lo) < 1.f ? 1.f + lo : 1.f);
    f.wt = t.wt;
    f.ratios = f.ws > 1e-30f && f.ws < 1e30f && (f.wt > 1e-30f || R == -kInf) && f.wt < 1e30f;
    f.at = f.b = 0.f;
    if (f.ratios) {
        f.q = t.q;
        f.d = (f.ws - f.wt) * f.q / (1.f + f.ws);
    } else {
        if (has_tail && has_top) f.b = (logf(t.zsum) - logf(S0)) - gap * kLn2;
        else f.b = has_top ? kInf : -kInf;
        f.at = t.tsum > 0.f ? (t.tmax * a.scale - R) + logf(t.tsum) : -kInf;   // R = -inf: +inf
        f.q = sigmoid(f.at);
        f.d = sigmoid_diff(-f.b, -f.at);             // p_T - q_T
        lost = !(S0 + t.zsum >= 0.f);                // then ws is no ratio within range either
    }
    f.dead = f.code || !(has_tail || has_top || lost);
    f.bias = has_tail ? M + log2f(S0) : 0.f;         // of the tail's gradient: 2^(z k2 - bias); no tail: any
    f.lt = has_tail ? f.bias * kLn2 : -kInf;
    if (lost) f.q = f.d = f.lt = __int_as_float(0x7FC00000);
    return f;
}

// tau^2 KL from the row's masses and the entries' sum of qh phi; NaN where there is no loss.
__device__ __forceinline__ float loss_of(const Args& a, const Finish& f, float kl_top) {
    float x1, x2, P, pT, qT;                         // log P/Q, log p_T/q_T
    if (f.ratios) {
        const float d = f.ws - f.wt, r = f.ws / f.wt;
        const float q = -d / (1.f + f.ws);
        x1 = q > -0.5f && q < 1.f ? log1pf(q) : log1pf(f.wt) - log1pf(f.ws);
        x2 = x1 + (r > 0.5f && r < 2.f ? log1pf(d / f.wt) : logf(r));
        P = 1.f / (1.f + f.ws);
        pT = f.ws * P;
        qT = f.wt * f.q;
    } else {
        x1 = softplus_f(-f.at) - softplus_f(-f.b);
        x2 = softplus_f(f.at) - softplus_f(f.b);
        P = sigmoid(f.b);
        pT = sigmoid(-f.b);
        qT = sigmoid(-f.at);
    }
    float kl = q_phi(f.q, P, x1) + q_phi(qT, pT, x2);
    if (f.q > 0.f) kl += f.q * kl_top;
    return f.dead || f.q != f.q ? __int_as_float(0x7FC00000) : a.tau * a.tau * kl;
}

// ---- one pass over rows longer than shared memory ----------------------------------------------------
//
// One cluster of eight blocks a row, every slice streamed twice (the second time mostly from L2): the
// entries' columns are left out of the sums by a bitmap, a word per consumer thread and stage.

template <typename S, typename O>
__global__ void __launch_bounds__(kThreads, 2) k_distill_long(const __grid_constant__ Args a) {
    constexpr int G = Elt<S>::kGroup;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* bufs = smem;
    uint32_t* marks = reinterpret_cast<uint32_t*>(smem + a.nbuf * kStageBytes);
    Entry* entry = reinterpret_cast<Entry*>(marks + a.max_stages * kConsumers);
    Ctl& ctl = *reinterpret_cast<Ctl*>(reinterpret_cast<uint8_t*>(entry) + (a.K * (int)sizeof(Entry) + 15) / 16 * 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = a.cluster;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int64_t row = blockIdx.x / C;
    const Row r = make_row<S>(a.logits, row, a.ld, a.V);
    const Slice sl = make_slice(r, C, rank);
    start_next();
    const int64_t* ids = a.ids + row * a.K;
    O* grow = static_cast<O*>(a.grad) + row * a.ld_g;
    const bool vec = grads_aligned<S, O>(r, grow);

    // A row without a teacher or with the ignored label: nothing of it is read (all blocks alike; were the
    // teacher written meanwhile they might not be, so one thread looks for a block, and a block that skips the
    // row stays while others may write into it).
    if (tid == 0) ctl.skip = ids[0] == -1 || (a.labels && a.labels[row] == a.ignore_index);
    __syncthreads();
    if (ctl.skip) {
        if (rank == 0 && tid == 0) {
            a.loss_rows[row] = 0.f;
            a.row_stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        fill_grads<S, O>(r, sl, grow, vec, tid, kThreads);
        if (a.red == VCE_RED_MEAN) wait_previous();
        if (C > 1)
            for (int i = 0; i < 3; ++i) cluster_arrive(), cluster_wait();   // as many as below
        return;
    }

    // the slice is copied twice; of its second round, the ring's first fill goes out before the
    // statistics are done (later stages wait for the gradient to release theirs)
    const int total = 2 * sl.nst - (a.withhold == rank + 1);
    const int early = min(total, sl.nst + a.nbuf);
    int issued = 0;
    if (tid == kProducerWarp * 32) {
        init_barriers(ctl.bar, a.nbuf);
        ctl.code = 0;
        for (; issued < min(sl.nst, a.nbuf); ++issued)
            issue_stage(bufs, ctl.bar, a.nbuf, r, sl, issued, issued, a.wait_ns);
    }
    if (C > 1) cluster_arrive();                     // this block runs: peers may write into it
    for (int i = tid; i < sl.nst * kConsumers; i += kThreads) marks[i] = 0;
    __syncthreads();

    // the entries: columns, marks
    int col[kPerLane];
    if (warp == kTopWarp) {
        int bad = 0;
        int64_t id[kPerLane];
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) id[i] = lane + 32 * i < a.K ? ids[lane + 32 * i] : -1;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            col[i] = id[i] >= 0 && id[i] < a.V ? (int)id[i] : -1;
            bad |= id[i] != -1 && col[i] < 0;
            if (col[i] >= 0) {
                const int at = col[i] + r.shift, v = at / G - sl.v0;
                if (v >= 0 && v < sl.n) {
                    const int j = v / kStageVecs, w = v % kStageVecs;
                    const uint32_t bit = 1u << ((w / kConsumers) * G + at % G);
                    bad |= (atomicOr(&marks[j * kConsumers + w % kConsumers], bit) & bit) != 0;
                }
            }
        }
        if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) ctl.code = VCE_ERR_TEACHER;
    }
    __syncthreads();

    if (warp == kProducerWarp) {
        if (lane == 0) {
            for (; issued < early; ++issued) {
                const int j = issued < sl.nst ? issued : issued - sl.nst;
                if (!issue_stage(bufs, ctl.bar, a.nbuf, r, sl, j, issued, a.wait_ns)) break;
            }
        }
    } else if (warp == kTopWarp) {
        // all arithmetic on the K entries, while the columns stream
        float z[kPerLane], t[kPerLane];
        const S* zrow = static_cast<const S*>(a.logits) + row * a.ld;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            const int k = lane + 32 * i;
            z[i] = t[i] = -kInf;
            if (col[i] >= 0) {
                z[i] = Elt<S>::load1(zrow + col[i]);
                t[i] = a.tbf16 ? Elt<uint16_t>::load1(static_cast<const uint16_t*>(a.tvals) + row * a.K + k)
                               : Elt<float>::load1(static_cast<const float*>(a.tvals) + row * a.K + k);
            }
        }
        const Top top = top_arithmetic(a, a.K, lane, col, z, t, entry, a.tail ? a.tail[row] : -kInf);
        if (lane == 0) ctl.top = top;
    } else {
        float m = -kInf, s = 0.f;
        for (int j = 0; j < sl.nst; ++j) {
            const uint32_t word = marks[j * kConsumers + tid];
            wait_stage(ctl.bar, a.nbuf, j, a.wait_ns);
            uint4 x[kU];
            load_stage<S>(bufs, a.nbuf, r, sl, j, j, tid, x);
            float v[kU][G];
#pragma unroll
            for (int u = 0; u < kU; ++u) Elt<S>::unpack(x[u], v[u]);
            if (word) {   // the entries' columns are left out
#pragma unroll
                for (int u = 0; u < kU; ++u)
#pragma unroll
                    for (int k = 0; k < G; ++k)
                        if ((word >> (u * G + k)) & 1u) v[u][k] = -kInf;
            }
            pair_push<G>(v, m, s, a.k2);
            release_stage(ctl.bar, a.nbuf, j);
        }
        pair_warp_reduce(m, s);
        if (lane == 0) {
            ctl.red_m[warp] = m;
            ctl.red_s[warp] = s;
        }
    }
    __syncthreads();

    // ---- the row's statistics, by every thread alike ----
    float M = -kInf, S0 = 0.f;
    for (int w = 0; w < kConsumerWarps; ++w) pair_merge(M, S0, ctl.red_m[w], ctl.red_s[w]);
    int code = ctl.bar.err ? ctl.bar.err : ctl.code;
    if (C > 1) {
        cluster_wait();                              // every peer runs
        if (tid < C) st_peer(peer_addr(&ctl.slot[rank], tid), make_float4(M, S0, __int_as_float(code), 0.f));
        cluster_arrive();
        cluster_wait();
        M = -kInf;
        S0 = 0.f;
        code = 0;
        for (int p = 0; p < C; ++p) {                // the same order in every block
            const float4 o = ctl.slot[p];
            pair_merge(M, S0, o.x, o.y);
            code = max(code, __float_as_int(o.z));
        }
    }
    const Finish f = finish_row(a, M, S0, ctl.top, a.tail ? a.tail[row] : -kInf, code);
    const bool dead = f.dead;
    if (rank == 0 && tid == kProducerWarp * 32) {
        a.loss_rows[row] = loss_of(a, f, ctl.top.kl);
        // weight: 1, negative for a row with an error, until the reduction writes it
        a.row_stats[row] = make_float4(f.lt, dead ? 0.f : f.d, 0.f, f.code ? -(float)f.code : 1.f);
    }
    if (C > 1) cluster_arrive();                     // the first block has written the loss
    if (dead) fill_grads<S, O>(r, sl, grow, vec, tid, kThreads);
    // k_distill_count: every block, with a gradient or without one, since the reduction waits for this kernel
    // alone and writes the word that the count does
    if (a.red == VCE_RED_MEAN) wait_previous();
    if (!dead) {
        const float c = a.go[a.red == VCE_RED_NONE ? row : 0] * (a.red == VCE_RED_MEAN ? *a.inv_n : 1.f) * a.tau;
        if (warp < kConsumerWarps) {
            const float coef = c * f.d, bias = f.bias;
            for (int j = 0; j < sl.nst; ++j) {
                const int q = sl.nst + j;
                wait_stage(ctl.bar, a.nbuf, q, a.wait_ns);
                uint4 x[kU];
                load_stage<S>(bufs, a.nbuf, r, sl, j, q, tid, x);
                write_grads<S, O, kU, kConsumers>(x, r, sl, j, tid, grow, vec, coef, a.k2, bias);
                release_stage(ctl.bar, a.nbuf, q);
            }
        } else if (tid == kProducerWarp * 32) {
            for (; issued < total; ++issued)
                if (!issue_stage(bufs, ctl.bar, a.nbuf, r, sl, issued - sl.nst, issued, a.wait_ns)) break;
        }
        __syncthreads();                             // the entries' gradients go over the tail's
        for (int k = tid; k < a.K; k += kThreads) {
            const Entry e = entry[k];
            const int v = e.col >= 0 ? (e.col + r.shift) / G - sl.v0 : -1;
            if (v >= 0 && v < sl.n && dbg::ok(e.col < a.V, dbg::kCols))
                Elt<O>::store1(grow + e.col, c * (f.q * e.diff - f.d * e.r));
        }
    }
    // copies that nothing waited for (after an abort, or of a row without a gradient) land first
    if ((ctl.bar.abort || dead) && tid == kProducerWarp * 32) drain(ctl.bar, a.nbuf, issued);
    // a wait for the second round gave up: the row's error, over what the first block wrote
    __syncthreads();
    if (C > 1) cluster_wait();
    if (ctl.bar.abort && tid == 0) {
        a.loss_rows[row] = __int_as_float(0x7FC00000);
        a.row_stats[row].w = -(float)ctl.bar.err;
    }
}

// ---- many rows: a persistent kernel -----------------------------------------------------------------
//
// Each block (a cluster of C of them per row) walks the rows cid, cid + ncl, ... with the copies
// of the next rows always in flight.  Its warps have roles, which hand rows on through mbarriers,
// everything that belongs to a row doubled by the parity of its number in the
// block's sequence (the entries by top warp):
//   producer        copies the rows' slices into the stage ring, running ahead as stages are released
//   patch           overwrites the entries' columns in the loaded stages with -inf, and writes the row's
//                   partial first and last vectors there, so the consumers' sums need not know of either
//   top 0 ..        (two, or four: each takes every second or fourth row) the arithmetic on the K entries
//   consumers       the tail's pair of a row; in one pass then the first stages of the next row, while
//                   this row's statistics are exchanged, this row's gradient from the held stages,
//                   releasing each, and the rest of the next row
//   stats           merges the warps' pairs and the cluster's, finishes the row, and writes the
//                   entries' gradients (in one pass once the consumers have written the row)
// Every role walks the same rows by itself (a lane looks at each of the next 32 rows' label and first
// id), so nothing has to be handed on about rows that are skipped.

namespace ring {

// Four forms, each direction's for rows of kLongRow bytes and more (kBig) and for shorter ones.
//  - Forward: of a long row one block an SM, 16 consumer warps and 32 KB stages (less to do per stage).
//    A short row costs a block's consumers about 1 us beside its columns (the merge of their pairs, the
//    hand-over, the next row's extent); so two blocks an SM take them, with 8 warps and 16 KB stages, and
//    each covers the other's (4096 x 32000 bf16: 80 us a call, and 102 with one block).
//  - One pass: one block an SM, whose shared memory holds a row and the beginning of the next (two blocks
//    at 4096 x 32000 bf16, measured when stages were released ahead of their use: 194 us against 125);
//    16 KB stages, so that a held row gives them back in small steps.  Two top warps have time enough for long
//    rows, short ones take four (16384 x 128256 bf16: 1427 us a call with two, 1526 with four; 1023 x 32001
//    bf16 to fp32: 75 and 65).
constexpr int64_t kLongRow = 131072;
template <bool kGrad, bool kBig>
struct Form {
    static constexpr bool kPair = !kGrad && !kBig;                            // two blocks an SM
    static constexpr int kBlocks = kPair ? 2 : 1;
    static constexpr int kWarps = kPair ? 8 : 16, kNT = kWarps * 32;          // consumers
    static constexpr int kTops = kGrad && !kBig ? 4 : 2;                      // top warps
    static constexpr int kProducer = kWarps, kPatch = kWarps + 1, kStats = kWarps + 2, kTop = kWarps + 3;
    static constexpr int kThreads = (kTop + kTops) * 32;
    static constexpr int kU = kGrad ? 2 : 4;                                  // vectors of a stage per consumer thread
    static constexpr int kVecs = kU * kNT, kBytes = kVecs * 16;               // of a stage
    static constexpr int kBufs = kGrad ? 13 : 6;
    static constexpr int kHeld = 8;                                           // stages of a slice that is held, at most
};
constexpr uint32_t kSuspend = 10000;                // ns a poll may sleep: waiting warps leave the issue slots to others
enum { kErrRow = 107, kErrPartials = 108, kErrCoefs = 109 };

struct TopStats {
    Top top;
    int code;
};
struct Coefs {                   // of the tail's gradient
    float coef, bias;            // coef 2^(z k2 - bias)
    int dead;
};

template <int kTops, int kWarps, int kBufs>
struct alignas(16) RingCtl {
    float4 slot[2][kMaxCluster];
    uint64_t full[kBufs], ready[kBufs], empty[kBufs];   // of the stages: copied, patched, released
    uint64_t topped[kTops];      // the entries' arithmetic (a top warp)
    uint64_t freed[kTops];       // the stats warp is done with the entries
    uint64_t paired[2];          // the consumer warps' pairs
    uint64_t exchanged[2];       // the cluster's pairs
    uint64_t finished[2];        // the row's coefficients (stats)
    uint64_t written[2];         // the tail's gradient (consumer warps)
    TopStats top[kTops];
    Coefs coefs[2];
    float red_m[2][kWarps], red_s[2][kWarps];
    int abort, err;
};

// A top warp's entries take at least as much room as its table of columns (for ids given twice), which
// lies there before: at least 2 K slots of 4 bytes, a power of two, 32 or more.
__host__ __device__ constexpr int entry_stride(int K) { return K > 8 ? K : 8; }

template <typename F>
using CtlOf = RingCtl<F::kTops, F::kWarps, F::kBufs>;

template <typename F>
__host__ __device__ constexpr int ring_smem(int K) {
    return F::kBufs * F::kBytes + F::kTops * entry_stride(K) * (int)sizeof(Entry) + (int)sizeof(CtlOf<F>) + 16;
}

// make_row without its address, in 32-bit arithmetic: what the consumers need of a row, each warp by itself.
template <typename S>
__device__ __forceinline__ Row row_extent(const Args& a, int64_t row) {
    constexpr int G = Elt<S>::kGroup;
    Row r;
    r.base = nullptr;
    r.V = a.V;
    const uint32_t off = ((uint32_t)reinterpret_cast<uintptr_t>(a.logits) + (uint32_t)row * ((uint32_t)a.ld * (uint32_t)sizeof(S))) & 15u;
    r.shift = (int)(off / sizeof(S));
    r.nv = ((int)a.V + r.shift + G - 1) / G;
    r.iv0 = r.shift ? 1 : 0;
    r.iv1 = ((int)a.V + r.shift) / G;
    return r;
}

// make_slice in stages of the ring.
template <typename F>
__device__ __forceinline__ Slice ring_slice(const Row& r, int parts, int part) {
    Slice s;
    const int per = (r.nv + parts - 1) >> (31 - __clz(parts));   // parts: a power of two
    s.v0 = min(r.nv, part * per);
    s.n = min(r.nv - s.v0, per);
    s.nst = (s.n + F::kVecs - 1) / F::kVecs;
    return s;
}

// A position of the ring, moved on stage by stage (a division by the number of stages, twice a stage in
// every consumer thread, took a fifth of the issue slots).
template <int N>
struct Cursor {
    int st;
    uint32_t phase;
    __device__ __forceinline__ void step() {
        if (++st == N) {
            st = 0;
            phase ^= 1;
        }
    }
};

// The rows cid, cid + ncl, ... that have a teacher and are not ignored (a warp, in step); of the others,
// skipped(row).  The labels and first ids of the next 32 rows are on their way while a batch is in use.
struct Walk {
    int64_t base, step;
    uint32_t left;
    int64_t id, label;           // of this lane's row of the next batch
};

__device__ __forceinline__ void walk_load(Walk& w, const Args& a, int64_t row) {
    w.id = row < a.T ? a.ids[row * a.K] : -1;
    w.label = row < a.T && a.labels ? a.labels[row] : 0;
}
__device__ __forceinline__ void walk_start(Walk& w, const Args& a, int64_t cid, int64_t ncl) {
    w.step = ncl;
    w.base = cid - 32 * ncl;
    w.left = 0;
    walk_load(w, a, cid + (int64_t)(threadIdx.x & 31) * ncl);
}
// The next row, or -1 behind the last.
template <typename F>
__device__ __forceinline__ int64_t walk_next(Walk& w, const Args& a, F skipped) {
    while (!w.left) {
        w.base += 32 * w.step;
        if (w.base >= a.T) return -1;
        w.left = __ballot_sync(0xFFFFFFFFu, w.id != -1 && !(a.labels && w.label == a.ignore_index));
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, w.base + (int64_t)(threadIdx.x & 31) * w.step < a.T);
        for (uint32_t no = there & ~w.left; no; no &= no - 1) skipped(w.base + (int64_t)(__ffs(no) - 1) * w.step);
        walk_load(w, a, w.base + (int64_t)(32 + (threadIdx.x & 31)) * w.step);
    }
    const int b = __ffs(w.left) - 1;
    w.left &= w.left - 1;
    return w.base + (int64_t)b * w.step;
}
__device__ __forceinline__ int64_t walk_next(Walk& w, const Args& a) {
    return walk_next(w, a, [](int64_t) {});
}

__device__ __forceinline__ void arrive_peer(uint32_t bar_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar_addr) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(tc::smem_u32(bar)), "r"(parity), "r"(10000)
        : "memory");
    return ok != 0;
}

// This thread's vectors of stage j of the slice; -inf beyond its end.
template <typename S, int U, int kNT>
__device__ __forceinline__ void ring_load(const uint8_t* buf8, const Slice& s, int j, int tid, uint4 (&x)[U]) {
    const uint4* buf = reinterpret_cast<const uint4*>(buf8) + tid;
    const int left = s.n - j * (U * kNT);
    if (left >= U * kNT) {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = tc::lds16(buf + u * kNT);
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = tid + u * kNT < left ? tc::lds16(buf + u * kNT) : stage::neg_inf16<S>();
    }
}

template <typename S, typename O, bool kGrad, bool kBig>
__global__ void __launch_bounds__(Form<kGrad, kBig>::kThreads, Form<kGrad, kBig>::kBlocks)
    k_distill_ring(const __grid_constant__ Args a) {
    constexpr int G = Elt<S>::kGroup;
    extern __shared__ __align__(128) uint8_t smem[];
    using F = Form<kGrad, kBig>;
    constexpr int nbuf = F::kBufs, U = F::kU, kRingVecs = F::kVecs, kRingBytes = F::kBytes;
    constexpr int kWarps = F::kWarps, kNT = F::kNT, kTops = F::kTops, kTop = F::kTop, kProducer = F::kProducer;
    constexpr int kPatch = F::kPatch, kStats = F::kStats, kRingThreads = F::kThreads;
    const int K = a.K, KS = entry_stride(a.K), C = a.cluster;
    Entry* entries = reinterpret_cast<Entry*>(smem + nbuf * kRingBytes);   // [kTops][KS]
    CtlOf<F>& ctl = *reinterpret_cast<CtlOf<F>*>((reinterpret_cast<uintptr_t>(entries + kTops * KS) + 15) / 16 * 16);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int64_t cid = blockIdx.x / C, ncl = gridDim.x / C;
    auto wait = [&](uint64_t* bar, int64_t e, int code) {   // the phase of row e of a barrier doubled by parity
        return tc::mbar_wait(bar, (uint32_t)(e >> 1) & 1, &ctl.abort, &ctl.err, code, a.wait_ns, kSuspend);
    };
    auto wait_top = [&](uint64_t* bar, int64_t e) {         // the phase of row e of one of kTops barriers
        return tc::mbar_wait(bar + e % kTops, (uint32_t)(e / kTops) & 1, &ctl.abort, &ctl.err, kErrRow, a.wait_ns, kSuspend);
    };

    start_next();
    if (tid == 0) {
        for (int i = 0; i < nbuf; ++i) {
            tc::mbar_init(&ctl.full[i], 1);
            tc::mbar_init(&ctl.ready[i], 1);
            tc::mbar_init(&ctl.empty[i], kWarps);
        }
        for (int p = 0; p < 2; ++p) {
            tc::mbar_init(&ctl.paired[p], kWarps);
            tc::mbar_init(&ctl.exchanged[p], C);
            tc::mbar_init(&ctl.finished[p], 1);
            tc::mbar_init(&ctl.written[p], kWarps);
        }
        for (int p = 0; p < kTops; ++p) {
            tc::mbar_init(&ctl.topped[p], 1);
            tc::mbar_init(&ctl.freed[p], 1);
        }
        ctl.abort = ctl.err = 0;
        tc::fence_mbar_init();
    }
    if (C > 1) cluster_arrive(), cluster_wait();
    else __syncthreads();

    Walk walk;
    walk_start(walk, a, cid, ncl);

    if (warp == kProducer) {
        Cursor<nbuf> at{0, 1};                         // waits for "released" start a phase back
        int q = 0;
        for (;;) {
            const int64_t row = walk_next(walk, a);
            if (row < 0 || *reinterpret_cast<volatile int*>(&ctl.abort)) break;
            if (lane == 0) {
                const Row r = make_row<S>(a.logits, row, a.ld, a.V);
                const Slice sl = ring_slice<F>(r, C, rank);
                for (int j = 0; j < sl.nst; ++j, ++q, at.step()) {
                    const int st = at.st;
                    if (!tc::mbar_wait(&ctl.empty[st], at.phase, &ctl.abort, &ctl.err, kErrEmpty, a.wait_ns)) break;
                    const int v = sl.v0 + j * kRingVecs;
                    const int lo = max(v, r.iv0), hi = min(min(v + kRingVecs, sl.v0 + sl.n), r.iv1);
                    if (hi > lo && dbg::ok(lo >= 0 && hi <= r.nv, dbg::kCols)) {
                        tc::mbar_arrive_expect_tx(&ctl.full[st], (uint32_t)(hi - lo) * 16);
                        tc::bulk_load(smem + st * kRingBytes + (lo - v) * 16, r.base + (int64_t)lo * 16,
                                      (uint32_t)(hi - lo) * 16, &ctl.full[st]);
                    } else {
                        tc::mbar_arrive(&ctl.full[st]);
                    }
                }
            }
            __syncwarp();
        }
        // after an abort, copies in flight land before the block may leave
        if (lane == 0 && *reinterpret_cast<volatile int*>(&ctl.abort)) {
            int never = 0;
            for (int p = max(0, q - nbuf); p < q; ++p)
                tc::mbar_wait(&ctl.full[p % nbuf], (p / nbuf) & 1, &never, nullptr, 0, a.wait_ns);
        }
        __syncwarp();
    } else if (warp == kPatch) {
        Cursor<nbuf> at{0, 0};
        const S neg = sizeof(S) == 2 ? (S)0xFF80u : (S)-kInf;
        // the ids of the next row are on their way while this one's stages are patched
        int64_t id[kPerLane];
        auto load_ids = [&](int64_t row) {
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                if (32 * i >= K) break;
                id[i] = lane + 32 * i < K ? a.ids[row * K + lane + 32 * i] : -1;
            }
        };
        int64_t next = walk_next(walk, a);
        if (next >= 0) load_ids(next);
        for (bool ok = true; ok && next >= 0;) {
            const int64_t row = next;
            const Row r = make_row<S>(a.logits, row, a.ld, a.V);
            const Slice sl = ring_slice<F>(r, C, rank);
            // the entries' places among the slice's elements; anything else is in no stage
            uint32_t place[kPerLane];
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                place[i] = 0xFFFFFFFFu;
                if (32 * i >= K) continue;
                if (id[i] >= 0 && id[i] < a.V) place[i] = (uint32_t)((int)id[i] + r.shift - sl.v0 * G);
            }
            next = walk_next(walk, a);
            if (next >= 0) load_ids(next);
            // lanes 0 .. G - 1: the first vector, if it is partial and the slice's; G .. 2 G - 1: the last
            const int edge = lane < G ? (r.shift ? 0 : -1) : (r.iv1 < r.nv && (r.nv > 1 || !r.shift) ? r.nv - 1 : -1);
            const int64_t ecol = (int64_t)edge * G - r.shift + lane % G;
            const bool mine = lane < 2 * G && edge >= sl.v0 && edge < sl.v0 + sl.n;
            S evalue = neg;
            if (mine && ecol >= 0 && ecol < a.V) evalue = static_cast<const S*>(a.logits)[row * a.ld + ecol];
            const uint32_t eplace = mine ? (uint32_t)((edge - sl.v0) * G + lane % G) : 0xFFFFFFFFu;
            for (int j = 0; j < sl.nst; ++j, at.step()) {
                ok = tc::mbar_wait(&ctl.full[at.st], at.phase, &ctl.abort, &ctl.err, kErrFull, a.wait_ns, kSuspend);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                S* buf = reinterpret_cast<S*>(smem + at.st * kRingBytes);
                const uint32_t first = (uint32_t)(j * kRingVecs * G);
                if (eplace - first < (uint32_t)(kRingVecs * G)) buf[eplace - first] = evalue;
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kPerLane; ++i) {
                    if (32 * i >= K) break;
                    if (place[i] - first < (uint32_t)(kRingVecs * G)) buf[place[i] - first] = neg;
                }
                // these writes before the next copy into the stage, which goes through another proxy
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl.ready[at.st]);
            }
        }
    } else if (warp >= kTop) {
        const int par = warp - kTop;
        Entry* en = entries + par * KS;
        uint32_t* seen = reinterpret_cast<uint32_t*>(en);
        int slots = 32;
        while (slots < 2 * K) slots *= 2;
        int64_t last = -1;
        for (int64_t e = 0;; ++e) {
            const int64_t row = walk_next(walk, a);
            if (row < 0) break;
            if (e % kTops != par) continue;
            const float R = a.tail ? a.tail[row] : -kInf;
            const int64_t* ids = a.ids + row * K;
            const S* zrow = static_cast<const S*>(a.logits) + row * a.ld;
            int64_t id[kPerLane];
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                if (32 * i >= K) break;
                id[i] = lane + 32 * i < K ? ids[lane + 32 * i] : -1;
            }
            int bad = 0;
            int col[kPerLane];
            float z[kPerLane], t[kPerLane];
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                const int k = lane + 32 * i;
                col[i] = -1;
                z[i] = t[i] = -kInf;
                if (32 * i >= K) continue;
                if (id[i] >= 0 && id[i] < a.V) {
                    col[i] = (int)id[i];
                    z[i] = Elt<S>::load1(zrow + col[i]);
                    t[i] = a.tbf16 ? Elt<uint16_t>::load1(static_cast<const uint16_t*>(a.tvals) + row * K + k)
                                   : Elt<float>::load1(static_cast<const float*>(a.tvals) + row * K + k);
                } else {
                    bad |= id[i] != -1;
                }
            }
            if (last >= 0 && !wait_top(ctl.freed, last)) break;
            last = e;
            // a column twice: the table (at most half full) already holds it
            for (int i = lane; i < slots; i += 32) seen[i] = 0xFFFFFFFFu;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kPerLane; ++i) {
                if (32 * i >= K) break;
                if (col[i] < 0) continue;
                uint32_t at = ((uint32_t)col[i] * 2654435761u) >> 8 & (slots - 1);
                uint32_t was;
                while ((was = atomicCAS(seen + at, 0xFFFFFFFFu, (uint32_t)col[i])) != 0xFFFFFFFFu && was != (uint32_t)col[i])
                    at = (at + 1) & (slots - 1);
                bad |= was == (uint32_t)col[i];
            }
            bad = __any_sync(0xFFFFFFFFu, bad);          // (and the table has been read)
            const Top top = top_arithmetic(a, K, lane, col, z, t, en, R);
            __syncwarp();
            if (lane == 0) {
                ctl.top[par] = TopStats{top, bad ? VCE_ERR_TEACHER : 0};
                tc::mbar_arrive(&ctl.topped[par]);
            }
        }
    } else if (warp == kStats) {
        if (kGrad && a.red == VCE_RED_MEAN) wait_previous();   // k_distill_count
        const float inv_n = kGrad && a.red == VCE_RED_MEAN ? *a.inv_n : 1.f;
        // The losses take longer than anything a consumer waits for: each lane keeps a row, and 32 rows'
        // are worked out at once.
        Finish kept{};
        int64_t kept_row = 0;
        float kept_kl = 0.f;
        int pending = 0;
        auto flush = [&]() {
            if (lane < pending && rank == 0) {
                a.loss_rows[kept_row] = loss_of(a, kept, kept_kl);
                a.row_stats[kept_row] =
                    make_float4(kept.lt, kept.dead ? 0.f : kept.d, 0.f, kept.code ? -(float)kept.code : 1.f);
            }
            pending = 0;
        };
        for (int64_t e = 0;; ++e) {
            const int par = (int)(e & 1);
            const int64_t row = walk_next(walk, a, [&](int64_t no) {   // an ignored row
                if (rank != 0) return;
                if (lane == 0) {
                    a.loss_rows[no] = 0.f;
                    a.row_stats[no] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                if (!kGrad)
                    for (int k = lane; k < K; k += 32) a.top_grads[no * K + k] = 0.f;
            });
            if (row < 0) break;
            const float go = kGrad ? a.go[a.red == VCE_RED_NONE ? row : 0] * inv_n * a.tau : 0.f;
            const float R = a.tail ? a.tail[row] : -kInf;
            if (!wait(&ctl.paired[par], e, kErrPartials)) break;
            float M = lane < kWarps ? ctl.red_m[par][lane] : -kInf;
            float S0 = lane < kWarps ? ctl.red_s[par][lane] : 0.f;
            pair_warp_reduce(M, S0);
            if (!wait_top(ctl.topped, e)) break;
            const TopStats ts = ctl.top[e % kTops];
            int code = ts.code;
            if (C > 1) {
                if (lane < C) {
                    st_peer(peer_addr(&ctl.slot[par][rank], lane), make_float4(M, S0, __int_as_float(code), 0.f));
                    arrive_peer(peer_addr(&ctl.exchanged[par], lane));
                }
                __syncwarp();
                const uint64_t t0 = tc::globaltimer();
                bool ok = true;
                while (!try_wait_cluster(&ctl.exchanged[par], (uint32_t)(e >> 1) & 1)) {
                    ok = !*reinterpret_cast<volatile int*>(&ctl.abort);
                    if (ok && tc::globaltimer() - t0 > a.wait_ns) {
                        ctl.abort = 1;
                        atomicCAS(&ctl.err, 0, (int)kErrRow);
                        ok = false;
                    }
                    if (!ok) break;
                }
                if (!__all_sync(0xFFFFFFFFu, ok)) break;
                M = -kInf;
                S0 = 0.f;
                code = 0;
                for (int p = 0; p < C; ++p) {   // the same order in every block
                    const float4 o = ctl.slot[par][p];
                    pair_merge(M, S0, o.x, o.y);
                    code = max(code, __float_as_int(o.z));
                }
            }
            const Finish f = finish_row(a, M, S0, ts.top, R, code);
            if (lane == 0) {
                ctl.coefs[par] = Coefs{go * f.d, f.bias, f.dead};
                if (a.withhold != rank + 1) tc::mbar_arrive(&ctl.finished[par]);
            }
            if (lane == pending) {
                kept = f;
                kept_row = row;
                kept_kl = ts.top.kl;
            }
            if (++pending == 32) flush();
            __syncwarp();
            if (kGrad && !wait(&ctl.written[par], e, kErrCoefs)) break;
            const Row r = make_row<S>(a.logits, row, a.ld, a.V);
            const Slice sl = ring_slice<F>(r, C, rank);
            const float c = kGrad ? go : a.tau;
            for (int k = lane; k < K; k += 32) {
                const Entry en = entries[(e % kTops) * KS + k];
                const float g = f.dead || en.col < 0 ? 0.f : c * (f.q * en.diff - f.d * en.r);
                if (!kGrad) {
                    if (rank == 0) a.top_grads[row * K + k] = g;
                } else if (en.col >= 0 && !f.dead) {
                    const int v = (en.col + r.shift) / G - sl.v0;
                    if (v >= 0 && v < sl.n) Elt<O>::store1(static_cast<O*>(a.grad) + row * a.ld_g + en.col, g);
                }
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.freed[e % kTops]);
        }
        flush();
    } else {
        // ---------------- consumers ----------------
        struct Pair {
            float m, s;
        };
        // A stage is released behind what is done with it, but by the short rows' forward, which keeps
        // only small stages (4096 x 32000 bf16: 79.8 us a call, 81.8 behind; 4096 x 128256 164.9 before, 163.3
        // behind; one pass 16384 x 128256 1483 before, 1424 behind).
        constexpr bool kEarly = !kGrad && !kBig;
        auto release = [&](int st) {
            reads_done();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.empty[st]);
        };
        // stages [j0, j1) of a row, at ring positions from `at` on
        auto forward = [&](Cursor<nbuf>& at, int j0, int j1, const Slice& sl, Pair& p) {
            for (int j = j0; j < j1; ++j, at.step()) {
                tc::mbar_wait(&ctl.ready[at.st], at.phase, &ctl.abort, &ctl.err, kErrFull, a.wait_ns, kSuspend);
                uint4 x[U];
                ring_load<S, U, kNT>(smem + at.st * kRingBytes, sl, j, tid, x);
                if (kEarly) release(at.st);
                float v[U][G];
#pragma unroll
                for (int u = 0; u < U; ++u) Elt<S>::unpack(x[u], v[u]);
                pair_push<G>(v, p.m, p.s, a.k2);
                if (!kGrad && !kEarly) release(at.st);
            }
        };
        auto publish = [&](int64_t e, Pair p) {
            const int par = (int)(e & 1);
            pair_warp_reduce(p.m, p.s);
            // row e - 2's pairs have been read (in one pass that follows from its gradient)
            if (!kGrad && e >= 2) wait(&ctl.finished[par], e - 2, kErrCoefs);
            if (lane == 0) {
                ctl.red_m[par][warp] = p.m;
                ctl.red_s[par][warp] = p.s;
                tc::mbar_arrive(&ctl.paired[par]);
            }
            __syncwarp();
        };
        Cursor<nbuf> at{0, 0}, back{0, 0};             // the next stage to sum, and to turn into gradients
        auto next = [&]() {
            return walk_next(walk, a, [&](int64_t no) {    // an ignored row
                if (!kGrad) return;
                const Row r = row_extent<S>(a, no);
                O* g = static_cast<O*>(a.grad) + no * a.ld_g;
                fill_grads<S, O>(r, ring_slice<F>(r, C, rank), g, grads_aligned<S, O>(r, g), tid, kNT);
            });
        };
        int64_t row = -1, row2 = next();                   // the row held, and the next one
        Row r{};
        Slice sl{};
        sl.nst = 0;
        for (int64_t e = -1; (row >= 0 || row2 >= 0) && !*reinterpret_cast<volatile int*>(&ctl.abort); ++e) {
            Row r2{};
            Slice sl2{};
            Pair p{-kInf, 0.f};
            int pre = 0;
            if (row2 >= 0) {
                r2 = row_extent<S>(a, row2);
                sl2 = ring_slice<F>(r2, C, rank);
                // the next row's stages that fit beside this one's (forward alone: all of them)
                pre = kGrad ? min(sl2.nst, nbuf - sl.nst) : sl2.nst;
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {         // the next row's first stages, this row, the rest
                if (row2 >= 0) forward(at, half ? pre : 0, half ? sl2.nst : pre, sl2, p);
                if (!kGrad || half || row < 0) continue;
                const int par = (int)(e & 1);
                if (!wait(&ctl.finished[par], e, kErrCoefs)) break;
                const Coefs cf = ctl.coefs[par];
                O* grow = static_cast<O*>(a.grad) + row * a.ld_g;
                const bool vec = grads_aligned<S, O>(r, grow);
                for (int j = 0; j < sl.nst; ++j, back.step()) {
                    uint4 x[U];
                    ring_load<S, U, kNT>(smem + back.st * kRingBytes, sl, j, tid, x);
                    write_grads<S, O, U, kNT>(x, r, sl, j, tid, grow, vec, cf.coef, a.k2, cf.bias, cf.dead);
                    release(back.st);
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl.written[par]);
            }
            if (row2 >= 0) publish(e + 1, p);
            row = row2;
            r = r2;
            sl = sl2;
            if (row2 >= 0) row2 = next();
        }
    }
    // after an abort: no row of this block is known to be right, nor of its cluster, whose first block has
    // written its losses by then
    __syncthreads();
    if (C > 1) cluster_arrive(), cluster_wait();       // and no block leaves while a peer may write into it
    if (ctl.abort)
        for (int64_t row = cid + (int64_t)tid * ncl; row < a.T; row += (int64_t)kRingThreads * ncl) {
            a.loss_rows[row] = __int_as_float(0x7FC00000);
            a.row_stats[row].w = -(float)(ctl.err ? ctl.err : kErrRow);
        }
}

}  // namespace ring

// ---- the gradient from saved statistics --------------------------------------------------------------

struct BwdArgs {
    const void* logits;
    int64_t T, V, ld;
    const int64_t* ids;
    int K;
    float tau, k2;
    int red;
    const float4* row_stats;
    const float* top_grads;
    const float* go;
    void* grad;
    int64_t ld_g;
    int parts, nbuf;
    uint64_t wait_ns;            // as Args
    int withhold;                // 1 (test hook): a row's last block waits for its last stage in vain
};

// One thread reads the row's statistics for the block: were they written meanwhile (a caller that does not
// wait for the forward's stream), threads that read for themselves could part ways at the row's weight, some
// of them gone before the barriers are set up that the others use.
struct alignas(16) BwdCtl {
    float4 st;
    Barriers bar;
};

template <typename S, typename O>
__global__ void __launch_bounds__(kConsumers + 32, 3) k_distill_bwd(const __grid_constant__ BwdArgs a) {
    constexpr int G = Elt<S>::kGroup;
    extern __shared__ __align__(128) uint8_t smem[];
    BwdCtl& ctl = *reinterpret_cast<BwdCtl*>(smem + a.nbuf * kStageBytes);
    Barriers& bar = ctl.bar;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t row = blockIdx.x / a.parts;
    const Row r = make_row<S>(a.logits, row, a.ld, a.V);
    const int part = (int)(blockIdx.x - row * a.parts);
    const Slice sl = make_slice(r, a.parts, part);
    O* grow = static_cast<O*>(a.grad) + row * a.ld_g;
    const bool vec = grads_aligned<S, O>(r, grow);
    const int copies = sl.nst - (a.withhold && part == a.parts - 1);
    int issued = 0;
    if (tid == kConsumers) {
        const float4 st = a.row_stats[row];
        ctl.st = st;
        init_barriers(bar, a.nbuf);
        if (st.w != 0.f)
            for (; issued < min(copies, a.nbuf); ++issued)
                issue_stage(smem, bar, a.nbuf, r, sl, issued, issued, a.wait_ns);
    }
    const float go = a.go[a.red == VCE_RED_NONE ? row : 0];
    __syncthreads();
    const float4 st = ctl.st;
    if (st.w == 0.f) {
        fill_grads<S, O>(r, sl, grow, vec, tid, kConsumers + 32);
        return;
    }
    const float cw = go * st.w;
    if (warp == kConsumerWarps) {
        if (tid == kConsumers)
            for (; issued < copies; ++issued)
                if (!issue_stage(smem, bar, a.nbuf, r, sl, issued, issued, a.wait_ns)) break;
    } else {
        const float coef = cw * a.tau * st.y, bias = st.x == -kInf ? 0.f : st.x * kLog2e;
        for (int j = 0; j < sl.nst; ++j) {
            wait_stage(bar, a.nbuf, j, a.wait_ns);
            uint4 x[kU];
            load_stage<S>(smem, a.nbuf, r, sl, j, j, tid, x);
            write_grads<S, O, kU, kConsumers>(x, r, sl, j, tid, grow, vec, coef, a.k2, bias);
            release_stage(bar, a.nbuf, j);
        }
    }
    __syncthreads();
    if (bar.abort) {                                   // there is no status word: NaN shows what was not worked out
        fill_grads<S, O>(r, sl, grow, vec, tid, kConsumers + 32, __int_as_float(0x7FC00000));
        if (tid == kConsumers) drain(bar, a.nbuf, issued);
        return;
    }
    for (int k = tid; k < a.K; k += kConsumers + 32) {
        const int64_t id = a.ids[row * a.K + k];
        if (id < 0 || id >= a.V) continue;
        const int v = (int)(id + r.shift) / G - sl.v0;
        if (v >= 0 && v < sl.n) Elt<O>::store1(grow + id, cw * a.top_grads[row * a.K + k]);
    }
}

// ---- N before a one-pass MEAN, and the losses' sum ----------------------------------------------------

constexpr int kReduceThreads = 1024;

// block sum of one integer per thread
__device__ __forceinline__ long long block_count(long long n, long long* sm) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = n;
    __syncthreads();
    long long t = 0;
    for (int w = 0; w < kReduceThreads / 32; ++w) t += sm[w];
    return t;
}

struct CountArgs {
    const int64_t* ids;
    int K;
    const int64_t* labels;
    int64_t ignore_index, T;
    float* inv_n;
};

__global__ void __launch_bounds__(kReduceThreads) k_distill_count(const __grid_constant__ CountArgs a) {
    __shared__ long long sm[kReduceThreads / 32];
    start_next();
    long long n = 0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < a.T; i += kReduceThreads)
        n += a.ids[i * a.K] != -1 && !(a.labels && a.labels[i] == a.ignore_index);
    n = block_count(n, sm);
    if (threadIdx.x == 0) *a.inv_n = n > 0 ? (float)(1.0 / (double)n) : 0.f;
}

// loss_out, status, and the rows' weights (1, a negative error code or 0 on entry; read only where
// MEAN needs N, the codes always).
struct ReduceArgs {
    const float* loss_rows;
    float4* row_stats;
    int64_t T;
    int red;
    float* loss_out;
    int32_t* status;
};

__global__ void __launch_bounds__(kReduceThreads) k_distill_reduce(const __grid_constant__ ReduceArgs a) {
    __shared__ long long sm[kReduceThreads / 32];
    __shared__ float sum[kReduceThreads / 32], comp[kReduceThreads / 32];
    __shared__ int code;
    wait_previous();
    if (threadIdx.x == 0) code = 0;
    __syncthreads();
    long long n = 0;
    int mine = 0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < a.T; i += kReduceThreads) {
        const float w = a.row_stats[i].w;
        n += w != 0.f;
        if (w < 0.f) mine = max(mine, (int)-w);
    }
    if (mine) atomicMax(&code, mine);
    n = block_count(n, sm);
    const float weight = a.red == VCE_RED_MEAN ? (n > 0 ? (float)(1.0 / (double)n) : 0.f) : 1.f;
    if (weight != 1.f || code) {               // else the weights stand as they are
#pragma unroll 8
        for (int64_t i = threadIdx.x; i < a.T; i += kReduceThreads) {
            const float w = a.row_stats[i].w;
            a.row_stats[i].w = w > 0.f ? weight : 0.f;
        }
    }
    if (a.red != VCE_RED_NONE) fold::sum_losses<kReduceThreads>(a.loss_rows, a.T, n, a.red, a.loss_out, sum, comp);
    if (threadIdx.x == 0) *a.status = code;
}

// ---- host ----------------------------------------------------------------------------------------------

// The persistent kernel's blocks of a row; 0: rows too long to hold.
template <typename F, bool kGrad>
int ring_cluster(int64_t T, int64_t V, int G, int sms) {
    const int64_t nv = (V + 2 * G - 2) / G;
    auto st = [&](int c) { return (int)(((nv + c - 1) / c + F::kVecs - 1) / F::kVecs); };
    int C = 1;
    while (C < kMaxCluster && ((kGrad && st(C) > F::kHeld) || (T * C < sms && st(C) > 1))) C *= 2;
    return kGrad && st(C) > F::kHeld ? 0 : C;
}

// In one pass with MEAN the row kernel starts while k_distill_count runs.
template <bool kGrad>
bool early_start(const Args& a) {
    return kGrad && a.red == VCE_RED_MEAN;
}

template <typename S, typename O, bool kGrad, bool kBig>
cudaError_t run_ring(Args& a, int sms, cudaStream_t s) {
    using F = ring::Form<kGrad, kBig>;
    constexpr auto kern = ring::k_distill_ring<S, O, kGrad, kBig>;
    a.cluster = ring_cluster<F, kGrad>(a.T, a.V, Elt<S>::kGroup, sms);
    if (a.withhold) a.withhold = a.cluster;
    const int bytes = ring::ring_smem<F>(a.K);
    const int64_t clusters = std::min<int64_t>(
        a.T, resident_clusters<kern>(a.cluster, F::kThreads, bytes, sms * (a.cluster == 1 ? F::kBlocks : 1)));
    if (clusters < 1) return cudaErrorInvalidConfiguration;   // not one cluster of that size fits
    return launch_clusters<kern>(clusters * a.cluster, a.cluster, F::kThreads, bytes, s, a, early_start<kGrad>(a));
}

template <typename S, typename O>
cudaError_t run_long(Args& a, cudaStream_t s) {
    const int64_t nv = (a.V + 2 * Elt<S>::kGroup - 2) / Elt<S>::kGroup;
    a.cluster = kMaxCluster;
    if (a.withhold) a.withhold = a.cluster;
    a.max_stages = (int)(((nv + kMaxCluster - 1) / kMaxCluster + kStageVecs - 1) / kStageVecs);
    a.nbuf = 4;
    return launch_clusters<k_distill_long<S, O>>(a.T * a.cluster, a.cluster, kThreads,
                                                 smem_bytes(a.nbuf, a.max_stages, a.K), s, a, early_start<true>(a));
}

template <typename S, typename O, bool kGrad>
cudaError_t run(Args& a, int sms, cudaStream_t s) {
    if constexpr (kGrad) {
        if (ring_cluster<ring::Form<true, true>, true>(a.T, a.V, Elt<S>::kGroup, sms) == 0) return run_long<S, O>(a, s);
    }
    return a.V * (int64_t)sizeof(S) >= ring::kLongRow ? run_ring<S, O, kGrad, true>(a, sms, s)
                                                      : run_ring<S, O, kGrad, false>(a, sms, s);
}

template <typename S, typename O>
cudaError_t run_bwd(BwdArgs& a, cudaStream_t s) {
    constexpr int G = Elt<S>::kGroup;
    const int64_t nv = (a.V + 2 * G - 2) / G;
    a.parts = (int)((nv + 4 * kStageVecs - 1) / (4 * kStageVecs));   // four stages a block
    a.nbuf = (int)std::min<int64_t>(4, (nv + kStageVecs - 1) / kStageVecs);
    const int bytes = a.nbuf * kStageBytes + (int)sizeof(BwdCtl);
    return launch_clusters<k_distill_bwd<S, O>>(a.T * a.parts, 1, kConsumers + 32, bytes, s, a);
}

int check_shape(int dt, int64_t T, int64_t V, int64_t ld, int K, float tau, int red) {
    if (dt != VCE_F32 && dt != VCE_BF16) return VCE_ERR_DTYPE;
    if (red != VCE_RED_NONE && red != VCE_RED_SUM && red != VCE_RED_MEAN) return VCE_ERR_DTYPE;
    // blocks of a launch stay within the grid's 2^31
    if (T < 0 || T > VCE_MAX_TOPK_T || V < 1 || V > VCE_MAX_TOPK_V) return VCE_ERR_SHAPE;
    if (K < 1 || K > VCE_MAX_TOPK || K > V || !temperature_ok(tau)) return VCE_ERR_ARG;
    if (ld < V) return VCE_ERR_LD;
    if (!fits_bytes(T, ld, dt == VCE_BF16 ? 2 : 4)) return VCE_ERR_SHAPE;
    return VCE_OK;
}

}  // namespace distill

VCE_DEBUG_READER(debug_word_distill)

namespace {

using namespace distill;

int forward_checks(const Args& a, vce_dtype dt, vce_dtype tdt, float tau, const int32_t* status) {
    int rc = check_shape(dt, a.T, a.V, a.ld, a.K, tau, a.red);
    if (rc) return rc;
    if (tdt != VCE_F32 && tdt != VCE_BF16) return VCE_ERR_DTYPE;
    if (!status || (a.T && (!a.logits || !a.ids || !a.tvals || !a.loss_rows || !a.row_stats)))
        return VCE_ERR_NULL;
    if (!aligned(a.logits, dt == VCE_BF16 ? 2 : 4) || !aligned(a.ids, 8) || !aligned(a.tvals, tdt == VCE_BF16 ? 2 : 4) ||
        !aligned(a.tail, 4) || !aligned(a.labels, 8) || !aligned(a.loss_rows, 4) || !aligned(a.row_stats, 16) ||
        !aligned(status, 4))
        return VCE_ERR_ALIGN;
    return VCE_OK;
}

cudaError_t reduce(const Args& a, float* loss_out, int32_t* status, cudaStream_t s) {
    const ReduceArgs r{a.loss_rows, a.row_stats, a.T, a.red, loss_out, status};
    return launch_clusters<k_distill_reduce>(1, 1, kReduceThreads, 0, s, r, a.T > 0);
}

}  // namespace
}  // namespace vce

using namespace vce;

extern "C" int ce_distill_forward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                  const int64_t* teacher_ids, const void* teacher_values, vce_dtype tdt,
                                  const float* teacher_tail, int K, float temperature, const int64_t* labels,
                                  int64_t ignore_index, vce_reduction red, float* loss_rows, float* loss_out,
                                  float* row_stats, float* top_grads, int32_t* status, vce_stream_t s) {
    distill::Args a{};
    a.logits = logits, a.T = T, a.V = V, a.ld = ld;
    a.ids = teacher_ids, a.tvals = teacher_values, a.tail = teacher_tail, a.K = K, a.tbf16 = tdt == VCE_BF16;
    a.tau = temperature, a.scale = 1.f / temperature, a.k2 = (float)(1.4426950408889634 / (double)temperature);
    a.labels = labels, a.ignore_index = ignore_index, a.red = red;
    a.loss_rows = loss_rows, a.row_stats = reinterpret_cast<float4*>(row_stats), a.top_grads = top_grads;
    a.wait_ns = tc::kWaitNs;
    int rc = forward_checks(a, dt, tdt, temperature, status);
    if (rc) return rc;
    if (red != VCE_RED_NONE && !loss_out) return VCE_ERR_NULL;
    if (T && !top_grads) return VCE_ERR_NULL;
    if (!aligned(top_grads, 4) || !aligned(loss_out, 4)) return VCE_ERR_ALIGN;
    if ((rc = require_sm100())) return rc;
    cudaError_t e = cudaSuccess;
    if (T) {
        const int sms = device_sm_count();
        e = dt == VCE_BF16 ? distill::run<uint16_t, float, false>(a, sms, s) : distill::run<float, float, false>(a, sms, s);
    }
    if (e == cudaSuccess) e = reduce(a, loss_out, status, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

static int backward_call(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                         const int64_t* teacher_ids, int K, float temperature, vce_reduction red,
                         const float* row_stats, const float* top_grads, const float* grad_output, void* grad_logits,
                         vce_dtype grad_dt, int64_t ld_grad, uint64_t wait_ns, int withhold, vce_stream_t s) {
    int rc = distill::check_shape(dt, T, V, ld, K, temperature, red);
    if (rc) return rc;
    if (grad_dt != VCE_F32 && grad_dt != VCE_BF16) return VCE_ERR_DTYPE;
    if (ld_grad < V) return VCE_ERR_LD;
    const size_t es = dt == VCE_BF16 ? 2 : 4, gs = grad_dt == VCE_BF16 ? 2 : 4;
    if (!fits_bytes(T, ld_grad, gs)) return VCE_ERR_SHAPE;
    if (T == 0) return VCE_OK;
    if (!logits || !teacher_ids || !row_stats || !top_grads || !grad_output || !grad_logits) return VCE_ERR_NULL;
    if (!aligned(logits, es) || !aligned(grad_logits, gs) || !aligned(teacher_ids, 8) || !aligned(row_stats, 16) ||
        !aligned(top_grads, 4) || !aligned(grad_output, 4))
        return VCE_ERR_ALIGN;
    if (rs::overlap(logits, T, V, ld, es, grad_logits, ld_grad, gs)) return VCE_ERR_ARG;
    if ((rc = require_sm100())) return rc;
    distill::BwdArgs a{};
    a.logits = logits, a.T = T, a.V = V, a.ld = ld, a.ids = teacher_ids, a.K = K;
    a.tau = temperature, a.k2 = (float)(1.4426950408889634 / (double)temperature), a.red = red;
    a.row_stats = reinterpret_cast<const float4*>(row_stats), a.top_grads = top_grads, a.go = grad_output;
    a.grad = grad_logits, a.ld_g = ld_grad;
    a.wait_ns = wait_ns, a.withhold = withhold;
    cudaError_t e;
    if (dt == VCE_BF16)
        e = grad_dt == VCE_BF16 ? distill::run_bwd<uint16_t, uint16_t>(a, s) : distill::run_bwd<uint16_t, float>(a, s);
    else
        e = grad_dt == VCE_BF16 ? distill::run_bwd<float, uint16_t>(a, s) : distill::run_bwd<float, float>(a, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

extern "C" int ce_distill_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                   const int64_t* teacher_ids, int K, float temperature, vce_reduction red,
                                   const float* row_stats, const float* top_grads, const float* grad_output,
                                   void* grad_logits, vce_dtype grad_dt, int64_t ld_grad, vce_stream_t s) {
    return backward_call(logits, dt, T, V, ld, teacher_ids, K, temperature, red, row_stats, top_grads, grad_output,
                         grad_logits, grad_dt, ld_grad, tc::kWaitNs, 0, s);
}

static int one_pass_call(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                         const int64_t* teacher_ids, const void* teacher_values, vce_dtype tdt,
                         const float* teacher_tail, int K, float temperature, const int64_t* labels,
                         int64_t ignore_index, vce_reduction red, const float* grad_output, float* loss_rows,
                         float* loss_out, float* row_stats, void* grad_logits, vce_dtype grad_dt, int64_t ld_grad,
                         int32_t* status, uint64_t wait_ns, int withhold, vce_stream_t s) {
    distill::Args a{};
    a.logits = logits, a.T = T, a.V = V, a.ld = ld;
    a.ids = teacher_ids, a.tvals = teacher_values, a.tail = teacher_tail, a.K = K, a.tbf16 = tdt == VCE_BF16;
    a.tau = temperature, a.scale = 1.f / temperature, a.k2 = (float)(1.4426950408889634 / (double)temperature);
    a.labels = labels, a.ignore_index = ignore_index, a.red = red, a.go = grad_output, a.inv_n = loss_out;
    a.loss_rows = loss_rows, a.row_stats = reinterpret_cast<float4*>(row_stats);
    a.grad = grad_logits, a.ld_g = ld_grad;
    a.wait_ns = wait_ns, a.withhold = withhold;
    int rc = forward_checks(a, dt, tdt, temperature, status);
    if (rc) return rc;
    if (grad_dt != VCE_F32 && grad_dt != VCE_BF16) return VCE_ERR_DTYPE;
    if (ld_grad < V) return VCE_ERR_LD;
    const size_t gs = grad_dt == VCE_BF16 ? 2 : 4;
    if (!fits_bytes(T, ld_grad, gs)) return VCE_ERR_SHAPE;
    if (red != VCE_RED_NONE && !loss_out) return VCE_ERR_NULL;
    if (T && (!grad_output || !grad_logits)) return VCE_ERR_NULL;
    if (!aligned(grad_output, 4) || !aligned(grad_logits, gs) || !aligned(loss_out, 4)) return VCE_ERR_ALIGN;
    if (T && rs::overlap(logits, T, V, ld, dt == VCE_BF16 ? 2 : 4, grad_logits, ld_grad, gs)) return VCE_ERR_ARG;
    if ((rc = require_sm100())) return rc;
    cudaError_t e = cudaSuccess;
    if (T) {
        if (red == VCE_RED_MEAN) {
            const distill::CountArgs c{teacher_ids, K, labels, ignore_index, T, loss_out};
            e = rs::launch_clusters<distill::k_distill_count>(1, 1, distill::kReduceThreads, 0, s, c);
        }
        const int sms = device_sm_count();
        if (e != cudaSuccess) ;
        else if (dt == VCE_BF16)
            e = grad_dt == VCE_BF16 ? distill::run<uint16_t, uint16_t, true>(a, sms, s)
                                    : distill::run<uint16_t, float, true>(a, sms, s);
        else
            e = grad_dt == VCE_BF16 ? distill::run<float, uint16_t, true>(a, sms, s)
                                    : distill::run<float, float, true>(a, sms, s);
    }
    if (e == cudaSuccess) e = reduce(a, loss_out, status, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

extern "C" int ce_distill_forward_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                           const int64_t* teacher_ids, const void* teacher_values, vce_dtype tdt,
                                           const float* teacher_tail, int K, float temperature,
                                           const int64_t* labels, int64_t ignore_index, vce_reduction red,
                                           const float* grad_output, float* loss_rows, float* loss_out,
                                           float* row_stats, void* grad_logits, vce_dtype grad_dt, int64_t ld_grad,
                                           int32_t* status, vce_stream_t s) {
    return one_pass_call(logits, dt, T, V, ld, teacher_ids, teacher_values, tdt, teacher_tail, K, temperature, labels,
                         ignore_index, red, grad_output, loss_rows, loss_out, row_stats, grad_logits, grad_dt, ld_grad,
                         status, tc::kWaitNs, 0, s);
}

extern "C" int vce_test_distill_stall(const void* logits, int64_t T, int64_t V, const int64_t* teacher_ids,
                                      const float* teacher_values, int K, const float* grad_output, float* loss_rows,
                                      float* loss_out, float* row_stats, void* grad_logits, uint64_t wait_ns,
                                      int32_t* status, vce_stream_t s) {
    if (wait_ns < 1000000ull || wait_ns > tc::kWaitNs) return VCE_ERR_ARG;
    return one_pass_call(logits, VCE_BF16, T, V, V, teacher_ids, teacher_values, VCE_F32, nullptr, K, 1.f, nullptr, 0,
                         VCE_RED_SUM, grad_output, loss_rows, loss_out, row_stats, grad_logits, VCE_BF16, V, status,
                         wait_ns, 1, s);
}

extern "C" int vce_test_distill_bwd_stall(const void* logits, int64_t T, int64_t V, const int64_t* teacher_ids, int K,
                                          const float* row_stats, const float* top_grads, const float* grad_output,
                                          void* grad_logits, uint64_t wait_ns, vce_stream_t s) {
    if (wait_ns < 1000000ull || wait_ns > tc::kWaitNs) return VCE_ERR_ARG;
    return backward_call(logits, VCE_BF16, T, V, V, teacher_ids, K, 1.f, VCE_RED_SUM, row_stats, top_grads, grad_output,
                         grad_logits, VCE_BF16, V, wait_ns, 1, s);
}
