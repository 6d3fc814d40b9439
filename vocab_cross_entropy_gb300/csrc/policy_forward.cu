// Token log-probabilities, the policy loss and the preference loss: the forward kernels' forms, and what comes of the
// rows (the mathematics: logprob_rows.cuh; the kernels: policy_ring.cuh, policy_held.cuh).
//
// A call is the rows' kernel, for the preference loss one block a pair, and one block that sums the losses in a fixed
// order, writes the status word and, for a mean, scales the saved coefficients; each starts while the one ahead of it
// runs (programmatic dependent launch).  Nothing is shared between calls.
//
// What bounds them, bf16: the forward reads the logits once (16384 x 128256: 606 us, 6.9 TB/s, 1.02 of the measured
// copy; with entropies 635 us, and 4096 x 128256 169 us, 6.2 TB/s, one fma and one maximum more a column); short rows
// cost about 1 us beside their columns (4096 x 32000: 53 us, 4.9 TB/s).  Few rows are latency: one of 128256 takes 7.2 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ce_fold.cuh"
#include "policy_held.cuh"
#include "policy_ring.cuh"

namespace vce {
namespace lp {

using namespace rs;

// ---- what comes of the rows ------------------------------------------------------------------------

constexpr int kFinishThreads = 1024;

struct FinishArgs {
    const int64_t* ids;
    int64_t ignore_index, T;
    float4* row_stats;
    const float* losses;         // of the rows (kPolicy) or pairs, n_losses of them
    int64_t n_losses;
    int mode, red;
    int scale_stats;             // kPolicy, MEAN: the saved coefficients by 1 / N
    float* loss_out;
    int32_t* status;
    const int64_t* offsets;      // kPreference
    int64_t P;
    float *pair_losses, *rewards;
};

// block sum of one integer per thread
__device__ __forceinline__ long long block_count(long long n, long long* sm) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = n;
    __syncthreads();
    long long t = 0;
    for (int w = 0; w < kFinishThreads / 32; ++w) t += sm[w];
    return t;
}

struct CountArgs {
    const int64_t* ids;
    int64_t ignore_index, T;
    float* inv_n;
};

// 1 / N before a one-pass call with MEAN.
__global__ void __launch_bounds__(kFinishThreads) k_loss_count(const __grid_constant__ CountArgs a) {
    __shared__ long long sm[kFinishThreads / 32];
    start_next();
    long long n = 0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < a.T; i += kFinishThreads) n += a.ids[i] != a.ignore_index;
    n = block_count(n, sm);
    if (threadIdx.x == 0) *a.inv_n = n > 0 ? (float)(1.0 / (double)n) : 0.f;
}

// The losses' sum, the status word, and the saved coefficients' mean.
__global__ void __launch_bounds__(kFinishThreads) k_loss_finish(const __grid_constant__ FinishArgs a) {
    __shared__ long long sm[kFinishThreads / 32];
    __shared__ float sum[kFinishThreads / 32], comp[kFinishThreads / 32];
    __shared__ int code, stray;                      // the rows' largest code; offsets that bound no sequences
    if (threadIdx.x == 0) code = stray = 0;
    __syncthreads();
    long long n = 0;
    if (a.mode == kPolicy && a.red == VCE_RED_MEAN)
        for (int64_t i = threadIdx.x; i < a.T; i += kFinishThreads) n += a.ids[i] != a.ignore_index;
    int mine = 0;
    if (a.mode == kPreference)
        for (int64_t i = threadIdx.x; i < 2 * a.P; i += kFinishThreads)
            if (!(a.offsets[i] >= 0 && a.offsets[i] <= a.offsets[i + 1] && a.offsets[i + 1] <= a.T)) stray = 1;
    wait_previous();
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < a.T; i += kFinishThreads) {
        const float4 st = a.row_stats[i];
        if (st.x == kInf) mine = max(mine, (int)-st.y);
    }
    if (mine) atomicMax(&code, mine);
    n = block_count(n, sm);                          // (and the code is known)
    if (stray) {                                     // sequences that are none: no loss and no gradient
        for (int64_t i = threadIdx.x; i < a.T; i += kFinishThreads) a.row_stats[i] = make_float4(kInf, 0.f, 0.f, 0.f);
        for (int64_t i = threadIdx.x; i < a.P; i += kFinishThreads) {
            a.pair_losses[i] = a.rewards[2 * i] = a.rewards[2 * i + 1] = nan_f();
        }
        __syncthreads();
    }
    if (a.scale_stats && n > 0) {
        const float w = (float)(1.0 / (double)n);
#pragma unroll 4
        for (int64_t i = threadIdx.x; i < a.T; i += kFinishThreads) {
            float4 st = a.row_stats[i];
            if (st.x != kInf) a.row_stats[i] = make_float4(st.x, st.y * w, st.z * w, st.w * w);
        }
    }
    if (a.mode != kLogprobs && a.red != VCE_RED_NONE)
        fold::sum_losses<kFinishThreads>(a.losses, a.n_losses, a.mode == kPolicy ? n : a.P, a.red, a.loss_out, sum, comp);
    if (threadIdx.x == 0) *a.status = stray ? max(code, (int)VCE_ERR_OFFSETS) : code;
}

// ---- pairs of sequences ------------------------------------------------------------------------------

struct PairArgs {
    const int64_t* offsets;
    int64_t T;
    const float* ref;
    float4* row_stats;
    int kind, average;
    float beta, eps, margin, inv_tau;
    float *pair_losses, *rewards;
};

constexpr int kPairThreads = 256;

// Block p: the sums of pair p's two sequences (as fp32 pairs with two-sum steps), its loss, and its rows'
// gradient coefficients.
__global__ void __launch_bounds__(kPairThreads) k_pairs(const __grid_constant__ PairArgs a) {
    __shared__ float sum[2][kPairThreads / 32], comp[2][kPairThreads / 32];
    __shared__ int count[2], wrong[2];               // rows, and whether one of them has an error or nothing but masks
    __shared__ float slope[2];
    start_next();
    wait_previous();
    const int64_t p = blockIdx.x;
    int64_t o[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) o[i] = min(max(a.offsets[2 * p + i], (int64_t)0), a.T);
    if (threadIdx.x < 2) count[threadIdx.x] = wrong[threadIdx.x] = 0;
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float s = 0.f, c = 0.f;
        int n = 0, code = 0;
        for (int64_t i = o[q] + threadIdx.x; i < o[q + 1]; i += kPairThreads) {
            const float4 st = a.row_stats[i];
            if (st.x == kInf) {
                if (st.y == 0.f && st.w == 0.f) continue;   // left out
                code = 1;
                continue;
            }
            const float d = a.ref ? st.z - a.ref[i] : st.z;   // exact, or nearly so: both near each other
            fold::add(s, c, d);
            if (a.ref) {                                     // what that difference rounded away
                const float bb = d - st.z;
                c += (st.z - (d - bb)) + (-a.ref[i] - bb);
            }
            c += st.w;
            ++n;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            const float s2 = __shfl_xor_sync(0xFFFFFFFFu, s, off), c2 = __shfl_xor_sync(0xFFFFFFFFu, c, off);
            fold::add(s, c, s2);
            c += c2;
            n += __shfl_xor_sync(0xFFFFFFFFu, n, off);
        }
        if (lane == 0) {
            sum[q][warp] = s;
            comp[q][warp] = c;
            if (n) atomicAdd(&count[q], n);
        }
        if (code) wrong[q] = 1;
    }
    __syncthreads();
    const bool bad = wrong[0] || wrong[1];
    if (threadIdx.x == 0) {
        float S[2], share[2];
        for (int q = 0; q < 2; ++q) {
            float s = 0.f, c = 0.f;
            for (int w = 0; w < kPairThreads / 32; ++w) {
                fold::add(s, c, sum[q][w]);
                c += comp[q][w];
            }
            S[q] = fabsf(s) < kInf ? s + c : s;
            share[q] = a.average && count[q] > 0 ? 1.f / (float)count[q] : 1.f;
            if (a.average && count[q] > 0) S[q] = S[q] / (float)count[q];
            S[q] = wrong[q] ? nan_f() : S[q] * a.beta;
        }
        const float x = (S[0] - S[1]) - a.margin;
        float loss, g;
        if (a.kind == VCE_PREF_SIGMOID) {
            const float e = expf(-fabsf(x)), l = log1pf(e), d = 1.f / (1.f + e);
            const float below = x >= 0.f ? e * d : d, above = x >= 0.f ? d : e * d;   // sigma(-x), sigma(x)
            loss = (1.f - a.eps) * (l + fmaxf(-x, 0.f)) + (a.eps != 0.f ? a.eps * (l + fmaxf(x, 0.f)) : 0.f);
            g = -(1.f - a.eps) * below + a.eps * above;
        } else if (a.kind == VCE_PREF_HINGE) {
            loss = 1.f - x > 0.f ? 1.f - x : 0.f;
            g = x < 1.f ? -1.f : 0.f;
        } else {
            const float d = (x - 0.5f) / a.beta;
            loss = d * d;
            g = 2.f * d / a.beta;
        }
        if (x != x) loss = g = nan_f();
        a.pair_losses[p] = loss;
        a.rewards[2 * p] = S[0];
        a.rewards[2 * p + 1] = S[1];
        slope[0] = a.beta * g * share[0];
        slope[1] = -a.beta * g * share[1];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q)
        for (int64_t i = o[q] + threadIdx.x; i < o[q + 1]; i += kPairThreads) {
            const float4 st = a.row_stats[i];
            if (st.x == kInf) continue;
            const Coefs c = coefs(st.y, st.z, 0.f, slope[q], 0.f, a.inv_tau);
            a.row_stats[i] = bad ? make_float4(kInf, 0.f, 0.f, 0.f) : make_float4(st.x, c.c0, __int_as_float((int)p), c.gt);
        }
}

// ---- host ----------------------------------------------------------------------------------------------

// The forward's forms (us a call in a graph, bf16):
//  - Rows of at most 16 KB, a row for every SM at least, are held in registers (8192 x 4000: 19.5, and 28.4 in the
//    ring; 8192 x 8000: 30.8 and 39.8).  At 32 KB it depends on the rows' alignment (8192 x 16000: 55.4 and 59.4; 4096 x
//    8001 fp32: 31.0 and 28.9), so those stay with the ring.  Rows of at most 4 KB are held however few they are.
//  - Few rows are shared by clusters of up to eight blocks, so that every SM streams (one of 128256: 8.1).
//  - Rows below 128 KB take four blocks an SM of 4 consumer warps and 8 KB stages: what a row costs beside its columns
//    (about 1 us of merges and hand-overs) runs under the other blocks' columns.  4096 x 32000: 57.4, and 59.6 with two
//    blocks of 8 warps and 16 KB stages, 74.5 with one of 16 and 32 KB.
//  - Longer rows take two blocks an SM of 8 warps and 16 KB stages.  4096 x 128256: 162, and 168 with four blocks, 185
//    with one.
constexpr int64_t kLongRow = 131072;
using Long = ring::Form<8, 2, 4, 6, 0>;
using Short = ring::Form<4, 4, 4, 6, 0>;

template <typename S, bool kEnt, typename F>
cudaError_t run_form(Args& a, int64_t blocks, cudaStream_t s) {
    constexpr auto kern = ring::k_loss_ring<S, float, false, kEnt, F>;
    return launch_clusters<kern>(blocks, a.cluster, F::kThreads, ring::smem_bytes<F>(), s, a);
}

template <typename S, bool kEnt>
cudaError_t run_rows(Args& a, cudaStream_t s) {
    constexpr int G = Elt<S>::kGroup;
    const int sms = device_sm_count();
    const int64_t nv = (a.V + 2 * G - 2) / G;
    a.cluster = 1;
    if (nv <= held::Warp::kVecs || (nv <= held::Block16::kVecs && a.T >= sms)) return held::run<S, float, false, kEnt>(a, nv, s);
    int C = 1;
    while (C < kMaxCluster && a.T * C < sms && (nv + C - 1) / C > 512) C *= 2;
    a.cluster = C;
    a.per = (int)((nv + C - 1) / C);
    if (C == 1 && a.V * (int64_t)sizeof(S) < kLongRow)
        return run_form<S, kEnt, Short>(a, std::min<int64_t>(a.T, (int64_t)sms * Short::kBlocks), s);
    constexpr auto kern = ring::k_loss_ring<S, float, false, kEnt, Long>;
    const int64_t fit = std::min<int64_t>(
        a.T, resident_clusters<kern>(C, Long::kThreads, ring::smem_bytes<Long>(), sms * (C == 1 ? Long::kBlocks : 1)));
    if (fit < 1) return cudaErrorInvalidConfiguration;   // not one cluster of that size fits
    return run_form<S, kEnt, Long>(a, fit * C, s);
}

cudaError_t finish_rows(const Args& a, float* loss_out, int32_t* status, int scale_stats, cudaStream_t s) {
    FinishArgs f{};
    f.ids = a.ids, f.ignore_index = a.ignore_index, f.T = a.T, f.row_stats = a.row_stats, f.losses = a.loss_rows;
    f.n_losses = a.T, f.mode = a.mode, f.red = a.red, f.scale_stats = scale_stats, f.loss_out = loss_out, f.status = status;
    return launch_clusters<k_loss_finish>(1, 1, kFinishThreads, 0, s, f, a.T > 0);
}

int rows_checks(const Args& a, vce_dtype dt, float tau, const int32_t* status) {
    int rc = check_shape(dt, a.T, a.V, a.ld, tau);
    if (rc) return rc;
    if (!status || (a.T && (!a.logits || !a.ids || !a.logprobs || !a.row_stats))) return VCE_ERR_NULL;
    if (!aligned(a.logits, dt == VCE_BF16 ? 2 : 4) || !aligned(a.ids, 8) || !aligned(a.logprobs, 4) ||
        !aligned(a.entropy, 4) || !aligned(a.row_stats, 16) || !aligned(status, 4))
        return VCE_ERR_ALIGN;
    return VCE_OK;
}

int policy_checks(Args& a, const vce_policy_params* p, float* loss_out) {
    if (a.red != VCE_RED_NONE && a.red != VCE_RED_SUM && a.red != VCE_RED_MEAN) return VCE_ERR_DTYPE;
    if (!p || (a.red != VCE_RED_NONE && !loss_out) || (a.T && (!a.adv || !a.loss_rows))) return VCE_ERR_NULL;
    if (!(p->clip_low >= 0.f) || !(p->clip_high >= 0.f) || !(p->dual_clip == 0.f || p->dual_clip >= 1.f) ||
        !std::isfinite(p->kl_coef) || !std::isfinite(p->entropy_coef) || (p->kl_coef != 0.f && !a.ref))
        return VCE_ERR_ARG;
    if (!aligned(a.old, 4) || !aligned(a.adv, 4) || !aligned(a.ref, 4) || !aligned(a.weights, 4) ||
        !aligned(a.loss_rows, 4) || !aligned(loss_out, 4))
        return VCE_ERR_ALIGN;
    a.lo = 1.f - p->clip_low, a.hi = 1.f + p->clip_high, a.dual = p->dual_clip, a.kl = p->kl_coef;
    a.ent = p->entropy_coef;
    return VCE_OK;
}

}  // namespace lp

VCE_DEBUG_READER(debug_word_policy)

}  // namespace vce

using namespace vce;

static lp::Args rows_args(const void* logits, int64_t T, int64_t V, int64_t ld, const int64_t* ids, int64_t ignore_index,
                          float tau, int mode, float* logprobs, float* entropy, float* row_stats) {
    lp::Args a{};
    a.logits = logits, a.T = T, a.V = V, a.ld = ld, a.ids = ids, a.ignore_index = ignore_index, a.mode = mode;
    a.k2 = lp::k2_of(tau), a.k2_lo = lp::k2_rest(tau), a.inv_tau = 1.f / tau, a.logprobs = logprobs, a.entropy = entropy;
    a.row_stats = reinterpret_cast<float4*>(row_stats), a.wait_ns = tc::kWaitNs;
    return a;
}

static cudaError_t run(vce_dtype dt, lp::Args& a, cudaStream_t s) {
    if (!a.T) return cudaSuccess;
    const bool ent = a.entropy || (a.mode == lp::kPolicy && a.ent != 0.f);
    if (dt == VCE_BF16) return ent ? lp::run_rows<uint16_t, true>(a, s) : lp::run_rows<uint16_t, false>(a, s);
    return ent ? lp::run_rows<float, true>(a, s) : lp::run_rows<float, false>(a, s);
}

extern "C" int ce_logprobs_forward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                   const int64_t* ids, int64_t ignore_index, float temperature, float* logprobs,
                                   float* entropy, float* row_stats, int32_t* status, vce_stream_t s) {
    lp::Args a = rows_args(logits, T, V, ld, ids, ignore_index, temperature, lp::kLogprobs, logprobs, entropy, row_stats);
    int rc = lp::rows_checks(a, dt, temperature, status);
    if (rc || (rc = require_sm100())) return rc;
    cudaError_t e = run(dt, a, s);
    if (e == cudaSuccess) e = lp::finish_rows(a, nullptr, status, 0, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

extern "C" int policy_loss_forward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                   const int64_t* actions, int64_t ignore_index, float temperature,
                                   const float* old_logprobs, const float* advantages, const float* ref_logprobs,
                                   const float* weights, const vce_policy_params* p, vce_reduction red, float* loss_rows,
                                   float* loss_out, float* logprobs, float* entropy, float* row_stats, int32_t* status,
                                   vce_stream_t s) {
    lp::Args a = rows_args(logits, T, V, ld, actions, ignore_index, temperature, lp::kPolicy, logprobs, entropy, row_stats);
    a.old = old_logprobs, a.adv = advantages, a.ref = ref_logprobs, a.weights = weights, a.red = red, a.loss_rows = loss_rows;
    int rc = lp::rows_checks(a, dt, temperature, status);
    if (rc || (rc = lp::policy_checks(a, p, loss_out)) || (rc = require_sm100())) return rc;
    cudaError_t e = run(dt, a, s);
    if (e == cudaSuccess) e = lp::finish_rows(a, loss_out, status, red == VCE_RED_MEAN, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

static int one_pass_call(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                          const int64_t* actions, int64_t ignore_index, float temperature,
                          const float* old_logprobs, const float* advantages,
                          const float* ref_logprobs, const float* weights, const vce_policy_params* p,
                          vce_reduction red, const float* grad_output, float* loss_rows,
                          float* loss_out, float* logprobs, float* entropy, float* row_stats,
                          void* grad_logits, vce_dtype grad_dt, int64_t ld_grad, int32_t* status,
                          uint64_t wait_ns, int withhold, vce_stream_t s) {
    lp::Args a = rows_args(logits, T, V, ld, actions, ignore_index, temperature, lp::kPolicy, logprobs, entropy, row_stats);
    a.old = old_logprobs, a.adv = advantages, a.ref = ref_logprobs, a.weights = weights, a.red = red, a.loss_rows = loss_rows;
    a.wait_ns = wait_ns, a.withhold = withhold;
    int rc = lp::rows_checks(a, dt, temperature, status);
    if (rc || (rc = lp::policy_checks(a, p, loss_out))) return rc;
    if ((rc = lp::check_grad(dt, logits, T, V, ld, grad_logits, grad_dt, ld_grad))) return rc;
    if (T && !grad_output) return VCE_ERR_NULL;
    if (!aligned(grad_output, 4)) return VCE_ERR_ALIGN;
    if ((rc = require_sm100())) return rc;
    cudaError_t e = cudaSuccess;
    const bool held = lp::one_pass_holds(dt, V);
    if (T && !held) {                                  // a row no cluster holds is read twice
        e = run(dt, a, s);
    } else if (T) {
        a.go = grad_output, a.inv_n = loss_out, a.grad = grad_logits, a.ld_g = ld_grad;
        if (red == VCE_RED_MEAN) {
            const lp::CountArgs c{actions, ignore_index, T, loss_out};
            e = rs::launch_clusters<lp::k_loss_count>(1, 1, lp::kFinishThreads, 0, s, c);
        }
        if (e == cudaSuccess) e = lp::launch_one_pass(dt, grad_dt, a, s);
    }
    if (e == cudaSuccess) e = lp::finish_rows(a, loss_out, status, !held && red == VCE_RED_MEAN, s);
    if (e == cudaSuccess && T && !held) {
        lp::GradArgs g{};
        g.logits = logits, g.T = T, g.V = V, g.ld = ld, g.ids = actions, g.mode = lp::kPolicy, g.k2 = a.k2;
        g.inv_tau = a.inv_tau, g.row_stats = a.row_stats, g.go = grad_output, g.go_each = red == VCE_RED_NONE;
        g.scale = 1.f, g.grad = grad_logits, g.ld_g = ld_grad, g.wait_ns = tc::kWaitNs;
        e = lp::launch_grad(dt, grad_dt, g, s);
    }
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

extern "C" int policy_loss_forward_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                            const int64_t* actions, int64_t ignore_index, float temperature,
                                            const float* old_logprobs, const float* advantages,
                                            const float* ref_logprobs, const float* weights, const vce_policy_params* p,
                                            vce_reduction red, const float* grad_output, float* loss_rows,
                                            float* loss_out, float* logprobs, float* entropy, float* row_stats,
                                            void* grad_logits, vce_dtype grad_dt, int64_t ld_grad, int32_t* status,
                                            vce_stream_t s) {
    return one_pass_call(logits, dt, T, V, ld, actions, ignore_index, temperature, old_logprobs, advantages, ref_logprobs,
                         weights, p, red, grad_output, loss_rows, loss_out, logprobs, entropy, row_stats, grad_logits,
                         grad_dt, ld_grad, status, tc::kWaitNs, 0, s);
}

extern "C" int vce_test_policy_stall(const void* logits, int64_t T, int64_t V, const int64_t* actions,
                                     const float* advantages, const float* grad_output, float* loss_rows,
                                     float* loss_out, float* logprobs, float* row_stats, void* grad_logits,
                                     uint64_t wait_ns, int32_t* status, vce_stream_t s) {
    if (wait_ns < 1000000ull || wait_ns > tc::kWaitNs) return VCE_ERR_ARG;
    const vce_policy_params p{0.2f, 0.2f, 0.f, 0.f, 0.f};
    return one_pass_call(logits, VCE_BF16, T, V, V, actions, -100, 1.f, nullptr, advantages, nullptr, nullptr, &p,
                         VCE_RED_SUM, grad_output, loss_rows, loss_out, logprobs, nullptr, row_stats, grad_logits,
                         VCE_BF16, V, status, wait_ns, 1, s);
}

extern "C" int preference_loss_forward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                       const int64_t* labels, int64_t ignore_index, float temperature,
                                       const int64_t* offsets, int64_t P, const float* ref_logprobs,
                                       const vce_preference_params* p, vce_reduction red, float* pair_losses,
                                       float* loss_out, float* rewards, float* logprobs, float* row_stats,
                                       int32_t* status, vce_stream_t s) {
    lp::Args a = rows_args(logits, T, V, ld, labels, ignore_index, temperature, lp::kPreference, logprobs, nullptr, row_stats);
    a.offsets = offsets, a.P = P, a.red = red;
    int rc = lp::rows_checks(a, dt, temperature, status);
    if (rc) return rc;
    if (red != VCE_RED_NONE && red != VCE_RED_SUM && red != VCE_RED_MEAN) return VCE_ERR_DTYPE;
    if (P < 0 || P > VCE_MAX_PAIRS) return VCE_ERR_SHAPE;
    if (!p || !offsets || (P && (!pair_losses || !rewards)) || (red != VCE_RED_NONE && !loss_out)) return VCE_ERR_NULL;
    if (p->kind != VCE_PREF_SIGMOID && p->kind != VCE_PREF_HINGE && p->kind != VCE_PREF_IPO) return VCE_ERR_ARG;
    if (!(p->beta > 0.f) || !std::isfinite(p->beta) || !std::isfinite(1.f / p->beta) || !std::isfinite(p->margin) ||
        !(p->label_smoothing >= 0.f && p->label_smoothing <= 0.5f) ||
        (p->kind != VCE_PREF_SIGMOID && p->label_smoothing != 0.f) || (p->average != 0 && p->average != 1))
        return VCE_ERR_ARG;
    if (!aligned(offsets, 8) || !aligned(ref_logprobs, 4) || !aligned(pair_losses, 4) || !aligned(rewards, 4) ||
        !aligned(loss_out, 4))
        return VCE_ERR_ALIGN;
    if ((rc = require_sm100())) return rc;
    cudaError_t e = run(dt, a, s);
    if (e == cudaSuccess && P) {
        const lp::PairArgs b{offsets, T, ref_logprobs, a.row_stats, (int)p->kind, p->average, p->beta,
                             p->label_smoothing, p->margin, a.inv_tau, pair_losses, rewards};
        e = rs::launch_clusters<lp::k_pairs>(P, 1, lp::kPairThreads, 0, s, b, T > 0);
    }
    if (e == cudaSuccess) {
        lp::FinishArgs f{};
        f.ids = labels, f.ignore_index = ignore_index, f.T = T, f.row_stats = a.row_stats, f.losses = pair_losses;
        f.n_losses = P, f.mode = lp::kPreference, f.red = red, f.loss_out = loss_out, f.status = status;
        f.offsets = offsets, f.P = P, f.pair_losses = pair_losses, f.rewards = rewards;
        e = rs::launch_clusters<lp::k_loss_finish>(1, 1, lp::kFinishThreads, 0, s, f, T > 0 || P > 0);
    }
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}
