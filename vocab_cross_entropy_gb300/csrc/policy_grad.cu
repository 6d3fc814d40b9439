// The gradient of the post-training losses w.r.t. the logits from the statistics that a forward saved:
// one read of the logits, one write of the gradient (the formulas: logprob_rows.cuh).
//
// A block takes up to four 16 KB stages of one row, streamed through shared memory by bulk copies while
// its warps turn the stages that have landed into gradients; three blocks share an SM, so that one's
// copies run under another's stores.  Nothing is shared between blocks.  The rows go from the last to the first:
// where a forward has just read them, the last are in L2 still (forward and backward of 4096 x 32000 bf16: 130 us, and
// 140 in ascending order).
//
// It runs at the copy's speed: 6144 x 128256 bf16 452 us, 7.0 TB/s; 4096 x 32000 bf16 83 us, 6.3 TB/s.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "logprob_rows.cuh"
#include "policy_rows.h"
#include "row_grads.cuh"

namespace vce {
namespace lp {

using namespace rs;

// One thread reads what belongs to the row for the block: were it written meanwhile, threads that read for
// themselves could part ways at it.
struct alignas(16) GradCtl {
    float4 st;
    Coefs c;
    float bias;
    int target;
    int none;
    Barriers bar;
};

template <typename S, typename O>
__global__ void __launch_bounds__(kConsumers + 32, 3) k_row_grads(const __grid_constant__ GradArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    GradCtl& ctl = *reinterpret_cast<GradCtl*>(smem + a.nbuf * kStageBytes);
    Barriers& bar = ctl.bar;
    const int tid = threadIdx.x, warp = tid >> 5;
    const int64_t row = a.T - 1 - blockIdx.x / a.parts;
    const rs::Row r = make_row<S>(a.logits, row, a.ld, a.V);
    const int part = (int)(blockIdx.x % a.parts);
    const Slice sl = make_slice(r, a.parts, part);
    O* grow = static_cast<O*>(a.grad) + row * a.ld_g;
    const bool vec = grads_aligned<S, O>(r, grow);
    const int copies = sl.nst - (a.withhold && part == a.parts - 1);
    int issued = 0;
    if (tid == kConsumers) {
        const float4 st = a.row_stats[row];
        const int64_t t = a.ids[row];
        ctl.none = st.x == kInf;
        if (a.mode == kPreference) {                   // statistics of another call may name a pair that is not there
            const int64_t pair = (int64_t)__float_as_int(st.z);
            ctl.none = ctl.none || pair < 0 || pair >= a.P;
        }
        init_barriers(bar, a.nbuf);
        if (!ctl.none)
            for (; issued < min(copies, a.nbuf); ++issued)
                issue_stage(smem, bar, a.nbuf, r, sl, issued, issued, a.wait_ns);
        Coefs c;
        if (a.mode == kLogprobs) {
            c = coefs(st.y, st.z, st.w, a.ga ? a.ga[row] : 0.f, a.gb ? a.gb[row] : 0.f, a.inv_tau);
        } else {
            const int64_t i = !a.go_each ? 0 : a.mode == kPreference ? (int64_t)__float_as_int(st.z) : row;
            const float go = ctl.none ? 0.f : a.go[i] * a.scale;
            c = Coefs{go * st.y, a.mode == kPreference ? 0.f : go * st.z, go * st.w};
        }
        ctl.c = c;
        ctl.bias = st.x;
        ctl.target = t >= 0 && t < a.V ? (int)t : -1;
    }
    __syncthreads();
    if (ctl.none) {
        fill_grads<S, O>(r, sl, grow, vec, tid, kConsumers + 32);
        return;
    }
    if (warp == kConsumerWarps) {
        if (tid == kConsumers)
            for (; issued < copies; ++issued)
                if (!issue_stage(smem, bar, a.nbuf, r, sl, issued, issued, a.wait_ns)) break;
    } else {
        const Coefs c = ctl.c;
        const float bias = ctl.bias;
        const bool whole = vec && !beyond(bias);
        const int target = ctl.target;
        for (int j = 0; j < sl.nst; ++j) {
            wait_stage(bar, a.nbuf, j, a.wait_ns);
            uint4 x[kU];
            load_stage<S>(smem, a.nbuf, r, sl, j, j, tid, x);
            const int v0 = sl.v0 + j * kStageVecs, v1 = sl.v0 + sl.n;
            const bool fast = whole && v0 >= r.iv0 && v0 + kStageVecs <= min(r.iv1, v1);
            if (c.c1 != 0.f)
                write_grads<S, O, kU, kConsumers, true>(x, r, v0 + tid, v1, fast, grow, whole, c, bias, a.k2);
            else
                write_grads<S, O, kU, kConsumers, false>(x, r, v0 + tid, v1, fast, grow, whole, c, bias, a.k2);
            // the token's entry, over what its thread has just written there
            const int rel = target >= 0 ? (target + r.shift) / Elt<S>::kGroup - v0 - tid : -1;
            if (rel >= 0 && rel < kStageVecs && rel % kConsumers == 0 && v0 + tid + rel < v1)
                Elt<O>::store1(grow + target, c.gt);
            release_stage(bar, a.nbuf, j);
        }
    }
    __syncthreads();
    if (bar.abort) {                                   // there is no status word: NaN shows what was not worked out
        fill_grads<S, O>(r, sl, grow, vec, tid, kConsumers + 32, nan_f());
        if (tid == kConsumers) drain(bar, a.nbuf, issued);
    }
}

template <typename S, typename O>
cudaError_t run_grad(GradArgs& a, cudaStream_t s) {
    constexpr int G = Elt<S>::kGroup;
    const int64_t nv = (a.V + 2 * G - 2) / G;
    a.parts = (int)((nv + 4 * kStageVecs - 1) / (4 * kStageVecs));   // four stages a block
    a.nbuf = (int)std::min<int64_t>(4, (nv + kStageVecs - 1) / kStageVecs);
    const int bytes = a.nbuf * kStageBytes + (int)sizeof(GradCtl);
    return launch_clusters<k_row_grads<S, O>>(a.T * a.parts, 1, kConsumers + 32, bytes, s, a);
}

cudaError_t launch_grad(vce_dtype dt, vce_dtype gdt, GradArgs& a, cudaStream_t s) {
    if (dt == VCE_BF16) return gdt == VCE_BF16 ? run_grad<uint16_t, uint16_t>(a, s) : run_grad<uint16_t, float>(a, s);
    return gdt == VCE_BF16 ? run_grad<float, uint16_t>(a, s) : run_grad<float, float>(a, s);
}

}  // namespace lp

VCE_DEBUG_READER(debug_word_policy_grad)

}  // namespace vce

using namespace vce;

static int backward(vce_dtype dt, vce_dtype gdt, lp::GradArgs& a, float tau, cudaStream_t s) {
    int rc = lp::check_shape(dt, a.T, a.V, a.ld, tau);
    if (rc || (rc = lp::check_grad(dt, a.logits, a.T, a.V, a.ld, a.grad, gdt, a.ld_g))) return rc;
    if (a.T == 0) return VCE_OK;
    if (!a.ids || !a.row_stats || (a.mode != lp::kLogprobs && !a.go)) return VCE_ERR_NULL;
    if (!aligned(a.ids, 8) || !aligned(a.row_stats, 16) || !aligned(a.go, 4) || !aligned(a.ga, 4) || !aligned(a.gb, 4))
        return VCE_ERR_ALIGN;
    if ((rc = require_sm100())) return rc;
    a.k2 = lp::k2_of(tau), a.inv_tau = 1.f / tau;
    if (!a.wait_ns) a.wait_ns = tc::kWaitNs;
    return record_cuda(lp::launch_grad(dt, gdt, a, s)) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

extern "C" int ce_logprobs_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                    const int64_t* ids, float temperature, const float* row_stats,
                                    const float* grad_logprobs, const float* grad_entropy, void* grad_logits,
                                    vce_dtype grad_dt, int64_t ld_grad, vce_stream_t s) {
    lp::GradArgs a{};
    a.logits = logits, a.T = T, a.V = V, a.ld = ld, a.ids = ids, a.mode = lp::kLogprobs;
    a.row_stats = reinterpret_cast<const float4*>(row_stats), a.ga = grad_logprobs, a.gb = grad_entropy;
    a.grad = grad_logits, a.ld_g = ld_grad;
    return backward(dt, grad_dt, a, temperature, s);
}

extern "C" int policy_loss_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                    const int64_t* actions, float temperature, vce_reduction red,
                                    const float* row_stats, const float* grad_output, void* grad_logits,
                                    vce_dtype grad_dt, int64_t ld_grad, vce_stream_t s) {
    if (red != VCE_RED_NONE && red != VCE_RED_SUM && red != VCE_RED_MEAN) return VCE_ERR_DTYPE;
    lp::GradArgs a{};
    a.logits = logits, a.T = T, a.V = V, a.ld = ld, a.ids = actions, a.mode = lp::kPolicy;
    a.row_stats = reinterpret_cast<const float4*>(row_stats), a.go = grad_output, a.go_each = red == VCE_RED_NONE;
    a.scale = 1.f, a.grad = grad_logits, a.ld_g = ld_grad;
    return backward(dt, grad_dt, a, temperature, s);
}

extern "C" int preference_loss_backward(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                                        const int64_t* labels, float temperature, int64_t P, vce_reduction red,
                                        const float* row_stats, const float* grad_output, void* grad_logits,
                                        vce_dtype grad_dt, int64_t ld_grad, vce_stream_t s) {
    if (red != VCE_RED_NONE && red != VCE_RED_SUM && red != VCE_RED_MEAN) return VCE_ERR_DTYPE;
    if (P < 0 || P > VCE_MAX_PAIRS) return VCE_ERR_SHAPE;
    lp::GradArgs a{};
    a.logits = logits, a.T = T, a.V = V, a.ld = ld, a.ids = labels, a.mode = lp::kPreference;
    a.row_stats = reinterpret_cast<const float4*>(row_stats), a.go = grad_output, a.go_each = red == VCE_RED_NONE, a.P = P;
    a.scale = red == VCE_RED_MEAN && P > 0 ? (float)(1.0 / (double)P) : 1.f, a.grad = grad_logits, a.ld_g = ld_grad;
    return backward(dt, grad_dt, a, temperature, s);
}

extern "C" int vce_test_policy_bwd_stall(const void* logits, int64_t T, int64_t V, const int64_t* actions,
                                         const float* row_stats, const float* grad_output, void* grad_logits,
                                         uint64_t wait_ns, vce_stream_t s) {
    if (wait_ns < 1000000ull || wait_ns > tc::kWaitNs) return VCE_ERR_ARG;
    lp::GradArgs a{};
    a.logits = logits, a.T = T, a.V = V, a.ld = V, a.ids = actions, a.mode = lp::kPolicy;
    a.row_stats = reinterpret_cast<const float4*>(row_stats), a.go = grad_output, a.scale = 1.f, a.grad = grad_logits;
    a.ld_g = V, a.wait_ns = wait_ns, a.withhold = 1;
    return backward(VCE_BF16, VCE_BF16, a, 1.f, s);
}
