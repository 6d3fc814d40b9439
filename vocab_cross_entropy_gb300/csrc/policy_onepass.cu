// The policy loss and its gradient with one read of the logits (the kernel: policy_ring.cuh).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "policy_ring.cuh"

namespace vce {
namespace lp {

using namespace rs;

using Held = ring::Form<16, 1, 2, 13, 8>;

template <typename S, typename O, bool kEnt>
cudaError_t run_held(Args& a, cudaStream_t s) {
    using F = Held;
    constexpr auto kern = ring::k_loss_ring<S, O, true, kEnt, F>;
    constexpr int G = Elt<S>::kGroup;
    const int sms = device_sm_count();
    const int64_t nv = (a.V + 2 * G - 2) / G;
    auto stages = [&](int c) { return (int)(((nv + c - 1) / c + F::kVecs - 1) / F::kVecs); };
    int C = 1;
    while (C < kMaxCluster && (stages(C) > F::kHeld || (a.T * C < sms && stages(C) > 1))) C *= 2;
    a.cluster = C;
    if (a.withhold) a.withhold = C;
    const int64_t fit = std::min<int64_t>(a.T, resident_clusters<kern>(C, F::kThreads, ring::smem_bytes<F>(), sms));
    if (fit < 1) return cudaErrorInvalidConfiguration;   // not one cluster of that size fits
    return launch_clusters<kern>(fit * C, C, F::kThreads, ring::smem_bytes<F>(), s, a, a.red == VCE_RED_MEAN);
}

// Whether a cluster's shared memory holds a row.
static bool holds(int64_t V, int G) {
    const int64_t nv = (V + 2 * G - 2) / G;
    return ((nv + kMaxCluster - 1) / kMaxCluster + Held::kVecs - 1) / Held::kVecs <= Held::kHeld;
}

template <typename S, typename O>
cudaError_t run_types(Args& a, cudaStream_t s) {
    return a.entropy || a.ent != 0.f ? run_held<S, O, true>(a, s) : run_held<S, O, false>(a, s);
}

bool one_pass_holds(vce_dtype dt, int64_t V) { return holds(V, dt == VCE_BF16 ? 8 : 4); }

cudaError_t launch_one_pass(vce_dtype dt, vce_dtype gdt, Args& a, cudaStream_t s) {
    if (dt == VCE_BF16) return gdt == VCE_BF16 ? run_types<uint16_t, uint16_t>(a, s) : run_types<uint16_t, float>(a, s);
    return gdt == VCE_BF16 ? run_types<float, uint16_t>(a, s) : run_types<float, float>(a, s);
}

}  // namespace lp

VCE_DEBUG_READER(debug_word_policy_onepass)

}  // namespace vce
