// The policy loss and its gradient with one read of the logits (the kernels: policy_held.cuh,
// policy_ring.cuh).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "policy_held.cuh"
#include "policy_ring.cuh"

namespace vce {
namespace lp {

using namespace rs;

// Short rows are held in registers, rows of at most 4 KB by a warp, of at most 16 KB by a block of 128 threads; longer
// ones in the ring's stages.
using Warp = held::Form<32, 8, 4>;
using Block = held::Form<128, 8, 8>;
// Rows (or a cluster's slices of one) of up to 64 KB: two blocks an SM, four consumer warps each, so that what a row
// costs beside its columns runs under the other block's columns; longer ones have a whole SM.
using Pair = ring::Form<4, 2, 8, 6, 4>;
using Whole = ring::Form<14, 1, 2, 15, 10>;
constexpr int64_t kLongRow = 65536;

template <typename S>
int64_t vectors(int64_t V) { return (V + 2 * Elt<S>::kGroup - 2) / Elt<S>::kGroup; }

template <typename S, typename O, bool kEnt, typename F>
cudaError_t run_held(Args& a, cudaStream_t s) {
    a.cluster = 1;
    const int64_t blocks = (a.T + F::kPer - 1) / F::kPer;
    return launch_clusters<held::k_loss_held<S, O, true, kEnt, F>>(blocks, 1, F::kThreads, 0, s, a, a.red == VCE_RED_MEAN);
}

template <typename F>
int stages(int64_t nv, int C) { return (int)(((nv + C - 1) / C + F::kVecs - 1) / F::kVecs); }

template <typename S, typename O, bool kEnt, typename F>
cudaError_t run_ring(Args& a, cudaStream_t s) {
    constexpr auto kern = ring::k_loss_ring<S, O, true, kEnt, F>;
    const int sms = device_sm_count();
    const int64_t nv = vectors<S>(a.V);
    int C = 1;
    while (C < kMaxCluster && (stages<F>(nv, C) > F::kHeld || (a.T * C < sms && stages<F>(nv, C) > 1))) C *= 2;
    a.cluster = C;
    a.per = (int)((nv + C - 1) / C);
    if (a.withhold) a.withhold = C;
    const int64_t fit = std::min<int64_t>(
        a.T, resident_clusters<kern>(C, F::kThreads, ring::smem_bytes<F>(), sms * (C == 1 ? F::kBlocks : 1)));
    if (fit < 1) return cudaErrorInvalidConfiguration;   // not one cluster of that size fits
    return launch_clusters<kern>(fit * C, C, F::kThreads, ring::smem_bytes<F>(), s, a, a.red == VCE_RED_MEAN);
}

template <typename S, typename O, bool kEnt>
cudaError_t run_rows(Args& a, cudaStream_t s) {
    const int64_t nv = vectors<S>(a.V);
    if (!a.withhold && nv <= Warp::kVecs) return run_held<S, O, kEnt, Warp>(a, s);
    if (!a.withhold && nv <= Block::kVecs && a.T >= device_sm_count()) return run_held<S, O, kEnt, Block>(a, s);
    return a.V * (int64_t)sizeof(S) > kLongRow ? run_ring<S, O, kEnt, Whole>(a, s) : run_ring<S, O, kEnt, Pair>(a, s);
}

template <typename S, typename O>
cudaError_t run_types(Args& a, cudaStream_t s) {
    return a.entropy || a.ent != 0.f ? run_rows<S, O, true>(a, s) : run_rows<S, O, false>(a, s);
}

bool one_pass_holds(vce_dtype dt, int64_t V) {
    return stages<Whole>(dt == VCE_BF16 ? vectors<uint16_t>(V) : vectors<float>(V), kMaxCluster) <= Whole::kHeld;
}

cudaError_t launch_one_pass(vce_dtype dt, vce_dtype gdt, Args& a, cudaStream_t s) {
    if (dt == VCE_BF16) return gdt == VCE_BF16 ? run_types<uint16_t, uint16_t>(a, s) : run_types<uint16_t, float>(a, s);
    return gdt == VCE_BF16 ? run_types<float, uint16_t>(a, s) : run_types<float, float>(a, s);
}

}  // namespace lp

VCE_DEBUG_READER(debug_word_policy_onepass)

}  // namespace vce
