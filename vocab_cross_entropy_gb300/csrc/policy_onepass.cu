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

// The forms (us a call, bf16 to bf16):
//  - Rows of at most 32 KB, a row for every SM at least, are held in registers (8192 x 4000: 34 in a graph, and 62 in
//    the ring; 8192 x 8000: 53 and 78; 8192 x 16000: 96 and 115; at 64 KB 100 and 101, but 2048 x 32001 to fp32 99 and
//    83).  Rows of at most 4 KB are held however few they are.
//  - Rows below 64 KB take two blocks an SM, four consumer warps each, so that what a row costs beside its columns runs
//    under the other block's columns (4096 x 32000: 101 in a graph; 128 with one block of 14 warps).
//  - Longer rows have a whole SM, or a cluster of them: 14 consumer warps, so that with the two others four are on each
//    scheduler and have 128 registers (16 had 96 and spilled); 15 stages of 14 KB, ten of which a row may take, so
//    that the next row's first stages are summed while this row's statistics are exchanged and finished (2048 x
//    64000: 107, and 122 with two blocks; 4096 x 128256: 368 and 435).
// What bounds the last: 16384 x 128256 1402 us, 6.0 TB/s, 0.90 of the measured copy, a column's two exponentials and the
// instructions around them; with an entropy term 1577 us, 0.80, where a column takes two maxima and two products more.
// The row's statistics take about 1.5 us from the last sum to the first gradient, of which the next row's first stages
// hide most (a release at cluster scope and functions worked out twice there cost 20 us of 387 at 4096 rows).
using Pair = ring::Form<4, 2, 8, 6, 4>;
using Whole = ring::Form<14, 1, 2, 15, 10>;
constexpr int64_t kLongRow = 65536;

template <typename S>
int64_t vectors(int64_t V) { return (V + 2 * Elt<S>::kGroup - 2) / Elt<S>::kGroup; }

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
    if (!a.withhold && (nv <= held::Warp::kVecs || (nv <= held::Block32::kVecs && a.T >= device_sm_count())))
        return held::run<S, O, true, kEnt>(a, nv, s, a.red == VCE_RED_MEAN);
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
