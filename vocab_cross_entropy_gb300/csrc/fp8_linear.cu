// Logits of a head in e4m3 with block scales on the tensor cores (tcgen05, kind::f8f6f4):
//     out[t][v] = sum_b xs[t][b] ws[v / 128][b] sum_{k in block b} x[t][k] w[v][k]
//
// The scales change every 128 columns of K and differ along t and v, so a block's products are summed by the
// tensor cores into a fresh accumulator of tensor memory (four MMAs of K = 32), and the block's sum is scaled and
// added to the running sum in registers, while the tensor cores work on the next block in the other accumulator.
//
//   k_linear_pair  T > 128: CTA pairs (cta_group::2) on 256 x 256 tiles, 128 rows of x and half of the tile's rows
//                  of w per CTA and K block.  8 epilogue warps, each 32 rows x 128 columns in registers: per K
//                  block and SM 32768 fma (256 cycles of the fma pipe) against the MMAs' 512 cycles.
//   k_linear_few   T <= 128: bound by reading w.  The roles change sides: w's rows are the MMA's 128, the rows of x
//                  its N (16 to 128 wide), so a stage is w's 16 KB and the few rows of x.  Where w has fewer tiles
//                  than there are SMs, a cluster's CTAs each take a part of K and add their sums in order.
// What bounds them.  8192 x 4096 by 128256 to bf16: 3.87-4.04 ms, 2220 TFLOP/s (0.59 of twice the bf16 product's
// measured burst rate), the tensor pipe 45% active at 1.91 GHz.  At 2048 x 4096 by 32768, 263 us: the copies out of
// L2 with a quarter of the MMAs take 168 us (1024 tiles of 32 blocks of 64 KB, 12.8 TB/s), copies and MMAs with nobody
// waiting for an accumulator 209, with the accumulators handed over but not read 236.  The hand-over (a block's MMAs
// done, both CTAs told, the sums read, the even CTA told: some 1300 cycles, of which the other accumulator's block hides
// 500) is what keeps the tensor pipe waiting.  N = 128 accumulators, four of them, would hide it but read x's tile twice
// as often from shared memory, which is then the limit (319 us).  16 epilogue warps of 64 columns spill at 104 registers
// (548 us).
// All this is for scales of any value.  Powers of two, as quantize_fp8 makes them, could be handed to the block-scaled
// form of the MMA as bytes, which would add up all of K in one accumulator; that needs operands of a type of their own
// and is not built.
// T = 1: 83-85 us in a graph, 6.2-6.3 TB/s of w (0.93-0.95 of the measured copy); T = 64: 90 us, T = 128: 109.  A block
// takes no less than its copies, some 1.5 ns a row of 128 bytes (0.2 us for w's 128 rows), however few SMs work, and
// 0.38 us where all do, which is the memory's rate.  Each SM the same number of rows, the last tile in copies of 32:
// 1 x 4096 by 128256 85.5 us to 87.7, 64 x 2064 by 32001 21.4 to 20.3; in copies of 8 slower everywhere.
// Every wait is bounded (2 s); where one gives up, the CTA's tiles become NaN.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "row_launch.h"
#include "tc_launch.cuh"
#include "vce_check.cuh"
#include "vce_fp8.h"
#include "vce_host.h"

namespace vce {
namespace fp8 {

using namespace tc;

constexpr int kBlock = VCE_FP8_BLOCK;                // K columns (bytes) of a block

struct LinearArgs {
    const float* xs;
    const float* ws;
    int64_t T, V;
    int nd;                      // blocks of K
    void* out;
    int64_t ld;
    int tiles_m, tiles_n;        // k_linear_pair
    int split;                   // k_linear_few: CTAs that share a tile's K
    int x_rows;                  // k_linear_few: rows of x in a copy
    int aligned;                 // out's rows start on 16-byte boundaries
    uint32_t tx_extra;           // 0; > 0 only in the test hook (no stage ever completes)
    uint64_t wait_ns;            // bound of every wait
};

// One lane of a whole warp, the same at every call.  The issuing warps stay whole and elect a lane for the MMAs and
// commits: issued by lane 0 in a loop of its own, whose operands the compiler cannot take for the warp's, a block's
// four MMAs and two commits cost 640 cycles (1 x 65536 by 1000 25.6 us for 20.2, 8192 x 4096 by 128256 3930 for 3868).
__device__ __forceinline__ bool elect_one() {
    uint32_t is;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(is));
    return is != 0;
}

template <bool kCta2>
__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    if constexpr (kCta2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, e4m3 A and B (format 0), both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {   // ties r to the wait, as tmem_wait_ld
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Arrive on a barrier of either CTA of a pair.  What it orders is tensor memory (its loads have been waited for, and
// tcgen05.fence stands before), nothing that a release at cluster scope would have to flush: that one held the
// epilogue warps for two fifths of their time (2670 cycles a K block, 1375 without it).
__device__ __forceinline__ void arrive_either(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// Arrive on the barrier at this shared-memory address in both CTAs of a pair once every MMA issued so far is done.
__device__ __forceinline__ void commit_both(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ uint4 ld_cluster16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// Scales k .. k + 3 of a row of nd (0 behind its end).
__device__ __forceinline__ float4 four_scales(const float* s, int k, int nd) {
    if (nd % 4 == 0 && (reinterpret_cast<uintptr_t>(s) & 15u) == 0) return __ldg(reinterpret_cast<const float4*>(s + k));
    return make_float4(__ldg(s + k), k + 1 < nd ? __ldg(s + k + 1) : 0.f, k + 2 < nd ? __ldg(s + k + 2) : 0.f,
                       k + 3 < nd ? __ldg(s + k + 3) : 0.f);
}

// (c0, c1) += (a[0] b0, a[1] b1), in one packed instruction.
__device__ __forceinline__ void fma_scaled(const uint32_t* a, uint32_t b0, uint32_t b1, float& c0, float& c1) {
    asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
        "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\tmov.b64 pc, {%0, %1};\n\t"
        "fma.rn.f32x2 pc, pa, pb, pc;\n\tmov.b64 {%0, %1}, pc;\n\t}"
        : "+f"(c0), "+f"(c1)
        : "r"(a[0]), "r"(a[1]), "r"(b0), "r"(b1));
}

// (c0, c1) += (a0, a1) * b, in one packed instruction.
__device__ __forceinline__ void fma_pair(uint32_t a0, uint32_t a1, float b, float& c0, float& c1) {
    asm("{\n\t.reg .b64 pa, pb, pc;\n\t"
        "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %4};\n\tmov.b64 pc, {%0, %1};\n\t"
        "fma.rn.f32x2 pc, pa, pb, pc;\n\tmov.b64 {%0, %1}, pc;\n\t}"
        : "+f"(c0), "+f"(c1)
        : "r"(a0), "r"(a1), "f"(b));
}

template <typename O>
__device__ __forceinline__ void store_nan(const LinearArgs& a, int64_t t, int64_t v) {
    if (t < a.T && v < a.V) Elt<O>::store1(static_cast<O*>(a.out) + t * a.ld + v, __int_as_float(0x7FC00000));
}

// ---- CTA pairs ----------------------------------------------------------------------------------------

constexpr int kM = 128, kN = 256;                    // rows of x per CTA, rows of w per tile
constexpr int kEpiWarps = 8, kEpi0 = 4, kProducer = 0, kIssuer = 1;   // warps 2 and 3 are there for the warpgroup
constexpr int kCols = 4 * kN / kEpiWarps;            // columns of an epilogue warp
constexpr int kPairThreads = (kEpi0 + kEpiWarps) * 32;
// Registers of a thread: at launch, and of the two kinds of warpgroups once they are split.  An epilogue thread holds
// 128 running sums and two loads of 32 columns.
constexpr int kLaunchRegs = 168, kRoleRegs = 56, kEpiRegs = 224;
static_assert(128 * kRoleRegs + 32 * kEpiWarps * kEpiRegs <= kPairThreads * kLaunchRegs, "the split fits what the launch has");
constexpr int kStages = 6;
constexpr int kTileBytes = kM * kBlock;              // 16 KB: x's rows, and this CTA's half of w's
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kScratch = 32 * 17 * 4;                // per epilogue warp, for the stores
constexpr int kPairSmem = kStages * kStageBytes + kEpiWarps * kScratch + 1024 /*alignment*/ + 256 /*barriers*/;
static_assert(kPairSmem <= kMaxSmem, "shared memory");

template <typename O>
__global__ void __launch_bounds__(kPairThreads, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapW,
                  const __grid_constant__ LinearArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scratch = reinterpret_cast<float*>(smem + kStages * kStageBytes);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes + kEpiWarps * kScratch);
    uint64_t* empty = full + kStages;
    uint64_t* acc_full = empty + kStages;
    uint64_t* acc_free = acc_full + 2;
    uint64_t* drain = acc_free + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 2 * kEpiWarps);   // one arrival per epilogue warp of both CTAs
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_map(&mapX);
        prefetch_map(&mapW);
    }
    if (warp == kProducer) {
        tmem_alloc<true>(tmem_slot, 2 * kN);
        tmem_relinquish<true>();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (threadIdx.x == 0 && rank == 1 && ld_cluster_u32(cluster_addr(tmem_slot, 0)) != tmem) *abort_flag = 1;
    __syncthreads();
    const int ntiles = a.tiles_m * a.tiles_n;        // of the pair; tiles that run at once share w's rows
    const int tile0 = (int)(blockIdx.x >> 1), tstep = (int)(gridDim.x >> 1);

    if (warp < kEpi0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
        if (warp == kProducer && lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int tile = tile0; tile < ntiles && !*abort_flag; tile += tstep) {
                const int t0 = (tile % a.tiles_m * 2 + (int)rank) * kM, v0 = tile / a.tiles_m * kN + (int)rank * (kN / 2);
                for (int kb = 0; kb < a.nd; ++kb) {
                    if (!wait_bar<false>(&empty[stage], phase ^ 1u, abort_flag, nullptr, 0, a.wait_ns)) break;
                    const uint32_t fb = cluster_addr(&full[stage], 0);   // the even CTA counts both CTAs' bytes
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes + a.tx_extra);
                    uint8_t* at = smem + stage * kStageBytes;
                    tma_load<true>(at, &mapX, fb, kb * kBlock, t0);
                    tma_load<true>(at + kTileBytes, &mapW, fb, kb * kBlock, v0);
                    issued = issued < kStages ? issued + 1 : kStages;
                    if (++stage == kStages) stage = 0, phase ^= 1u;
                }
            }
            if (*abort_flag) {   // copies in flight land before the CTA may leave
                const uint64_t t0 = globaltimer();
                if (rank == 0) {
                    for (int i = 0; i < issued; ++i) {
                        if (--stage < 0) stage = kStages - 1, phase ^= 1u;
                        while (!mbar_try_wait(&full[stage], phase) && globaltimer() - t0 < a.wait_ns) {
                        }
                    }
                } else {         // these complete on the even CTA's barriers: give them time
                    while (globaltimer() - t0 < 1000000ull) {
                    }
                }
            }
        } else if (warp == kIssuer && rank == 0) {
            constexpr uint32_t idesc = idesc_e4m3_f32(2 * kM, kN);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            const uint32_t base = smem_u32(smem);
            for (int tile = tile0; tile < ntiles && !*abort_flag; tile += tstep) {
                for (int kb = 0; kb < a.nd; ++kb) {
                    if (!__all_sync(0xFFFFFFFFu,
                                    wait_bar<false>(&full[stage], phase, abort_flag, nullptr, 0, a.wait_ns) &&
                                        wait_bar<false>(&acc_free[acc], acc_phase ^ 1u, abort_flag, nullptr, 0, a.wait_ns)))
                        break;
                    tc_fence_after();
                    const uint64_t ad = desc_kmajor_sw128(base + stage * kStageBytes);
                    const uint64_t bd = desc_kmajor_sw128(base + stage * kStageBytes + kTileBytes);
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kBlock / 32; ++k)   // 32 bytes of K a step
                            mma_e4m3<true>(tmem + (uint32_t)(acc * kN), ad + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
                        commit_both(smem_u32(&acc_full[acc]));
                        commit_both(smem_u32(&empty[stage]));
                    }
                    __syncwarp();
                    if (++stage == kStages) stage = 0, phase ^= 1u;
                    acc ^= 1;
                    if (acc == 0) acc_phase ^= 1u;
                }
            }
            // every MMA this thread issued has finished before tensor memory can be released
            if (elect_one()) mma_commit<true>(smem_u32(drain));
            __syncwarp();
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < a.wait_ns) {
            }
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
        const int sub = warp & 3, cg = (warp - kEpi0) >> 2;   // this warp's 32 rows and kCols columns of the CTA's tile
        const uint32_t taddr = tmem + ((uint32_t)(sub * 32) << 16) + (uint32_t)(cg * kCols);
        float* mine = scratch + (warp - kEpi0) * (kScratch / 4);
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int tile = tile0; tile < ntiles && ok; tile += tstep) {
            const int64_t t0 = (int64_t)(tile % a.tiles_m * 2 + (int)rank) * kM + sub * 32;
            const int64_t v0 = (int64_t)(tile / a.tiles_m) * kN + cg * kCols;
            const bool active = t0 < a.T && v0 < a.V;
            // the scales of four blocks at a time, the next four on their way: a thread's row has its own, so each load
            // touches 32 lines (one block at a time, the epilogue waited for them longer than for the MMAs)
            const float* xs = a.xs + (t0 + lane < a.T ? t0 + lane : 0) * a.nd;
            const float* ws = a.ws + (active ? v0 / kBlock : 0) * a.nd;
            float c[kCols];
#pragma unroll
            for (int i = 0; i < kCols; ++i) c[i] = 0.f;
            float4 sc = make_float4(0.f, 0.f, 0.f, 0.f), xn = sc, wn = sc;
            if (active) xn = four_scales(xs, 0, a.nd), wn = four_scales(ws, 0, a.nd);
            for (int kb = 0; kb < a.nd; ++kb) {
                if (kb % 4 == 0) {
                    sc = make_float4(xn.x * wn.x, xn.y * wn.y, xn.z * wn.z, xn.w * wn.w);
                    if (active && kb + 4 < a.nd) xn = four_scales(xs, kb + 4, a.nd), wn = four_scales(ws, kb + 4, a.nd);
                }
                const float s = sc.x;
                sc = make_float4(sc.y, sc.z, sc.w, 0.f);
                ok = __all_sync(0xFFFFFFFFu, wait_bar<false>(&acc_full[acc], acc_phase, abort_flag, nullptr, 0, a.wait_ns));
                if (!ok) break;
                tc_fence_after();
                const uint32_t to = cluster_addr(&acc_free[acc], 0);
                auto release = [&]() {               // every load of this accumulator has landed
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_either(to);
                };
                if (active) {
                    uint32_t r[2][32];
                    const uint32_t at = taddr + (uint32_t)(acc * kN);
                    tmem_ld32(at, r[0]);
#pragma unroll
                    for (int q = 0; q < kCols / 32; ++q) {
                        tmem_wait_ld(r[q & 1]);
                        if (q + 1 < kCols / 32) tmem_ld32(at + (q + 1) * 32, r[(q + 1) & 1]);
                        else release();
#pragma unroll
                        for (int i = 0; i < 32; i += 2) fma_pair(r[q & 1][i], r[q & 1][i + 1], s, c[q * 32 + i], c[q * 32 + i + 1]);
                    }
                } else {
                    release();
                }
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
            if (!ok || !active) continue;
            O* out = static_cast<O*>(a.out) + t0 * a.ld + v0;
            if (a.aligned && v0 + kCols <= a.V) {   // each lane its row
                if (t0 + lane < a.T && dbg::ok(v0 + kCols <= a.ld, dbg::kTile)) {
                    O* p = out + lane * a.ld;
#pragma unroll
                    for (int i = 0; i < kCols; i += 8) {
                        const float g[8] = {c[i], c[i + 1], c[i + 2], c[i + 3], c[i + 4], c[i + 5], c[i + 6], c[i + 7]};
                        GroupStore<O, 8>::run(p + i, g);
                    }
                }
            } else {                                 // rows of any alignment: 16 columns at a time through shared memory
                const int rows = (int)min((int64_t)32, a.T - t0);
#pragma unroll
                for (int q = 0; q < kCols / 16; ++q) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) mine[lane * 17 + i] = c[q * 16 + i];
                    __syncwarp();
                    const int64_t v = v0 + q * 16 + (lane & 15);
                    if (v < a.V && dbg::ok(v < a.ld, dbg::kTile))
                        for (int i = lane >> 4; i < rows; i += 2)
                            Elt<O>::store1(out + i * a.ld + q * 16 + (lane & 15), mine[i * 17 + (lane & 15)]);
                    __syncwarp();
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (*abort_flag)
        for (int tile = tile0; tile < ntiles; tile += tstep)
            for (int i = threadIdx.x; i < kM * kN; i += kPairThreads)
                store_nan<O>(a, (int64_t)(tile % a.tiles_m * 2 + (int)rank) * kM + i / kN,
                             (int64_t)(tile / a.tiles_m) * kN + i % kN);
    // neither CTA releases its tensor memory or leaves while the other's MMAs, copies or arrivals may reach it
    cluster_sync_all();
    if (warp == kProducer) {
        tc_fence_after();
        tmem_dealloc<true>(tmem, 2 * kN);
    }
}

// ---- few rows of x --------------------------------------------------------------------------------------

constexpr int kMaxSplit = 8;                         // CTAs that share a tile's K, at most
constexpr int kScales = 8;                           // K blocks' scales in flight
constexpr int kAccs = 4;                             // accumulators: an MMA waits for what an epilogue three blocks before freed
template <int N>
struct Few {
    static constexpr int kEach = N > 32 ? N / 2 : N;                 // rows of x of an epilogue warp
    static constexpr int kEpi = 4 * (N / kEach);                     // epilogue warps
    static constexpr int kProducer = kEpi, kIssuer = kEpi + 1, kScaler = kEpi + 2, kThreads = (kEpi + 3) * 32;
    static constexpr int kStage = kTileBytes + N * kBlock;
    static constexpr int kBufs = (kMaxSmem - 1536 - kScales * N * 4) / kStage < 12 ? (kMaxSmem - 1536 - kScales * N * 4) / kStage : 12;
    static constexpr int kSmem = kBufs * kStage + 1024 + 512 + kScales * N * 4;
    static constexpr int kCols = kAccs * N;                          // of tensor memory
    static_assert(kBufs * kStage >= N * kM * 4, "a CTA's sums lie in its stages");
    static_assert(kCols >= 32 && kCols <= 512 && N % kMaxSplit == 0, "tile");
};

template <typename O, int N>
__global__ void __launch_bounds__(Few<N>::kThreads, 1)
    k_linear_few(const __grid_constant__ CUtensorMap mapX, const __grid_constant__ CUtensorMap mapW,
                 const __grid_constant__ LinearArgs a) {
    using F = Few<N>;
    constexpr int S = F::kBufs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* scales = reinterpret_cast<float*>(smem + S * F::kStage);   // [kScales][N]
    uint64_t* full = reinterpret_cast<uint64_t*>(scales + kScales * N);
    uint64_t* empty = full + S;
    uint64_t* acc_full = empty + S;
    uint64_t* acc_free = acc_full + kAccs;
    uint64_t* sc_full = acc_free + kAccs;
    uint64_t* sc_free = sc_full + kScales;
    uint64_t* drain = sc_free + kScales;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = a.split > 1 ? (int)cluster_ctarank() : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < kAccs; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], F::kEpi);
        }
        for (int i = 0; i < kScales; ++i) {
            mbar_init(&sc_full[i], 1);
            mbar_init(&sc_free[i], F::kEpi);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_map(&mapX);
        prefetch_map(&mapW);
    }
    if (warp == F::kProducer) {
        tmem_alloc<false>(tmem_slot, F::kCols);
        tmem_relinquish<false>();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int ntiles = (int)((a.V + kM - 1) / kM);
    const int tile0 = (int)blockIdx.x / a.split, tstep = (int)gridDim.x / a.split;
    const int per = (a.nd + a.split - 1) / a.split, k0 = min(a.nd, rank * per), k1 = min(a.nd, k0 + per);

    constexpr int NC = F::kEach;
    const int half = warp / 4 * NC;                  // the first row of x of this epilogue warp
    float c[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) c[i] = 0.f;
    if (warp == F::kProducer) {
        if (lane == 0) {
            int stage = 0, issued = 0;
            uint32_t phase = 0;
            for (int tile = tile0; tile < ntiles && !*abort_flag; tile += tstep) {
                for (int kb = k0; kb < k1; ++kb) {
                    if (!wait_bar<false>(&empty[stage], phase ^ 1u, abort_flag, nullptr, 0, a.wait_ns)) break;
                    mbar_arrive_expect_tx(&full[stage], kTileBytes + a.x_rows * kBlock + a.tx_extra);
                    uint8_t* at = smem + stage * F::kStage;
                    tma_load<false>(at, &mapW, smem_u32(&full[stage]), kb * kBlock, tile * kM);
                    tma_load<false>(at + kTileBytes, &mapX, smem_u32(&full[stage]), kb * kBlock, 0);
                    issued = issued < S ? issued + 1 : S;
                    if (++stage == S) stage = 0, phase ^= 1u;
                }
            }
            if (*abort_flag) {
                const uint64_t t0 = globaltimer();
                for (int i = 0; i < issued; ++i) {
                    if (--stage < 0) stage = S - 1, phase ^= 1u;
                    while (!mbar_try_wait(&full[stage], phase) && globaltimer() - t0 < a.wait_ns) {
                    }
                }
            }
        }
        __syncwarp();
    } else if (warp == F::kIssuer) {
        constexpr uint32_t idesc = idesc_e4m3_f32(kM, N);
        int stage = 0, acc = 0;
        uint32_t phase = 0, acc_phase = 0;
        const uint32_t base = smem_u32(smem);
        for (int tile = tile0; tile < ntiles && !*abort_flag; tile += tstep) {
            for (int kb = k0; kb < k1; ++kb) {
                if (!__all_sync(0xFFFFFFFFu,
                                wait_bar<false>(&acc_free[acc], acc_phase ^ 1u, abort_flag, nullptr, 0, a.wait_ns) &&
                                    wait_bar<false>(&full[stage], phase, abort_flag, nullptr, 0, a.wait_ns)))
                    break;
                tc_fence_after();
                const uint64_t ad = desc_kmajor_sw128(base + stage * F::kStage);
                const uint64_t bd = desc_kmajor_sw128(base + stage * F::kStage + kTileBytes);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBlock / 32; ++k)
                        mma_e4m3<false>(tmem + (uint32_t)(acc * N), ad + 2 * k, bd + 2 * k, idesc, k ? 1u : 0u);
                    mma_commit<false>(smem_u32(&acc_full[acc]));
                }
                __syncwarp();
                if (++stage == S) stage = 0, phase ^= 1u;
                if (++acc == kAccs) acc = 0, acc_phase ^= 1u;
            }
        }
        if (elect_one()) mma_commit<false>(smem_u32(drain));
        __syncwarp();
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(drain, 0) && globaltimer() - t0 < a.wait_ns) {
        }
        __syncwarp();
    } else if (warp == F::kScaler) {
        // the scales of a K block for every row of x, times the tile's, where the epilogue reads them four at a time (out
        // of the lanes by shuffles they cost T = 64 a tenth of its time)
        int slot = 0;
        uint32_t phase = 0;
        for (int tile = tile0; tile < ntiles && !*abort_flag; tile += tstep) {
            const float* ws = a.ws + (int64_t)tile * a.nd;
            for (int kb = k0; kb < k1; ++kb) {
                float x[(N + 31) / 32];
                const float w = __ldg(ws + kb);
#pragma unroll
                for (int i = 0; i < (N + 31) / 32; ++i) {
                    const int t = i * 32 + lane;
                    x[i] = t < a.T ? __ldg(a.xs + (int64_t)t * a.nd + kb) : 0.f;
                }
                if (!__all_sync(0xFFFFFFFFu, wait_bar<false>(&sc_free[slot], phase ^ 1u, abort_flag, nullptr, 0, a.wait_ns))) break;
#pragma unroll
                for (int i = 0; i < (N + 31) / 32; ++i)
                    if (i * 32 + lane < N) scales[slot * N + i * 32 + lane] = x[i] * w;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_full[slot]);
                if (++slot == kScales) slot = 0, phase ^= 1u;
            }
        }
    } else {
        // a thread holds row v of w against NC rows of x
        const uint32_t taddr = tmem + ((uint32_t)(warp % 4 * 32) << 16) + (uint32_t)half;
        int acc = 0, slot = 0, stage = 0;
        uint32_t acc_phase = 0, phase = 0;
        bool ok = true;
        for (int tile = tile0; tile < ntiles && ok; tile += tstep) {
#pragma unroll
            for (int i = 0; i < NC; ++i) c[i] = 0.f;
            for (int kb = k0; kb < k1; ++kb) {
                ok = __all_sync(0xFFFFFFFFu, wait_bar<false>(&sc_full[slot], phase, abort_flag, nullptr, 0, a.wait_ns) &&
                                                 wait_bar<false>(&acc_full[acc], acc_phase, abort_flag, nullptr, 0, a.wait_ns));
                if (!ok) break;
                if (threadIdx.x == 0) mbar_arrive(&empty[stage]);     // the MMAs are done with the stage, too (a second
                                                                      // commit: 20.2 us for 18.9, 1 x 65536 by 1000)
                if (++stage == S) stage = 0;
                tc_fence_after();
                uint32_t r[NC / 16][16];
#pragma unroll
                for (int q = 0; q < NC / 16; ++q) tmem_ld16(taddr + (uint32_t)(acc * N + q * 16), r[q]);
#pragma unroll
                for (int q = 0; q < NC / 16; ++q) tmem_wait16(r[q]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_free[acc]);
                const float* s = scales + slot * N + half;
#pragma unroll
                for (int i = 0; i < NC; i += 4) {
                    const uint4 f = lds16(s + i);
                    fma_scaled(r[i / 16] + i % 16, f.x, f.y, c[i], c[i + 1]);
                    fma_scaled(r[i / 16] + i % 16 + 2, f.z, f.w, c[i + 2], c[i + 3]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sc_free[slot]);
                if (++acc == kAccs) acc = 0, acc_phase ^= 1u;
                if (++slot == kScales) slot = 0, phase ^= 1u;
            }
            const int64_t v = (int64_t)tile * kM + warp % 4 * 32 + lane;
            if (ok && a.split == 1 && v < a.V && dbg::ok(v < a.ld, dbg::kTile)) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (half + i < a.T) Elt<O>::store1(static_cast<O*>(a.out) + (half + i) * a.ld + v, c[i]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (a.split > 1) {
        // the parts of K: every CTA's sums into its own stages (its copies have landed and been read), and each CTA adds
        // up a share of x's rows out of all of them, in the CTAs' order, 16 bytes a load (128 x 2048 by 8000 10.0 us;
        // 12.9 with 4 bytes, whose loads wait for one another; stored into the first CTA one at a time 39).
        float* own = reinterpret_cast<float*>(smem);          // [rows of x][128]
        if (warp < F::kEpi) {
            const bool bad = *abort_flag != 0;
#pragma unroll
            for (int i = 0; i < NC; ++i) own[(half + i) * kM + warp % 4 * 32 + lane] = bad ? __int_as_float(0x7FC00000) : c[i];
        }
        cluster_sync_all();
        const int share = N / a.split * kM, first = rank * share;
        for (int e = threadIdx.x * 4; e < share; e += F::kThreads * 4) {
            const int t = (first + e) / kM;
            const int64_t v = (int64_t)tile0 * kM + e % kM;
            if (t >= a.T || v >= a.V) continue;
            uint4 part[kMaxSplit];
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
                if (q < a.split) part[q] = ld_cluster16(cluster_addr(own + first + e, q));
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q)
                if (q < a.split) {
                    sum[0] += __uint_as_float(part[q].x), sum[1] += __uint_as_float(part[q].y);
                    sum[2] += __uint_as_float(part[q].z), sum[3] += __uint_as_float(part[q].w);
                }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v + i < a.V && dbg::ok(v + i < a.ld, dbg::kTile))
                    Elt<O>::store1(static_cast<O*>(a.out) + t * a.ld + v + i, sum[i]);
        }
        cluster_sync_all();                                   // no CTA leaves while another reads its sums
    }
    if (*abort_flag && rank == 0)
        for (int tile = tile0; tile < ntiles; tile += tstep)
            for (int i = threadIdx.x; i < kM * N; i += F::kThreads) store_nan<O>(a, i / kM, (int64_t)tile * kM + i % kM);
    if (warp == F::kProducer) {
        tc_fence_after();
        tmem_dealloc<false>(tmem, F::kCols);
    }
}

// ---- host --------------------------------------------------------------------------------------------------

// 2-D map over a row-major byte matrix with boxes of 128 bytes (the swizzle span) x box_rows rows.
bool make_byte_map(CUtensorMap* map, const void* base, int64_t inner, int64_t outer, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
    cuuint64_t strides[1] = {(cuuint64_t)inner};
    cuuint32_t box[2] = {(cuuint32_t)kBlock, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class K>
cudaError_t launch(K kern, int blocks, int cluster, int threads, int smem, cudaStream_t s, const CUtensorMap& mx,
                   const CUtensorMap& mw, const LinearArgs& a) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, mx, mw, a);
}

template <typename O>
cudaError_t run_pair(const void* x, const void* w, int64_t D, LinearArgs& a, cudaStream_t s) {
    CUtensorMap mx, mw;
    if (!make_byte_map(&mx, x, D, a.T, kM) || !make_byte_map(&mw, w, D, a.V, kN / 2)) return cudaErrorInvalidValue;
    a.tiles_m = (int)((a.T + 2 * kM - 1) / (2 * kM));
    a.tiles_n = (int)((a.V + kN - 1) / kN);
    if ((int64_t)a.tiles_m * a.tiles_n > INT32_MAX / 2) return cudaErrorInvalidValue;
    static std::atomic<int> ready[kMaxDevices];
    int clusters = 0;
    cudaError_t e = prepare_kernel(k_linear_pair<O>, kPairSmem, true, ready, &clusters);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    // the warpgroups' split waits for registers that the launch has to have
    static std::atomic<int> regs{0};
    int r = regs.load();
    if (r == 0) {
        cudaFuncAttributes f;
        if ((e = cudaFuncGetAttributes(&f, k_linear_pair<O>)) != cudaSuccess) return e;
        regs.store(r = f.numRegs);
    }
    if (r * kPairThreads < 128 * kRoleRegs + 32 * kEpiWarps * kEpiRegs) return cudaErrorInvalidConfiguration;
    const int pairs = std::min(a.tiles_m * a.tiles_n, clusters);
    return launch(k_linear_pair<O>, 2 * pairs, 2, kPairThreads, kPairSmem, s, mx, mw, a);
}

template <typename O, int N>
cudaError_t run_few(const void* x, const void* w, int64_t D, LinearArgs& a, cudaStream_t s) {
    CUtensorMap mx, mw;
    // x's rows and no more than 7 behind them (copies cost by the row); what the MMA's other columns hold is not stored
    a.x_rows = (int)(a.T + 7) / 8 * 8;
    if (!make_byte_map(&mx, x, D, a.T, a.x_rows) || !make_byte_map(&mw, w, D, a.V, kM)) return cudaErrorInvalidValue;
    static std::atomic<int> ready[kMaxDevices];
    int none = 0;
    cudaError_t e = prepare_kernel(k_linear_few<O, N>, Few<N>::kSmem, false, ready, &none);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count();
    const int64_t tiles = (a.V + kM - 1) / kM;
    // As many CTAs to a tile as there are SMs for, with two blocks of K each at least (1 x 4096 by 4000: 10.7 us with
    // one, 8.0 with two, 6.4 with four; 128 x 1024 by 4000: 8.6, 8.8, 7.3), but eight only where they take no more than
    // half the SMs (1 x 4096 by 1000: 6.3 with four, 5.5 with eight; 1 x 16384 by 2048, 128 CTAs of 152: 15.2 and 18.1 when
    // tried, the clusters of eight not all finding a place at once).  Below eight blocks the joining costs more than it
    // saves (1 and 64 x 512 by 4000: 4.3 and 5.4 with one, 4.7 and 6.0 with two).
    a.split = 1;
    while (a.split < kMaxSplit && tiles * a.split * (a.split < 4 ? 2 : 4) <= sms && a.nd >= std::max(8, 4 * a.split)) a.split *= 2;
    const int blocks = a.split > 1 ? (int)tiles * a.split : (int)std::min<int64_t>(tiles, sms);
    return launch(k_linear_few<O, N>, blocks, a.split, Few<N>::kThreads, Few<N>::kSmem, s, mx, mw, a);
}

template <typename O>
cudaError_t run(const void* x, const void* w, int64_t D, LinearArgs& a, cudaStream_t s) {
    if (a.T > 128) return run_pair<O>(x, w, D, a, s);
    if (a.T > 64) return run_few<O, 128>(x, w, D, a, s);
    if (a.T > 32) return run_few<O, 64>(x, w, D, a, s);
    if (a.T > 16) return run_few<O, 32>(x, w, D, a, s);
    return run_few<O, 16>(x, w, D, a, s);
}

}  // namespace fp8

VCE_DEBUG_READER(debug_word_fp8)

}  // namespace vce

using namespace vce;

static int linear_call(const void* x, const float* x_scales, const void* w, const float* w_scales, int64_t T, int64_t D,
                       int64_t V, void* out, vce_dtype out_dt, int64_t ld, uint32_t tx_extra, uint64_t wait_ns,
                       vce_stream_t s) {
    if (out_dt != VCE_F32 && out_dt != VCE_BF16) return VCE_ERR_DTYPE;
    if (T < 0 || T > (int64_t)1 << 24 || V < 1 || V > (int64_t)1 << 24 || D < 16 || D > 65536 || D % 16) return VCE_ERR_SHAPE;
    if (ld < V) return VCE_ERR_LD;
    const size_t es = out_dt == VCE_BF16 ? 2 : 4;
    if (!fits_bytes(T, ld, es)) return VCE_ERR_SHAPE;
    if (T == 0) return VCE_OK;
    if (!x || !x_scales || !w || !w_scales || !out) return VCE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(out, es))
        return VCE_ERR_ALIGN;
    const int64_t nd = (D + 127) / 128, no = ((T - 1) * ld + V) * (int64_t)es;
    if (overlap_bytes(out, no, x, T * D) || overlap_bytes(out, no, w, V * D) || overlap_bytes(out, no, x_scales, T * nd * 4) ||
        overlap_bytes(out, no, w_scales, (V + 127) / 128 * nd * 4))
        return VCE_ERR_ARG;                          // tiles are read while others are written
    int rc = require_sm100();
    if (rc) return rc;
    fp8::LinearArgs a{};
    a.xs = x_scales, a.ws = w_scales, a.T = T, a.V = V, a.nd = (int)nd, a.out = out, a.ld = ld, a.split = 1;
    a.aligned = aligned(out, 16) && ld * (int64_t)es % 16 == 0;
    a.tx_extra = tx_extra, a.wait_ns = wait_ns;
    const cudaError_t e = out_dt == VCE_BF16 ? fp8::run<uint16_t>(x, w, D, a, s) : fp8::run<float>(x, w, D, a, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

extern "C" int vce_linear_fp8(const void* x, const float* x_scales, const void* w, const float* w_scales, int64_t T,
                              int64_t D, int64_t V, void* out, vce_dtype out_dt, int64_t ld, vce_stream_t s) {
    return linear_call(x, x_scales, w, w_scales, T, D, V, out, out_dt, ld, 0, tc::kWaitNs, s);
}

extern "C" int vce_test_linear_fp8_stall(const void* x, const float* x_scales, const void* w, const float* w_scales,
                                         int64_t T, int64_t D, int64_t V, float* out, uint64_t wait_ns, vce_stream_t s) {
    if (wait_ns < 1000000ull || wait_ns > tc::kWaitNs) return VCE_ERR_ARG;
    return linear_call(x, x_scales, w, w_scales, T, D, V, out, VCE_F32, V, 16, wait_ns, s);
}
