// ce_topk: a row's K largest logits in order, with the log-sum-exp of the row and of the columns
// left out.
//
// One pass over the logits.  The row (or its slice, in a thread-block cluster) streams through
// shared memory (row_stream.cuh); of every group of 16 or 32 values -- a consumer thread's vectors
// of a stage -- only the maximum and the sum of exponentials relative to it are kept.  The K-th
// largest group maximum is a lower bound t of the K-th largest value: K groups hold a value >= t,
// and every value >= t lies in a group whose maximum is >= t.  So
//   1. t: a binary search over the bits of the maxima's order keys (counts of keys >= t), stopped
//      as soon as no more than K + K/4 groups remain;
//   2. the groups with a maximum >= t are read once more (from L2): their values >= t become
//      candidates, and the group's pair is rebuilt from the other values, so the candidates are
//      left out of the tail's sum without a subtraction;
//   3. the candidates (about 1.1 K of them) are ranked by counting, as 64-bit keys (order key,
//      reversed column), all different, so ties go to the lowest column and the result does not
//      depend on the order in which candidates were found; those ranked K or later join the tail;
//   4. the blocks of a cluster merge their sorted lists the same way (ranks by binary search).
// Where the bound admits too many values (few columns per K, or many equal values), the K-th
// largest value itself is found by the same search over all values, read from L2, and the values
// equal to it are taken in column order.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "row_launch.h"
#include "row_stream.cuh"
#include "vce_logits.h"

namespace vce {
namespace topk {

using namespace rs;

constexpr int kThreads = kConsumers + 32;   // the last warp: producer
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCand = 1024;              // candidates of a block
constexpr int kMaxSel = 512;                // groups read again
constexpr uint32_t kKeyMin = 0x00800000u;   // order key of the lowest finite value

// Scratch over the stage buffers, once the columns have streamed through.
constexpr int kCandAt = 0;                                   // [kMaxCand] candidates
constexpr int kListAt = kCandAt + kMaxCand * 8;              // [kMaxCand] candidates by rank (read by peers)
constexpr int kSelAt = kListAt + kMaxCand * 8;               // [kMaxSel] group numbers
constexpr int kPartAt = kSelAt + kMaxSel * 4;                // [kMaxSel * kU] pairs of the vectors read again
constexpr int kPartEnd = kPartAt + kMaxSel * kU * 8;
constexpr int kInAt = kSelAt;                                // [cluster * K] the cluster's lists
constexpr int kOutAt = kInAt + kMaxCluster * VCE_MAX_TOPK * 8;   // the same by rank
constexpr int kScratch = kOutAt + kMaxCluster * VCE_MAX_TOPK * 8;
static_assert(kScratch <= 3 * kStageBytes && kPartEnd <= 3 * kStageBytes && kMaxCand >= VCE_MAX_TOPK, "scratch");

struct Args {
    const void* logits;
    int64_t T, V, ld;
    int K;
    float scale, k2;
    float* values;
    int64_t* ids;
    float *lse, *tail;
    int cluster, nbuf, max_stages;
};

struct alignas(16) Ctl {
    float4 tail;                    // the block's pair of the columns left out (read by peers)
    Barriers bar;
    float red_m[kWarps], red_s[kWarps];
    int count[2][kWarps];
    int nsel, ncand, neq;
};

__host__ __device__ constexpr int smem_bytes(int nbuf, int max_stages) {
    const int b = nbuf * kStageBytes;
    return (b > kScratch ? b : kScratch) + max_stages * kConsumers * 8 + (int)sizeof(Ctl);
}

// Keys in the order of the values (larger value, larger key); -0 as +0.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}
// Candidates: key above, reversed column below; 0: none.
__device__ __forceinline__ uint64_t cand_of(uint32_t key, int col) {
    return ((uint64_t)key << 32) | (0xFFFFFFFFu - (uint32_t)col);
}
__device__ __forceinline__ uint32_t cand_key(uint64_t c) { return (uint32_t)(c >> 32); }
__device__ __forceinline__ int cand_col(uint64_t c) { return (int)(0xFFFFFFFFu - (uint32_t)c); }

// Sum over the block of each thread's n (call number it picks one of two buffers, so one barrier
// a call is enough).
__device__ __forceinline__ int block_sum(int n, Ctl& ctl, int it) {
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if ((threadIdx.x & 31) == 0) ctl.count[it & 1][threadIdx.x >> 5] = n;
    __syncthreads();
    int t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += ctl.count[it & 1][w];
    return t;
}

// The pair of G values, -inf left out.
template <int G>
__device__ __forceinline__ float2 pair_of(const float (&v)[G], float k2) {
    float m = v[0];
#pragma unroll
    for (int k = 1; k < G; ++k) m = fmaxf(m, v[k]);
    if (m == -kInf) return make_float2(-kInf, 0.f);
    const float mb = m * k2;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) s += ex2(fmaf(v[k], k2, -mb));
    return make_float2(m, s);
}

// The K largest of the slice by the exact K-th value, every value read from global memory as often
// as its search takes: for slices where the bound from the groups admits too many.  Candidates go
// to cand (ctl.ncand of them), everything else into this thread's pair (tm, ts).
template <typename S>
__device__ __noinline__ void exact_threshold(const Args& a, const Row& r, const Slice& sl, Ctl& ctl, uint64_t* cand,
                                             float& tm, float& ts) {
    constexpr int G = Elt<S>::kGroup;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int it = 0;
    auto count_from = [&](uint32_t t) {
        int n = 0;
        for (int i = tid; i < sl.n; i += kThreads) {
            float v[G];
            Elt<S>::unpack(load_vector<S>(r, sl.v0 + i), v);
#pragma unroll
            for (int k = 0; k < G; ++k) n += key_of(v[k]) >= t;
        }
        return block_sum(n, ctl, it++);
    };
    uint32_t t = kKeyMin;
    if (count_from(kKeyMin) >= a.K) {
        t = 0;
        for (int bit = 31; bit >= 0; --bit)
            if (count_from(t | (1u << bit)) >= a.K) t |= 1u << bit;
    }
    if (tid == 0) ctl.ncand = 0;
    __syncthreads();
    // above t: candidates; equal: counted; below: the tail
    int eq = 0;
    for (int i = tid; i < sl.n; i += kThreads) {
        float v[G];
        Elt<S>::unpack(load_vector<S>(r, sl.v0 + i), v);
#pragma unroll
        for (int k = 0; k < G; ++k) {
            const uint32_t key = key_of(v[k]);
            if (key > t) {
                const int at = atomicAdd(&ctl.ncand, 1);
                if (at < kMaxCand) cand[at] = cand_of(key, (sl.v0 + i) * G - r.shift + k);
            }
            eq += key == t;
            if (key >= t) v[k] = -kInf;
        }
        const float2 p = pair_of<G>(v, a.k2);
        pair_merge(tm, ts, p.x, p.y, a.k2);
    }
    const int total_eq = block_sum(eq, ctl, it++);
    const int above = min(ctl.ncand, kMaxCand);
    const int want = min(total_eq, a.K - above);
    __syncthreads();
    // the first `want` values equal to t, in column order: vectors i = base + tid
    int found = 0;
    for (int base = 0; base < sl.n && found < want; base += kThreads) {
        const int i = base + tid;
        uint32_t hits = 0;
        if (i < sl.n) {
            float v[G];
            Elt<S>::unpack(load_vector<S>(r, sl.v0 + i), v);
#pragma unroll
            for (int k = 0; k < G; ++k) hits |= (key_of(v[k]) == t ? 1u : 0u) << k;
        }
        int n = __popc(hits), before = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {   // inclusive sums of the warp
            const int o = __shfl_up_sync(0xFFFFFFFFu, before, off);
            if (lane >= off) before += o;
        }
        if (lane == 31) ctl.count[0][warp] = before;
        before += found - n;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += ctl.count[0][w];
            all += ctl.count[0][w];
        }
        for (; hits && before < want; hits &= hits - 1, ++before)
            cand[above + before] = cand_of(t, (sl.v0 + i) * G - r.shift + __ffs(hits) - 1);
        found += all;
        __syncthreads();
    }
    if (tid == 0) {
        ctl.ncand = above + want;
        if (total_eq > want) pair_merge(tm, ts, value_of(t), (float)(total_eq - want), a.k2);
    }
    __syncthreads();
}

template <typename S>
__global__ void __launch_bounds__(kThreads, 3) k_topk(const __grid_constant__ Args a) {
    constexpr int G = Elt<S>::kGroup;
    extern __shared__ __align__(128) uint8_t smem[];
    const int over = max(a.nbuf * kStageBytes, kScratch);
    float* gm = reinterpret_cast<float*>(smem + over);
    float* gs = gm + a.max_stages * kConsumers;
    Ctl& ctl = *reinterpret_cast<Ctl*>(gs + a.max_stages * kConsumers);
    uint64_t* cand = reinterpret_cast<uint64_t*>(smem + kCandAt);
    uint64_t* list = reinterpret_cast<uint64_t*>(smem + kListAt);
    int* sel = reinterpret_cast<int*>(smem + kSelAt);
    float2* part = reinterpret_cast<float2*>(smem + kPartAt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = a.cluster, K = a.K;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int64_t row = blockIdx.x / C;
    const Row r = make_row<S>(a.logits, row, a.ld, a.V);
    const Slice sl = make_slice(r, C, rank);

    int issued = 0;
    if (tid == kConsumers) {
        init_barriers(ctl.bar, a.nbuf);
        ctl.nsel = ctl.ncand = 0;
        for (; issued < min(sl.nst, a.nbuf); ++issued) issue_stage(smem, ctl.bar, a.nbuf, r, sl, issued, issued);
    }
    __syncthreads();
    if (warp == kConsumerWarps) {
        if (lane == 0)
            for (; issued < sl.nst; ++issued)
                if (!issue_stage(smem, ctl.bar, a.nbuf, r, sl, issued, issued)) break;
    } else {
        for (int j = 0; j < sl.nst; ++j) {
            wait_stage(ctl.bar, a.nbuf, j);
            uint4 x[kU];
            load_stage<S>(smem, a.nbuf, r, sl, j, j, tid, x);
            release_stage(ctl.bar, a.nbuf, j);
            float v[kU][G];
#pragma unroll
            for (int u = 0; u < kU; ++u) Elt<S>::unpack(x[u], v[u]);
            const float m = max_of<G>(v);
            gm[j * kConsumers + tid] = m;
            gs[j * kConsumers + tid] = m == -kInf ? 0.f : sum_exp<G>(v, a.k2, m * a.k2);
        }
    }
    __syncthreads();
    const bool ok = !ctl.bar.abort;
    if (!ok && tid == kConsumers) drain(ctl.bar, a.nbuf, issued);
    if (!ok) __syncthreads();                  // the scratch overlies the stages

    // ---- 1. the bound t from the groups' maxima (a thread's own: no barrier before reading them) ----
    const bool consumer = tid < kConsumers;
    int it = 0;
    auto groups_from = [&](uint32_t t) {
        int n = 0;
        if (consumer)
            for (int j = 0; j < sl.nst; ++j) n += key_of(gm[j * kConsumers + tid]) >= t;
        return block_sum(n, ctl, it++);
    };
    uint32_t t = kKeyMin;
    if (groups_from(kKeyMin) >= K) {
        t = 0;
        for (int bit = 31; bit >= (sizeof(S) == 2 ? 16 : 0); --bit) {
            const int n = groups_from(t | (1u << bit));
            if (n >= K) {
                t |= 1u << bit;
                if (n <= K + K / 4) break;
            }
        }
        t = max(t, kKeyMin);
    }
    // ---- 2. candidates ----
    if (consumer)
        for (int j = 0; j < sl.nst; ++j)
            if (key_of(gm[j * kConsumers + tid]) >= t) {
                const int at = atomicAdd(&ctl.nsel, 1);
                if (at < kMaxSel) sel[at] = j * kConsumers + tid;
            }
    __syncthreads();
    const int nsel = ctl.nsel;
    float tm = -kInf, ts = 0.f;                // this thread's pair of the columns left out
    if (nsel <= kMaxSel) {
        for (int task = tid; task < nsel * kU; task += kThreads) {
            const int g = sel[task / kU];
            const int i = (g / kConsumers) * kStageVecs + g % kConsumers + (task % kU) * kConsumers;
            float2 p = make_float2(-kInf, 0.f);
            if (i < sl.n) {
                float v[G];
                Elt<S>::unpack(load_vector<S>(r, sl.v0 + i), v);
#pragma unroll
                for (int k = 0; k < G; ++k) {
                    const uint32_t key = key_of(v[k]);
                    if (key >= t) {
                        const int at = atomicAdd(&ctl.ncand, 1);
                        if (at < kMaxCand) cand[at] = cand_of(key, (sl.v0 + i) * G - r.shift + k);
                        v[k] = -kInf;
                    }
                }
                p = pair_of<G>(v, a.k2);
            }
            part[task] = p;
        }
        __syncthreads();
    }
    if (nsel > kMaxSel || ctl.ncand > kMaxCand) {
        exact_threshold<S>(a, r, sl, ctl, cand, tm, ts);
    } else {
        for (int i = tid; i < nsel; i += kThreads) {
            float m = -kInf, s = 0.f;
#pragma unroll
            for (int u = 0; u < kU; ++u) pair_merge(m, s, part[i * kU + u].x, part[i * kU + u].y, a.k2);
            gm[sel[i]] = m;
            gs[sel[i]] = s;
        }
        __syncthreads();
        if (consumer)
            for (int j = 0; j < sl.nst; ++j)
                pair_merge(tm, ts, gm[j * kConsumers + tid], gs[j * kConsumers + tid], a.k2);
    }
    // ---- 3. ranks ----
    const int n = min(ctl.ncand, kMaxCand);
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t c = cand[i];
        int rk = 0;
#pragma unroll 8
        for (int q = 0; q < n; ++q) rk += cand[q] > c;
        list[rk] = c;
    }
    for (int i = n + tid; i < K; i += kThreads) list[i] = 0;
    __syncthreads();
    for (int i = K + tid; i < n; i += kThreads) pair_merge(tm, ts, value_of(cand_key(list[i])), 1.f, a.k2);
    auto block_pair = [&](float& m, float& s) {
        pair_warp_reduce(m, s, a.k2);
        if (lane == 0) {
            ctl.red_m[warp] = m;
            ctl.red_s[warp] = s;
        }
        __syncthreads();
        m = -kInf;
        s = 0.f;
        for (int w = 0; w < kWarps; ++w) pair_merge(m, s, ctl.red_m[w], ctl.red_s[w], a.k2);
    };
    block_pair(tm, ts);
    bool all_ok = ok;
    const uint64_t* top = list;
    // ---- 4. the cluster's lists ----
    if (C > 1) {
        if (tid == 0) ctl.tail = make_float4(tm, ts, ok ? 1.f : 0.f, 0.f);
        cluster_arrive();
        cluster_wait();
        uint64_t* in = reinterpret_cast<uint64_t*>(smem + kInAt);
        uint64_t* out = reinterpret_cast<uint64_t*>(smem + kOutAt);
        if (rank == 0) {
            for (int i = tid; i < C * K; i += kThreads) {
                const int p = i / K;
                in[i] = ld_peer_u64(peer_addr(list + (i - p * K), (uint32_t)p));
                out[i] = 0;
            }
            tm = -kInf;
            ts = 0.f;
            for (int p = 0; p < C; ++p) {
                const float4 o = ld_peer_f4(peer_addr(&ctl.tail, (uint32_t)p));
                if (tid == 0) pair_merge(tm, ts, o.x, o.y, a.k2);
                all_ok = all_ok && o.z != 0.f;
            }
        }
        cluster_arrive();                      // the peers may leave
        cluster_wait();
        if (rank != 0) return;
        __syncthreads();
        for (int i = tid; i < C * K; i += kThreads) {
            const uint64_t c = in[i];
            if (!c) continue;
            int rk = i % K;
            for (int p = 0; p < C; ++p) {
                if (p == i / K) continue;
                const uint64_t* l = in + p * K;
                int lo = 0, hi = K;            // entries of l above c
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (l[mid] > c) lo = mid + 1;
                    else hi = mid;
                }
                rk += lo;
            }
            out[rk] = c;
        }
        __syncthreads();
        for (int i = K + tid; i < C * K; i += kThreads)
            if (out[i]) pair_merge(tm, ts, value_of(cand_key(out[i])), 1.f, a.k2);
        block_pair(tm, ts);
        top = out;
    }
    // ---- outputs ----
    for (int k = tid; k < K; k += kThreads) {
        const uint64_t c = top[k];
        a.values[row * K + k] = all_ok ? (c ? value_of(cand_key(c)) : -kInf) : __int_as_float(0x7FC00000);
        a.ids[row * K + k] = all_ok && c ? cand_col(c) : -1;
    }
    if (warp == 0) {
        float m = top[0] ? value_of(cand_key(top[0])) : -kInf, s = 0.f;
        for (int k = lane; k < K; k += 32)
            if (top[k]) s += ex2((value_of(cand_key(top[k])) - m) * a.k2);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
        pair_merge(m, s, tm, ts, a.k2);
        if (lane == 0) {
            const float bad = __int_as_float(0x7FC00000);
            a.lse[row] = !all_ok ? bad : s > 0.f ? m * a.scale + logf(s) : -kInf;
            a.tail[row] = !all_ok ? bad : ts > 0.f ? tm * a.scale + logf(ts) : -kInf;
        }
    }
}

template <typename S>
cudaError_t run(Args& a, int sms, cudaStream_t s) {
    constexpr int G = Elt<S>::kGroup;
    const int64_t nv = (a.V + 2 * G - 2) / G;
    auto st = [&](int c) { return (int)(((nv + c - 1) / c + kStageVecs - 1) / kStageVecs); };
    // few rows: blocks for the SMs; long rows: groups that leave room for two blocks an SM
    int C = 1;
    while (C < kMaxCluster && ((a.T * C < 2 * sms && st(C) > 1) || smem_bytes(3, st(C)) > 116000)) C *= 2;
    a.cluster = C;
    a.max_stages = st(C);
    a.nbuf = std::min(3, st(C));
    return launch_clusters<k_topk<S>>(a.T * C, C, kThreads, smem_bytes(a.nbuf, a.max_stages), s, a);
}

}  // namespace topk

VCE_DEBUG_READER(debug_word_topk)

}  // namespace vce

using namespace vce;

extern "C" int ce_topk(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld, int K, float temperature,
                       float* values, int64_t* ids, float* lse, float* tail_lse, vce_stream_t s) {
    if (dt != VCE_F32 && dt != VCE_BF16) return VCE_ERR_DTYPE;
    if (T < 0 || T > VCE_MAX_TOPK_T || V < 1 || V > VCE_MAX_TOPK_V) return VCE_ERR_SHAPE;
    if (K < 1 || K > VCE_MAX_TOPK || K > V || !rs::temperature_ok(temperature)) return VCE_ERR_ARG;
    if (ld < V) return VCE_ERR_LD;
    const size_t es = dt == VCE_BF16 ? 2 : 4;
    if (!fits_bytes(T, ld, es)) return VCE_ERR_SHAPE;
    if (T == 0) return VCE_OK;
    if (!logits || !values || !ids || !lse || !tail_lse) return VCE_ERR_NULL;
    if (!aligned(logits, es) || !aligned(values, 4) || !aligned(ids, 8) || !aligned(lse, 4) || !aligned(tail_lse, 4))
        return VCE_ERR_ALIGN;
    const int rc = require_sm100();
    if (rc) return rc;
    topk::Args a{logits, T, V, ld, K, 1.f / temperature, kLog2e / temperature, values, ids, lse, tail_lse, 1, 1, 1};
    const int sms = device_sm_count();
    const cudaError_t e = dt == VCE_BF16 ? topk::run<uint16_t>(a, sms, s) : topk::run<float>(a, sms, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}
