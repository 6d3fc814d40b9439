// ce_topk: a row's K largest logits in order, with the log-sum-exp of the row and of the columns
// left out.
//
// One pass over the logits.  The row (or its slice, in a thread-block cluster) streams through
// shared memory (row_stream.cuh); of every group of 16 or 32 values -- a consumer thread's vectors
// of a stage -- only the maximum and the sum of exponentials relative to it are kept.  The K-th
// largest group maximum is a lower bound t of the K-th largest value (K groups hold a value >= t), and
// every value >= t lies in a group whose maximum is >= t.  So
//   1. t: a binary search over the bits of the maxima's order keys (counts of keys >= t), among the
//      largest maxima of 512 sets of groups;
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
//
// What bounds it: many rows (k_topk_rows) the stream, with the selection of a row beside the next
// one's copies (8192 x 128256 bf16, K 64: 394 us, 5.4 TB/s, 0.79 of the measured copy); few rows (k_topk)
// the chain of a launch: copies, maxima, search, read again, rank, merge (one row of 128256: 11 us;
// 64 x 32001 fp32: 13.8 us, 0.6 TB/s).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "row_launch.h"
#include "row_stream.cuh"
#include "vce_logits.h"

namespace vce {
namespace topk {

using namespace rs;

constexpr int kThreads = kConsumers + 32;   // k_topk: consumers, which also select, and the producer warp
constexpr int kSets = 512;                  // sets of groups among whose maxima the bound is searched
constexpr int kMaxCand = 1024;              // candidates of a block
constexpr int kMaxSel = 512;                // groups read again
constexpr uint32_t kKeyMin = 0x00800000u;   // order key of the lowest finite value (-inf is one below)

// Scratch of a selection (in k_topk over the stage buffers, once the columns have streamed through).
constexpr int kCandAt = 0;                                   // [kMaxCand] candidates
constexpr int kSelAt = kCandAt + kMaxCand * 8;               // [kMaxSel] group numbers; before, [kSets] maxima
constexpr int kPartAt = kSelAt + kMaxSel * 4;                // [kMaxSel * kU] pairs of the vectors read again
constexpr int kListAt = kPartAt;                             // then [kMaxCand] candidates by rank (read by peers)
constexpr int kScratch = kPartAt + kMaxSel * kU * 8;
constexpr int kOutAt = kCandAt;                              // at last, [cluster * K] the cluster's lists by rank
static_assert(kMaxCluster * VCE_MAX_TOPK * 8 <= kScratch && kMaxCand * 8 <= kMaxSel * kU * 8 && kSets * 4 <= kMaxSel * 4 && kMaxCand >= VCE_MAX_TOPK, "scratch");

struct Args {
    const void* logits;
    int64_t T, V, ld;
    int K;
    float k2;                       // log2(e) / temperature
    float* values;
    int64_t* ids;
    float *lse, *tail;
    int cluster, nbuf, max_stages;
    uint64_t wait_ns;               // bound of every wait
    int withhold;                   // 1 (test hook): the last stage of a slice is not copied
};

constexpr int kRowsPerSm = 2;               // rows for each SM from which the persistent kernel runs

// What the selecting threads share.
struct alignas(16) SelCtl {
    float4 tail[kMaxCluster];       // in a cluster's first block: each block's rest (m, s, largest) and whether its copies landed
    float4 rest[8];                 // by the selecting warp
    int count[2][8];
    int nsel, ncand;
    float bound;
};

struct alignas(16) Ctl {
    SelCtl sel;
    Barriers bar;
};

// The scratch lies over the stage buffers, or behind them where they hold the whole slice (which is
// then read again from there).
__host__ __device__ constexpr int scratch_at(int nbuf, int max_stages) {
    return max_stages <= nbuf ? nbuf * kStageBytes : 0;
}
__host__ __device__ constexpr int scratch_end(int nbuf, int max_stages) {
    const int b = nbuf * kStageBytes, e = scratch_at(nbuf, max_stages) + kScratch;
    return b > e ? b : e;
}
__host__ __device__ constexpr int smem_bytes(int nbuf, int max_stages, int cluster, int K) {
    return scratch_end(nbuf, max_stages) + max_stages * kConsumers * 8 + (int)sizeof(Ctl) +
           (cluster > 1 ? cluster * K * 8 : 0);
}

// NS threads (whole warps of consecutive numbers, tid counted from the first) select together; a
// barrier of theirs, number `id`.
template <int NS>
struct Team {
    static_assert(NS % 32 == 0 && NS <= 256 && kSets % NS == 0, "selecting threads");
    static constexpr int kThreads = NS, kWarps = NS / 32;
    int tid, id;
    __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(NS) : "memory"); }
    __device__ __forceinline__ int warp() const { return tid >> 5; }
    __device__ __forceinline__ int lane() const { return tid & 31; }
};

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

// Sum over the selecting threads of each one's n (call number it picks one of two buffers, so one
// barrier a call is enough).
template <int NS>
__device__ __forceinline__ int block_sum(const Team<NS>& tm, int n, SelCtl& ctl, int it) {
    n = __reduce_add_sync(0xFFFFFFFFu, n);
    if (tm.lane() == 0) ctl.count[it & 1][tm.warp()] = n;
    tm.sync();
    int t = 0;
#pragma unroll
    for (int w = 0; w < Team<NS>::kWarps; ++w) t += ctl.count[it & 1][w];
    return t;
}
// The columns left out: their pair, and the largest of them, which stands for their log-sum-exp where
// its product with k2 passes fp32 (masks of the type's lowest value; such values are in no pair).
struct Rest {
    float m, s, top;
    __device__ __forceinline__ void merge(float m2, float s2, float top2) {
        pair_merge(m, s, m2, s2);
        top = fmaxf(top, top2);
    }
    // a value, `times` over
    __device__ __forceinline__ void add(float v, float k2, float times = 1.f) {
        const float r = v * k2;
        if (r > -kInf) pair_merge(m, s, r, times * ex2(fmaf(v, k2, -r)));
        top = fmaxf(top, v);
    }
    __device__ __forceinline__ float lse(float scale) const { return s > 0.f ? m * kLn2 + logf(s) : top * scale; }
};

// Merges the selecting threads' rests; every thread has the result.
__device__ __forceinline__ void warp_rest(Rest& t) {
    pair_warp_reduce(t.m, t.s);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t.top = fmaxf(t.top, __shfl_xor_sync(0xFFFFFFFFu, t.top, off));
}
template <int NS>
__device__ __forceinline__ void block_rest(const Team<NS>& team, Rest& t, SelCtl& ctl) {
    warp_rest(t);
    if (team.lane() == 0) ctl.rest[team.warp()] = make_float4(t.m, t.s, t.top, 0.f);
    team.sync();
    t = Rest{-kInf, 0.f, -kInf};
    for (int w = 0; w < Team<NS>::kWarps; ++w) t.merge(ctl.rest[w].x, ctl.rest[w].y, ctl.rest[w].z);
}

template <int G>
__device__ __forceinline__ float max_of_vector(const float (&v)[G]) {
    float m = v[0];
#pragma unroll
    for (int k = 1; k < G; ++k) m = fmaxf(m, v[k]);
    return m;
}

// The pair of G values (the reference: the largest times k2), -inf left out.
template <int G>
__device__ __forceinline__ float2 pair_of(const float (&v)[G], float k2) {
    const float m = max_of_vector<G>(v) * k2;
    if (m == -kInf) return make_float2(-kInf, 0.f);
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < G; ++k) s += ex2(fmaf(v[k], k2, -m));
    return make_float2(m, s);
}

// The K largest of the slice by the exact K-th value, every value read from global memory as often
// as its search takes: for slices where the bound from the groups admits too many.  Candidates go
// to cand (ctl.ncand of them), everything else into this thread's rest.
template <typename S, int NS>
__device__ __noinline__ void exact_threshold(const Args& a, const Row& r, const Slice& sl, SelCtl& ctl, uint64_t* cand,
                                             Team<NS> team, Rest& rest) {
    constexpr int G = Elt<S>::kGroup;
    const int tid = team.tid, lane = team.lane(), warp = team.warp();
    int it = 0;
    auto count_from = [&](uint32_t t) {
        int n = 0;
        for (int i = tid; i < sl.n; i += NS) {
            float v[G];
            Elt<S>::unpack(load_vector<S>(r, sl.v0 + i), v);
#pragma unroll
            for (int k = 0; k < G; ++k) n += key_of(v[k]) >= t;
        }
        return block_sum(team, n, ctl, it++);
    };
    team.sync();                                // ctl.count of the caller's search has been read
    uint32_t t = kKeyMin;
    if (count_from(kKeyMin) >= a.K) {
        t = 0;
        for (int bit = 31; bit >= 0; --bit)
            if (count_from(t | (1u << bit)) >= a.K) t |= 1u << bit;
    }
    if (tid == 0) ctl.ncand = 0;
    team.sync();
    // above t: candidates; equal: counted; below: the tail
    int eq = 0;
    for (int i = tid; i < sl.n; i += NS) {
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
            rest.top = fmaxf(rest.top, v[k]);
        }
        const float2 p = pair_of<G>(v, a.k2);
        rest.merge(p.x, p.y, -kInf);
    }
    const int total_eq = block_sum(team, eq, ctl, it++);
    const int above = min(ctl.ncand, kMaxCand);
    const int want = min(total_eq, a.K - above);
    team.sync();
    // the first `want` values equal to t, in column order: vectors i = base + tid
    int found = 0;
    for (int base = 0; base < sl.n && found < want; base += NS) {
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
        team.sync();
        int all = 0;
        for (int w = 0; w < Team<NS>::kWarps; ++w) {
            if (w < warp) before += ctl.count[0][w];
            all += ctl.count[0][w];
        }
        for (; hits && before < want; hits &= hits - 1, ++before)
            cand[above + before] = cand_of(t, (sl.v0 + i) * G - r.shift + __ffs(hits) - 1);
        found += all;
        team.sync();
    }
    if (tid == 0) {
        ctl.ncand = above + want;
        if (total_eq > want) rest.add(value_of(t), a.k2, (float)(total_eq - want));
    }
    team.sync();
}

// The K largest of a slice whose groups' maxima and sums are in gm and gs ([stages][GT], group t of
// stage j holding the vectors j GT kU + t + u GT), by a team: the sorted
// candidates, at least K places with 0 behind the last, in the scratch's list, and the pair of the
// columns that are not among the first K (the same in every thread).  held: the slice's vectors in
// shared memory, if they are all there.
template <typename S, int GT, int NS>
__device__ __forceinline__ void select(const Args& a, const Row& r, const Slice& sl, int stages, SelCtl& ctl,
                                       uint8_t* scratch, float* gm, float* gs, const Team<NS>& team, Rest& rest,
                                       const uint8_t* held = nullptr) {
    constexpr int G = Elt<S>::kGroup;
    static_assert(GT % NS == 0, "whole rounds of groups");
    constexpr int SP = kSets / NS;             // sets of a thread
    const int tid = team.tid, lane = team.lane(), warp = team.warp();
    const int K = a.K, rounds = stages * (GT / NS), groups = stages * GT;
    uint64_t* cand = reinterpret_cast<uint64_t*>(scratch + kCandAt);
    uint64_t* list = reinterpret_cast<uint64_t*>(scratch + kListAt);
    int* sel = reinterpret_cast<int*>(scratch + kSelAt);
    float2* part = reinterpret_cast<float2*>(scratch + kPartAt);
    // ---- 1. the bound t ----
    // Each thread's groups are tid + i NS, round i in its set i mod SP.  The largest values of the kSets
    // sets are values of as many columns, so the K-th largest of them bounds the K-th largest value from
    // below nearly as well as that of all groups (K = 64: 73 groups are read again instead of 64), and
    // one warp finds it in registers, without barriers.
    float most_of[SP];
#pragma unroll
    for (int q = 0; q < SP; ++q) most_of[q] = -kInf;
    for (int i = 0; i < rounds; i += SP) {
#pragma unroll
        for (int q = 0; q < SP; ++q)
            if (i + q < rounds) most_of[q] = fmaxf(most_of[q], gm[(i + q) * NS + tid]);
    }
    uint32_t* tops = reinterpret_cast<uint32_t*>(scratch + kSelAt);   // [kSets]
    float most_mine = -kInf;
#pragma unroll
    for (int q = 0; q < SP; ++q) {
        tops[q * NS + tid] = key_of(most_of[q]);
        most_mine = fmaxf(most_mine, most_of[q]);
    }
    team.sync();
    if (warp == 0) {
        constexpr int N = kSets / 32;
        uint32_t k[N], most = 0;
        int n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            k[i] = tops[lane + 32 * i];
            most = max(most, k[i]);
            n += k[i] >= kKeyMin;
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        uint32_t t = kKeyMin;
        if (__reduce_add_sync(0xFFFFFFFFu, n) >= K) {
            t = 0;
            for (int bit = 31; bit >= (sizeof(S) == 2 ? 16 : 0); --bit) {
                const uint32_t c = t | (1u << bit);
                if (c > most) continue;        // none is as large
                int part4[4] = {};
#pragma unroll
                for (int i = 0; i < N; ++i) part4[i % 4] += k[i] >= c;
                n = __reduce_add_sync(0xFFFFFFFFu, (part4[0] + part4[1]) + (part4[2] + part4[3]));
                if (n >= K) t = c;
                if (n >= K && n <= K + K / 2) break;   // near enough: a few more groups are read again
            }
            t = max(t, kKeyMin);
        }
        if (lane == 0) {
            ctl.bound = value_of(t);
            ctl.nsel = ctl.ncand = 0;
        }
    }
    team.sync();
    const float t = ctl.bound;
    // ---- 2. candidates ----
    // the groups with a value >= t: a place on the list for each lane's, one atomic a warp (and for each 64
    // rounds: a slice of the longest fp32 rows has 65)
    auto list_rounds = [&](int i0, int i1) {
        uint64_t mine = 0;                     // bit i: group tid + (i0 + i) NS
        if (most_mine >= t) {
#pragma unroll 4
            for (int i = i0; i < i1; ++i) mine |= (uint64_t)(gm[i * NS + tid] >= t) << (i - i0);
        }
        const int n = __popcll(mine);
        int at = n;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, at, off);
            if (lane >= off) at += o;
        }
        int base = 0;
        if (lane == 31 && at) base = atomicAdd(&ctl.nsel, at);
        at += __shfl_sync(0xFFFFFFFFu, base, 31) - n;
        for (; mine; mine &= mine - 1, ++at)
            if (at < kMaxSel) sel[at] = tid + (i0 + __ffsll((long long)mine) - 1) * NS;
    };
    list_rounds(0, min(rounds, 64));
    if (rounds > 64) list_rounds(64, rounds);
    team.sync();
    const int nsel = ctl.nsel;
    rest = Rest{-kInf, 0.f, -kInf};            // this thread's columns left out
    if (nsel <= kMaxSel) {
        // vectors of the listed groups, two in flight a thread
        const int tasks = nsel * kU;
        for (int task0 = tid; task0 < tasks; task0 += 2 * NS) {
            uint4 x[2];
            int at[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int task = task0 + h * NS;
                at[h] = -1;
                if (task >= tasks) continue;
                const int g = sel[task / kU];
                const int i = (g / GT) * (GT * kU) + g % GT + (task % kU) * GT;
                if (i >= sl.n) continue;
                at[h] = i;
                const int v = sl.v0 + i;
                x[h] = held && v >= r.iv0 && v < r.iv1 ? tc::lds16(held + (size_t)i * 16) : load_vector<S>(r, v);
            }
#pragma unroll 1
            for (int h = 0; h < 2 && task0 + h * NS < tasks; ++h) {
                float2 p = make_float2(-kInf, 0.f);   // the largest value left, and its sum of exponentials
                if (at[0] >= 0) {
                    float v[G];
                    Elt<S>::unpack(x[0], v);
                    uint32_t hits = 0;
#pragma unroll
                    for (int k = 0; k < G; ++k) hits |= (v[k] >= t ? 1u : 0u) << k;
                    if (hits) {
                        int n = atomicAdd(&ctl.ncand, __popc(hits));
#pragma unroll
                        for (int k = 0; k < G; ++k)
                            if ((hits >> k) & 1u) {
                                if (n < kMaxCand) cand[n] = cand_of(key_of(v[k]), (sl.v0 + at[0]) * G - r.shift + k);
                                ++n;
                                v[k] = -kInf;
                            }
                    }
                    p = pair_of<G>(v, a.k2);
                    p.x = max_of_vector<G>(v);
                }
                part[task0 + h * NS] = p;
                x[0] = x[1];
                at[0] = at[1];
            }
        }
        team.sync();
    }
    if (nsel > kMaxSel || ctl.ncand > kMaxCand) {
        exact_threshold<S, NS>(a, r, sl, ctl, cand, team, rest);
    } else {
        for (int i = tid; i < nsel; i += NS) {
            float top = -kInf;
#pragma unroll
            for (int u = 0; u < kU; ++u) top = fmaxf(top, part[i * kU + u].x);
            gm[sel[i]] = top;
            const float ref = top * a.k2;
            float s = 0.f;
            if (ref > -kInf) {
#pragma unroll
                for (int u = 0; u < kU; ++u) s += part[i * kU + u].y * ex2(part[i * kU + u].x * a.k2 - ref);   // 0 * 0 for -inf
            }
            gs[sel[i]] = s;
        }
        team.sync();
#pragma unroll 4
        for (int g = tid; g < groups; g += NS) rest.top = fmaxf(rest.top, gm[g]);
        rest.m = rest.top * a.k2;
        if (rest.m > -kInf) {
#pragma unroll 4
            for (int g = tid; g < groups; g += NS) rest.s += gs[g] * ex2(gm[g] * a.k2 - rest.m);   // 0 * 0 for -inf
        }
    }
    // ---- 3. ranks ----
    const int n = min(ctl.ncand, kMaxCand);
    for (int i = tid; i < n; i += NS) {
        const uint64_t c = cand[i];
        int rk = 0;
#pragma unroll 8
        for (int q = 0; q < n; ++q) rk += cand[q] > c;
        list[rk] = c;
    }
    for (int i = n + tid; i < K; i += NS) list[i] = 0;
    team.sync();
    for (int i = K + tid; i < n; i += NS) rest.add(value_of(cand_key(list[i])), a.k2);
    block_rest(team, rest, ctl);
}

// The row's outputs from its sorted list and the pair of the rest (of the team's first warp), by a team.
template <int NS>
__device__ __forceinline__ void outputs(const Args& a, int64_t row, const uint64_t* top, bool ok, Rest rest,
                                        const Team<NS>& team) {
    const int tid = team.tid;
    const float bad = __int_as_float(0x7FC00000);
    for (int k = tid; k < a.K; k += NS) {
        const uint64_t c = top[k];
        a.values[row * a.K + k] = ok ? (c ? value_of(cand_key(c)) : -kInf) : bad;
        a.ids[row * a.K + k] = ok && c ? cand_col(c) : -1;
    }
    if (tid < 32) {
        const float scale = a.k2 * kLn2;
        const float bad = __int_as_float(0x7FC00000);
        Rest all{-kInf, 0.f, top[0] ? value_of(cand_key(top[0])) : -kInf};
        all.m = all.top * a.k2;
        if (all.m > -kInf)
            for (int k = tid; k < a.K; k += 32)
                if (top[k]) all.s += ex2(fmaf(value_of(cand_key(top[k])), a.k2, -all.m));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) all.s += __shfl_xor_sync(0xFFFFFFFFu, all.s, off);
        all.merge(rest.m, rest.s, rest.top);
        if (tid == 0) {
            a.lse[row] = ok ? all.lse(scale) : bad;
            a.tail[row] = ok ? rest.lse(scale) : bad;
        }
    }
}

// A group's maximum and the sum of its exponentials relative to it (to its product with k2, as rounded).
template <typename S>
__device__ __forceinline__ void group_of(const uint4 (&x)[kU], float k2, float& m, float& s) {
    constexpr int G = Elt<S>::kGroup;
    const float top = max_of_loaded<S>(x);
    float v[kU][G];
#pragma unroll
    for (int u = 0; u < kU; ++u) Elt<S>::unpack(x[u], v[u]);
    m = top;
    const float ref = top * k2;
    s = ref == -kInf ? 0.f : sum_exp<G>(v, k2, ref);
}

// ---- one cluster per row -------------------------------------------------------------------------

template <typename S>
__global__ void __launch_bounds__(kThreads, 3) k_topk(const __grid_constant__ Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* scratch = smem + scratch_at(a.nbuf, a.max_stages);
    float* gm = reinterpret_cast<float*>(smem + scratch_end(a.nbuf, a.max_stages));
    float* gs = gm + a.max_stages * kConsumers;
    Ctl& ctl = *reinterpret_cast<Ctl*>(gs + a.max_stages * kConsumers);
    uint64_t* in = reinterpret_cast<uint64_t*>(&ctl + 1);   // [cluster][K] in the cluster's first block
    uint64_t* list = reinterpret_cast<uint64_t*>(scratch + kListAt);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int NS = kConsumers;             // the consumers select
    const Team<NS> team{tid, 1};
    const int C = a.cluster, K = a.K;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int64_t row = blockIdx.x / C;
    const Row r = make_row<S>(a.logits, row, a.ld, a.V);
    const Slice sl = make_slice(r, C, rank);

    const int copies = sl.nst - a.withhold;
    int issued = 0;
    if (tid == kConsumers) {
        init_barriers(ctl.bar, a.nbuf);
        for (; issued < min(copies, a.nbuf); ++issued)
            issue_stage(smem, ctl.bar, a.nbuf, r, sl, issued, issued, a.wait_ns);
    }
    if (C > 1) cluster_arrive_relaxed();       // this block runs: peers may write into it
    __syncthreads();
    if (warp == kConsumerWarps) {
        if (lane == 0)
            for (; issued < copies; ++issued)
                if (!issue_stage(smem, ctl.bar, a.nbuf, r, sl, issued, issued, a.wait_ns)) break;
    } else {
        for (int j = 0; j < sl.nst; ++j) {
            wait_stage(ctl.bar, a.nbuf, j, a.wait_ns);
            uint4 x[kU];
            load_stage<S>(smem, a.nbuf, r, sl, j, j, tid, x);
            group_of<S>(x, a.k2, gm[j * kConsumers + tid], gs[j * kConsumers + tid]);
            release_stage(ctl.bar, a.nbuf, j);
        }
    }
    __syncthreads();
    const bool ok = !ctl.bar.abort;
    if (!ok && tid == kConsumers) drain(ctl.bar, a.nbuf, issued);
    if (!ok) __syncthreads();                  // the scratch overlies the stages

    Rest rest{-kInf, 0.f, -kInf};
    if (tid < NS) select<S, kConsumers, NS>(a, r, sl, sl.nst, ctl.sel, scratch, gm, gs, team, rest,
                                               a.max_stages <= a.nbuf ? smem : nullptr);
    if (C == 1) {
        if (tid < NS) outputs(a, row, list, ok, rest, team);
        return;
    }
    // ---- 4. every block's list and pair into the first block, which merges them ----
    cluster_wait();                            // the first block runs
    if (tid < NS)
        for (int i = tid; i < K; i += NS) st_peer_u64(peer_addr(in + rank * K + i, 0), list[i]);
    if (tid == 0) st_peer(peer_addr(&ctl.sel.tail[rank], 0), make_float4(rest.m, rest.s, rest.top, ok ? 1.f : 0.f));
    cluster_arrive();
    cluster_wait();
    if (rank != 0 || tid >= NS) return;
    uint64_t* out = reinterpret_cast<uint64_t*>(scratch + kOutAt);
    const int n = C * K;
    for (int i = tid; i < n; i += NS) out[i] = 0;
    team.sync();
    for (int i = tid; i < n; i += NS) {
        const uint64_t c = in[i];
        if (!c) continue;
        int rk = 0;
        if (n <= 512) {
#pragma unroll 8
            for (int q = 0; q < n; ++q) rk += in[q] > c;
        } else {                               // ranks in the other lists, which are sorted
            const int own = i / K;
            rk = i - own * K;
            for (int p = 0; p < C; ++p) {
                const uint64_t* l = in + p * K;
                int lo = 0, hi = p == own ? 0 : K;   // entries of l above c
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (l[mid] > c) lo = mid + 1;
                    else hi = mid;
                }
                rk += lo;
            }
        }
        out[rk] = c;
    }
    team.sync();
    // the columns left out, by the warp that writes their log-sum-exp: the blocks' and the lists' rest
    bool all_ok = true;
    for (int p = 0; p < C; ++p) all_ok = all_ok && ctl.sel.tail[p].w != 0.f;
    if (tid < 32) {
        rest = Rest{-kInf, 0.f, -kInf};
        if (tid < C) rest.merge(ctl.sel.tail[tid].x, ctl.sel.tail[tid].y, ctl.sel.tail[tid].z);
        for (int i = K + tid; i < n; i += 32)
            if (out[i]) rest.add(value_of(cand_key(out[i])), a.k2);
        warp_rest(rest);
    }
    outputs(a, row, out, all_ok, rest, team);
}

// ---- many rows: a persistent kernel -----------------------------------------------------------------
//
// One block per SM walks the rows blockIdx.x, blockIdx.x + gridDim.x, ...: consumers reduce a row's
// groups while two teams of selecting warps work on the rows before (even and odd ones), so the copies
// never stop for a selection, and a selection's waits are covered by the other's.

constexpr int kPWarps = 16, kPNT = kPWarps * 32;             // consumers
constexpr int kPVecs = kPNT * kU, kPBytes = kPVecs * 16;     // a stage: 32 KB
constexpr int kPBufs = 3, kPStages = 8;                      // stages of the ring and, at most, of a row
constexpr int kPProducer = kPWarps, kPSelect = kPWarps + 1;
constexpr int kPTeam = 128;                                  // selecting threads of a team
constexpr int kPThreads = (kPWarps + 1) * 32 + 2 * kPTeam;
constexpr uint32_t kSuspend = 10000;                         // ns a poll may sleep

struct alignas(16) PCtl {
    SelCtl sel[2];
    uint64_t full[kPBufs], empty[kPBufs];
    uint64_t grouped[2], taken[2];   // a row's groups are there; have been selected from
    int abort, err;
};
constexpr int kPSmem = kPBufs * kPBytes + 2 * kScratch + 2 * kPStages * kPNT * 8 + (int)sizeof(PCtl);

template <typename S>
__global__ void __launch_bounds__(kPThreads, 1) k_topk_rows(const __grid_constant__ Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* scratch = smem + kPBufs * kPBytes;                     // [2]
    float* groups = reinterpret_cast<float*>(scratch + 2 * kScratch);   // [2][maxima, sums][kPStages][kPNT]
    PCtl& ctl = *reinterpret_cast<PCtl*>(groups + 4 * kPStages * kPNT);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &ctl.abort;
    if (tid == 0) {
        for (int i = 0; i < kPBufs; ++i) {
            tc::mbar_init(&ctl.full[i], 1);
            tc::mbar_init(&ctl.empty[i], kPWarps);
        }
        for (int p = 0; p < 2; ++p) {
            tc::mbar_init(&ctl.grouped[p], kPWarps);
            tc::mbar_init(&ctl.taken[p], kPTeam / 32);
        }
        ctl.abort = ctl.err = 0;
        tc::fence_mbar_init();
    }
    __syncthreads();
    auto slice_of = [&](const Row& r) { return Slice{0, r.nv, (r.nv + kPVecs - 1) / kPVecs}; };
    int st = 0;
    uint32_t phase = 0;
    auto step = [&]() {
        if (++st == kPBufs) {
            st = 0;
            phase ^= 1;
        }
    };
    if (warp == kPProducer) {
        if (lane == 0) {
            int q = 0;
            for (int64_t row = blockIdx.x; row < a.T && !*abort; row += gridDim.x) {
                const Row r = make_row<S>(a.logits, row, a.ld, a.V);
                const Slice sl = slice_of(r);
                for (int j = 0; j < sl.nst; ++j, ++q, step()) {
                    if (!tc::mbar_wait(&ctl.empty[st], phase ^ 1, &ctl.abort, &ctl.err, kErrEmpty, a.wait_ns, kSuspend)) break;
                    if (a.withhold && j == sl.nst - 1) continue;
                    const int lo = max(j * kPVecs, r.iv0), hi = min((j + 1) * kPVecs, r.iv1);
                    if (hi > lo && dbg::ok(lo >= 0 && hi <= r.nv, dbg::kCols)) {
                        tc::mbar_arrive_expect_tx(&ctl.full[st], (uint32_t)(hi - lo) * 16);
                        tc::bulk_load(smem + st * kPBytes + (lo - j * kPVecs) * 16, r.base + (int64_t)lo * 16,
                                      (uint32_t)(hi - lo) * 16, &ctl.full[st]);
                    } else {
                        tc::mbar_arrive(&ctl.full[st]);
                    }
                }
            }
            if (*abort) {                      // copies in flight land before the block may leave
                int never = 0;
                for (int p = max(0, q - kPBufs); p < q; ++p)
                    tc::mbar_wait(&ctl.full[p % kPBufs], (p / kPBufs) & 1, &never, nullptr, 0, a.wait_ns);
            }
        }
        __syncwarp();
    } else if (warp < kPWarps) {
        int64_t e = 0;
        for (int64_t row = blockIdx.x; row < a.T && !*abort; row += gridDim.x, ++e) {
            const int par = (int)(e & 1);
            const Row r = make_row<S>(a.logits, row, a.ld, a.V);
            const Slice sl = slice_of(r);
            // row e - 2's groups have been selected from
            if (e >= 2) tc::mbar_wait(&ctl.taken[par], (uint32_t)((e - 2) >> 1) & 1, &ctl.abort, &ctl.err, kErrEmpty,
                                      a.wait_ns, kSuspend);
            float* gm = groups + par * 2 * kPStages * kPNT + tid;
            for (int j = 0; j < sl.nst; ++j, step()) {
                tc::mbar_wait(&ctl.full[st], phase, &ctl.abort, &ctl.err, kErrFull, a.wait_ns, kSuspend);
                const uint4* buf = reinterpret_cast<const uint4*>(smem + st * kPBytes) + tid;
                const int at = j * kPVecs + tid;
                uint4 x[kU];
                if (j * kPVecs >= r.iv0 && (j + 1) * kPVecs <= r.iv1) {
#pragma unroll
                    for (int u = 0; u < kU; ++u) x[u] = tc::lds16(buf + u * kPNT);
                } else {
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const int v = at + u * kPNT;
                        x[u] = stage::neg_inf16<S>();
                        if (v < r.nv) x[u] = v >= r.iv0 && v < r.iv1 ? tc::lds16(buf + u * kPNT) : load_partial<S>(r, v);
                    }
                }
                reads_done();                  // before the sums: 395 us at 8192 x 128256, behind them 402
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl.empty[st]);
                group_of<S>(x, a.k2, gm[j * kPNT], gm[(kPStages + j) * kPNT]);
            }
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.grouped[par]);
        }
    } else {
        const int par = (tid - kPSelect * 32) / kPTeam;
        const Team<kPTeam> team{(tid - kPSelect * 32) % kPTeam, 1 + par};
        uint8_t* mine = scratch + par * kScratch;
        float* gm = groups + par * 2 * kPStages * kPNT;
        uint32_t phase_of = 0;
        for (int64_t row = blockIdx.x + (int64_t)par * gridDim.x; row < a.T; row += 2 * (int64_t)gridDim.x, phase_of ^= 1) {
            const Row r = make_row<S>(a.logits, row, a.ld, a.V);
            const Slice sl = slice_of(r);
            tc::mbar_wait(&ctl.grouped[par], phase_of, &ctl.abort, &ctl.err, kErrFull, a.wait_ns, kSuspend);
            Rest rest;
            select<S, kPNT, kPTeam>(a, r, sl, sl.nst, ctl.sel[par], mine, gm, gm + kPStages * kPNT, team, rest);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.taken[par]);
            outputs(a, row, reinterpret_cast<const uint64_t*>(mine + kListAt), !*abort, rest, team);
            team.sync();                       // the list has been read
        }
    }
}

template <typename S>
cudaError_t run(Args& a, int sms, cudaStream_t s) {
    constexpr int G = Elt<S>::kGroup;
    const int64_t nv = (a.V + 2 * G - 2) / G;
    if (a.T >= kRowsPerSm * sms && nv > kPVecs && nv <= kPStages * kPVecs)
        return launch_clusters<k_topk_rows<S>>(sms, 1, kPThreads, kPSmem, s, a);
    auto st = [&](int c) { return (int)(((nv + c - 1) / c + kStageVecs - 1) / kStageVecs); };
    // few rows: as many blocks as run at once, two an SM; long rows: groups that leave room for two
    int C = 1;
    while (C < kMaxCluster && ((2 * C * a.T <= 2 * sms && st(C) > 1) || smem_bytes(3, st(C), C, a.K) > 116000)) C *= 2;
    a.cluster = C;
    a.max_stages = st(C);
    a.nbuf = std::min(3, st(C));
    return launch_clusters<k_topk<S>>(a.T * C, C, kThreads, smem_bytes(a.nbuf, a.max_stages, C, a.K), s, a);
}

}  // namespace topk

VCE_DEBUG_READER(debug_word_topk)

}  // namespace vce

using namespace vce;

static int topk_call(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld, int K, float temperature,
                     float* values, int64_t* ids, float* lse, float* tail_lse, uint64_t wait_ns, int withhold,
                     vce_stream_t s) {
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
    topk::Args a{logits, T, V, ld, K, (float)(1.4426950408889634 / (double)temperature), values, ids, lse, tail_lse, 1, 1, 1,
                 wait_ns, withhold};
    const int sms = device_sm_count();
    const cudaError_t e = dt == VCE_BF16 ? topk::run<uint16_t>(a, sms, s) : topk::run<float>(a, sms, s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

extern "C" int ce_topk(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld, int K, float temperature,
                       float* values, int64_t* ids, float* lse, float* tail_lse, vce_stream_t s) {
    return topk_call(logits, dt, T, V, ld, K, temperature, values, ids, lse, tail_lse, tc::kWaitNs, 0, s);
}

extern "C" int vce_test_topk_stall(const void* logits, int64_t T, int64_t V, int K, float* values, int64_t* ids,
                                   float* lse, float* tail_lse, uint64_t wait_ns, vce_stream_t s) {
    if (wait_ns < 1000000ull || wait_ns > tc::kWaitNs) return VCE_ERR_ARG;
    return topk_call(logits, VCE_BF16, T, V, V, K, 1.f, values, ids, lse, tail_lse, wait_ns, 1, s);
}
