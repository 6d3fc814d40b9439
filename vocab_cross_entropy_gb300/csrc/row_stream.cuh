// Streaming of one row's columns (or a slice of them) through shared memory, shared by the
// top-K and distillation kernels (ce_topk.cu, ce_distill.cu).
//
// A row of any alignment and length is taken as the 16-byte vectors of global memory that hold
// it: vector v holds the columns v * G - shift + k, k < G, where shift is the row's distance from
// the 16-byte boundary below it.  Every vector but possibly the first and the last lies wholly in
// the row and is copied by bulk asynchronous copies (cp.async.bulk, 16-byte aligned at both ends
// by construction); the elements of a partial first or last vector are loaded one by one, by the
// thread that owns the vector, and read as -inf outside the row.  So rows of every layout run the
// same code, at the same speed.
//
// A block has kConsumers threads that work on the columns and a producer warp, whose first lane
// keeps up to nbuf stages of 16 KB in flight, each with a mbarrier for "loaded" and one for
// "released".  Consumer thread t owns the vectors t + u * kConsumers, u < kU, of every stage.
// Every wait is bounded (2 s; less in the test hooks); one that gives up records its code and sets the
// block's abort flag, after which every role stops waiting, and the producer lets its copies in flight
// land.  Kernels look at the flag once everything is written, and mark what may be wrong.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "ce_stage.cuh"
#include "vce_async.cuh"
#include "vce_check.cuh"
#include "vce_device.cuh"

namespace vce {
namespace rs {

constexpr int kConsumerWarps = 8;
constexpr int kConsumers = kConsumerWarps * 32;
constexpr int kU = 4;                                // vectors of a stage per consumer thread
constexpr int kStageVecs = kU * kConsumers;          // 1024
constexpr int kStageBytes = kStageVecs * 16;         // 16 KB
constexpr int kMaxBufs = 12;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxCluster = 8;
enum { kErrEmpty = 105, kErrFull = 106 };

// A row's vectors: base is the 16-byte aligned address of vector 0, [iv0, iv1) the whole ones.
struct Row {
    const char* base;
    int64_t V;
    int nv, iv0, iv1, shift;
};

template <typename S>
__device__ __forceinline__ Row make_row(const void* p, int64_t row, int64_t ld, int64_t V) {
    constexpr int G = Elt<S>::kGroup;
    const char* at = static_cast<const char*>(p) + row * ld * (int64_t)sizeof(S);
    Row r;
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(at) & 15u);
    r.base = at - off;
    r.shift = (int)(off / sizeof(S));
    r.V = V;
    r.nv = (int)((V + r.shift + G - 1) / G);
    r.iv0 = r.shift ? 1 : 0;
    r.iv1 = (int)((V + r.shift) / G);
    return r;
}

// The vectors [v0, v0 + n) of a row that one block takes, in nst stages.
struct Slice {
    int v0, n, nst;
};

__device__ __forceinline__ Slice make_slice(const Row& r, int parts, int part) {
    const int per = (r.nv + parts - 1) / parts;
    Slice s;
    s.v0 = min(r.nv, part * per);
    s.n = min(r.nv - s.v0, per);
    s.nst = (s.n + kStageVecs - 1) / kStageVecs;
    return s;
}

struct Barriers {
    uint64_t full[kMaxBufs], empty[kMaxBufs];
    int abort;
    int err;
};

__device__ __forceinline__ void init_barriers(Barriers& b, int nbuf) {
    for (int i = 0; i < nbuf; ++i) {
        tc::mbar_init(&b.full[i], 1);
        tc::mbar_init(&b.empty[i], kConsumerWarps);
    }
    b.abort = 0;
    b.err = 0;
    tc::fence_mbar_init();
}

// Copies stage j of the slice into ring position q (one thread).  False: a wait gave up.
__device__ __forceinline__ bool issue_stage(uint8_t* bufs, Barriers& b, int nbuf, const Row& r, const Slice& s, int j,
                                            int q, uint64_t wait_ns) {
    const int st = q % nbuf;
    if (q >= nbuf && !tc::mbar_wait(&b.empty[st], ((q / nbuf) & 1) ^ 1, &b.abort, &b.err, kErrEmpty, wait_ns)) return false;
    const int a = s.v0 + j * kStageVecs;
    const int lo = max(a, r.iv0), hi = min(min(a + kStageVecs, s.v0 + s.n), r.iv1);
    if (hi > lo && dbg::ok(lo >= 0 && (int64_t)hi * 16 <= (int64_t)r.nv * 16, dbg::kCols)) {
        tc::mbar_arrive_expect_tx(&b.full[st], (uint32_t)(hi - lo) * 16);
        tc::bulk_load(bufs + st * kStageBytes + (lo - a) * 16, r.base + (int64_t)lo * 16, (uint32_t)(hi - lo) * 16,
                      &b.full[st]);
    } else {
        tc::mbar_arrive(&b.full[st]);
    }
    return true;
}

// After an abort: waits (bounded) until the copies of ring positions [0, q) have landed.
__device__ __forceinline__ void drain(Barriers& b, int nbuf, int q) {
    int never = 0;
    for (int p = max(0, q - nbuf); p < q; ++p) tc::mbar_wait(&b.full[p % nbuf], (p / nbuf) & 1, &never, nullptr, 0);
}

__device__ __forceinline__ bool wait_stage(Barriers& b, int nbuf, int q, uint64_t wait_ns) {
    return tc::mbar_wait(&b.full[q % nbuf], (q / nbuf) & 1, &b.abort, &b.err, kErrFull, wait_ns);
}

// This thread's reads of a stage come before the copy that is issued once the stage has been released: the
// copy writes through another proxy, which the release alone does not order behind reads that are still
// on their way (behind a thread's stores they take long).
__device__ __forceinline__ void reads_done() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// A consumer warp is done with ring position q.
__device__ __forceinline__ void release_stage(Barriers& b, int nbuf, int q) {
    reads_done();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&b.empty[q % nbuf]);
}

template <typename S>
__device__ __forceinline__ uint32_t bits_of(S v);
template <>
__device__ __forceinline__ uint32_t bits_of<uint16_t>(uint16_t v) { return v; }
template <>
__device__ __forceinline__ uint32_t bits_of<float>(float v) { return __float_as_uint(v); }

// A partial vector: its elements in the row one by one, -inf elsewhere.
template <typename S>
__device__ __noinline__ uint4 load_partial(const Row& r, int v) {
    constexpr int G = Elt<S>::kGroup, B = (int)sizeof(S) * 8;
    uint32_t w[4];
    const S* p = reinterpret_cast<const S*>(r.base) + (int64_t)v * G;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i] = 0;
#pragma unroll
        for (int k = 0; k < G / 4; ++k) {
            const int e = i * (G / 4) + k;
            const int64_t col = (int64_t)v * G - r.shift + e;
            const uint32_t x = col >= 0 && col < r.V ? bits_of<S>(p[e]) : (B == 16 ? 0xFF80u : 0xFF800000u);
            w[i] |= x << (B == 16 ? 16 * k : 0);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A vector of the row from global memory, whole or partial.
template <typename S>
__device__ __forceinline__ uint4 load_vector(const Row& r, int v) {
    if (v >= r.iv0 && v < r.iv1) return ld_stream16(r.base + (int64_t)v * 16);
    return load_partial<S>(r, v);
}

// This thread's vectors of stage j, landed in ring position q; -inf beyond the slice.
template <typename S>
__device__ __forceinline__ void load_stage(const uint8_t* bufs, int nbuf, const Row& r, const Slice& s, int j, int q,
                                           int tid, uint4 (&x)[kU]) {
    const uint4* buf = reinterpret_cast<const uint4*>(bufs + (q % nbuf) * kStageBytes);
    const int a = s.v0 + j * kStageVecs;
    if (a >= r.iv0 && a + kStageVecs <= min(s.v0 + s.n, r.iv1)) {
#pragma unroll
        for (int u = 0; u < kU; ++u) x[u] = tc::lds16(buf + tid + u * kConsumers);
    } else {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = tid + u * kConsumers, v = a + i;
            x[u] = stage::neg_inf16<S>();
            if (v < s.v0 + s.n) x[u] = v >= r.iv0 && v < r.iv1 ? tc::lds16(buf + i) : load_partial<S>(r, v);
        }
    }
}

// ---- (reference, sum-exp) pairs: s * 2^m = sum 2^(z k2), k2 = log2(e) / temperature
//
// As vce_device.cuh's pairs, but the reference m is in the exponent's units: whatever fp32 number it is,
// z k2 - m is one fma with one rounding, where a reference among the logits would round its product with
// k2 alike in every term.

__device__ __forceinline__ void pair_merge(float& m, float& s, float m2, float s2) {
    const float M = fmaxf(m, m2);
    const float a = (m == M) ? 1.f : ex2(m - M);
    const float b = (m2 == M) ? 1.f : ex2(m2 - M);
    s = s * a + s2 * b;
    m = M;
}

// The warp's pairs merged, in every lane: to the largest reference first, then one sum.
__device__ __forceinline__ void pair_warp_reduce(float& m, float& s) {
    float M = m;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, off));
    s *= (m == M) ? 1.f : ex2(m - M);
    m = M;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
}

// (d0, d1) = (a0 + b0, a1 + b1), in one packed instruction; each sum rounds as the scalar one.
__device__ __forceinline__ void fadd2(float a0, float a1, float b0, float b1, float& d0, float& d1) {
    asm("{\n\t.reg .b64 pa, pb, pd;\n\t"
        "mov.b64 pa, {%2, %3};\n\tmov.b64 pb, {%4, %5};\n\t"
        "add.rn.f32x2 pd, pa, pb;\n\tmov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// sum of 2^(v k2 - m) over a thread's vectors of a stage: exponents and sums two at a time (even and
// odd values summed apart), since the issue slots are what these kernels run short of
template <int G, int U>
__device__ __forceinline__ float sum_exp(const float (&v)[U][G], float k2, float m) {
    constexpr int N = U * G;
    float e[N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < G; k += 2) {
            float a0, a1;
            ffma2(v[u][k], v[u][k + 1], k2, -m, a0, a1);
            e[u * G + k] = ex2(a0);
            e[u * G + k + 1] = ex2(a1);
        }
#pragma unroll
    for (int w = 2; w < N; w *= 2)
#pragma unroll
        for (int k = 0; k + w < N; k += 2 * w) fadd2(e[k], e[k + 1], e[k + w], e[k + w + 1], e[k], e[k + 1]);
    return e[0] + e[1];
}

// The largest value; NaN if there is one (which fmaxf would pass over).
template <int G, int U>
__device__ __forceinline__ float max_of(const float (&v)[U][G]) {
    float m = v[0][0];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < G; ++k)
            if (u || k) asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(v[u][k]));
    return m;
}

// References of this size and more are large.  Below it the exponent of the reference's own logit, which is what the
// product with k2 was rounded by, is 2^6 at most; against a mask of -1e10 it would be 2^9, which no power of two holds.
constexpr float kLarge = 2147483648.f;               // 2^31
__device__ __forceinline__ bool beyond(float m) { return fabsf(m) >= kLarge; }

// How many products with k2 round to m, the largest of them (+inf: NaN).
template <int G, int U>
__device__ __forceinline__ float count_of(const float (&v)[U][G], float k2, float m) {
    float n = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < G; ++k) n += v[u][k] * k2 == m ? 1.f : 0.f;
    return m < kInf ? n : __int_as_float(0x7FC00000);
}

// Adds a stage's values to a pair whose reference moves only when a term would pass 2^32 (it is then one
// of the values', so s is about 1 or more and nothing overflows).  Values whose product with k2 is -2^31 or less
// (masks) count as -inf.  A NaN, or a product of 2^31 or more, makes s NaN.
template <int G, int U>
__device__ __forceinline__ void pair_push(const float (&v)[U][G], float& m, float& s, float k2) {
    if (m == -kInf) {
        m = max_of<G>(v) * k2;
        if (m <= -kLarge) {
            m = -kInf;
            return;
        }
        if (m >= kLarge) s = __int_as_float(0x7FC00000);
    }
    float t;
#pragma unroll 1
    for (int again = 0;; again = 1) {   // one copy of the sum's code, for the instruction cache
        t = sum_exp<G>(v, k2, m);
        if (again || t < 4294967296.f) break;
        const float vm = fmaxf(m, max_of<G>(v) * k2);   // a value far above the reference: take the new maximum
        if (vm >= kLarge) s = __int_as_float(0x7FC00000);
        s *= ex2(m - vm);
        m = vm;
    }
    s += t;
}

// The largest of a thread's vectors of a stage as they were loaded (bf16: two at a time).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <typename S, int U>
__device__ __forceinline__ float max_of_loaded(const uint4 (&x)[U]) {
    if (sizeof(S) == 2) {
        uint32_t m = x[0].x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u) m = max_bf16x2(m, x[u].x);
            m = max_bf16x2(max_bf16x2(m, x[u].y), max_bf16x2(x[u].z, x[u].w));
        }
        return fmaxf(bf16_lo(m), bf16_hi(m));
    }
    float m = __uint_as_float(x[0].x);
#pragma unroll
    for (int u = 0; u < U; ++u)
        m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(x[u].x)), fmaxf(__uint_as_float(x[u].y), __uint_as_float(x[u].z))),
                  __uint_as_float(x[u].w));
    return m;
}

// ---- programmatic dependent launch: the next kernel of the stream may start; the previous one has ended
__device__ __forceinline__ void start_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- thread-block clusters -------------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
// Without ordering memory: for a barrier that only keeps blocks alive or known to run.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void st_peer_u64(uint32_t addr, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

}  // namespace rs
}  // namespace vce
