// The rows' sums, and for the policy loss their gradients in the same pass: a persistent kernel whose warps
// have roles.  A block (a cluster of C of them per row) walks the rows cid, cid + ncl, ... with the
// copies of the next rows always in flight; what belongs to a row is doubled by the parity of its number in
// the block's sequence and handed on through mbarriers:
//   producer        copies the rows' slices into the stage ring, running ahead as stages are released, and
//                   writes a row's partial first and last vectors there, so the consumers need not know of
//                   them (the elements of the next row's are on their way while this one's copies wait)
//   consumers       a row's sums, the token's column left out; with a gradient then the first stages of the
//                   next row, while this row's statistics are exchanged, this row's gradient from the held
//                   stages, releasing each, and the rest of the next row
//   stats           merges the warps' sums and the cluster's and finishes the row: at once where the
//                   consumers wait for its gradient's coefficients, else 32 rows together, a lane each
// Every role walks the same rows by itself (a lane looks at each of the next 32 rows' tokens), so nothing
// has to be handed on about rows that are left out.  Every wait is bounded; one that gives up sets the
// block's abort flag, every role stops at its next wait, and the rows of the block become NaN.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "logprob_rows.cuh"
#include "policy_finish.cuh"
#include "policy_rows.h"
#include "row_grads.cuh"

namespace vce {
namespace lp {
namespace ring {

using namespace rs;

template <int kWarps_, int kBlocks_, int kU_, int kBufs_, int kHeld_>
struct Form {
    static constexpr int kWarps = kWarps_, kNT = kWarps * 32;                 // consumers
    static constexpr int kBlocks = kBlocks_;                                  // of an SM
    static constexpr int kSpan = kWarps > 16 ? 32 : kWarps > 8 ? 16 : 8;      // lanes that merge the warps' sums
    static constexpr int kProducer = kWarps, kStats = kWarps + 1;
    static constexpr int kThreads = (kWarps + 2) * 32;
    static constexpr int kU = kU_;                                            // vectors of a stage per consumer thread
    static constexpr int kVecs = kU * kNT, kBytes = kVecs * 16;               // of a stage
    static constexpr int kBufs = kBufs_;
    static constexpr int kHeld = kHeld_;                                      // stages of a slice that is held, at most
};

constexpr uint32_t kSuspend = 10000;                // ns a poll may sleep: waiting warps leave the issue slots to others
enum { kErrRow = 107, kErrPartials = 108, kErrCoefs = 109 };

struct RowCoefs {
    Coefs c;
    float bias;
    int none;                    // no gradient (nothing but masks)
};

template <int kWarps, int kBufs>
struct alignas(16) Ctl {
    float4 slot[2][kMaxCluster];
    uint64_t full[kBufs], empty[kBufs];
    uint64_t paired[2];          // the consumer warps' sums
    uint64_t exchanged[2];       // the cluster's
    uint64_t finished[2];        // the sums have been read; with a gradient: its coefficients are there
    Sums red[2][kWarps];
    RowCoefs coefs[2];
    int abort, err;
};

template <typename F>
__host__ __device__ constexpr int smem_bytes() {
    return F::kBufs * F::kBytes + (int)sizeof(Ctl<F::kWarps, F::kBufs>);
}

// make_row without its address, in 32-bit arithmetic: what the consumers need of a row, each warp by itself.
template <typename S>
__device__ __forceinline__ rs::Row row_extent(const Args& a, int64_t row) {
    constexpr int G = Elt<S>::kGroup;
    rs::Row r;
    r.base = nullptr;
    r.V = a.V;
    const uint32_t off =
        ((uint32_t) reinterpret_cast<uintptr_t>(a.logits) + (uint32_t)row * ((uint32_t)a.ld * (uint32_t)sizeof(S))) & 15u;
    r.shift = (int)(off / sizeof(S));
    r.nv = ((int)a.V + r.shift + G - 1) / G;
    r.iv0 = r.shift ? 1 : 0;
    r.iv1 = ((int)a.V + r.shift) / G;
    return r;
}

// The vectors of a row that a block takes, per of them, in stages of the ring.
template <typename F>
__device__ __forceinline__ Slice ring_slice(const rs::Row& r, int per, int part) {
    Slice s;
    s.v0 = min(r.nv, part * per);
    s.n = min(r.nv - s.v0, per);
    s.nst = (s.n + F::kVecs - 1) / F::kVecs;
    return s;
}

// A position of the ring, moved on stage by stage.
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

// The rows cid, cid + ncl, ... whose token is a column (a warp, in step); of the others, skipped(row).  The
// tokens of the next 32 rows are on their way while a batch is in use.
struct Walk {
    int64_t base, step, first, end;
    uint32_t left, next_left;
    int64_t id;                  // of this lane's row of the next batch
    int64_t token;               // of this lane's row of this one
};

__device__ __forceinline__ void walk_load(Walk& w, const Args& a, int64_t row) {
    w.id = row < a.T ? a.ids[row] : -1;
}
__device__ __forceinline__ void walk_start(Walk& w, const Args& a, int64_t cid, int64_t ncl) {
    w.step = ncl;
    w.base = cid - 32 * ncl;
    w.left = 0;
    w.token = 0;
    w.first = a.offsets ? a.offsets[0] : 0;
    w.end = a.offsets ? a.offsets[2 * a.P] : a.T;
    walk_load(w, a, cid + (int64_t)(threadIdx.x & 31) * ncl);
}
// The next row and its token, or -1 behind the last.  skipped(row, code): a row that is left out (code 0) or
// whose token is no column.
template <typename F>
__device__ __forceinline__ int64_t walk_next(Walk& w, const Args& a, int& token, F skipped) {
    const int lane = threadIdx.x & 31;
    while (!w.left) {
        w.base += 32 * w.step;
        if (w.base >= a.T) return -1;
        const int64_t row = w.base + (int64_t)lane * w.step;
        const bool out = w.id == a.ignore_index || row < w.first || row >= w.end;
        w.left = __ballot_sync(0xFFFFFFFFu, row < a.T && !out && w.id >= 0 && w.id < a.V);
        w.token = w.id;
        const uint32_t there = __ballot_sync(0xFFFFFFFFu, row < a.T), bad = __ballot_sync(0xFFFFFFFFu, !out);
        for (uint32_t no = there & ~w.left; no; no &= no - 1) {
            const int b = __ffs(no) - 1;
            skipped(w.base + (int64_t)b * w.step, (bad >> b) & 1u ? VCE_ERR_LABEL : 0);
        }
        walk_load(w, a, w.base + (int64_t)(32 + lane) * w.step);
    }
    const int b = __ffs(w.left) - 1;
    w.left &= w.left - 1;
    token = (int)__shfl_sync(0xFFFFFFFFu, w.token, b);
    return w.base + (int64_t)b * w.step;
}
__device__ __forceinline__ int64_t walk_next(Walk& w, const Args& a, int& token) {
    return walk_next(w, a, token, [](int64_t, int) {});
}

// Four floats into a peer's shared memory, counted as 16 bytes on its barrier: no release that would wait for this
// warp's stores to global memory.
__device__ __forceinline__ void send_peer(uint32_t addr, float4 v, uint32_t bar_addr) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar_addr)
                 : "memory");
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

template <typename S, typename O, bool kGrad, bool kEnt, typename F>
__global__ void __launch_bounds__(F::kThreads, F::kBlocks) k_loss_ring(const __grid_constant__ Args a) {
    constexpr int G = Elt<S>::kGroup;
    // with a gradient the sums are taken against the same scale as its entries, and no mean is needed
    constexpr int kKind = kEnt ? kEntropy : kGrad ? kSum : kMean;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int nbuf = F::kBufs, U = F::kU, B = U < 4 ? U : 4, kVecs = F::kVecs, kWarps = F::kWarps, kNT = F::kNT;
    Ctl<kWarps, nbuf>& ctl = *reinterpret_cast<Ctl<kWarps, nbuf>*>(smem + nbuf * F::kBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = a.cluster;
    const int rank = C > 1 ? (int)cluster_rank() : 0;
    const int64_t cid = blockIdx.x / C, ncl = gridDim.x / C;
    auto wait = [&](uint64_t* bar, int64_t e, int code) {   // the phase of row e of a barrier doubled by parity
        return tc::mbar_wait(bar, (uint32_t)(e >> 1) & 1, &ctl.abort, &ctl.err, code, a.wait_ns, kSuspend);
    };

    start_next();
    if (tid == 0) {
        for (int i = 0; i < nbuf; ++i) {
            tc::mbar_init(&ctl.full[i], 1);
            tc::mbar_init(&ctl.empty[i], kWarps);
        }
        for (int p = 0; p < 2; ++p) {
            tc::mbar_init(&ctl.paired[p], kWarps);
            tc::mbar_init(&ctl.exchanged[p], 1);
            tc::mbar_init(&ctl.finished[p], 1);
        }
        ctl.abort = ctl.err = 0;
        tc::fence_mbar_init();
    }
    if (C > 1) cluster_arrive(), cluster_wait();
    else __syncthreads();

    Walk walk;
    walk_start(walk, a, cid, ncl);
    int token = 0;

    if (warp == F::kProducer) {
        Cursor<nbuf> at{0, 1};                         // waits for "released" start a phase back
        int q = 0;
        const S neg = sizeof(S) == 2 ? (S)0xFF80u : (S)-kInf;
        // lanes 0 .. G - 1: the slice's first vector, if it is partial; G .. 2 G - 1: the row's last
        struct Edge {
            uint32_t place;
            S value;
        };
        auto load_edge = [&](int64_t row) {
            Edge e{0xFFFFFFFFu, neg};
            if (row < 0) return e;
            const rs::Row r = row_extent<S>(a, row);
            const Slice sl = ring_slice<F>(r, a.per, rank);
            const int edge = lane < G ? (r.shift ? 0 : -1) : (r.iv1 < r.nv && (r.nv > 1 || !r.shift) ? r.nv - 1 : -1);
            if (lane < 2 * G && edge >= sl.v0 && edge < sl.v0 + sl.n) {
                const int64_t col = (int64_t)edge * G - r.shift + lane % G;
                e.place = (uint32_t)((edge - sl.v0) * G + lane % G);
                if (col >= 0 && col < a.V) e.value = static_cast<const S*>(a.logits)[row * a.ld + col];
            }
            return e;
        };
        int64_t row = walk_next(walk, a, token);
        Edge edge = load_edge(row);
        while (row >= 0 && !*reinterpret_cast<volatile int*>(&ctl.abort)) {
            const rs::Row r = make_row<S>(a.logits, row, a.ld, a.V);
            const Slice sl = ring_slice<F>(r, a.per, rank);
            const int64_t next = walk_next(walk, a, token);
            const Edge later = load_edge(next);
            const bool edges = __any_sync(0xFFFFFFFFu, edge.place != 0xFFFFFFFFu);
            for (int j = 0; j < sl.nst; ++j, ++q, at.step()) {
                const int st = at.st;
                bool ok = true;
                if (lane == 0) ok = tc::mbar_wait(&ctl.empty[st], at.phase, &ctl.abort, &ctl.err, kErrEmpty, a.wait_ns);
                if (!__shfl_sync(0xFFFFFFFFu, (int)ok, 0)) break;
                if (edges) {
                    const uint32_t p = edge.place - (uint32_t)(j * kVecs * G);
                    if (p < (uint32_t)(kVecs * G)) {
                        reinterpret_cast<S*>(smem + st * F::kBytes)[p] = edge.value;
                        reads_done();                  // before the next copy into the stage, of another proxy
                    }
                    __syncwarp();
                }
                if (lane == 0) {
                    const int v = sl.v0 + j * kVecs;
                    const int lo = max(v, r.iv0), hi = min(min(v + kVecs, sl.v0 + sl.n), r.iv1);
                    if (hi > lo && dbg::ok(lo >= 0 && hi <= r.nv, dbg::kCols)) {
                        tc::mbar_arrive_expect_tx(&ctl.full[st], (uint32_t)(hi - lo) * 16);
                        tc::bulk_load(smem + st * F::kBytes + (lo - v) * 16, r.base + (int64_t)lo * 16,
                                      (uint32_t)(hi - lo) * 16, &ctl.full[st]);
                    } else {
                        tc::mbar_arrive(&ctl.full[st]);
                    }
                }
            }
            __syncwarp();
            row = next;
            edge = later;
        }
        // after an abort, copies in flight land before the block may leave
        if (lane == 0 && *reinterpret_cast<volatile int*>(&ctl.abort)) {
            int never = 0;
            for (int p = max(0, q - nbuf); p < q; ++p)
                tc::mbar_wait(&ctl.full[p % nbuf], (p / nbuf) & 1, &never, nullptr, 0, a.wait_ns);
        }
        __syncwarp();
    } else if (warp == F::kStats) {
        float inv_n = 1.f;
        if (kGrad && a.red == VCE_RED_MEAN) {
            wait_previous();                           // the count of the rows
            inv_n = *a.inv_n;
        }
        // without a gradient nobody waits for a row's results: each lane keeps a row, 32 are worked out at once
        Sums kept{-kInf, 0.f, 0.f};
        int64_t kept_row = 0;
        int kept_token = 0, pending = 0;
        auto flush = [&]() {
            if (!kGrad && lane < pending && rank == 0) {
                const RowIn in = row_in<S>(a, kept_row, kept_token);
                const Row r = finish<kKind>(kept, in.zt, Scale{a.k2, a.k2_lo});
                float loss = 0.f;
                const float4 st = row_result(a, r, in, 1.f, loss);
                write_result(a, kept_row, r, st, loss);
            }
            pending = 0;
        };
        for (int64_t e = 0;; ++e) {
            const int par = (int)(e & 1);
            const int64_t row = walk_next(walk, a, token, [&](int64_t no, int code) {
                if (rank == 0 && lane == 0) write_none(a, no, code);
            });
            if (row < 0) break;
            RowIn in{};
            float go = 0.f;
            if (kGrad) {                               // on their way while the row streams
                in = row_in<S>(a, row, token);
                go = a.go[a.red == VCE_RED_NONE ? row : 0] * inv_n;
            }
            if (!wait(&ctl.paired[par], e, kErrPartials)) break;
            Sums x = lane < kWarps ? ctl.red[par][lane] : Sums{-kInf, 0.f, 0.f};
            warp_merge<kKind, kGrad ? F::kSpan : 32>(x);  // (with a gradient lane 0 alone goes on with it)
            if (!kGrad) {                              // (every lane has read its warp's sums)
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&ctl.finished[par]);
            }
            if (C > 1) {
                if (lane == 0) tc::mbar_arrive_expect_tx(&ctl.exchanged[par], 16 * C);
                if (lane < C)                          // C <= kSpan: these lanes have the sums
                    send_peer(peer_addr(&ctl.slot[par][rank], lane), make_float4(x.m, x.s, x.w, 0.f),
                              peer_addr(&ctl.exchanged[par], lane));
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
                x = Sums{-kInf, 0.f, 0.f};
                if (lane < C) {
                    const float4 o = ctl.slot[par][lane];
                    x = Sums{o.x, o.y, o.z};
                }
                warp_merge<kKind, kGrad ? kMaxCluster : 32>(x);   // the same order in every block
            }
            if (kGrad) {
                const Row r = finish<kKind>(x, in.zt, Scale{a.k2, a.k2_lo});
                float loss = 0.f;
                const float4 st = row_result(a, r, in, go, loss);
                if (lane == 0) {
                    ctl.coefs[par] = RowCoefs{Coefs{st.y, st.z, st.w}, r.m, r.dead};
                    if (a.withhold != rank + 1) tc::mbar_arrive(&ctl.finished[par]);
                    if (rank == 0) write_result(a, row, r, st, loss);
                }
                __syncwarp();
            } else {
                if (lane == pending) {
                    kept = x;
                    kept_row = row;
                    kept_token = token;
                }
                if (++pending == 32) flush();
            }
        }
        flush();
    } else {
        // ---------------- consumers ----------------
        auto release = [&](int st) {
            reads_done();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&ctl.empty[st]);
        };
        // stages [j0, j1) of a row, at ring positions from `at` on; tv: the token's vector of the slice, tk: its
        // place there
        auto forward = [&](Cursor<nbuf>& at, int j0, int j1, const Slice& sl, int tv, int tk, Sums& x) {
            for (int j = j0; j < j1; ++j, at.step()) {
                tc::mbar_wait(&ctl.full[at.st], at.phase, &ctl.abort, &ctl.err, kErrFull, a.wait_ns, kSuspend);
                const uint4* buf = reinterpret_cast<const uint4*>(smem + at.st * F::kBytes) + tid;
                const int all = sl.n - j * kVecs, left = all - tid;     // vectors from the stage's, this thread's first on
                const int rel = tv - j * kVecs - tid;
                const bool token = rel >= 0 && rel < kVecs && rel % kNT == 0;
#pragma unroll 1
                for (int h = 0; h < U; h += B) {
                    if (h * kNT >= all) break;
                    uint4 raw[B];
                    if (left > (h + B - 1) * kNT) {
#pragma unroll
                        for (int u = 0; u < B; ++u) raw[u] = tc::lds16(buf + (h + u) * kNT);
                    } else {
#pragma unroll
                        for (int u = 0; u < B; ++u)
                            raw[u] = left > (h + u) * kNT ? tc::lds16(buf + (h + u) * kNT) : stage::neg_inf16<S>();
                    }
                    if (!kGrad && (h + B >= U || (h + B) * kNT >= all)) release(at.st);
                    float v[B][G];
#pragma unroll
                    for (int u = 0; u < B; ++u) Elt<S>::unpack(raw[u], v[u]);
                    if (token) {                                   // the token's column is left out
#pragma unroll
                        for (int u = 0; u < B; ++u)
#pragma unroll
                            for (int k = 0; k < G; ++k)
                                if (rel == (h + u) * kNT && k == tk) v[u][k] = -kInf;
                    }
                    push<G, B, kKind>(v, x, a.k2);
                }
            }
        };
        auto publish = [&](int64_t e, Sums x) {
            const int par = (int)(e & 1);
            warp_merge<kKind>(x);
            // row e - 2's sums have been read (with a gradient that follows from its coefficients)
            if (!kGrad && e >= 2) wait(&ctl.finished[par], e - 2, kErrCoefs);
            if (lane == 0) {
                ctl.red[par][warp] = x;
                tc::mbar_arrive(&ctl.paired[par]);
            }
            __syncwarp();
        };
        Cursor<nbuf> at{0, 0}, back{0, 0};             // the next stage to sum, and to turn into gradients
        auto next = [&](int& tok) {
            return walk_next(walk, a, tok, [&](int64_t no, int) {
                if (!kGrad) return;
                const rs::Row r = row_extent<S>(a, no);
                O* g = static_cast<O*>(a.grad) + no * a.ld_g;
                fill_grads<S, O>(r, ring_slice<F>(r, a.per, rank), g, grads_aligned<S, O>(r, g), tid, kNT);
            });
        };
        int tok = 0, tok2 = 0;
        int64_t row = -1, row2 = next(tok2);               // the row held, and the next one
        rs::Row r{};
        Slice sl{};
        sl.nst = 0;
        for (int64_t e = -1; (row >= 0 || row2 >= 0) && !*reinterpret_cast<volatile int*>(&ctl.abort); ++e) {
            rs::Row r2{};
            Slice sl2{};
            Sums x{-kInf, 0.f, 0.f};
            int pre = 0, tv = -1, tk = 0;
            if (row2 >= 0) {
                r2 = row_extent<S>(a, row2);
                sl2 = ring_slice<F>(r2, a.per, rank);
                const int p = tok2 + r2.shift;
                tv = p / G - sl2.v0;
                tk = p % G;
                // the next row's stages that fit beside this one's (forward alone: all of them)
                pre = kGrad ? min(sl2.nst, nbuf - sl.nst) : sl2.nst;
            }
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {         // the next row's first stages, this row, the rest
                if (row2 >= 0) forward(at, half ? pre : 0, half ? sl2.nst : pre, sl2, tv, tk, x);
                // the sums are handed on as soon as they are there: the statistics are exchanged and finished
                // under this row's gradient where the next row fits beside it
                if (row2 >= 0 && half == (pre < sl2.nst)) publish(e + 1, x);
                if (!kGrad || half || row < 0) continue;
                const int par = (int)(e & 1);
                if (!wait(&ctl.finished[par], e, kErrCoefs)) continue;
                const RowCoefs cf = ctl.coefs[par];
                O* grow = static_cast<O*>(a.grad) + row * a.ld_g;
                const bool vec = grads_aligned<S, O>(r, grow) && !beyond(cf.bias);
                const int fast0 = vec ? r.iv0 : r.nv, fast1 = min(r.iv1, sl.v0 + sl.n);
                for (int j = 0; j < sl.nst; ++j, back.step()) {
                    const uint4* buf = reinterpret_cast<const uint4*>(smem + back.st * F::kBytes) + tid;
                    const int first = sl.v0 + j * kVecs;
                    if (cf.none) {
                        fill_grads<S, O>(r, Slice{first, min(sl.n - j * kVecs, kVecs), 1}, grow, vec, tid, kNT);
                    } else {
#pragma unroll 1
                        for (int h = 0; h < U; h += B) {
                            const int v0 = first + h * kNT, v1 = sl.v0 + sl.n;
                            if (v0 >= v1) break;
                            uint4 raw[B];
#pragma unroll
                            for (int u = 0; u < B; ++u) raw[u] = tc::lds16(buf + (h + u) * kNT);
                            const bool fast = v0 >= fast0 && v0 + B * kNT <= fast1;
                            if (kEnt && cf.c.c1 != 0.f)
                                write_grads<S, O, B, kNT, true>(raw, r, v0 + tid, v1, fast, grow, vec, cf.c, cf.bias, a.k2);
                            else
                                write_grads<S, O, B, kNT, false>(raw, r, v0 + tid, v1, fast, grow, vec, cf.c, cf.bias, a.k2);
                        }
                        // the token's entry, over what its thread has just written there
                        const int rel = (tok + r.shift) / G - first - tid;
                        if (rel >= 0 && rel < kVecs && rel % kNT == 0 && first + tid + rel < sl.v0 + sl.n)
                            Elt<O>::store1(grow + tok, cf.c.gt);
                    }
                    release(back.st);
                }
            }
            row = row2;
            r = r2;
            sl = sl2;
            tok = tok2;
            if (row2 >= 0) row2 = next(tok2);
        }
    }
    // after an abort: no row of this block is known to be right, nor of its cluster, whose first block has
    // written its results by then
    __syncthreads();
    if (C > 1) {                                       // and no block leaves while a peer may write into it
        cluster_arrive(), cluster_wait();
        if (ctl.abort) {                               // nobody waited for what a peer has sent since: time to land
            const uint64_t t0 = tc::globaltimer();
            while (tc::globaltimer() - t0 < 1000000ull) {
            }
        }
    }
    if (ctl.abort) {
        for (int64_t row = cid + (int64_t)tid * ncl; row < a.T; row += (int64_t)F::kThreads * ncl)
            write_none(a, row, ctl.err ? ctl.err : kErrRow);
        if (kGrad)                                     // nor is any of its columns' gradients
            for (int64_t row = cid; row < a.T; row += ncl) {
                const rs::Row r = row_extent<S>(a, row);
                O* g = static_cast<O*>(a.grad) + row * a.ld_g;
                fill_grads<S, O>(r, ring_slice<F>(r, a.per, rank), g, grads_aligned<S, O>(r, g), tid, F::kThreads, nan_f());
            }
    }
}

}  // namespace ring
}  // namespace lp
}  // namespace vce
