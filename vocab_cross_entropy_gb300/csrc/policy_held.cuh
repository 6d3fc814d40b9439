// Rows held in registers: a block (a cluster of C of them, or a warp of a block for the shortest rows) loads
// all of a row at once, U vectors a thread, sums it, finishes it, and turns the registers into the gradient.
// No stage is staged, nothing is read again, and several blocks share an SM, so that one's loads run under
// another's exchange and stores.
//
// Of a row's vectors thread t of NT takes t, t + NT, ... of its block's slice.  The cluster's blocks exchange
// their sums through distributed shared memory, ordered by the cluster's hardware barrier.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "logprob_rows.cuh"
#include "policy_finish.cuh"
#include "policy_rows.h"
#include "row_grads.cuh"

namespace vce {
namespace lp {
namespace held {

using namespace rs;

template <int kNT_, int kU_, int kBlocks_>
struct Form {
    static constexpr int kNT = kNT_, kU = kU_, kBlocks = kBlocks_;
    static constexpr int kPer = kNT == 32 ? 4 : 1;                // rows of a block
    static constexpr int kThreads = kNT * kPer;
    static constexpr int kVecs = kNT * kU;                        // of a slice, at most
};

struct RowCoefs {
    Coefs c;
    float bias;
    int none;
};

template <typename S, typename O, bool kGrad, bool kEnt, typename F>
__global__ void __launch_bounds__(F::kThreads, F::kBlocks) k_loss_held(const __grid_constant__ Args a) {
    constexpr int G = Elt<S>::kGroup, NT = F::kNT, U = F::kU, kWarps = NT / 32;
    static_assert(U % 2 == 0, "vectors go in pairs");
    constexpr int kKind = kEnt ? kEntropy : kGrad ? kSum : kMean;    // as the ring's
    __shared__ Sums part[kWarps > 1 ? kWarps : 1];
    __shared__ float4 slot[kMaxCluster];
    __shared__ RowCoefs coefs_of_row;
    __shared__ int64_t token_of_row;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tid = threadIdx.x % NT;
    const int C = a.cluster;
    const int rank = kWarps > 1 && C > 1 ? (int)cluster_rank() : 0;
    const int64_t row = F::kPer > 1 ? (int64_t)blockIdx.x * F::kPer + warp : blockIdx.x / C;
    start_next();
    if (F::kPer > 1 && row >= a.T) return;

    // one thread's look at the row's token decides for all (it might be written meanwhile, by a caller's mistake)
    int64_t t;
    if (kWarps > 1) {
        if (threadIdx.x == 0) {
            t = a.ids[row];
            if (a.offsets && (row < a.offsets[0] || row >= a.offsets[2 * a.P])) t = a.ignore_index;
            token_of_row = t;
        }
        __syncthreads();
        t = token_of_row;
    } else {
        if (lane == 0) {
            t = a.ids[row];
            if (a.offsets && (row < a.offsets[0] || row >= a.offsets[2 * a.P])) t = a.ignore_index;
        }
        t = __shfl_sync(0xFFFFFFFFu, t, 0);
    }
    const rs::Row r = make_row<S>(a.logits, row, a.ld, a.V);
    const Slice sl = make_slice(r, C, rank);
    O* grow = kGrad ? static_cast<O*>(a.grad) + row * a.ld_g : nullptr;
    const bool vec = kGrad && grads_aligned<S, O>(r, grow);
    if (kWarps > 1 && C > 1) cluster_arrive_relaxed();               // this block runs: peers may write into it

    if (t == a.ignore_index || t < 0 || t >= a.V) {
        if (rank == 0 && tid == 0) write_none(a, row, t == a.ignore_index ? 0 : VCE_ERR_LABEL);
        if (kGrad) fill_grads<S, O>(r, sl, grow, vec, tid, NT);
        if (kGrad && a.red == VCE_RED_MEAN) wait_previous();
        if (kWarps > 1 && C > 1) cluster_wait(), cluster_arrive(), cluster_wait();   // as many as below
        return;
    }

    // all of the slice is on its way before any of it is used
    const bool inside = sl.v0 >= r.iv0 && sl.v0 + sl.n <= r.iv1;     // no partial vector
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = sl.v0 + tid + u * NT;
        x[u] = stage::neg_inf16<S>();
        if (v < sl.v0 + sl.n && (inside || (v >= r.iv0 && v < r.iv1))) x[u] = ld_stream16(r.base + (int64_t)v * 16);
    }
    RowIn in{};
    float go = 0.f;
    if (warp == 0 || F::kPer > 1) {
        in = row_in<S>(a, row, (int)t);
        if (kGrad) go = a.go[a.red == VCE_RED_NONE ? row : 0];
    }
    if (!inside) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int v = sl.v0 + tid + u * NT;
            if (v < sl.v0 + sl.n && (v < r.iv0 || v >= r.iv1)) x[u] = load_partial<S>(r, v);
        }
    }

    // the sums, the token's column left out
    const int at = (int)t + r.shift, tv = at / G - sl.v0 - tid, tk = at % G;
    const int tu = tv >= 0 && tv < F::kVecs && tv % NT == 0 ? tv / NT : -1;
    Sums sum{-kInf, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < U; u += 2) {
        float v[2][G];
        Elt<S>::unpack(x[u], v[0]);
        Elt<S>::unpack(x[u + 1], v[1]);
        if (tu == u || tu == u + 1) {
#pragma unroll
            for (int k = 0; k < G; ++k) {
                if (k == tk && tu == u) v[0][k] = -kInf;
                if (k == tk && tu == u + 1) v[1][k] = -kInf;
            }
        }
        push<G, 2, kKind>(v, sum, a.k2);
    }
    warp_merge<kKind>(sum);
    if (kWarps > 1) {
        if (lane == 0) part[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            sum = lane < kWarps ? part[lane] : Sums{-kInf, 0.f, 0.f};
            warp_merge<kKind>(sum);
        }
        if (C > 1) {
            cluster_wait();                                          // every peer runs
            if (warp == 0 && lane < C) st_peer(peer_addr(&slot[rank], lane), make_float4(sum.m, sum.s, sum.w, 0.f));
            cluster_arrive();
            cluster_wait();
            if (warp == 0) {
                sum = Sums{-kInf, 0.f, 0.f};
                if (lane < C) {
                    const float4 o = slot[lane];
                    sum = Sums{o.x, o.y, o.z};
                }
                warp_merge<kKind>(sum);                               // the same order in every block
            }
        }
    }

    // the row's scalars: one warp works them out
    RowCoefs cf{};
    if (warp == 0 || F::kPer > 1) {
        if (kGrad && a.red == VCE_RED_MEAN) {
            wait_previous();                                         // the count of the rows
            go *= *a.inv_n;
        }
        const lp::Row res = finish<kKind>(sum, in.zt, Scale{a.k2, a.k2_lo});
        float loss = 0.f;
        const float4 st = row_result(a, res, in, kGrad ? go : 1.f, loss);
        cf = RowCoefs{Coefs{st.y, st.z, st.w}, res.m, res.dead};
        if (kGrad && kWarps > 1 && lane == 0) coefs_of_row = cf;
        if (rank == 0 && lane == 0) write_result(a, row, res, st, loss);
    } else if (kGrad && a.red == VCE_RED_MEAN) {
        wait_previous();
    }
    if (!kGrad) return;
    if (kWarps > 1) {
        __syncthreads();
        cf = coefs_of_row;
    }
    // the vectors are unpacked anew: kept unpacked since the sums, they would take twice the registers
#pragma unroll
    for (int u = 0; u < U; ++u) asm volatile("" : "+r"(x[u].x), "+r"(x[u].y), "+r"(x[u].z), "+r"(x[u].w));
    if (cf.none) {
        fill_grads<S, O>(r, sl, grow, vec, tid, NT);
        return;
    }
    const int v0 = sl.v0, v1 = sl.v0 + sl.n;
    const bool fast = vec && v0 >= r.iv0 && v0 + F::kVecs <= min(r.iv1, v1);
    if (kEnt && cf.c.c1 != 0.f)
        write_grads<S, O, U, NT, true>(x, r, v0 + tid, v1, fast, grow, vec, cf.c, cf.bias, a.k2);
    else
        write_grads<S, O, U, NT, false>(x, r, v0 + tid, v1, fast, grow, vec, cf.c, cf.bias, a.k2);
    if (tu >= 0 && sl.v0 + tid + tu * NT < v1) Elt<O>::store1(grow + t, cf.c.gt);   // over what this thread wrote there
}

}  // namespace held
}  // namespace lp
}  // namespace vce
