// Short rows held in registers: a block (or a warp of a block for the shortest) loads all of a row at once, U
// vectors a thread, sums it, finishes it, and turns the registers into the gradient.  There is nothing to
// stage or to hand on, and many blocks share an SM, so that one's loads run under the others' scalars and
// stores.  Of a row's vectors thread t of NT takes t, t + NT, ...
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
    static constexpr int kVecs = kNT * kU;                        // of a row, at most
};

struct RowCoefs {
    Coefs c;
    float bias;
    int none;
};

// A warp for rows of at most 4 KB, then blocks of 64, 128 and 256 threads for 8, 16 and 32 KB.
using Warp = Form<32, 8, 4>;
using Block8 = Form<64, 8, 16>;
using Block16 = Form<128, 8, 8>;
using Block32 = Form<256, 8, 4>;

template <typename S, typename O, bool kGrad, bool kEnt, typename F>
__global__ void __launch_bounds__(F::kThreads, F::kBlocks) k_loss_held(const __grid_constant__ Args a) {
    constexpr int G = Elt<S>::kGroup, NT = F::kNT, U = F::kU, kWarps = NT / 32;
    static_assert(U % 2 == 0, "vectors go in pairs");
    constexpr int kKind = kEnt ? kEntropy : kGrad ? kSum : kMean;    // as the ring's
    // a call where the registers allow it (8192 x 8000 bf16 one pass 50.0 us, 51.0 inlined; 4096 x 2000 fp32 with
    // an entropy term 17.8, 16.6 inlined)
    constexpr bool kCall = !(G == 4 && kGrad && kEnt);
    __shared__ Sums part[kWarps > 1 ? kWarps : 1];
    __shared__ RowCoefs coefs_of_row;
    __shared__ int64_t token_of_row;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tid = threadIdx.x % NT;
    const int64_t row = F::kPer > 1 ? (int64_t)blockIdx.x * F::kPer + warp : blockIdx.x;
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
    const Slice sl{0, r.nv, 1};
    O* grow = kGrad ? static_cast<O*>(a.grad) + row * a.ld_g : nullptr;
    const bool vec = kGrad && grads_aligned<S, O>(r, grow);

    if (t == a.ignore_index || t < 0 || t >= a.V) {
        if (tid == 0) write_none(a, row, t == a.ignore_index ? 0 : VCE_ERR_LABEL);
        if (kGrad) fill_grads<S, O>(r, sl, grow, vec, tid, NT);
        if (kGrad && a.red == VCE_RED_MEAN) wait_previous();
        return;
    }

    // all of the row is on its way before any of it is used
    const bool inside = r.iv0 == 0 && r.iv1 == r.nv;                 // no partial vector
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int v = tid + u * NT;
        x[u] = stage::neg_inf16<S>();
        if (v < r.nv && (inside || (v >= r.iv0 && v < r.iv1))) x[u] = ld_stream16(r.base + (int64_t)v * 16);
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
            const int v = tid + u * NT;
            if (v < r.nv && (v < r.iv0 || v >= r.iv1)) x[u] = load_partial<S>(r, v);
        }
    }

    // the sums, the token's column left out
    const int at = (int)t + r.shift, tv = at / G - tid, tk = at % G;
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
        push<G, 2, kKind, kCall>(v, sum, a.k2);
    }
    warp_merge<kKind>(sum);
    if (kWarps > 1) {
        if (lane == 0) part[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            sum = lane < kWarps ? part[lane] : Sums{-kInf, 0.f, 0.f};
            warp_merge<kKind>(sum);
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
        if (lane == 0) write_result(a, row, res, st, loss);
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
    const bool whole = vec && !beyond(cf.bias);
    const bool fast = whole && inside && F::kVecs <= r.nv;
    if (kEnt && cf.c.c1 != 0.f)
        write_grads<S, O, U, NT, true>(x, r, tid, r.nv, fast, grow, whole, cf.c, cf.bias, a.k2);
    else
        write_grads<S, O, U, NT, false>(x, r, tid, r.nv, fast, grow, whole, cf.c, cf.bias, a.k2);
    if (tu >= 0 && tid + tu * NT < r.nv) Elt<O>::store1(grow + t, cf.c.gt);   // over what this thread wrote there
}

// early: the kernel may start before the one ahead of it has ended (the count of a mean's rows).
template <typename S, typename O, bool kGrad, bool kEnt, typename F>
cudaError_t launch(Args& a, cudaStream_t s, bool early) {
    const int64_t blocks = (a.T + F::kPer - 1) / F::kPer;
    return launch_clusters<k_loss_held<S, O, kGrad, kEnt, F>>(blocks, 1, F::kThreads, 0, s, a, early);
}

// By the smallest form that holds a row of nv vectors (the largest is for one pass alone).
template <typename S, typename O, bool kGrad, bool kEnt>
cudaError_t run(Args& a, int64_t nv, cudaStream_t s, bool early = false) {
    if (nv <= Warp::kVecs) return launch<S, O, kGrad, kEnt, Warp>(a, s, early);
    if (nv <= Block8::kVecs) return launch<S, O, kGrad, kEnt, Block8>(a, s, early);
    if constexpr (kGrad) {
        if (nv > Block16::kVecs) return launch<S, O, kGrad, kEnt, Block32>(a, s, early);
    }
    return launch<S, O, kGrad, kEnt, Block16>(a, s, early);
}

}  // namespace held
}  // namespace lp
}  // namespace vce
