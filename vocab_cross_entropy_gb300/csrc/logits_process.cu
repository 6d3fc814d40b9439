// logits_process: repeated-token penalties, biases, temperature and masks on [T, V] logits, and
// the gradient through them.
//
// One read and one write of a row; masked vectors are written without being read.  What makes it
// more than a scaling is the row's history: a list of up to many thousands of tokens with repeats,
// of which the penalties need every column's count.  A row is taken by a thread-block cluster; each
// block owns a slice of the columns with a 32-bit word for each in shared memory (bits 0..29 the
// count behind the prompt, bit 30 a column with a bias, bit 31 seen in the prompt).  The blocks
// share the history out among their threads and add each token to its owner's word through
// distributed shared memory, so the list is read once whatever the number of blocks; after a cluster
// barrier each block streams its slice with its words beside it.  Integer adds: the order does not
// matter.  Columns with a bias are left out of the stream and handled entry by entry, so the
// logits may be processed in place.  Rows without lists skip all of this.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "row_launch.h"
#include "row_stream.cuh"
#include "vce_logits.h"

namespace vce {
namespace process {

using rs::Row;

constexpr int kThreads = 512;
constexpr int kUnroll = 4;                    // 16-byte vectors in flight per thread
constexpr int kMaxCluster = 8;
constexpr int kMaxSlice = 16384;              // columns of a block's slice: 64 KB of words
constexpr uint32_t kPrompt = 0x80000000u, kBias = 0x40000000u, kCount = 0x3FFFFFFFu;

struct Args {
    const void* in;                           // the logits; backward: the upstream gradient
    int64_t T, V, ld;
    const void* z;                            // backward: the logits (read at the history's columns)
    int64_t ld_z;
    int z_bf16;
    const float *temperature, *repetition, *frequency, *presence;
    const int64_t* hist;
    int64_t n_hist;
    const int64_t *hist_off, *prompt;
    const int64_t* bias_ids;
    const float* bias;
    int64_t n_bias;
    const int64_t* bias_off;
    const uint32_t* mask;
    int64_t mask_ld;
    void* out;
    int64_t ld_out;
    int32_t* row_status;
    int cluster, windows, slice;              // vectors of a block's slice in one window
};

struct alignas(16) Ctl {
    int code;                                 // rank 0: the row's first error
    int pad[3];
};

// A row's factors.
struct Rule {
    float inv_t, r, f, p;
};

__device__ __forceinline__ void red_add_peer(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void red_or_peer(uint32_t addr, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void red_max_peer(uint32_t addr, int v) {
    asm volatile("red.relaxed.cluster.shared::cluster.max.s32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// One processed logit; w: its column's word.
__device__ __forceinline__ float process_one(float z, uint32_t w, const Rule& u, float bias) {
    float y = z;
    const uint32_t n = w & kCount;
    if (n || (w & kPrompt)) y = z > 0.f ? z / u.r : z * u.r;
    if (n) y = (y - u.f * (float)n) - u.p;
    return (y + bias) * u.inv_t;
}

// Loads of the row: plain ones, since it may be processed in place (a location is read once, by the
// thread that then writes it).
__device__ __forceinline__ uint4 load16(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ float load_one(const float* p) { return *reinterpret_cast<const volatile float*>(p); }
__device__ __forceinline__ float load_one(const uint16_t* p) {
    return __uint_as_float((uint32_t)*reinterpret_cast<const volatile uint16_t*>(p) << 16);
}

// Whether each of the G columns from c0 (a whole vector of the row) is allowed, bit k for c0 + k.
template <int G>
__device__ __forceinline__ uint32_t allowed_bits(const uint32_t* mrow, int64_t c0) {
    const uint32_t sh = (uint32_t)c0 & 31u;
    const uint32_t* m = mrow + (c0 >> 5);
    uint32_t b = m[0] >> sh;
    if (sh + G > 32) b |= m[1] << (32 - sh);
    return b & ((1u << G) - 1u);
}

template <typename S, typename O, bool kBack, bool kLists>
__global__ void __launch_bounds__(kThreads) k_process(const __grid_constant__ Args a) {
    constexpr int G = Elt<S>::kGroup;
    extern __shared__ __align__(16) uint8_t smem[];
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + sizeof(Ctl));   // [slice * G]
    const int tid = threadIdx.x, C = a.cluster;
    const int rank = kLists ? (C > 1 ? (int)rs::cluster_rank() : 0) : (int)(blockIdx.x % C);
    const int64_t row = blockIdx.x / C;
    const Row r = rs::make_row<S>(a.in, row, a.ld, a.V);
    const S* irow = static_cast<const S*>(a.in) + row * a.ld;
    O* orow = static_cast<O*>(a.out) + row * a.ld_out;
    const uint32_t* mrow = a.mask ? a.mask + row * a.mask_ld : nullptr;
    const bool vec = (reinterpret_cast<uintptr_t>(orow - r.shift) % (GroupStore<O, G>::kAlign)) == 0;
    const float kMasked = kBack ? 0.f : -kInf;

    int code = 0;
    Rule u{1.f, 1.f, 0.f, 0.f};
    const float nan = __int_as_float(0x7FC00000);
    if (a.temperature) {
        const float t = a.temperature[row];
        const bool good = t > 0.f && t < kInf && 1.f / t < kInf;
        u.inv_t = good ? 1.f / t : nan;
        if (!good) code = VCE_ERR_PARAM;
    }
    int64_t h0 = 0, h1 = 0, prompt_end = 0, b0 = 0, b1 = 0;
    if (kLists) {
        if (a.hist) {
            if (a.repetition) {
                u.r = a.repetition[row];
                if (!(u.r > 0.f && u.r < kInf)) {
                    u.r = nan;
                    code = VCE_ERR_PARAM;
                }
            }
            if (!kBack && a.frequency) u.f = a.frequency[row];
            if (!kBack && a.presence) u.p = a.presence[row];
            h0 = a.hist_off[row];
            h1 = a.hist_off[row + 1];
            if (h0 < 0 || h1 < h0 || h1 > a.n_hist) {
                h0 = h1 = 0;
                code = VCE_ERR_OFFSETS;
            }
            const int64_t np = a.prompt ? a.prompt[row] : 0;
            prompt_end = h0 + (np < 0 ? 0 : np > h1 - h0 ? h1 - h0 : np);
        }
        if (!kBack && a.bias_ids) {
            b0 = a.bias_off[row];
            b1 = a.bias_off[row + 1];
            if (b0 < 0 || b1 < b0 || b1 > a.n_bias) {
                b0 = b1 = 0;
                code = VCE_ERR_OFFSETS;
            }
        }
    }
    const bool lists = kLists && (h1 > h0 || b1 > b0);   // the same in every block of the row
    if (kLists && tid == 0) ctl.code = 0;

    for (int win = 0; win < a.windows; ++win) {
        // this block's vectors [v0, v1) of the row in this window
        const int first = win * C * a.slice;
        const int v0 = min(r.nv, first + rank * a.slice), v1 = min(r.nv, v0 + a.slice);
        if (lists) {
            uint4* w4 = reinterpret_cast<uint4*>(words);
            for (int i = tid; i < (v1 - v0) * G / 4; i += kThreads) w4[i] = make_uint4(0, 0, 0, 0);
            if (C > 1) rs::cluster_arrive(), rs::cluster_wait();
            else __syncthreads();
            // the history, shared out over the cluster's threads: four tokens in flight each
            const int64_t step = (int64_t)C * kThreads;
            int bad = 0;
            for (int64_t i0 = h0 + (int64_t)rank * kThreads + tid; i0 < h1; i0 += 4 * step) {
                int64_t id[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) id[q] = i0 + q * step < h1 ? a.hist[i0 + q * step] : 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t i = i0 + q * step;
                    if (i >= h1) break;
                    if (id[q] < 0 || id[q] >= a.V) {
                        bad = VCE_ERR_LABEL;
                        continue;
                    }
                    const int64_t at = id[q] + r.shift;              // element of the row's vectors
                    const int v = (int)(at / G) - first;             // vector of the window
                    if (v < 0 || v >= C * a.slice) continue;
                    const int owner = v / a.slice;
                    uint32_t* w = words + (int64_t)(v - owner * a.slice) * G + at % G;
                    if (C > 1) {
                        const uint32_t peer = rs::peer_addr(w, (uint32_t)owner);
                        if (i < prompt_end) red_or_peer(peer, kPrompt);
                        else red_add_peer(peer, 1u);
                    } else if (i < prompt_end) {
                        atomicOr(w, kPrompt);
                    } else {
                        atomicAdd(w, 1u);
                    }
                }
            }
            // biases: every block looks through the row's entries for its own
            for (int64_t i = b0 + tid; i < b1; i += kThreads) {
                const int64_t id = a.bias_ids[i];
                if (id < 0 || id >= a.V || (i > b0 && a.bias_ids[i - 1] >= id)) {
                    bad = VCE_ERR_LABEL;
                    continue;
                }
                const int64_t at = id + r.shift;
                const int v = (int)(at / G);
                if (v >= v0 && v < v1) atomicOr(words + (int64_t)(v - v0) * G + at % G, kBias);
            }
            if (bad) {
                if (C > 1) red_max_peer(rs::peer_addr(&ctl.code, 0), bad);
                else atomicMax(&ctl.code, bad);
            }
            if (C > 1) rs::cluster_arrive(), rs::cluster_wait();
            else __syncthreads();
        }

        // the stream: kUnroll vectors in flight a thread
        for (int vb = v0 + tid; vb < v1; vb += kUnroll * kThreads) {
            uint4 x[kUnroll];
            uint32_t ok[kUnroll];
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) {
                const int v = vb + q * kThreads;
                const bool whole = v < v1 && v >= r.iv0 && v < r.iv1;
                ok[q] = (1u << G) - 1u;
                if (whole && mrow) ok[q] = allowed_bits<G>(mrow, (int64_t)v * G - r.shift);
                x[q] = make_uint4(0, 0, 0, 0);
                if (whole && ok[q]) x[q] = load16(r.base + (int64_t)v * 16);
            }
#pragma unroll
            for (int q = 0; q < kUnroll; ++q) {
                const int v = vb + q * kThreads;
                if (v >= v1) break;
                const int64_t c0 = (int64_t)v * G - r.shift;
                const bool whole = v >= r.iv0 && v < r.iv1;
                float z[G];
                Elt<S>::unpack(x[q], z);
                if (!whole) {                 // a partial first or last vector, by elements
                    ok[q] = 0;
#pragma unroll
                    for (int k = 0; k < G; ++k) {
                        const int64_t c = c0 + k;
                        z[k] = 0.f;
                        if (c < 0 || c >= a.V) continue;
                        if (!mrow || (mrow[c >> 5] >> (c & 31)) & 1u) {
                            ok[q] |= 1u << k;
                            z[k] = load_one(irow + c);
                        }
                    }
                }
                uint32_t skip = 0;            // columns that the bias entries write
                uint32_t w[G];
                uint32_t any = 0;
                if (lists) {
                    const uint4* wp = reinterpret_cast<const uint4*>(words + (int64_t)(v - v0) * G);
#pragma unroll
                    for (int k = 0; k < G / 4; ++k) {
                        const uint4 t = wp[k];
                        w[4 * k] = t.x, w[4 * k + 1] = t.y, w[4 * k + 2] = t.z, w[4 * k + 3] = t.w;
                        any |= t.x | t.y | t.z | t.w;
                    }
                }
                if (any) {
#pragma unroll
                    for (int k = 0; k < G; ++k) {
                        if (w[k] & kBias) skip |= 1u << k;
                        if (kBack) {
                            float g = z[k] * u.inv_t;
                            if (w[k] && ((ok[q] >> k) & 1u)) {
                                const float lz = a.z_bf16
                                                     ? Elt<uint16_t>::load1(static_cast<const uint16_t*>(a.z) +
                                                                            row * a.ld_z + c0 + k)
                                                     : Elt<float>::load1(static_cast<const float*>(a.z) +
                                                                         row * a.ld_z + c0 + k);
                                g = lz > 0.f ? g / u.r : g * u.r;
                            }
                            z[k] = g;
                        } else {
                            z[k] = process_one(z[k], w[k], u, 0.f);
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < G; ++k) z[k] *= u.inv_t;
                }
#pragma unroll
                for (int k = 0; k < G; ++k)
                    if (!((ok[q] >> k) & 1u)) z[k] = kMasked;
                if (whole && vec && !skip) {
                    GroupStore<O, G>::run(orow + c0, z);
                } else {
#pragma unroll
                    for (int k = 0; k < G; ++k)
                        if (c0 + k >= 0 && c0 + k < a.V && !((skip >> k) & 1u)) Elt<O>::store1(orow + c0 + k, z[k]);
                }
            }
        }
        // the columns with a bias
        if (lists && !kBack) {
            for (int64_t i = b0 + tid; i < b1; i += kThreads) {
                const int64_t id = a.bias_ids[i];
                if (id < 0 || id >= a.V || (i > b0 && a.bias_ids[i - 1] >= id)) continue;
                const int64_t at = id + r.shift;
                const int v = (int)(at / G);
                if (v < v0 || v >= v1) continue;
                float y = kMasked;
                if (!mrow || (mrow[id >> 5] >> (id & 31)) & 1u)
                    y = process_one(load_one(irow + id), words[(int64_t)(v - v0) * G + at % G], u, a.bias[i]);
                Elt<O>::store1(orow + id, y);
            }
        }
        if (lists && win + 1 < a.windows) __syncthreads();   // the words are written again
    }
    if (rank == 0 && tid == 0) a.row_status[row] = lists && ctl.code ? ctl.code : code;
}

template <typename S, typename O, bool kBack>
cudaError_t run(Args& a, int sms, cudaStream_t s) {
    constexpr int G = Elt<S>::kGroup;
    const int64_t nv = (a.V + 2 * G - 2) / G;
    const bool lists = a.hist || a.bias_ids;
    if (!lists) {   // independent blocks of four rounds of vectors
        const int per = (int)std::min<int64_t>(nv, kUnroll * kThreads);
        a.slice = per;
        a.cluster = (int)((nv + per - 1) / per);   // blocks of a row
        a.windows = 1;
        return rs::launch_clusters(k_process<S, O, kBack, false>, a.T * a.cluster, 1, kThreads, 0, s, a);
    }
    int C = 1;
    auto cols = [&](int c) { return (nv + c - 1) / c * G; };
    while (C < kMaxCluster && (cols(C) > kMaxSlice || (a.T * C < 2 * sms && cols(C) > 4096))) C *= 2;
    a.cluster = C;
    const int64_t per = (nv + C - 1) / C;
    a.slice = (int)std::min<int64_t>(per, kMaxSlice / G);
    a.windows = (int)((nv + (int64_t)C * a.slice - 1) / ((int64_t)C * a.slice));
    const int smem = (int)sizeof(Ctl) + a.slice * G * 4;
    return rs::launch_clusters(k_process<S, O, kBack, true>, a.T * C, C, kThreads, smem, s, a);
}

template <bool kBack>
cudaError_t dispatch(Args& a, vce_dtype dt, vce_dtype odt, int sms, cudaStream_t s) {
    if (dt == VCE_BF16)
        return odt == VCE_BF16 ? run<uint16_t, uint16_t, kBack>(a, sms, s) : run<uint16_t, float, kBack>(a, sms, s);
    return odt == VCE_BF16 ? run<float, uint16_t, kBack>(a, sms, s) : run<float, float, kBack>(a, sms, s);
}

// The checks that the forward and the backward share.
int check(const Args& a, vce_dtype dt, vce_dtype odt) {
    if ((dt != VCE_F32 && dt != VCE_BF16) || (odt != VCE_F32 && odt != VCE_BF16)) return VCE_ERR_DTYPE;
    if (a.T < 0 || a.T > VCE_MAX_TOPK_T || a.V < 1 || a.V > ((int64_t)1 << 30) / 4 || a.n_hist < 0 || a.n_bias < 0 ||
        a.n_hist >= ((int64_t)1 << 60) || a.n_bias >= ((int64_t)1 << 60))
        return VCE_ERR_SHAPE;
    if (a.ld < a.V || a.ld_out < a.V) return VCE_ERR_LD;
    if (a.mask && a.mask_ld < (a.V + 31) / 32) return VCE_ERR_LD;
    const size_t es = dt == VCE_BF16 ? 2 : 4, os = odt == VCE_BF16 ? 2 : 4;
    if (!fits_bytes(a.T, a.ld, es) || !fits_bytes(a.T, a.ld_out, os) || (a.mask && !fits_bytes(a.T, a.mask_ld, 4)))
        return VCE_ERR_SHAPE;
    // blocks of a launch: at most T * ceil(V / 1024)
    if (a.T * ((a.V + 1023) / 1024 + 1) >= ((int64_t)1 << 31)) return VCE_ERR_SHAPE;
    if (a.T == 0) return VCE_OK;
    if (!a.in || !a.out || !a.row_status) return VCE_ERR_NULL;
    if ((a.hist != nullptr) != (a.hist_off != nullptr) || (a.bias_ids != nullptr) != (a.bias_off != nullptr) ||
        (a.bias_ids != nullptr) != (a.bias != nullptr))
        return VCE_ERR_NULL;
    if (!a.hist && (a.repetition || a.frequency || a.presence || a.prompt)) return VCE_ERR_NULL;   // penalties of nothing
    if (!aligned(a.in, es) || !aligned(a.out, os) || !aligned(a.row_status, 4) || !aligned(a.temperature, 4) ||
        !aligned(a.repetition, 4) || !aligned(a.frequency, 4) || !aligned(a.presence, 4) || !aligned(a.hist, 8) ||
        !aligned(a.hist_off, 8) || !aligned(a.prompt, 8) || !aligned(a.bias_ids, 8) || !aligned(a.bias_off, 8) ||
        !aligned(a.bias, 4) || !aligned(a.mask, 4))
        return VCE_ERR_ALIGN;
    // in place, or apart
    const bool same = a.in == a.out && es == os && (a.ld == a.ld_out || a.T == 1);
    if (!same && rs::overlap(a.in, a.T, a.V, a.ld, es, a.out, a.ld_out, os)) return VCE_ERR_ARG;
    return VCE_OK;
}

}  // namespace process

VCE_DEBUG_READER(debug_word_process)

}  // namespace vce

using namespace vce;

extern "C" int logits_process(const void* logits, vce_dtype dt, int64_t T, int64_t V, int64_t ld,
                              const float* temperature, const float* repetition, const float* frequency,
                              const float* presence, const int64_t* history_ids, int64_t n_history,
                              const int64_t* history_offsets, const int64_t* prompt_lens, const int64_t* bias_ids,
                              const float* bias_values, int64_t n_bias, const int64_t* bias_offsets,
                              const int32_t* mask, int64_t mask_ld, void* out, vce_dtype out_dt, int64_t ld_out,
                              int32_t* row_status, vce_stream_t s) {
    process::Args a{};
    a.in = logits, a.T = T, a.V = V, a.ld = ld;
    a.temperature = temperature, a.repetition = repetition, a.frequency = frequency, a.presence = presence;
    a.hist = history_ids, a.n_hist = n_history, a.hist_off = history_offsets, a.prompt = prompt_lens;
    a.bias_ids = bias_ids, a.bias = bias_values, a.n_bias = n_bias, a.bias_off = bias_offsets;
    a.mask = reinterpret_cast<const uint32_t*>(mask), a.mask_ld = mask_ld;
    a.out = out, a.ld_out = ld_out, a.row_status = row_status;
    int rc = process::check(a, dt, out_dt);
    if (rc || T == 0) return rc;
    if ((rc = require_sm100())) return rc;
    const cudaError_t e = process::dispatch<false>(a, dt, out_dt, device_sm_count(), s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}

extern "C" int logits_process_backward(const void* grad_out, vce_dtype gdt, int64_t T, int64_t V, int64_t ld_gout,
                                       const void* logits, vce_dtype dt, int64_t ld, const float* temperature,
                                       const float* repetition, const int64_t* history_ids, int64_t n_history,
                                       const int64_t* history_offsets, const int32_t* mask, int64_t mask_ld,
                                       void* grad_logits, vce_dtype grad_dt, int64_t ld_grad, int32_t* row_status,
                                       vce_stream_t s) {
    process::Args a{};
    a.in = grad_out, a.T = T, a.V = V, a.ld = ld_gout;
    a.z = logits, a.ld_z = ld, a.z_bf16 = dt == VCE_BF16;
    a.temperature = temperature, a.repetition = repetition;
    a.hist = history_ids, a.n_hist = n_history, a.hist_off = history_offsets;
    a.mask = reinterpret_cast<const uint32_t*>(mask), a.mask_ld = mask_ld;
    a.out = grad_logits, a.ld_out = ld_grad, a.row_status = row_status;
    int rc = process::check(a, gdt, grad_dt);
    if (rc || T == 0) return rc;
    if (history_ids) {
        if (dt != VCE_F32 && dt != VCE_BF16) return VCE_ERR_DTYPE;
        if (!logits) return VCE_ERR_NULL;
        if (ld < V) return VCE_ERR_LD;
        if (!fits_bytes(T, ld, dt == VCE_BF16 ? 2 : 4)) return VCE_ERR_SHAPE;
        const size_t zs = dt == VCE_BF16 ? 2 : 4;
        if (!aligned(logits, zs)) return VCE_ERR_ALIGN;
        if (rs::overlap(logits, T, V, ld, zs, grad_logits, ld_grad, grad_dt == VCE_BF16 ? 2 : 4)) return VCE_ERR_ARG;
    }
    if ((rc = require_sm100())) return rc;
    const cudaError_t e = process::dispatch<true>(a, gdt, grad_dt, device_sm_count(), s);
    return record_cuda(e) == cudaSuccess ? VCE_OK : VCE_ERR_CUDA;
}
