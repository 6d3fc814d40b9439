// logits_process: repeated-token penalties, biases, temperature and masks on [T, V] logits, and
// the gradient through them.
//
// One read and one write of a row, and vectors that the mask leaves nothing of are written without
// being read.  What makes it more than a scaling is the row's history: a list of up to many thousands
// of tokens with repeats, of which the penalties need every column's count.
//
// A block takes a row, or a range of its columns where rows are few, in these steps:
//   count    its range's tokens into shared memory: a word per column (bits 0..29 the count behind
//            the prompt, bit 30 a bias, bit 31 seen in the prompt), in an open-addressing hash table,
//            or one for every column where the range is short.  Integer atomics: the order of the
//            tokens does not matter.  The columns named go on a list.
//   fetch    (backward) the logits at the listed columns into L2, without waiting for them
//   stream   the range's vectors: temperature and mask alone, four in flight a thread
//   touch    the listed columns' results, over the vectors just written
// so the stream runs without a look at the history, and the scattered reads and writes of the touch
// come to lines in L2 that the stream has just read and written.
// A range with more columns named than its hash table takes is done in windows, a word for every
// column.
//
// Measured at 4096 x 32000 bf16, backward, 384 tokens a row, half of the rows masked but for 50
// columns: 104 us, 71 without the history (a copy of the matrix: 79).  The rest is the touch: three
// scattered accesses a column, one of them to logits that nothing else reads (64 bytes of DRAM
// each).  A stream that looked at the words beside its vectors took 190 us (most warps meet one of
// the columns), a second kernel for the listed columns 151 us.  At 256 x 128256 bf16 with about
// 3000 tokens a row: 40 us; 26 for the same launch when no row has a token, 24 in the form for short
// histories, 18 without lists.  At 37 x 32001 fp32 with 15000: 11.9 us; 4.5, 4.2 and 3.3.  What the tokens
// cost is their instructions (each of a row's blocks looks at all of them) and the wait for them behind
// other blocks' streams.  Tried at these two shapes: a range's own tokens sorted out first, so that full
// warps count them, 52 and 25 us; the tokens shared out among a cluster's blocks, which count into one
// another's shared memory, 15.5 us at the second.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "row_launch.h"
#include "row_stream.cuh"
#include "vce_logits.h"

namespace vce {
namespace process {

using rs::Row;

constexpr int kThreads = 256, kLongThreads = 512;
constexpr int kLong = 1024;                   // tokens a row, on average, from which a block has kLongThreads
constexpr int kUnroll = 4;                    // 16-byte vectors a thread has in flight
constexpr int kBlocksPerSm = 4;               // blocks wanted for each SM before rows are taken whole
constexpr int kTokens = 4, kDenseTokens = 4;  // tokens a thread has in flight (hash table, a word a column)
constexpr int kDense = 8192;                  // columns of a range, at most, that all have a word
constexpr int kMinSlots = 1024, kMaxSlots = 16384;   // of a hash table (8 bytes each)
constexpr int kList = 2048;                   // listed columns; beyond, all words are looked through
constexpr uint32_t kPrompt = 0x80000000u, kBias = 0x40000000u, kCount = 0x3FFFFFFFu;
constexpr uint32_t kFree = 0xFFFFFFFFu;       // a slot without a column

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
    int parts, slice;                         // blocks of a row, vectors of a block
    int slots;                                // 8-byte slots of shared memory
    float masked;                             // -inf, or 0 in the backward
};

// A row's factors: 1 / temperature, the repetition penalty and its reciprocal, f, p.
struct Rule {
    float inv_t, r, inv_r, f, p;
};

struct alignas(16) Ctl {
    int code;                                 // an error among the tokens
    int n;                                    // columns named
    int full;                                 // the hash table has no room
    int status;                               // of the parameters and offsets
    int64_t h0, b0, b1;                       // the row's tokens from h0, its biases [b0, b1)
    int tokens, prompt;                       // its tokens, and how many of them are its prompt
    Rule rule;
    uint16_t list[kList];                     // the first of them: slots, or columns of the window
};

// One processed logit; w: its column's word.
__device__ __forceinline__ float process_one(float z, uint32_t w, const Rule& u, float bias) {
    const uint32_t n = w & kCount;
    float y = z * (n | (w & kPrompt) ? (z > 0.f ? u.inv_r : u.r) : 1.f);
    y = n ? (y - u.f * (float)n) - u.p : y;
    return (y + bias) * u.inv_t;
}

// Whether each of the G columns from c0 (a whole vector of the row) is allowed, bit k for c0 + k.
// kAligned: c0 is a multiple of G, so the bits lie in one word.
template <int G, bool kAligned>
__device__ __forceinline__ uint32_t allowed_bits(const uint32_t* mrow, uint32_t c0) {
    const uint32_t sh = c0 & 31u;
    const uint32_t* m = mrow + (c0 >> 5);
    uint32_t b = m[0] >> sh;
    if (!kAligned && sh + G > 32) b |= m[1] << (32 - sh);
    return b & ((1u << G) - 1u);
}

// The row's 1 / temperature; NaN and an error code if it is unusable.
__device__ __forceinline__ float inv_temperature(const Args& a, int64_t row, int& code) {
    if (!a.temperature) return 1.f;
    const float t = a.temperature[row];
    if (t > 0.f && t < kInf && 1.f / t < kInf) return 1.f / t;
    code = VCE_ERR_PARAM;
    return __int_as_float(0x7FC00000);
}

// z * inv_t where allowed (bits ok), `masked` elsewhere.  kWhole: vectors that the mask leaves whole, most
// of those that are read, skip the selection (512 threads, 256 x 128256 bf16: 40.2 against 42.9 us; with 256
// threads, the backward at 4096 x 32000: 109 against 104).
template <typename S, bool kWhole>
__device__ __forceinline__ void scale(uint4 x, uint32_t ok, float inv_t, float masked, float (&z)[Elt<S>::kGroup]) {
    constexpr int G = Elt<S>::kGroup;
    Elt<S>::unpack(x, z);
#pragma unroll
    for (int k = 0; k < G; k += 2) fmul2(z[k], z[k + 1], inv_t, z[k], z[k + 1]);
    if (kWhole && (ok & ((1u << G) - 1)) == (1u << G) - 1) return;
#pragma unroll
    for (int k = 0; k < G; ++k) z[k] = ((ok >> k) & 1u) ? z[k] : masked;
}

// kUnroll whole vectors of each thread, at vectors vs + q * NT of the row (kFull: all below
// `end`): loads first.
template <typename S, typename O, int NT, bool kMask, bool kAligned, bool kFull>
__device__ __forceinline__ void stream_batch(const Row& r, O* out0, const uint32_t* mrow, float inv_t, float masked,
                                             uint32_t vs, uint32_t end) {
    constexpr int G = Elt<S>::kGroup;
    uint4 x[kUnroll];
    uint32_t ok[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
        const uint32_t v = vs + q * NT;
        ok[q] = kMask && (kFull || v < end) ? allowed_bits<G, kAligned>(mrow, v * G - r.shift) : kMask ? 0u : 1u;
    }
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
        const uint32_t v = vs + q * NT;
        if ((!kMask || ok[q]) && (kFull || v < end)) x[q] = ld_stream16(r.base + (size_t)v * 16);
    }
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
        const uint32_t v = vs + q * NT;
        if (!kFull && v >= end) break;
        float z[G];
        if (kMask && !ok[q]) {
#pragma unroll
            for (int k = 0; k < G; ++k) z[k] = masked;
        } else {
            scale<S, NT == kLongThreads>(x[q], kMask ? ok[q] : 0xFFFFFFFFu, inv_t, masked, z);
        }
        if (dbg::ok((int)v >= r.iv0 && (int)v < r.iv1, dbg::kCols)) GroupStore<O, G>::run(out0 + (size_t)v * G, z);
    }
}

template <typename S, typename O, int NT, bool kMask, bool kAligned>
__device__ __forceinline__ void stream_whole(const Row& r, O* out0, const uint32_t* mrow, float inv_t, float masked,
                                             int wa, int wb) {
    constexpr int B = kUnroll * NT;
    int vs = wa;
#pragma unroll 1
    for (; vs + B <= wb; vs += B)
        stream_batch<S, O, NT, kMask, kAligned, true>(r, out0, mrow, inv_t, masked, vs + threadIdx.x, wb);
    if (vs < wb) stream_batch<S, O, NT, kMask, kAligned, false>(r, out0, mrow, inv_t, masked, vs + threadIdx.x, wb);
}

// Reads, processes (temperature and mask) and writes the vectors [va, vb) of the row.
template <typename S, typename O, int NT>
__device__ __forceinline__ void stream(const Args& a, const Row& r, const S* irow, O* orow, const uint32_t* mrow,
                                       float inv_t, int va, int vb) {
    constexpr int G = Elt<S>::kGroup;
    const bool vec = (reinterpret_cast<uintptr_t>(orow - r.shift) % (GroupStore<O, G>::kAlign)) == 0;
    const int wa = max(va, r.iv0), wb = min(vb, r.iv1);   // the whole ones
    O* out0 = orow - r.shift;
    if (vec && !mrow) {
        stream_whole<S, O, NT, false, true>(r, out0, mrow, inv_t, a.masked, wa, wb);
    } else if (vec && !r.shift) {
        stream_whole<S, O, NT, true, true>(r, out0, mrow, inv_t, a.masked, wa, wb);
    } else if (vec) {
        stream_whole<S, O, NT, true, false>(r, out0, mrow, inv_t, a.masked, wa, wb);
    } else {   // the output's rows are aligned unlike the input's: stores by elements
        for (int v = wa + threadIdx.x; v < wb; v += NT) {
            const uint32_t ok = mrow ? allowed_bits<G, false>(mrow, (uint32_t)v * G - r.shift) : 0xFFFFFFFFu;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (ok) x = ld_stream16(r.base + (size_t)v * 16);
            float z[G];
            scale<S, false>(x, ok, inv_t, a.masked, z);
#pragma unroll
            for (int k = 0; k < G; ++k) Elt<O>::store1(out0 + (size_t)v * G + k, z[k]);
        }
    }
    const int head = va < r.iv0 ? min((int64_t)G - r.shift, a.V) : 0;          // columns [0, head)
    const int tail = va <= r.iv1 && vb > r.iv1 && r.iv1 >= r.iv0 ? r.iv1 * G - r.shift : (int)a.V;   // columns [tail, V)
    if ((int)threadIdx.x < 2 * G) {
        const int c = (int)threadIdx.x < G ? (int)threadIdx.x : tail + (int)threadIdx.x - G;
        if ((int)threadIdx.x < G ? c < head : c < a.V) {
            const bool ok = !mrow || (mrow[c >> 5] >> (c & 31)) & 1u;
            Elt<O>::store1(orow + c, ok ? Elt<S>::load1(irow + c) * inv_t : a.masked);
        }
    }
}

// The row's parameters, tokens and biases (one thread).
template <bool kBack>
__device__ __forceinline__ void read_row(const Args& a, int64_t row, float inv_t, int status, Ctl& ctl) {
    Rule u{inv_t, 1.f, 1.f, 0.f, 0.f};
    int64_t h0 = 0, h1 = 0, np = 0, b0 = 0, b1 = 0;
    if (a.hist) {
        h0 = a.hist_off[row];
        h1 = a.hist_off[row + 1];
        if (a.prompt) np = a.prompt[row];
        if (a.repetition) u.r = a.repetition[row];
        if (!kBack && a.frequency) u.f = a.frequency[row];
        if (!kBack && a.presence) u.p = a.presence[row];
    }
    if (!kBack && a.bias_ids) {
        b0 = a.bias_off[row];
        b1 = a.bias_off[row + 1];
    }
    if (!(u.r > 0.f && u.r < kInf)) {
        u.r = __int_as_float(0x7FC00000);
        status = VCE_ERR_PARAM;
    }
    u.inv_r = 1.f / u.r;
    if (h0 < 0 || h1 < h0 || h1 > a.n_hist || h1 - h0 > (int64_t)kCount) {
        h0 = h1 = 0;
        status = VCE_ERR_OFFSETS;
    }
    if (b0 < 0 || b1 < b0 || b1 > a.n_bias || b1 - b0 > (int64_t)kCount) {
        b0 = b1 = 0;
        status = VCE_ERR_OFFSETS;
    }
    ctl.code = ctl.full = 0;
    ctl.status = status;
    ctl.h0 = h0;
    ctl.tokens = (int)(h1 - h0);
    ctl.prompt = (int)(np < 0 ? 0 : np > h1 - h0 ? h1 - h0 : np);
    ctl.b0 = b0;
    ctl.b1 = b1;
    ctl.rule = u;
}

// Lists a place; its number on the list.
__device__ __forceinline__ int enlist(Ctl& ctl, int at) {
    const int n = atomicAdd(&ctl.n, 1);
    if (n < kList) ctl.list[n] = (uint16_t)at;
    return n;
}

// One token (bits 0: one more) or bias at column c of the range.
template <int NT, bool kHash>
__device__ __forceinline__ void count_one(const Args& a, Ctl& ctl, uint32_t* words, uint32_t* cols, uint32_t c,
                                          uint32_t bits) {
    uint32_t at = c;
    if (kHash) {
        // a thread stops at its first insertion past `room`, so that probing always meets a free slot
        const int room = min(a.slots / 4 * 3, a.slots - NT - 1);
        if (*reinterpret_cast<volatile int*>(&ctl.full)) return;
        at = (c * 2654435761u >> 8) & (uint32_t)(a.slots - 1);   // Knuth's multiplicative hash
        for (;; at = (at + 1) & (uint32_t)(a.slots - 1)) {
            const uint32_t was = atomicCAS(cols + at, kFree, c);
            if (was == kFree && enlist(ctl, (int)at) >= room) ctl.full = 1;
            if (was == kFree || was == c) break;
        }
    }
    if (!dbg::ok(at < (uint32_t)(kHash ? a.slots : 2 * a.slots), dbg::kStage)) return;
    if (bits) atomicOr(words + at, bits);
    else atomicAdd(words + at, 1u);
}

// The bias of column c, an entry of the row's ascending ones.
__device__ __forceinline__ float bias_of(const Args& a, int64_t lo, int64_t hi, int64_t c) {
    --hi;
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (a.bias_ids[mid] < c) lo = mid + 1;
        else hi = mid;
    }
    return a.bias[lo];
}

// All steps for the vectors [va, vb) of the row, by every thread of the block: with a hash table of
// their columns, or a word for each of them.  False, with nothing written: the table has no room.
template <typename S, typename O, int NT, bool kBack, bool kHash>
__device__ __forceinline__ bool range(const Args& a, Ctl& ctl, uint32_t* words, const Row& r, int64_t row, float inv_t,
                                      int va, int vb) {
    constexpr int G = Elt<S>::kGroup;
    const int tid = threadIdx.x;
    uint32_t* cols = words + a.slots;
    const S* irow = static_cast<const S*>(a.in) + row * a.ld;
    O* orow = static_cast<O*>(a.out) + row * a.ld_out;
    const uint32_t* mrow = a.mask ? a.mask + row * a.mask_ld : nullptr;
    // the columns [lo, hi) of the vectors [va, vb)
    const int lo = max(0, va * G - r.shift), hi = max(lo, min((int)a.V, vb * G - r.shift));
    if (tid == 0) ctl.n = 0;
    if (kHash) {
#pragma unroll 1
        for (int i = tid; i < a.slots; i += NT) {
            words[i] = 0;
            cols[i] = kFree;
        }
    } else {
#pragma unroll 1
        for (int i = tid; i < hi - lo; i += NT) words[i] = 0;
    }
    __syncthreads();
    // ---- count ----
    // The tokens as (low, high) halves, several of them in flight.  Of a hash table one copy of the code
    // that counts them, the ids moving up to it (unrolled, it outgrows the instruction cache).
    const int n = ctl.tokens, np = ctl.prompt;
    const uint2* ids = reinterpret_cast<const uint2*>(a.hist + ctl.h0);
    const uint32_t ulo = (uint32_t)lo, width = (uint32_t)(hi - lo);
    constexpr int kAhead = kHash ? kTokens : kDenseTokens;
    bool bad = false;
#pragma unroll 1
    for (int i0 = tid; i0 < n; i0 += kAhead * NT) {
        uint2 id[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) id[q] = i0 + q * NT < n ? ids[i0 + q * NT] : make_uint2(ulo, 0);
        if constexpr (kHash) {
#pragma unroll 1
            for (int i = i0, q = 0; q < kAhead && i < n; ++q, i += NT) {
                const uint2 t = id[0];
#pragma unroll
                for (int k = 1; k < kAhead; ++k) id[k - 1] = id[k];
                if (t.y | (t.x >= (uint32_t)a.V)) bad = true;
                else if (t.x - ulo < width) count_one<NT, kHash>(a, ctl, words, cols, t.x - ulo, i < np ? kPrompt : 0u);
            }
        } else {
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int i = i0 + q * NT;
                const uint32_t c = id[q].x - ulo;
                bad |= id[q].y != 0 || id[q].x >= (uint32_t)a.V;
                if (c < width && id[q].y == 0 && dbg::ok(c < 2u * (uint32_t)a.slots, dbg::kStage)) {
                    if (i < np) atomicOr(words + c, kPrompt);
                    else if (i < n) atomicAdd(words + c, 1u);
                }
            }
        }
    }
    if (bad) ctl.code = VCE_ERR_LABEL;
    if (!kBack) {
#pragma unroll 1
        for (int64_t i = ctl.b0 + tid; i < ctl.b1; i += NT) {
            const int64_t id = a.bias_ids[i];
            if (id < 0 || id >= a.V || (i > ctl.b0 && a.bias_ids[i - 1] >= id)) ctl.code = VCE_ERR_LABEL;
            else if (id >= lo && id < hi) count_one<NT, kHash>(a, ctl, words, cols, (uint32_t)(id - lo), kBias);
        }
    }
    __syncthreads();
    if (kHash && ctl.full) return false;
    if (!kHash && n + (int)(ctl.b1 - ctl.b0)) {
#pragma unroll 1
        for (int i = tid; i < hi - lo; i += NT)
            if (words[i]) enlist(ctl, i);
        __syncthreads();
    }
    // the listed places, or, if they are too many for the list, all places with a word
    const bool listed = ctl.n <= kList;
    const int places = listed ? ctl.n : kHash ? a.slots : hi - lo;
    // ---- fetch ----
    if (kBack) {
#pragma unroll 1
        for (int i = tid; i < places; i += NT) {
            const int at = listed ? (int)ctl.list[i] : i;
            const int c = lo + (kHash ? (int)cols[at] : at);
            if (!dbg::ok(at < (kHash ? a.slots : 2 * a.slots), dbg::kStage)) continue;
            if (!words[at] || !dbg::ok(c >= lo && c < hi, dbg::kCols) || (mrow && !((mrow[c >> 5] >> (c & 31)) & 1u))) continue;
            const char* z = static_cast<const char*>(a.z) + (row * a.ld_z + c) * (a.z_bf16 ? 2 : 4);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(z));
        }
    }
    // ---- stream ----
    stream<S, O, NT>(a, r, irow, orow, mrow, inv_t, va, vb);
    __syncthreads();
    // ---- touch ----
#pragma unroll 1
    for (int i = tid; i < places; i += NT) {
        const int at = listed ? (int)ctl.list[i] : i;
        if (!dbg::ok(at < (kHash ? a.slots : 2 * a.slots), dbg::kStage)) continue;
        const uint32_t w = words[at];
        const int c = lo + (kHash ? (int)cols[at] : at);
        if (!w || !dbg::ok(c >= lo && c < hi, dbg::kCols) || (mrow && !((mrow[c >> 5] >> (c & 31)) & 1u))) continue;
        const float e = Elt<S>::load1(irow + c);
        const Rule& u = ctl.rule;
        float y;
        if (kBack) {
            const int64_t zc = row * a.ld_z + c;
            const float z = a.z_bf16 ? Elt<uint16_t>::load1(static_cast<const uint16_t*>(a.z) + zc)
                                     : Elt<float>::load1(static_cast<const float*>(a.z) + zc);
            y = e * inv_t * (z > 0.f ? u.inv_r : u.r);
        } else {
            y = process_one(e, w, u, w & kBias ? bias_of(a, ctl.b0, ctl.b1, c) : 0.f);
        }
        Elt<O>::store1(orow + c, y);
    }
    __syncthreads();
    return true;
}

// The vectors [v0, v1) in windows, after the hash table had no room for their columns.
template <typename S, typename O, int NT, bool kBack>
__device__ __noinline__ void windows(const Args& a, Ctl& ctl, uint32_t* words, int64_t row, float inv_t, int v0, int v1) {
    const Row r = rs::make_row<S>(a.in, row, a.ld, a.V);
    const int width = 2 * a.slots / Elt<S>::kGroup;
    for (int va = v0; va < v1; va += width) {
        __syncthreads();
        range<S, O, NT, kBack, false>(a, ctl, words, r, row, inv_t, va, min(v1, va + width));
    }
}

// The block's place: its row, its part of the row, and the vectors [v0, v1) of that.
struct Place {
    int64_t row;
    int part, v0, v1;
};
__device__ __forceinline__ Place place_of(const Args& a, int nv_of_row, int64_t row) {
    const int part = (int)(blockIdx.x - row * a.parts), v0 = min(nv_of_row, part * a.slice);
    return Place{row, part, v0, min(nv_of_row, v0 + a.slice)};
}

// Of a row with an error: every column of the block's NaN, or in the backward without a gradient, so that
// what was skipped or could not be worked out shows where nobody looks at the status.  Everything is
// worked out again here: values kept for it would cost the kernel's loops registers.
template <typename S, typename O, int NT, bool kBack>
__device__ __noinline__ void refuse(const Args& a) {
    constexpr int G = Elt<S>::kGroup;
    const int64_t row = blockIdx.x / a.parts;
    const Row r = rs::make_row<S>(a.in, row, a.ld, a.V);
    const Place p = place_of(a, r.nv, row);
    O* orow = static_cast<O*>(a.out) + row * a.ld_out;
    const int lo = max(0, p.v0 * G - r.shift), hi = min((int)a.V, p.v1 * G - r.shift);
    for (int c = lo + (int)threadIdx.x; c < hi; c += NT) Elt<O>::store1(orow + c, kBack ? 0.f : __int_as_float(0x7FC00000));
}

enum { kNoLists, kDenseRange, kHashed };

template <typename S, typename O, int NT, bool kBack, int kKind>
__global__ void __launch_bounds__(NT, NT == kThreads ? 5 : 3) k_process(const __grid_constant__ Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.parts;
    const Row r = rs::make_row<S>(a.in, row, a.ld, a.V);
    const Place p = place_of(a, r.nv, row);
    const int part = p.part, v0 = p.v0, v1 = p.v1;
    int code = 0;
    const float inv_t = inv_temperature(a, row, code);
    if (kKind == kNoLists) {
        const S* irow = static_cast<const S*>(a.in) + row * a.ld;
        O* orow = static_cast<O*>(a.out) + row * a.ld_out;
        if (code) refuse<S, O, NT, kBack>(a);
        else stream<S, O, NT>(a, r, irow, orow, a.mask ? a.mask + row * a.mask_ld : nullptr, inv_t, v0, v1);
        if (part == 0 && tid == 0) a.row_status[row] = code;
        return;
    }
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
    uint32_t* words = reinterpret_cast<uint32_t*>(smem + sizeof(Ctl));   // [slots], then a hash table's columns
    if (tid == 0) read_row<kBack>(a, row, inv_t, code, ctl);
    if (!range<S, O, NT, kBack, kKind == kHashed>(a, ctl, words, r, row, inv_t, v0, v1))
        windows<S, O, NT, kBack>(a, ctl, words, row, inv_t, v0, v1);
    const int error = max(ctl.status, ctl.code);   // every block of a row has seen all its tokens and biases
    if (error) refuse<S, O, NT, kBack>(a);
    if (part == 0 && tid == 0) a.row_status[row] = error;
}

template <typename S, typename O, int NT, bool kBack>
cudaError_t launch_lists(Args& a, bool dense, cudaStream_t s) {
    const int smem = (int)sizeof(Ctl) + (a.slots * 8 + 15) / 16 * 16;
    if (dense) return rs::launch_clusters<k_process<S, O, NT, kBack, kDenseRange>>(a.T * a.parts, 1, NT, smem, s, a);
    return rs::launch_clusters<k_process<S, O, NT, kBack, kHashed>>(a.T * a.parts, 1, NT, smem, s, a);
}

template <typename S, typename O, bool kBack>
cudaError_t run(Args& a, int sms, cudaStream_t s) {
    constexpr int G = Elt<S>::kGroup;
    const int64_t nv = (a.V + 2 * G - 2) / G;
    const int64_t most = (nv + kUnroll * kThreads - 1) / (kUnroll * kThreads);   // blocks of four rounds of vectors
    if (!a.hist && !a.bias_ids) {
        a.parts = (int)most;
        a.slice = kUnroll * kThreads;
        return rs::launch_clusters<k_process<S, O, kThreads, kBack, kNoLists>>(a.T * a.parts, 1, kThreads, 0, s, a);
    }
    // With lists a block takes a whole row where the rows fill the SMs, since every block of a row
    // reads its tokens.
    a.parts = (int)std::min<int64_t>(most, (kBlocksPerSm * sms + a.T - 1) / a.T);
    a.slice = (int)((nv + a.parts - 1) / a.parts);
    const int64_t mean = (a.n_hist + a.n_bias) / a.T;
    const bool dense = (int64_t)a.slice * G <= kDense;
    if (dense) {
        a.slots = (a.slice * G + 1) / 2;
    } else {                                  // room for the mean number of tokens twice
        a.slots = kMinSlots;
        while (a.slots < kMaxSlots && a.slots < 2 * (mean / a.parts)) a.slots *= 2;
    }
    // Long histories: more threads to count them (37 x 32001 fp32 with 15000 tokens a row: 13.6 against
    // 19.5 us); short ones: more blocks an SM (4096 x 32000 bf16 backward with 384: 104 against 115 us).
    return mean >= kLong ? launch_lists<S, O, kLongThreads, kBack>(a, dense, s) : launch_lists<S, O, kThreads, kBack>(a, dense, s);
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
    // blocks of a launch: at most T * (V / 4096 + 9)
    if (a.T * (a.V / 4096 + 9) >= ((int64_t)1 << 31)) return VCE_ERR_SHAPE;
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
    if (rs::overlap(a.in, a.T, a.V, a.ld, es, a.out, a.ld_out, os)) return VCE_ERR_ARG;
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
    a.out = out, a.ld_out = ld_out, a.row_status = row_status, a.masked = -kInf;
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
