/*
 * vce_fp8.h -- C ABI of the head in 8-bit floating point (libvce.so): the logits of a frozen
 * policy, reference or teacher whose hidden states and weights are e4m3 values (1 sign, 4 exponent,
 * 3 mantissa bits, largest 448) with an fp32 scale for each block of 128 columns.
 *
 *   vce_quantize_fp8   a matrix to e4m3 with block scales
 *   vce_linear_fp8     logits = (scaled hidden states) (scaled weights)^T
 *
 * The conventions of vce.h hold (device pointers owned by the caller, nothing allocated, work only
 * enqueued on `s`, VCE_OK or a negative host-detected error).
 */
#ifndef VCE_FP8_H
#define VCE_FP8_H

#include "vce.h"

#ifdef __cplusplus
extern "C" {
#endif

#define VCE_FP8_BLOCK 128

/*
 * vce_quantize_fp8 -- x [R, D] to q [R, D] e4m3 and scales [ceil(R / block_rows), ceil(D / 128)]:
 *   scale = the least power of two with max |x| <= 448 scale over the block of block_rows x 128
 *           elements (1 for a block of zeros, at least 2^-126),   q = x / scale rounded to nearest even
 * The scale is a power of two, so the division is exact and q carries one rounding.  A block with a
 * NaN or an infinity has the scale NaN and nothing but NaN in it.
 *   x, dt       fp32 or bf16, leading dimension ld >= D
 *   block_rows  1 (hidden states: a scale for every row) or 128 (weights)
 *   q           [R, D] bytes, leading dimension D, written;  scales  fp32, written; VCE_ERR_ARG if the extents of
 *               x, q and scales share a byte
 *   D           1 .. 2^24;  R <= 2^27
 */
VCE_API int vce_quantize_fp8(const void* x, vce_dtype dt, int64_t R, int64_t D, int64_t ld, int block_rows,
                             void* q, float* scales, vce_stream_t s);

/*
 * vce_linear_fp8 -- out[t][v] = sum_b x_scales[t][b] w_scales[v / 128][b] sum_{k in block b} x[t][k] w[v][k]
 * over the blocks b of 128 columns, on the tensor cores: a block's products are summed in fp32 there,
 * and the scaled blocks in fp32 beside them.  The scales may be any fp32 numbers; a row's and a block's are
 * multiplied first, so their product has to be one too.
 *   x         [T, D] e4m3, leading dimension D, 16-byte aligned
 *   x_scales  [T, ceil(D / 128)] fp32
 *   w         [V, D] e4m3, leading dimension D, 16-byte aligned
 *   w_scales  [ceil(V / 128), ceil(D / 128)] fp32
 *   T, V, D   T, V <= 2^24; D a multiple of 16, 16 .. 65536
 *   out       [T, ld] of dtype out_dt (bf16 or fp32), written; ld >= V; VCE_ERR_ARG if its extent shares a byte
 *             with an operand's
 * Tiles behind a device-side wait that gave up after 2 s hold NaN.
 */
VCE_API int vce_linear_fp8(const void* x, const float* x_scales, const void* w, const float* w_scales,
                           int64_t T, int64_t D, int64_t V, void* out, vce_dtype out_dt, int64_t ld,
                           vce_stream_t s);

/*
 * vce_test_linear_fp8_stall -- test hook: vce_linear_fp8 to fp32 (ld = V) with its producer announcing 16
 * more bytes per stage than its copies deliver, so no stage ever completes and every wait, bounded by
 * wait_ns (1 ms .. 2 s), gives up.  out is NaN; the context stays usable.
 */
VCE_API int vce_test_linear_fp8_stall(const void* x, const float* x_scales, const void* w, const float* w_scales,
                                      int64_t T, int64_t D, int64_t V, float* out, uint64_t wait_ns,
                                      vce_stream_t s);

#ifdef __cplusplus
}
#endif

#endif /* VCE_FP8_H */
