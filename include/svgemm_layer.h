/*
 * svgemm_layer.h -- C ABI of the steps of a decoder layer around the quantized
 * linears of svgemm.h: the norm in front of every activation quantization,
 * attention of a draft tree over a paged cache, and the cache's pages.
 *
 * Conventions are those of svgemm.h: device pointers owned by the caller,
 * asynchronous on `stream`, checked on the host before anything is enqueued
 * (svg_last_error(), outputs untouched on a failed check), nothing allocated
 * or synchronised, no memset recorded: every call may be captured in a HIP
 * graph.  The pointers belong to the current device.  What only the device
 * knows (lengths, page numbers, trees) is checked there, and each call says
 * what it does with a value out of range; none reads or writes out of bounds.
 */
#ifndef SVGEMM_LAYER_H
#define SVGEMM_LAYER_H

#include "svgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { SVG_F32 = 0, SVG_F16 = 1, SVG_BF16 = 2 }; /* element types */

/*
 * add_rmsnorm_quant_i8 -- residual addition, root-mean-square norm, rotation
 * and int8 quantization of activation rows, in one launch: what stands in
 * front of every projection of a decoder layer.
 *
 *  x         [M][K] of x_type, 16-byte aligned: the rows to add (the output of
 *            the projection before, or the embedding rows).
 *  residual  fp32 [M][K], 16-byte aligned, updated in place; NULL: none (the
 *            norm is of x itself).
 *  weight    [K] of w_type, 16-byte aligned.
 *  eps       > 0 and finite.
 *  M, K      M >= 0 rows (M == 0: nothing enqueued), M <= 2^24; K % block == 0, K <= 32768.
 *  signs, block   as for act_rht_quant_i8.
 *  y         fp32 [M][K], 16-byte aligned, or NULL: receives the normalised
 *            rows before the rotation (for a reader that is not quantized).
 *  xq, x_scale   codes and row scales as from act_rht_quant_i8.  Rows are
 *            taken 32 at a time: rows 32 b .. 32 b + 31 (the last ones fewer) are one slab
 *            buffer of their own at xq + 32 b K, so that a prompt's
 *            blocks go to the linears one after another.  M <= 32 is one buffer.
 *
 *  h = x + residual -> residual;  r = 1 / sqrt(sum_k h^2 / K + eps), the sum, the
 *  quotient and the root in 64 bits, rounded once to fp32;  u = (h * r) * weight
 *  -> y, each product rounded to fp32; then u as X in act_rht_quant_i8.  The
 *  codes are those of the separate steps bit for bit.
 *  Errors: SVG_EINVAL for a null required pointer, M < 0, K <= 0 or eps not a
 *  positive finite number; SVG_EUNSUPPORTED for a type, a block, K % 32, K % block,
 *  K > 32768, M > 2^24; SVG_EALIGN.
 */
svg_status add_rmsnorm_quant_i8(const void* x, int x_type, float* residual, const void* weight, int w_type,
                                double eps, int M, int K, const int8_t* signs, int block, float* y, int8_t* xq,
                                float* x_scale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SVGEMM_LAYER_H */
