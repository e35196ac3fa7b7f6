/*
 * svgemm_prompt.h -- C ABI of a prompt's pass through a decoder layer: many rows of many
 * requests at once, where svgemm.h and svgemm_layer.h run single tokens and draft trees.
 *
 * A pass: add_rmsnorm_quant_i8 (any number of rows), w4a8_prompt_linear or w8a8_prompt_linear,
 * rope_append, prompt_attention, gated_quant_i8 without a gate, the next linear, ..., gated_quant_i8 of
 * gate and up.  kv_row_map is called once for all layers, behind kv_reserve; afterwards the caller adds
 * the rows of each slot to len.  kv_row_map and rope_append serve draft trees as well.
 *
 * Conventions are those of svgemm_layer.h: device pointers owned by the caller, asynchronous on
 * `stream`, checked on the host before anything is enqueued, nothing allocated or synchronised, no memset
 * recorded; what only the device knows is checked there, and nothing is read or written out of bounds.
 */
#ifndef SVGEMM_PROMPT_H
#define SVGEMM_PROMPT_H

#include "svgemm_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kv_row_map -- where the rows of a step belong: of each slot its first row and their number, of each
 * row its slot, its position and its place in the cache's pages.  One launch.
 *
 *  n_new     int32 [n_slots]: new rows of each slot (below 1: none).
 *  parent    NULL, or int32 [n_slots][T] draft trees as for tree_attention (T in 1 .. SVG_TREE_MAX_NODES).
 *  T         0: the rows are packed, slot after slot.  T >= 1: T rows for each slot, row s * T + i is its row i, of which
 *            the nearest of 0 .. T to n_new[s] are in use.
 *  n_rows    rows of the step's buffers: n_slots * T, or for packed rows any number below 2^31 (rows past it have no place in
 *            the step: the slots' counts are cut).
 *  start     OUTPUT int32 [n_slots]: the first row of each slot (T = 0: the sum of the n_new before it, n_rows at most).
 *  count     OUTPUT int32 [n_slots]: its rows.
 *  slot      OUTPUT int32 [n_rows] or NULL: the slot of each row; -1 for a row of none (behind the last slot's, or not in use).
 *  pos       OUTPUT int32 [n_rows]: the position in its sequence: len[s] + i for row i of slot s; in a tree len[s] + the
 *            depth of node i (the root's is 0).  -1: a row of no slot, a node whose root path breaks the tree rule,
 *            a negative length, or a position past 2^31 - 1.
 *  place     OUTPUT int32 [n_rows]: table[s][p / page] * page + p % page for p = len[s] + i, where the row's key and value
 *            go (and kv_append puts them); -1 where pos is -1 and for every row that kv_append passes over.
 *  Reads table, pages, len, and refs where it is not NULL.
 *  Errors: SVG_EINVAL for a null required pointer, T < 0, n_rows < 0, n_rows other than n_slots * T (T >= 1), a parent
 *  with T = 0; SVG_EUNSUPPORTED for a cache outside its limits, a parent with T > SVG_TREE_MAX_NODES, n_slots * T >= 2^31;
 *  SVG_EALIGN.
 */
svg_status kv_row_map(const svg_kv_cache* cache, const int32_t* n_new, const int32_t* parent, int T, int n_rows, int32_t* start,
                      int32_t* count, int32_t* slot, int32_t* pos, int32_t* place, void* stream);

/*
 * svg_rope -- rotary positions: a host struct that a call reads during the call only.
 *
 *  freq         float64 [rot / 2], 8-byte aligned: the angle of pair i of a row at position pos is pos * freq[i] radians
 *               (one fp64 product; base^(-2 i / rot), divided or bent as the model's long contexts are).
 *  rot          rotated values of each head, its first ones: a multiple of 16, 16 .. dim; the others pass.
 *  interleaved  0: pair i is values i and i + rot / 2;  1: values 2 i and 2 i + 1.
 *  amplitude    finite; multiplies the cosines and sines (1 unless the long-context scaling has such a factor).
 */
typedef struct svg_rope {
    const double* freq;
    int rot, interleaved;
    float amplitude;
} svg_rope;

/*
 * rope_append -- rotate the queries and keys of a step's rows by their positions, and write keys and values
 * into the pages of one layer: between a projection and the attention.  One launch.
 *
 *  q, k, v    n_rows rows of x_type (SVG_F32, SVG_F16, SVG_BF16), of q_heads * dim, heads * dim and heads * dim values, rows ld_q /
 *             ld_k / ld_v values apart, each row 16-byte aligned (they may be parts of one projection's rows).
 *  q_heads    >= 0 (0: no queries; q and q_out may be NULL), at most 4096.
 *  n_rows     rows, below 2^31.
 *  pos, place int32 [n_rows] as from kv_row_map.  A row with pos < 0 is passed over.  One with place < 0 (or outside the
 *             cache's pages) has its queries rotated and its key and value passed over.  No two rows have the same place.
 *  q_out      [n_rows][q_heads * dim] of q_type: SVG_F32 (for tree_attention) or the cache's type (for prompt_attention),
 *             16-byte aligned.
 *
 *  Pair (a, b) becomes (a c - b s, b c + a s) with c, s the cosine and sine of the angle times amplitude, the angle
 *  reduced in fp64 and c and s within 2 units of fp32's last place of it; two fp32 operations, then one
 *  rounding to q_type or the cache's type.  Values that are not rotated and v are rounded once.  kv_append and
 *  this call write the same patterns for keys that are not rotated.
 *  Reads no table of the cache (k, v, type, heads, dim, page, n_pages, n_layers).
 *  Errors: SVG_EINVAL for a null required pointer, n_rows < 0, q_heads < 0, a layer outside the cache, or an amplitude that is
 *  not finite; SVG_EUNSUPPORTED for a cache outside its limits, an unknown type, rot, q_heads, a row stride below the row or of
 *  2^31 or more; SVG_EALIGN.
 */
svg_status rope_append(const svg_kv_cache* cache, int layer, const svg_rope* rope, const void* q, int64_t ld_q, int q_heads,
                       const void* k, int64_t ld_k, const void* v, int64_t ld_v, int x_type, int n_rows, const int32_t* pos,
                       const int32_t* place, void* q_out, int q_type, void* stream);

/*
 * prompt_attention -- causal attention of the rows of all slots over the cache, in one layer: the rows' own keys and
 * values have been written (rope_append, kv_append) behind the committed tokens, and len has not grown yet.
 *
 *  q          [n_rows] rows of q_heads * dim values of the cache's type, rows ld_q values apart, 16-byte aligned each.
 *  q_heads    a multiple of heads: query head a reads key/value head a / (q_heads / heads); at most 4096.
 *  n_rows     rows of q and out.
 *  start, count  int32 [n_slots] as from kv_row_map: rows start[s] .. start[s] + count[s] - 1 are slot s's (a start
 *             outside 0 .. n_rows - 1 is no row, and rows past n_rows are not computed).  Rows of out that belong to no slot
 *             are left as they were.  No row belongs to two.
 *  scale      finite; the scores are scale * q . k.
 *  out        [n_rows][q_heads * dim] of the cache's type, 16-byte aligned.
 *  workspace  prompt_attention_workspace() bytes, 256-byte aligned; its contents need not be set or kept.  Calls that may
 *             overlap need different ones.
 *
 *  Row i of slot s: o = sum_t p_t v_t / sum_t p_t, p_t = exp(scale * q . k_t), over the positions 0 .. len[s] + i.
 *  Scores, sums and accumulators are fp32; p enters the second product rounded to the cache's type (as v is held in it), so an
 *  output is off by its own rounding and by about as much again.  Of an fp16 cache a p below 2^-33 of the
 *  row's largest so far may be lost.  Finite scores and values of any size give finite rows (of a bf16 cache an output is off by up to
 *  2^-116 a token besides, which only its smallest values show).
 *  Keys and values of tokens that a row does not see never reach it, whatever they are.  Of those it sees: a key that gives a
 *  NaN or +infinite score makes the row NaN (-infinity leaves the token out, and a row all of whose tokens are left out is NaN);
 *  a value that is not finite makes its own element of the row NaN or infinite, and no other.
 *  NaN rows: a row that sees a page number outside the cache, or a position of the step's own (len[s] and on) in a page that
 *  other slots hold too; all of a slot whose pages do not cover len + count.
 *  Reads table, pages, len, and refs where it is not NULL.
 *  Errors: SVG_EINVAL for a null required pointer, n_rows < 0, q_heads < 1, a layer outside the cache, a scale that is
 *  not finite; SVG_EUNSUPPORTED for a cache outside its limits, q_heads, ld_q or n_rows * (q_heads / heads) >= 2^30;
 *  SVG_EALIGN.
 *
 * prompt_attention_workspace -- the bytes of that workspace (host only).
 */
svg_status prompt_attention_workspace(const svg_kv_cache* cache, int q_heads, int n_rows, uint64_t* bytes);
svg_status prompt_attention(const svg_kv_cache* cache, int layer, const void* q, int64_t ld_q, int q_heads, int n_rows,
                            const int32_t* start, const int32_t* count, float scale, void* out, void* workspace, void* stream);

/*
 * w4a8_prompt_linear, w8a8_prompt_linear -- y = x . W^T for any number of int8 activation rows: the linears of svgemm.h
 * without their limit on M, on the same weights.
 *
 *  xq, x_scale   M rows in 32-row slab buffers, as add_rmsnorm_quant_i8 and gated_quant_i8 write them: rows 32 b .. 32 b + 31 (the
 *                last ones fewer) at xq + 32 b K, code (row m, k) of a buffer of R rows at byte ((k / 32) * R + m % 32) * 32 + k % 32.
 *                xq 16-byte aligned.
 *  M, K, N       M >= 0 (M <= 2^24), K % 32 == 0 (W4: K % group == 0), K <= 131072, M * K < 2^40, 0 <= N <= 2^30; M == 0 or N == 0: nothing
 *                enqueued.
 *  wq, w_scale, w_zero, fmt, group   the tiled storage as for w4a8_linear / w8a8_linear (svg_weight_sizes), wq 16-byte aligned.  w_scale
 *                and w_zero 4-byte.  fp16 zeros are whole numbers 0 .. 15, as rht_rotate_weights writes them.
 *  y             [M][N] of y_type (SVG_F32, SVG_F16, SVG_BF16), row-major, 4-byte aligned.
 *
 *  W8: y[m][n] = x_scale[m] * s[n] * S[m][n];  W4: x_scale[m] * sum_g s[n][g] * S_g[m][n]; the integer sums are exact, the rest fp32,
 *  then one rounding to y_type.  A row's W8 results do not depend on M and on the other rows; W4's sum over the groups
 *  may be taken in another order for another M.
 *  Errors: SVG_EINVAL for a null required pointer, M, N < 0 or K <= 0; SVG_EUNSUPPORTED for an unknown y_type, fmt or group, K, M, N, M * K
 *  of 2^40 or M * N of 2^39 or more; SVG_EALIGN.
 */
svg_status w4a8_prompt_linear(const int8_t* xq, const float* x_scale, int M, int K, const uint8_t* wq, const uint16_t* w_scale,
                              const void* w_zero, int fmt, int group, int N, void* y, int y_type, void* stream);
svg_status w8a8_prompt_linear(const int8_t* xq, const float* x_scale, int M, int K, const int8_t* wq, const uint16_t* w_scale, int N,
                              void* y, int y_type, void* stream);

/*
 * gated_quant_i8 -- the gated activation, rotation and int8 quantization of many rows in one launch: what stands in front
 * of a down projection, and without a gate in front of an output projection.
 *
 *  x, gate     M rows of K values of x_type (SVG_F32, SVG_F16, SVG_BF16), rows ld_x / ld_gate values apart, each 16-byte aligned
 *              (they may be halves of one product's rows); gate NULL: none, ld_gate is not read.
 *  M, K        M >= 0 (M <= 2^24; 0: nothing enqueued), K % block == 0, K <= 32768.
 *  signs, block, xq, x_scale   as for add_rmsnorm_quant_i8 (32-row slab buffers).
 *
 *  u = the fp32 number nearest to x * gate / (1 + exp(-gate)), computed in 64 bits (within 2^-50 of itself before that one
 *  rounding); u = x without a gate.  Then u as X in act_rht_quant_i8, bit for bit.
 *  Errors: SVG_EINVAL for a null required pointer, M < 0 or K <= 0; SVG_EUNSUPPORTED for a type, a block, K % block, K > 32768,
 *  M > 2^24, a row stride below K or of 2^31 or more; SVG_EALIGN.
 */
svg_status gated_quant_i8(const void* x, int64_t ld_x, const void* gate, int64_t ld_gate, int x_type, int M, int K, const int8_t* signs,
                          int block, int8_t* xq, float* x_scale, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SVGEMM_PROMPT_H */
