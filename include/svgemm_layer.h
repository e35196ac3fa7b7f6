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

/*
 * svg_kv_cache -- a paged cache of keys and values and the slots that use it:
 * a host struct that every call below reads during the call only.
 *
 *  k, v      the pages of all layers, 16-byte aligned: page p of layer l of
 *            each starts at element (l * n_pages + p) * heads * page * dim.
 *  type      SVG_F16 or SVG_BF16.
 *  heads     key/value heads, 1 .. 1024.   dim   64, 128 or 256 values a head.
 *  page      tokens of a page: 32, 64 or 128.
 *  n_pages   1 .. 2^20.    n_layers  1 .. 65535.    n_slots  0 .. 1024 sequences.
 *  width     entries of a table row; width * page <= 2^25 tokens.
 *  table     int32 [n_slots][width]: the pages of a slot in token order; token t
 *            of slot s lies in page table[s][t / page], place t % page.
 *  pages     int32 [n_slots]: entries of each row that are in use.
 *  len       int32 [n_slots]: committed tokens of each slot.
 *  refs      int32 [n_pages]: the number of slots that hold each page; a page is
 *            free where it is 0.  A page that several slots hold (a count above 1) is never written but by
 *            kv_copy_pages, which goes by the page numbers that it is given.
 *  (table, pages, len, refs: 4-byte aligned.  Each call names the ones it needs.)
 *
 * A page holds head after head, page * dim values each, in the lane order of
 * the matrix instructions that read them (v_mfma_f32_16x16x32), so that a wave
 * reads 32 tokens of a head as contiguous KiB and needs no exchange:
 *   keys    value (t, d) is element ((t / 16) * (dim / 32) + d / 32) * 512
 *           + (16 * ((d % 32) / 8) + t % 16) * 8 + d % 8.
 *   values  value (t, d) is element ((t / 32) * (dim / 16) + d / 16) * 512
 *           + (16 * ((t % 16) / 4) + d % 16) * 8 + 4 * ((t % 32) / 16) + t % 4.
 */
typedef struct svg_kv_cache {
    void* k;
    void* v;
    int type, heads, dim, page, n_pages, n_layers, n_slots, width;
    int32_t* table;
    int32_t* pages;
    int32_t* len;
    int32_t* refs;
} svg_kv_cache;

/*
 * kv_append -- write the keys and values of new tokens behind the committed
 * ones of each slot, in one layer.  len does not change (kv_commit does that).
 *
 *  k, v      fp32 [n_slots * T] rows of heads * dim values, rows ld_k / ld_v
 *            values apart (a multiple of 4, >= heads * dim), 16-byte aligned: row
 *            s * T + i is token i of slot s, written to position len[s] + i, rounded to nearest (even) once.
 *  T         rows of each slot, >= 1.
 *  n_rows    int32 [n_slots] or NULL: rows of each slot that are written (the
 *            nearest of 0 .. T); NULL: all T.
 *  A row whose position is not inside the slot's pages, whose page number is not one of the cache's, or whose page
 *  other slots hold too (refs above 1: kv_reserve was not called, or refused the slot) is not written.
 *  Reads table, pages, len, and refs where it is not NULL (without it the caller sees to it that no page written is
 *  another slot's as well).  Errors: SVG_EINVAL for a null required pointer, T < 1 or a layer
 *  outside 0 .. n_layers - 1; SVG_EUNSUPPORTED for a cache outside the limits above, n_slots * T >= 2^31
 *  or ld_k / ld_v; SVG_EALIGN.
 */
svg_status kv_append(const svg_kv_cache* cache, int layer, const float* k, int64_t ld_k, const float* v, int64_t ld_v, int T,
                     const int32_t* n_rows, void* stream);

/*
 * kv_commit -- keep the accepted path of each slot's draft tree: its tokens move
 * together behind the root, in every layer, and the slot's length grows.
 *
 *  T         nodes of each slot's tree, 1 .. SVG_TREE_MAX_NODES: node i of slot s was
 *            appended at position len[s] + i.
 *  path      int32 [n_slots][T], n_emit int32 [n_slots]: as tree_accept_greedy writes
 *            them for each slot's tree (path rising node numbers below the root).
 *  len_out   int32 [n_slots]: len[s] + n_emit[s] (the root and the accepted nodes are
 *            committed); may be len itself.
 *  The token of node path[s][j] moves to position len[s] + 1 + j, j < n_emit[s] - 1.  A slot with
 *  n_emit outside 1 .. T, a path that is not rising inside 1 .. T - 1, or positions (the root's to the last accepted
 *  node's) outside its pages or in a page that other slots hold too keeps its tokens, and len_out[s] = len[s].
 *  Reads table, pages, len, and refs as kv_append does.  Errors as for kv_append.
 */
svg_status kv_commit(const svg_kv_cache* cache, int T, const int32_t* path, const int32_t* n_emit, int32_t* len_out,
                     void* stream);

/*
 * kv_fork -- give every slot the state of a slot: forking, keeping and freeing
 * in one call, as if all at once.
 *
 *  src       int32 [n_slots]: slot s becomes a fork of slot src[s]: it holds the pages of src[s]'s
 *            committed tokens (the last one may be partly filled) and has its length; its own
 *            pages are given up.  src[s] == s keeps the slot as it is; -1 frees it (no pages, length
 *            0); any other number outside 0 .. n_slots - 1 keeps it.
 *  cache     read: table, pages, len.   refs is updated (one count for each slot that holds a page).
 *  table_out, pages_out, len_out   the new tables, of the sizes of table, pages and len, and not
 *            these themselves.  Entries of table_out behind a row's pages_out are left as they were.
 *  No page is copied: kv_reserve does that for those that a fork writes to.  A tree that has been appended is committed
 *  before its slot is forked: the page that the fork then holds as well is not written any more, by kv_commit neither.
 *  Errors as for kv_append, and SVG_EINVAL where an output is its input.
 */
svg_status kv_fork(const svg_kv_cache* cache, const int32_t* src, int32_t* table_out, int32_t* pages_out,
                   int32_t* len_out, void* stream);

/*
 * kv_reserve -- make room: after it, the tokens len[s] .. len[s] + need[s] - 1 of each slot
 * lie in pages that no other slot holds.
 *
 *  need      int32 [n_slots]; a slot with need < 1 is left as it is.
 *  status    OUTPUT int32 [n_slots]: 0 done; 1 not enough free pages; 2 more than a table row holds, or
 *            a slot whose pages, length or last page number is not valid.  A slot with 1 or 2 is left as it was, and
 *            takes no part in a step until it has room: its n_rows, n_nodes and n_emit are to be 0.  (Otherwise the calls
 *            pass over what has no place of its own, and what it has room for is written and committed.)
 *  workspace SVG_KV_WORKSPACE_BYTES(n_slots) bytes, 8-byte aligned; its contents need not be kept.  Calls that
 *            may overlap need different ones (and may not share refs).
 *  The slots are served in order.  Where the page of token len - 1 is partly filled and other slots hold it too
 *  (refs > 1 when the slot's turn comes), a free page takes its place and its contents in every layer; then
 *  pages are added behind.  Each page taken is the free one with the lowest number.
 *  Updates table, pages, refs.  Errors as for kv_append.
 */
#define SVG_KV_WORKSPACE_BYTES(n_slots) (8 * (uint64_t)(n_slots) + 16)
svg_status kv_reserve(const svg_kv_cache* cache, const int32_t* need, int32_t* status, void* workspace, void* stream);

/*
 * kv_copy_pages -- copy page src[i] to page dst[i], i < n, in every layer (to compact a
 * pool, or to keep a copy).  The pages of dst are different ones, and none of them is in src.  A
 * pair with a number outside 0 .. n_pages - 1 is passed over.  Reads no table.
 *  Errors as for kv_append, and SVG_EINVAL for n < 0 (n == 0: nothing enqueued).
 */
svg_status kv_copy_pages(const svg_kv_cache* cache, const int32_t* src, const int32_t* dst, int n, void* stream);

/*
 * tree_attention -- attention of the draft trees of all slots over the cache, in
 * one layer: the keys and values of a tree's nodes have been appended
 * (kv_append) and are not committed yet.  Plain decoding is a tree of one node.
 *
 *  q         fp32 [n_slots * T] rows of q_heads * dim values, rows ld_q values apart (a multiple
 *            of 4, >= q_heads * dim), 16-byte aligned: row s * T + i is node i of slot s, whose key and
 *            value lie at position len[s] + i.
 *  q_heads   a multiple of heads: query head a reads key/value head a / (q_heads / heads); at most 4096.
 *  parent    int32 [n_slots][T]: parent[s][0] = -1, 0 <= parent[s][i] < i (as tree_accept_greedy);
 *            NULL: parent[i] = i - 1, a chain.
 *  T         nodes of a slot, 1 .. SVG_TREE_MAX_NODES.
 *  n_nodes   int32 [n_slots] or NULL: nodes of each slot (the nearest of 0 .. T; 0: the slot is
 *            idle); NULL: all T.  Behind a slot's nodes rows of q do not matter and rows of out are left as they were.
 *  shared    int32 [1] or NULL: a number of leading tokens that are the same pages in the
 *            table rows of all slots that are not idle (as after kv_fork).  They are read once for
 *            every 128 rows of a head (slots * T * query heads of it).  What is used is the largest
 *            multiple of 32 that neither this number nor any of those slots' len is below; it does not
 *            change what is computed.
 *  scale     finite; the scores are scale * q . k.
 *  out       fp32 [n_slots * T][q_heads * dim], 16-byte aligned.
 *  workspace tree_attention_workspace() bytes, 256-byte aligned; its contents need not be set or kept.
 *            Calls that may overlap need different ones.
 *
 *  Row (s, i, a): o = sum_t p_t v_t / sum_t p_t, p_t = exp(scale * q . k_t), over the positions t < len[s] and
 *  len[s] + j for the nodes j of i's root path, i included.  Sums and accumulators are fp32; q and p
 *  enter the 16-bit matrix products in parts.  A value of q is off by 2^-22 of itself or 2^-38 of its row's largest,
 *  whichever is more (fp16), or 2^-24 of itself (bf16).  A p carries at least 16 bits; with an fp16 cache it also
 *  loses up to 2^-36 of the largest that its wave has seen for the row, for each token of the wave's (long calls are
 *  spread over 512 waves and more: 131072 tokens of 8 heads lose up to 2^-25 in all, what the whole memory holds 2^-15).  Without
 *  that an output is within about 1e-5 of its row's largest |v| of an exact one while scores stay below about 50 (2^-22
 *  of a score is an error of its exponential, as in fp32).
 *  Keys and values of tokens that a row does not see never reach it, whatever they are.  Of those it sees (kv_append rounds
 *  what an fp16 cache cannot hold to infinity): a key that is not finite gives a NaN row where a score is NaN or
 *  +infinity, and may where it is -infinity, which by the definition only leaves the token out (the parts of q decide);
 *  a value that is not finite makes its own element of the row NaN or infinite (unless the token's p is small enough to
 *  be lost, see above), and no other.
 *  NaN rows: a node whose root path breaks the rule above, or meets a node in a page that other slots hold too (which
 *  kv_append has passed over); a row that reads a page number outside the cache; all of a slot whose pages do not cover
 *  len + n_nodes.
 *  Reads table, pages, len, and refs where it is not NULL (without it no node is passed over).
 *  Errors: SVG_EINVAL for a null required pointer, T < 1, q_heads < 1, a layer outside the cache or a scale that is not
 *  finite; SVG_EUNSUPPORTED for a cache outside its limits, T > SVG_TREE_MAX_NODES, q_heads, ld_q, or a table so large that
 *  n_slots * width * page * heads times the blocks of 128 rows of an item nears 2^36; SVG_EALIGN.
 *
 * tree_attention_workspace -- the bytes of that workspace (host only).
 */
#define SVG_ATTN_MAX_GROUPS 512
svg_status tree_attention_workspace(const svg_kv_cache* cache, int q_heads, int T, uint64_t* bytes);
svg_status tree_attention(const svg_kv_cache* cache, int layer, const float* q, int64_t ld_q, int q_heads, const int32_t* parent,
                          int T, const int32_t* n_nodes, const int32_t* shared, float scale, float* out, void* workspace,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SVGEMM_LAYER_H */
