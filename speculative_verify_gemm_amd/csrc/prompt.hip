// C ABI entry points of svgemm_prompt.h: host-side validation, then the launch.
#include "../../include/svgemm_prompt.h"

#include <cmath>

#include "svg_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == SVG_F32 || t == SVG_F16 || t == SVG_BF16; }
hipStream_t to_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
// Rows of `width` values `ld` apart: whether the stride is one (n rows), and whether each row is 16-byte aligned.
bool stride_ok(int64_t ld, int64_t width) { return ld >= width && ld < (1ll << 31); }
bool rows_aligned(const void* p, int64_t ld, int64_t n, int type) {
  return aligned(p, 16) && (n <= 1 || (ld * (type == SVG_F32 ? 4 : 2)) % 16 == 0);
}

svg_status check_linear(const char* fn, const void* xq, const void* x_scale, int64_t M, int64_t K, const void* wq, const void* w_scale,
                        int N, const void* y, int y_type) {
  if (M < 0 || N < 0) return svg_fail(SVG_EINVAL, fn, "M < 0 or N < 0");
  if (K <= 0) return svg_fail(SVG_EINVAL, fn, "K <= 0");
  if (!type_ok(y_type)) return svg_fail(SVG_EUNSUPPORTED, fn, "unknown y_type");
  if (K % 32 || K > 131072) return svg_fail(SVG_EUNSUPPORTED, fn, "K must be a multiple of 32, at most 131072");
  if (M > (1 << 24) || M * K >= (1ll << 40)) return svg_fail(SVG_EUNSUPPORTED, fn, "M > 2^24 or M * K >= 2^40");
  if (N > (1 << 30)) return svg_fail(SVG_EUNSUPPORTED, fn, "N > 2^30");
  if ((M + 15) / 16 * ((N + 15ll) / 16) >= (1ll << 31)) return svg_fail(SVG_EUNSUPPORTED, fn, "M * N past 2^39");
  if (M == 0 || N == 0) return SVG_OK;
  if (!xq || !x_scale || !wq || !w_scale || !y) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(xq, 16) || !aligned(wq, 16)) return svg_fail(SVG_EALIGN, fn, "xq and wq need 16-byte alignment");
  if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(y, 4))
    return svg_fail(SVG_EALIGN, fn, "x_scale, w_scale and y need 4-byte alignment");
  return SVG_OK;
}

}  // namespace

extern "C" {

svg_status kv_row_map(const svg_kv_cache* cache, const int32_t* n_new, const int32_t* parent, int T, int n_rows, int32_t* start,
                      int32_t* count, int32_t* slot, int32_t* pos, int32_t* place, void* stream) {
  static const char* fn = "kv_row_map";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen)) return st;
  if (T < 0 || n_rows < 0) return svg_fail(SVG_EINVAL, fn, "T < 0 or n_rows < 0");
  if (parent && T == 0) return svg_fail(SVG_EINVAL, fn, "trees need T >= 1 rows a slot");
  if (parent && T > SVG_TREE_MAX_NODES) return svg_fail(SVG_EUNSUPPORTED, fn, "T > SVG_TREE_MAX_NODES");
  if ((int64_t)cache->n_slots * T >= (1ll << 31)) return svg_fail(SVG_EUNSUPPORTED, fn, "n_slots * T >= 2^31");
  if (T > 0 && (int64_t)cache->n_slots * T != n_rows) return svg_fail(SVG_EINVAL, fn, "n_rows must be n_slots * T");
  if (cache->n_slots == 0 && n_rows == 0) return svg_ok();
  if ((cache->n_slots > 0 && (!n_new || !start || !count)) || (n_rows > 0 && (!pos || !place)))
    return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(n_new, 4) || !aligned(parent, 4) || !aligned(start, 4) || !aligned(count, 4) || !aligned(slot, 4) || !aligned(pos, 4) ||
      !aligned(place, 4))
    return svg_fail(SVG_EALIGN, fn, "n_new, parent and the outputs need 4-byte alignment");
  return svg_hip_status(fn, svg_launch_kv_row_map(*cache, n_new, parent, T, n_rows, start, count, slot, pos, place, to_stream(stream)));
}

svg_status rope_append(const svg_kv_cache* cache, int layer, const svg_rope* rope, const void* q, int64_t ld_q, int q_heads,
                       const void* k, int64_t ld_k, const void* v, int64_t ld_v, int x_type, int n_rows, const int32_t* pos,
                       const int32_t* place, void* q_out, int q_type, void* stream) {
  static const char* fn = "rope_append";
  if (const svg_status st = svg_check_cache(fn, cache, 0)) return st;
  if (!rope) return svg_fail(SVG_EINVAL, fn, "null rope");
  if (n_rows < 0 || q_heads < 0) return svg_fail(SVG_EINVAL, fn, "n_rows < 0 or q_heads < 0");
  if (layer < 0 || layer >= cache->n_layers) return svg_fail(SVG_EINVAL, fn, "layer outside the cache");
  if (!std::isfinite(rope->amplitude)) return svg_fail(SVG_EINVAL, fn, "amplitude must be finite");
  if (!type_ok(x_type)) return svg_fail(SVG_EUNSUPPORTED, fn, "unknown x_type");
  if (q_type != SVG_F32 && q_type != cache->type) return svg_fail(SVG_EUNSUPPORTED, fn, "q_type must be fp32 or the cache's type");
  if (rope->rot < 16 || rope->rot > cache->dim || rope->rot % 16)
    return svg_fail(SVG_EUNSUPPORTED, fn, "rot must be a multiple of 16, 16 .. dim");
  if (q_heads > 4096) return svg_fail(SVG_EUNSUPPORTED, fn, "q_heads > 4096");
  const int64_t row = (int64_t)cache->heads * cache->dim, q_row = (int64_t)q_heads * cache->dim;
  if ((q_heads && !stride_ok(ld_q, q_row)) || !stride_ok(ld_k, row) || !stride_ok(ld_v, row))
    return svg_fail(SVG_EUNSUPPORTED, fn, "ld_q, ld_k, ld_v must be at least a row and below 2^31");
  if (n_rows == 0) return svg_ok();
  if (!rope->freq || !k || !v || !pos || !place || (q_heads && (!q || !q_out))) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if ((q_heads && (!rows_aligned(q, ld_q, n_rows, x_type) || !aligned(q_out, 16))) || !rows_aligned(k, ld_k, n_rows, x_type) ||
      !rows_aligned(v, ld_v, n_rows, x_type))
    return svg_fail(SVG_EALIGN, fn, "rows of q, k, v and q_out need 16-byte alignment");
  if (!aligned(rope->freq, 8) || !aligned(pos, 4) || !aligned(place, 4))
    return svg_fail(SVG_EALIGN, fn, "freq needs 8-byte, pos and place 4-byte alignment");
  return svg_hip_status(fn, svg_launch_rope_append(*cache, layer, *rope, q, ld_q, q_heads, k, ld_k, v, ld_v, x_type, n_rows, pos, place,
                                                   q_out, q_type, to_stream(stream)));
}

static svg_status check_prompt(const char* fn, const svg_kv_cache* c, int q_heads, int n_rows) {
  if (n_rows < 0 || q_heads < 1) return svg_fail(SVG_EINVAL, fn, "n_rows < 0 or q_heads < 1");
  if (q_heads % c->heads || q_heads > 4096)
    return svg_fail(SVG_EUNSUPPORTED, fn, "q_heads must be a multiple of the cache's heads, at most 4096");
  if ((int64_t)n_rows * (q_heads / c->heads) >= (1ll << 30)) return svg_fail(SVG_EUNSUPPORTED, fn, "n_rows * (q_heads / heads) >= 2^30");
  return SVG_OK;
}

svg_status prompt_attention_workspace(const svg_kv_cache* cache, int q_heads, int n_rows, uint64_t* bytes) {
  static const char* fn = "prompt_attention_workspace";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen)) return st;
  if (const svg_status st = check_prompt(fn, cache, q_heads, n_rows)) return st;
  if (!bytes) return svg_fail(SVG_EINVAL, fn, "null bytes");
  *bytes = cache->n_slots && n_rows ? svg_prompt_attention_bytes(*cache) : 0;
  return svg_ok();
}

svg_status prompt_attention(const svg_kv_cache* cache, int layer, const void* q, int64_t ld_q, int q_heads, int n_rows,
                            const int32_t* start, const int32_t* count, float scale, void* out, void* workspace, void* stream) {
  static const char* fn = "prompt_attention";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen)) return st;
  if (const svg_status st = check_prompt(fn, cache, q_heads, n_rows)) return st;
  if (layer < 0 || layer >= cache->n_layers) return svg_fail(SVG_EINVAL, fn, "layer outside the cache");
  if (!std::isfinite(scale)) return svg_fail(SVG_EINVAL, fn, "scale must be finite");
  if (!stride_ok(ld_q, (int64_t)q_heads * cache->dim)) return svg_fail(SVG_EUNSUPPORTED, fn, "ld_q must be at least a row and below 2^31");
  if (cache->n_slots == 0 || n_rows == 0) return svg_ok();
  if (!q || !out || !start || !count || !workspace) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!rows_aligned(q, ld_q, n_rows, cache->type) || !aligned(out, 16))
    return svg_fail(SVG_EALIGN, fn, "rows of q and out need 16-byte alignment");
  if (!aligned(start, 4) || !aligned(count, 4)) return svg_fail(SVG_EALIGN, fn, "start and count need 4-byte alignment");
  if (!aligned(workspace, 256)) return svg_fail(SVG_EALIGN, fn, "workspace needs 256-byte alignment");
  return svg_hip_status(fn, svg_launch_prompt_attention(*cache, layer, q, ld_q, q_heads / cache->heads, n_rows, start, count, scale, out,
                                                        workspace, to_stream(stream)));
}

svg_status w4a8_prompt_linear(const int8_t* xq, const float* x_scale, int M, int K, const uint8_t* wq, const uint16_t* w_scale,
                              const void* w_zero, int fmt, int group, int N, void* y, int y_type, void* stream) {
  static const char* fn = "w4a8_prompt_linear";
  if (fmt != SVG_W4_ASYM_Z4 && fmt != SVG_W4_ASYM_Z16) return svg_fail(SVG_EUNSUPPORTED, fn, "fmt must be a 4-bit one");
  if (group != 32 && group != 64 && group != 128) return svg_fail(SVG_EUNSUPPORTED, fn, "group must be 32, 64 or 128");
  if (const svg_status st = check_linear(fn, xq, x_scale, M, K, wq, w_scale, N, y, y_type)) return st;
  if (K % group) return svg_fail(SVG_EUNSUPPORTED, fn, "K must be a multiple of group");
  if (M == 0 || N == 0) return svg_ok();
  if (!w_zero) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(w_zero, 4)) return svg_fail(SVG_EALIGN, fn, "w_zero needs 4-byte alignment");
  return svg_hip_status(fn, svg_launch_prompt_w4(xq, x_scale, M, K, wq, w_scale, w_zero, fmt == SVG_W4_ASYM_Z4, group, N, y, y_type,
                                                 to_stream(stream)));
}

svg_status w8a8_prompt_linear(const int8_t* xq, const float* x_scale, int M, int K, const int8_t* wq, const uint16_t* w_scale, int N,
                              void* y, int y_type, void* stream) {
  static const char* fn = "w8a8_prompt_linear";
  if (const svg_status st = check_linear(fn, xq, x_scale, M, K, wq, w_scale, N, y, y_type)) return st;
  if (M == 0 || N == 0) return svg_ok();
  return svg_hip_status(fn, svg_launch_prompt_w8(xq, x_scale, M, K, wq, w_scale, N, y, y_type, to_stream(stream)));
}

svg_status gated_quant_i8(const void* x, int64_t ld_x, const void* gate, int64_t ld_gate, int x_type, int M, int K, const int8_t* signs,
                          int block, int8_t* xq, float* x_scale, void* stream) {
  static const char* fn = "gated_quant_i8";
  if (M < 0) return svg_fail(SVG_EINVAL, fn, "M < 0");
  if (K <= 0) return svg_fail(SVG_EINVAL, fn, "K <= 0");
  if (!type_ok(x_type)) return svg_fail(SVG_EUNSUPPORTED, fn, "unknown x_type");
  if (block != 32 && block != 64) return svg_fail(SVG_EUNSUPPORTED, fn, "block must be 32 or 64");
  if (K % block) return svg_fail(SVG_EUNSUPPORTED, fn, "K must be a multiple of block");
  if (K > 32768) return svg_fail(SVG_EUNSUPPORTED, fn, "K > 32768");
  if (M > (1 << 24)) return svg_fail(SVG_EUNSUPPORTED, fn, "M > 2^24");
  if (!stride_ok(ld_x, K) || (gate && !stride_ok(ld_gate, K)))
    return svg_fail(SVG_EUNSUPPORTED, fn, "ld_x, ld_gate must be at least K and below 2^31");
  if (M == 0) return svg_ok();
  if (!x || !signs || !xq || !x_scale) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!rows_aligned(x, ld_x, M, x_type) || (gate && !rows_aligned(gate, ld_gate, M, x_type)) || !aligned(xq, 16))
    return svg_fail(SVG_EALIGN, fn, "rows of x and gate, and xq, need 16-byte alignment");
  if (!aligned(signs, 4) || !aligned(x_scale, 4)) return svg_fail(SVG_EALIGN, fn, "signs / x_scale need 4-byte alignment");
  return svg_hip_status(fn, svg_launch_gated_quant(x, ld_x, gate, ld_gate, x_type, M, K, signs, block, xq, x_scale, to_stream(stream)));
}

}  // extern "C"
