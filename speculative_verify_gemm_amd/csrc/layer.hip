// C ABI entry points of svgemm_layer.h: host-side validation, then the launch.
#include "../../include/svgemm_layer.h"

#include <cmath>

#include "svg_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == SVG_F32 || t == SVG_F16 || t == SVG_BF16; }
hipStream_t to_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

int svg_check_cache(const char* fn, const svg_kv_cache* c, int needs) {
  if (!c) return svg_fail(SVG_EINVAL, fn, "null cache");
  if (!c->k || !c->v) return svg_fail(SVG_EINVAL, fn, "null cache pages");
  if (c->type != SVG_F16 && c->type != SVG_BF16) return svg_fail(SVG_EUNSUPPORTED, fn, "cache type must be fp16 or bf16");
  if (c->dim != 64 && c->dim != 128 && c->dim != 256) return svg_fail(SVG_EUNSUPPORTED, fn, "dim must be 64, 128 or 256");
  if (c->page != 32 && c->page != 64 && c->page != 128)
    return svg_fail(SVG_EUNSUPPORTED, fn, "page must be 32, 64 or 128");
  if (c->heads < 1 || c->heads > 1024) return svg_fail(SVG_EUNSUPPORTED, fn, "heads must be 1 .. 1024");
  if (c->n_pages < 1 || c->n_pages > (1 << 20)) return svg_fail(SVG_EUNSUPPORTED, fn, "n_pages must be 1 .. 2^20");
  if (c->n_layers < 1 || c->n_layers > 65535) return svg_fail(SVG_EUNSUPPORTED, fn, "n_layers must be 1 .. 65535");
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return svg_fail(SVG_EALIGN, fn, "cache pages need 16-byte alignment");
  if (!needs) return SVG_OK;
  if (c->n_slots < 0 || c->width < 0) return svg_fail(SVG_EINVAL, fn, "n_slots < 0 or width < 0");
  if (c->n_slots > 1024) return svg_fail(SVG_EUNSUPPORTED, fn, "n_slots > 1024");
  if ((int64_t)c->width * c->page > (1ll << 25))
    return svg_fail(SVG_EUNSUPPORTED, fn, "width * page > 2^25");
  if (c->n_slots == 0) return SVG_OK;
  const struct { int bit; const void* p; const char* null; } fields[] = {{kTable, c->table, "null table"},
                                                                          {kPages, c->pages, "null pages"},
                                                                          {kLen, c->len, "null len"},
                                                                          {kRefs, c->refs, "null refs"}};
  for (const auto& f : fields) {
    if (!(needs & f.bit)) continue;
    if (!f.p) return svg_fail(SVG_EINVAL, fn, f.null);
    if (!aligned(f.p, 4)) return svg_fail(SVG_EALIGN, fn, "table, pages, len and refs need 4-byte alignment");
  }
  return SVG_OK;
}

extern "C" {

svg_status add_rmsnorm_quant_i8(const void* x, int x_type, float* residual, const void* weight, int w_type,
                                double eps, int M, int K, const int8_t* signs, int block, float* y, int8_t* xq,
                                float* x_scale, void* stream) {
  static const char* fn = "add_rmsnorm_quant_i8";
  if (M < 0) return svg_fail(SVG_EINVAL, fn, "M < 0");
  if (K <= 0) return svg_fail(SVG_EINVAL, fn, "K <= 0");
  if (!(eps > 0.0) || !std::isfinite(eps)) return svg_fail(SVG_EINVAL, fn, "eps must be a positive finite number");
  if (!type_ok(x_type) || !type_ok(w_type)) return svg_fail(SVG_EUNSUPPORTED, fn, "unknown x_type or w_type");
  if (block != 32 && block != 64) return svg_fail(SVG_EUNSUPPORTED, fn, "block must be 32 or 64");
  if (K % block) return svg_fail(SVG_EUNSUPPORTED, fn, "K must be a multiple of block");
  if (K > 32768) return svg_fail(SVG_EUNSUPPORTED, fn, "K > 32768");
  if (M > (1 << 24)) return svg_fail(SVG_EUNSUPPORTED, fn, "M > 2^24");
  if (M == 0) return svg_ok();  // an empty call needs no buffers
  if (!x || !weight || !signs || !xq || !x_scale) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(y, 16) || !aligned(xq, 16))
    return svg_fail(SVG_EALIGN, fn, "x, residual, weight, y and xq need 16-byte alignment");
  if (!aligned(signs, 4) || !aligned(x_scale, 4))
    return svg_fail(SVG_EALIGN, fn, "signs / x_scale need 4-byte alignment");
  return svg_hip_status(fn, svg_launch_norm_quant(x, x_type, residual, weight, w_type, eps, M, K, signs, block, y, xq,
                                                  x_scale, reinterpret_cast<hipStream_t>(stream)));
}

svg_status kv_append(const svg_kv_cache* cache, int layer, const float* k, int64_t ld_k, const float* v, int64_t ld_v, int T,
                     const int32_t* n_rows, void* stream) {
  static const char* fn = "kv_append";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen)) return st;
  if (T < 1) return svg_fail(SVG_EINVAL, fn, "T < 1");
  if (layer < 0 || layer >= cache->n_layers) return svg_fail(SVG_EINVAL, fn, "layer outside the cache");
  const int64_t row = (int64_t)cache->heads * cache->dim;
  if ((int64_t)cache->n_slots * T >= (1ll << 31)) return svg_fail(SVG_EUNSUPPORTED, fn, "n_slots * T >= 2^31");
  if (ld_k < row || ld_v < row || ld_k % 4 || ld_v % 4 || ld_k >= (1ll << 31) || ld_v >= (1ll << 31))
    return svg_fail(SVG_EUNSUPPORTED, fn, "ld_k, ld_v must be multiples of 4, at least heads * dim and below 2^31");
  if (cache->n_slots == 0) return svg_ok();
  if (!k || !v) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(k, 16) || !aligned(v, 16)) return svg_fail(SVG_EALIGN, fn, "k and v need 16-byte alignment");
  if (!aligned(n_rows, 4)) return svg_fail(SVG_EALIGN, fn, "n_rows needs 4-byte alignment");
  return svg_hip_status(fn, svg_launch_kv_append(*cache, layer, k, ld_k, v, ld_v, T, n_rows, to_stream(stream)));
}

svg_status kv_commit(const svg_kv_cache* cache, int T, const int32_t* path, const int32_t* n_emit, int32_t* len_out,
                     void* stream) {
  static const char* fn = "kv_commit";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen)) return st;
  if (T < 1) return svg_fail(SVG_EINVAL, fn, "T < 1");
  if (T > SVG_TREE_MAX_NODES) return svg_fail(SVG_EUNSUPPORTED, fn, "T > SVG_TREE_MAX_NODES");
  if (cache->n_slots == 0) return svg_ok();
  if (!path || !n_emit || !len_out) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(path, 4) || !aligned(n_emit, 4) || !aligned(len_out, 4))
    return svg_fail(SVG_EALIGN, fn, "path, n_emit and len_out need 4-byte alignment");
  return svg_hip_status(fn, svg_launch_kv_commit(*cache, T, path, n_emit, len_out, to_stream(stream)));
}

svg_status kv_fork(const svg_kv_cache* cache, const int32_t* src, int32_t* table_out, int32_t* pages_out,
                   int32_t* len_out, void* stream) {
  static const char* fn = "kv_fork";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen | kRefs)) return st;
  if (cache->n_slots == 0) return svg_ok();
  if (!src || !table_out || !pages_out || !len_out) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (table_out == cache->table || pages_out == cache->pages || len_out == cache->len)
    return svg_fail(SVG_EINVAL, fn, "an output is its input");
  if (!aligned(src, 4) || !aligned(table_out, 4) || !aligned(pages_out, 4) || !aligned(len_out, 4))
    return svg_fail(SVG_EALIGN, fn, "src and the outputs need 4-byte alignment");
  return svg_hip_status(fn, svg_launch_kv_fork(*cache, src, table_out, pages_out, len_out, to_stream(stream)));
}

svg_status kv_reserve(const svg_kv_cache* cache, const int32_t* need, int32_t* status, void* workspace, void* stream) {
  static const char* fn = "kv_reserve";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen | kRefs)) return st;
  if (cache->n_slots == 0) return svg_ok();
  if (!need || !status || !workspace) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(need, 4) || !aligned(status, 4)) return svg_fail(SVG_EALIGN, fn, "need and status need 4-byte alignment");
  if (!aligned(workspace, 8)) return svg_fail(SVG_EALIGN, fn, "workspace needs 8-byte alignment");
  return svg_hip_status(fn, svg_launch_kv_reserve(*cache, need, status, workspace, to_stream(stream)));
}

svg_status kv_copy_pages(const svg_kv_cache* cache, const int32_t* src, const int32_t* dst, int n, void* stream) {
  static const char* fn = "kv_copy_pages";
  if (const svg_status st = svg_check_cache(fn, cache, 0)) return st;
  if (n < 0) return svg_fail(SVG_EINVAL, fn, "n < 0");
  if (n == 0) return svg_ok();
  if (!src || !dst) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(src, 4) || !aligned(dst, 4)) return svg_fail(SVG_EALIGN, fn, "src and dst need 4-byte alignment");
  return svg_hip_status(fn, svg_launch_kv_copy(*cache, src, dst, n, to_stream(stream)));
}

static svg_status check_heads(const char* fn, const svg_kv_cache* c, int q_heads, int T) {
  if (T < 1 || q_heads < 1) return svg_fail(SVG_EINVAL, fn, "T < 1 or q_heads < 1");
  if (T > SVG_TREE_MAX_NODES) return svg_fail(SVG_EUNSUPPORTED, fn, "T > SVG_TREE_MAX_NODES");
  if (q_heads % c->heads || q_heads > 4096)
    return svg_fail(SVG_EUNSUPPORTED, fn, "q_heads must be a multiple of the cache's heads, at most 4096");
  if (c->n_slots && !svg_tree_attention_fits(*c, T, q_heads / c->heads))
    return svg_fail(SVG_EUNSUPPORTED, fn, "too much work for one call: n_slots * width * page * heads * row blocks of 128 past 2^36");
  return SVG_OK;
}

svg_status tree_attention_workspace(const svg_kv_cache* cache, int q_heads, int T, uint64_t* bytes) {
  static const char* fn = "tree_attention_workspace";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen)) return st;
  if (const svg_status st = check_heads(fn, cache, q_heads, T)) return st;
  if (!bytes) return svg_fail(SVG_EINVAL, fn, "null bytes");
  *bytes = cache->n_slots ? svg_tree_attention_bytes(*cache, T, q_heads / cache->heads) : 0;
  return svg_ok();
}

svg_status tree_attention(const svg_kv_cache* cache, int layer, const float* q, int64_t ld_q, int q_heads, const int32_t* parent,
                          int T, const int32_t* n_nodes, const int32_t* shared, float scale, float* out, void* workspace,
                          void* stream) {
  static const char* fn = "tree_attention";
  if (const svg_status st = svg_check_cache(fn, cache, kTable | kPages | kLen)) return st;
  if (const svg_status st = check_heads(fn, cache, q_heads, T)) return st;
  if (layer < 0 || layer >= cache->n_layers) return svg_fail(SVG_EINVAL, fn, "layer outside the cache");
  if (!std::isfinite(scale)) return svg_fail(SVG_EINVAL, fn, "scale must be finite");
  if (ld_q < (int64_t)q_heads * cache->dim || ld_q % 4 || ld_q >= (1ll << 31))
    return svg_fail(SVG_EUNSUPPORTED, fn, "ld_q must be a multiple of 4, at least q_heads * dim and below 2^31");
  if (cache->n_slots == 0) return svg_ok();
  if (!q || !out || !workspace) return svg_fail(SVG_EINVAL, fn, "null required pointer");
  if (!aligned(q, 16) || !aligned(out, 16)) return svg_fail(SVG_EALIGN, fn, "q and out need 16-byte alignment");
  if (!aligned(workspace, 256)) return svg_fail(SVG_EALIGN, fn, "workspace needs 256-byte alignment");
  if (!aligned(parent, 4) || !aligned(n_nodes, 4) || !aligned(shared, 4))
    return svg_fail(SVG_EALIGN, fn, "parent, n_nodes and shared need 4-byte alignment");
  return svg_hip_status(fn, svg_launch_tree_attention(*cache, layer, q, ld_q, q_heads / cache->heads, parent, T, n_nodes,
                                                      shared, scale, out, workspace, to_stream(stream)));
}

}  // extern "C"
