// C ABI entry points of svgemm_layer.h: host-side validation, then the launch.
#include "../../include/svgemm_layer.h"

#include <cmath>

#include "svg_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int t) { return t == SVG_F32 || t == SVG_F16 || t == SVG_BF16; }

}  // namespace

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

}  // extern "C"
