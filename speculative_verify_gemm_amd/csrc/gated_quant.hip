// The gated activation x * silu(gate), block Hadamard rotation and int8 quantization of activation rows in one
// launch, gfx950.
//
// u = x * gate / (1 + exp(-gate)) decides codes, so it is defined as one rounding of a 64-bit value and computed in
// fp64 here (its error there, below 2^-50, moves that rounding once in 2^25 values); the rotation and the codes are
// those of svg_act.h.  One workgroup owns a row and holds it in registers.
//
// Bound by vector instructions: about 63 a value with a gate, of which the gate is half and the rotation and the codes are the
// rest (4099 rows of 12288, bf16 halves of one product: 109 to 115 us, 2.3 TB/s, vector units busy 91 %; a table of 128 powers of two, which
// saves a third of the fp64 operations: 111 us), about 31 without one (4099 rows of 4096, fp16: 19 us, 2.6 TB/s, where a copy reaches
// 4.7; the instructions alone are about 13 of them); few rows by the chain of one load, a reduction and one store (40 rows of 4096: 4.1 us).
#include "../../include/svgemm_prompt.h"
#include "svg_act.h"
#include "svg_internal.h"

#pragma clang fp contract(off)

namespace {

struct GateArgs {
  const void *x, *gate;
  const int8_t* signs;
  int8_t* xq;
  float* x_scale;
  long ld_x, ld_gate;  // bytes
  int M, K, type;
};

// exp(y) for -745 <= y <= 709 within 2^-51 of itself: y = n ln 2 + r (ln 2 in two parts), a polynomial in r (Chebyshev
// interpolation of exp over |r| <= ln 2 / 2, off by 2^-56), the power of two put into the exponent.
SVG_DEV double exp_f64(double y) {
  const double n = rint(y * 1.4426950408889634);
  const double r = __builtin_fma(n, -1.9082149292705877e-10, __builtin_fma(n, -0.69314718036912382, y));
  double p = 2.51449546413054e-08;
  p = __builtin_fma(p, r, 2.7633231742717875e-07);
  p = __builtin_fma(p, r, 2.7557123950259445e-06);
  p = __builtin_fma(p, r, 2.480148370245139e-05);
  p = __builtin_fma(p, r, 0.00019841270034100182);
  p = __builtin_fma(p, r, 0.0013888888954182422);
  p = __builtin_fma(p, r, 0.008333333333240394);
  p = __builtin_fma(p, r, 0.041666666666480195);
  p = __builtin_fma(p, r, 0.16666666666666866);
  p = __builtin_fma(p, r, 0.500000000000002);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_ldexp(p, (int)n);
}
// x * g / (1 + exp(-g)), rounded once.  The exponential's argument stops where the result no longer changes.
SVG_DEV float gated(float x, float g) {
  const double d = 1.0 + exp_f64(fmax(fmin(-(double)g, 709.0), -745.0));
  double y = __builtin_amdgcn_rcp(d);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  return (float)((double)x * ((double)g * y));
}

// A launch has fewer than 2^32 work-items a dimension: rows go on in y.
constexpr int kRowsX = 1 << 20;

template <int NT, int CPT, int B>
__global__ __launch_bounds__(NT) void k_gated_quant(GateArgs a) {
  __shared__ float red[16];
  const int m = (int)(blockIdx.y * kRowsX + blockIdx.x), K = a.K;
  if (m >= a.M) return;
  const u32 tid = threadIdx.x, size = a.type == SVG_F32 ? 4u : 2u;
  const rsrc_t xr = make_rsrc(static_cast<const char*>(a.x) + m * a.ld_x, (u32)K * size);
  const rsrc_t gr = make_rsrc(static_cast<const char*>(a.gate) + (a.gate ? m * a.ld_gate : 0), a.gate ? (u32)K * size : 0u);
  const rsrc_t sr = make_rsrc(a.signs, (u32)K);
  RowRegs<CPT> r;
  float g[CPT][4];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const u32 c = tid + NT * i;
    load_chunk(xr, a.type, c, r.e[i]);
    load_chunk(gr, a.type, c, g[i]);
    r.sg[i] = (int)bload4(sr, c * 4u);
  }
  if (a.gate) {
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) r.e[i][j] = gated(r.e[i][j], g[i][j]);
  }
  // the row's 32-row slab buffer
  const int first = m & ~31, rows = a.M - first < 32 ? a.M - first : 32;
  const StoreGlobal st(a.xq + (size_t)first * K, m - first, rows, a.x_scale + m, K);
  act_quant_loaded<CPT, StoreGlobal, B, true>(r, K, st, red);
}

// As many threads as the row has chunks, up to 1024; many short rows: a row for 256 threads, so that a compute unit has several at
// different steps.  Measured (256 | 1024 threads): 4099 rows of 4096, fp16, no gate 18.6 | 25.3 us; 40 rows alike; longer rows gain
// nothing (1000 rows of 12288, fp32 with a gate: 37.6 | 32.2 us).
template <int B>
void launch(const GateArgs& a, hipStream_t stream) {
  const int nchunk = a.K / 4;
  const dim3 grid(a.M < kRowsX ? a.M : kRowsX, (a.M + kRowsX - 1) / kRowsX);
#define SVG_GATE(NT, CPT) hipLaunchKernelGGL((k_gated_quant<NT, CPT, B>), grid, dim3(NT), 0, stream, a)
  if (nchunk <= 256) SVG_GATE(256, 1);
  else if (nchunk <= 1024 && a.M >= 512) SVG_GATE(256, 4);
  else if (nchunk <= 512) SVG_GATE(512, 1);
  else if (nchunk <= 1024) SVG_GATE(1024, 1);
  else if (nchunk <= 2048) SVG_GATE(1024, 2);
  else if (nchunk <= 3 * 1024) SVG_GATE(1024, 3);
  else if (nchunk <= 4096) SVG_GATE(1024, 4);
  else SVG_GATE(1024, 8);
#undef SVG_GATE
}

}  // namespace

hipError_t svg_launch_gated_quant(const void* x, int64_t ld_x, const void* gate, int64_t ld_gate, int x_type, int M, int K,
                                  const int8_t* signs, int block, int8_t* xq, float* x_scale, hipStream_t stream) {
  const int size = x_type == SVG_F32 ? 4 : 2;
  const GateArgs a{x, gate, signs, xq, x_scale, ld_x * size, ld_gate * size, M, K, x_type};
  if (block == 64) launch<64>(a, stream);
  else launch<32>(a, stream);
  return hipGetLastError();
}
