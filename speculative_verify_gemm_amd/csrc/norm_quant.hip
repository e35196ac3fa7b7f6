// Residual addition, root-mean-square norm, block Hadamard rotation and int8
// quantization of activation rows in one launch, gfx950.
//
// Per row: h = x + residual (written back), r = 1 / sqrt(sum h^2 / K + eps),
// u = (h * r) * w, then the rotation and the codes of svg_act.h.  Everything
// that decides a code is one IEEE fp32 operation, except r: the sum of the
// squares is kept in 64 bits (a product of two fp32 values is exact there, and
// the order of the additions no longer reaches the fp32 rounding of r), so the
// codes do not depend on how the row is split over threads.
//
// One workgroup owns a row and holds it in registers between its two
// reductions (sum, then maximum), so every input is read once and every output
// written once.  Few rows are bound by the chain of one load, two reductions
// and one store (one row of 4096 3.8 us, 16 rows with y 4.8 us, of which the launch is 2 to 3);
// many rows by memory (4099 rows of 4096, fp16 in: 39 to 44 us, 4.7 TB/s).
#include "svg_act.h"
#include "svg_device.h"
#include "svg_internal.h"

#pragma clang fp contract(off)

namespace {

struct NormArgs {
  const void* x;
  float* residual;
  const void* weight;
  const int8_t* signs;
  float* y;
  int8_t* xq;
  float* x_scale;
  double eps;
  int M, K, x_type, w_type;
};

template <int CTRL>
SVG_DEV double dpp_f64(double v) {
  const int2 b = *reinterpret_cast<const int2*>(&v);
  int2 o;
  o.x = __builtin_amdgcn_update_dpp(0, b.x, CTRL, 0xF, 0xF, false);
  o.y = __builtin_amdgcn_update_dpp(0, b.y, CTRL, 0xF, 0xF, false);
  return *reinterpret_cast<const double*>(&o);
}
SVG_DEV double lane_f64(double v, int lane) {
  const int2 b = *reinterpret_cast<const int2*>(&v);
  int2 o;
  o.x = __builtin_amdgcn_readlane(b.x, lane);
  o.y = __builtin_amdgcn_readlane(b.y, lane);
  return *reinterpret_cast<const double*>(&o);
}
// Sum over the wave, the same in every lane: the exchanges of wave_max.
SVG_DEV double wave_sum_f64(double v) {
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x124>(v);
  v += dpp_f64<0x128>(v);
  return (lane_f64(v, 0) + lane_f64(v, 16)) + (lane_f64(v, 32) + lane_f64(v, 48));
}

// A launch has fewer than 2^32 work-items a dimension: rows go on in y.
constexpr int kRowsX = 1 << 20;
static_assert(1024ull * kRowsX < (1ull << 32), "work-items of a row of the grid");

template <int NT, int CPT, int B>
__global__ __launch_bounds__(NT) void k_norm_quant(NormArgs a) {
  __shared__ double sums[16];
  __shared__ float red[16];
  const int m = (int)(blockIdx.y * kRowsX + blockIdx.x), K = a.K;
  if (m >= a.M) return;
  const u32 nchunk = (u32)K >> 2, tid = threadIdx.x;
  const u32 xb = a.x_type == SVG_F32 ? 4u : 2u, wb = a.w_type == SVG_F32 ? 4u : 2u;
  const rsrc_t xr = make_rsrc(static_cast<const char*>(a.x) + (size_t)m * K * xb, (u32)K * xb);
  const rsrc_t rr = make_rsrc(a.residual + (a.residual ? (size_t)m * K : 0), a.residual ? (u32)K * 4u : 0u);
  const rsrc_t wr = make_rsrc(a.weight, (u32)K * wb);
  const rsrc_t sr = make_rsrc(a.signs, (u32)K);
  RowRegs<CPT> r;
  float w[CPT][4], res[CPT][4];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const u32 c = tid + NT * i;
    load_chunk(xr, a.x_type, c, r.e[i]);
    load_chunk(rr, SVG_F32, c, res[i]);  // zeros without a residual
    load_chunk(wr, a.w_type, c, w[i]);
    r.sg[i] = (int)bload4(sr, c * 4u);
  }
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    if (a.residual) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r.e[i][j] = r.e[i][j] + res[i][j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) ss = __builtin_fma((double)r.e[i][j], (double)r.e[i][j], ss);
  }
  ss = wave_sum_f64(ss);
  if ((tid & 63u) == 0) sums[tid >> 6] = ss;
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const u32 c = tid + NT * i;
      if (c < nchunk)
        *reinterpret_cast<float4*>(a.residual + (size_t)m * K + 4 * c) =
            make_float4(r.e[i][0], r.e[i][1], r.e[i][2], r.e[i][3]);
    }
  }
  __syncthreads();
  ss = sums[0];
#pragma unroll
  for (int v = 1; v < NT / 64; ++v) ss += sums[v];
  const float rn = (float)(1.0 / sqrt(ss / (double)K + a.eps));
#pragma unroll
  for (int i = 0; i < CPT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) r.e[i][j] = (r.e[i][j] * rn) * w[i][j];
  if (a.y) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const u32 c = tid + NT * i;
      if (c < nchunk)
        *reinterpret_cast<float4*>(a.y + (size_t)m * K + 4 * c) =
            make_float4(r.e[i][0], r.e[i][1], r.e[i][2], r.e[i][3]);
    }
  }
  // the row's 32-row slab buffer
  const int first = m & ~31, rows = a.M - first < 32 ? a.M - first : 32;
  const StoreGlobal st(a.xq + (size_t)first * K, m - first, rows, a.x_scale + m, K);
  act_quant_loaded<CPT, StoreGlobal, B, true>(r, K, st, red);
}

// Few rows: as many threads as the row has chunks (the chain of one row is all there is).  Many rows: a row for
// 256 threads, so that a compute unit has several at different steps.  Measured (fp16 rows with a residual, back to back,
// few | many): K = 4096: 256 rows 5.6 | 5.7 us, 512 rows 8.1 | 6.9 us, 4099 rows (cold) 45.7 | 39.2 us (4.7 TB/s);
// K = 8192: 512 rows 11.1 | 11.8 us, 1024 rows 18.1 | 17.7 us.
template <int B>
void launch(const NormArgs& a, hipStream_t stream) {
  const int nchunk = a.K / 4;
  const dim3 grid(a.M < kRowsX ? a.M : kRowsX, (a.M + kRowsX - 1) / kRowsX);
#define SVG_NORM(NT, CPT) hipLaunchKernelGGL((k_norm_quant<NT, CPT, B>), grid, dim3(NT), 0, stream, a)
  if (nchunk <= 2048 && a.M >= (nchunk <= 1024 ? 512 : 1024)) {
    if (nchunk <= 256) SVG_NORM(256, 1);
    else if (nchunk <= 512) SVG_NORM(256, 2);
    else if (nchunk <= 1024) SVG_NORM(256, 4);
    else SVG_NORM(256, 8);
  } else if (nchunk <= 256) SVG_NORM(256, 1);
  else if (nchunk <= 512) SVG_NORM(512, 1);
  else if (nchunk <= 1024) SVG_NORM(1024, 1);
  else if (nchunk <= 2048) SVG_NORM(1024, 2);
  else if (nchunk <= 4096) SVG_NORM(1024, 4);
  else SVG_NORM(1024, 8);
#undef SVG_NORM
}

}  // namespace

hipError_t svg_launch_norm_quant(const void* x, int x_type, float* residual, const void* weight, int w_type,
                                 double eps, int M, int K, const int8_t* signs, int block, float* y, int8_t* xq,
                                 float* x_scale, hipStream_t stream) {
  const NormArgs a{x, residual, weight, signs, y, xq, x_scale, eps, M, K, x_type, w_type};
  if (block == 64) launch<64>(a, stream);
  else launch<32>(a, stream);
  return hipGetLastError();
}
