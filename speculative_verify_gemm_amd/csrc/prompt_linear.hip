// y = x . W^T of many int8 activation rows against the tiled int8 or 4-bit weights, gfx950.
#include "../../include/svgemm_prompt.h"
#include "svg_cache.h"
#include "svg_internal.h"
#include "svg_lds.h"

#pragma clang fp contract(off)

namespace {

struct Args {
  const int8_t* xq;
  const float* x_scale;
  const char* wq;
  const uint16_t* w_scale;
  const char* w_zero;
  void* y;
  int M, N, K, y_type;
  int tiles_m, tiles_n;
};

typedef float f32x4 __attribute__((ext_vector_type(4)));

// Weight formats: kStep values of K a step; kX fragments of 16 x 64 activation codes in one.
struct W8 {
  static constexpr int kStep = 64, kX = 1, kParams = 0;
  static constexpr bool k4 = false;
  typedef v4i Acc;
};
SVG_DEV v4i mfma(u32x4 a, u32x4 b, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
}

// Codes 0 .. 15 of the low nibbles less their zero points (the same in every byte of z), as int8: no byte borrows.
SVG_DEV u32 less(u32 codes, u32 z) { return (((codes & 0x0F0F0F0Fu) | 0x80808080u) - z) ^ 0x80808080u; }

template <int G, bool Z4_>
struct W4 {
  static constexpr int kStep = 128, kX = 2, kGroup = G;
  static constexpr bool k4 = true, kZ4 = Z4_;
  // dwords of scales and of zeros that a row has in a step
  static constexpr int kS = G == 32 ? 2 : 1, kZ = G == 32 && !Z4_ ? 2 : 1, kParams = kS + kZ;
  static constexpr u32 kRow = 16 * (512 / G) * 2;  // bytes of scales of 16 rows and 512 values of K
  // first byte of a step's dword in a row's 512 values (4-bit zeros: of the row's dword; two rows of groups of 128 share one)
  SVG_DEV static u32 scale_at(int s) { return G == 32 ? s * 8u : (G == 64 ? s * 4u : (s >> 1) * 4u); }
  SVG_DEV static u32 zero_at(int s) { return G == 32 ? (s >> 1) * 4u : 0u; }
  typedef f32x4 Acc;
  // the zero point of the 16 values that a lane holds of half h of step s (of four in 512 values)
  SVG_DEV static u32 zero(const u32* word, int s, int h, int lane) {
    const int b = lane >> 5;  // which half of 64 values
    if constexpr (Z4_) {
      const int at = G == 64 ? 2 * s + h : (G == 128 ? 4 * (lane & 1) + s : 4 * (s & 1) + 2 * h + b);
      return (word[0] >> (4 * at)) & 15u;
    } else {
      const u32 w = G == 32 ? word[h] : word[0];
      const int hi = G == 64 ? h : (G == 128 ? s & 1 : b);
      return (u32)(int)half_bits_to_float((uint16_t)(hi ? w >> 16 : w & 0xFFFFu)) & 15u;
    }
  }
  template <int TM, int TN>
  SVG_DEV static void product(const u32x4 (&x)[TM][2], const u32x4 (&w)[2], const u32* word, int s, int lane, Acc (&acc)[TM][TN], int j) {
    const v4i none{};
    if constexpr (G == 128) {
      const float sc = half_bits_to_float((uint16_t)(s & 1 ? word[0] >> 16 : word[0] & 0xFFFFu));
#pragma unroll
      for (int i = 0; i < TM; ++i) add(acc[i][j], mfma(x[i][1], w[1], mfma(x[i][0], w[0], none)), sc);
    } else if constexpr (G == 64) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float sc = half_at(word, h);
#pragma unroll
        for (int i = 0; i < TM; ++i) add(acc[i][j], mfma(x[i][h], w[h], none), sc);
      }
    } else {
      // groups of 32: half the lanes' weights at a time
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float sc = half_at(word, q);
        u32x4 part = w[q >> 1];
        if ((lane >> 5) != (q & 1)) part = u32x4{};
#pragma unroll
        for (int i = 0; i < TM; ++i) add(acc[i][j], mfma(x[i][q >> 1], part, none), sc);
      }
    }
  }
  SVG_DEV static void add(Acc& to, v4i sum, float scale) {
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = __builtin_fmaf((float)sum[e], scale, to[e]);
  }
};

// 4 bytes a lane from global memory straight into LDS (256 bytes from `to` on), as load_to_lds.
SVG_DEV void load4_to_lds(const char* from, u32 lane4, u32 to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               ::"s"(__builtin_amdgcn_readfirstlane((int)to)), "v"(lane4), "s"(from) : "memory");
}
SVG_DEV u32 round_to(int type, float v) {
  return type == SVG_F16 ? kv_round<false>(v) : kv_round<true>(v);
}

template <class F, int WM, int WN, int TM, int TN, int STAGES>
__global__ __launch_bounds__(64 * WM * WN) void k_prompt_linear(Args a) {
  constexpr int WAVES = WM * WN, MF = WM * TM, NF = WN * TN;          // fragments of 16 rows, of 16 columns
  constexpr int FRAGS = NF + MF * F::kX;                              // KiB of a stage
  constexpr int PARAMS = F::k4 ? NF / 4 * F::kParams : 0;             // 256-byte loads of parameters
  constexpr int STAGE = FRAGS * 1024 + PARAMS * 256;
  static_assert(FRAGS % WAVES == 0 && (PARAMS == 0 || PARAMS <= WAVES), "loads of a wave");
  constexpr int LOADS = FRAGS / WAVES;
  __shared__ __attribute__((aligned(1024))) char lds[STAGES * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
  const u32 base = lds_at(lds);
  const int steps = (a.K + F::kStep - 1) / F::kStep, slabs = a.K >> 5;
  // tiles: every XCD takes a stretch of them, by columns inside groups of 8 tile rows
  const u32 total = (u32)a.tiles_m * (u32)a.tiles_n, per = total >> 3, more = total & 7u;
  const u32 xcd = blockIdx.x & 7u, t = xcd * per + (xcd < more ? xcd : more) + (blockIdx.x >> 3);
  const u32 group = t / (8u * a.tiles_n), in = t % (8u * a.tiles_n);
  const u32 rows_in = (u32)a.tiles_m - group * 8 < 8 ? (u32)a.tiles_m - group * 8 : 8;
  const int m0 = (int)(group * 8 + in % rows_in) * MF * 16, n0 = (int)(in / rows_in) * NF * 16;

  // this wave's fragments of a stage: number wave + i * WAVES, first the weights', then the activations'
  const char* wbase = a.wq + (size_t)(n0 >> 4) * steps * 1024;
  const char* xbase = reinterpret_cast<const char*>(a.xq) + (size_t)m0 * a.K;
  const int last_tile = ((a.N + 15) >> 4) - 1 - (n0 >> 4);
  u32 off[LOADS], stride[LOADS];
#pragma unroll
  for (int i = 0; i < LOADS; ++i) {
    const int f = wave + i * WAVES;
    if (f < NF) {
      off[i] = (u32)(f < last_tile ? f : last_tile) * (u32)steps * 1024u + lane * 16u;
      stride[i] = 1024u;
    } else {
      const int j = (f - NF) / F::kX, h = (f - NF) % F::kX, kb = lane >> 4;
      int m = m0 + 16 * j + (lane & 15);
      m = m < a.M ? m : a.M - 1;
      const int buf = m & ~31, R = a.M - buf < 32 ? a.M - buf : 32;
      off[i] = (u32)(buf - m0) * (u32)a.K + ((u32)(2 * h + (kb >> 1)) * R + (m & 31)) * 32u + (kb & 1) * 16u;
      stride[i] = (u32)R * (F::kStep == 64 ? 64u : 128u);
    }
  }
  // parameters: load number p brings one dword of 64 rows, of kind p / (NF / 4); waves below PARAMS have one each
  const char* pbase = nullptr;
  u32 poff = 0;
  if constexpr (F::k4) {
    const int kind = wave / (NF / 4), tile = wave % (NF / 4) * 4 + (lane >> 4);
    const u32 blocks = (u32)(a.K + 511) >> 9, row = (u32)(tile < last_tile ? tile : last_tile) * blocks * 16u + (lane & 15);
    if (kind < F::kS) {
      pbase = reinterpret_cast<const char*>(a.w_scale) + (size_t)(n0 >> 4) * blocks * F::kRow;
      poff = row * (F::kRow / 16) + 4u * kind;
    } else {
      constexpr u32 zrow = F::kZ4 ? F::kRow / 64 : F::kRow / 16;
      pbase = a.w_zero + (size_t)(n0 >> 4) * blocks * (zrow * 16u);
      poff = (row * zrow & ~3u) + 4u * (kind - F::kS);
    }
  }
  auto fetch = [&](int s) {
    const u32 to = base + (u32)(s % STAGES) * STAGE;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int f = wave + i * WAVES;
      u32 o = off[i] + (u32)s * stride[i];
      if (f >= NF) {
        // K's last slabs may be missing: any codes do, the weights there are zero
        const int slab = s * (F::kStep / 32) + (F::kX == 2 ? 2 * ((f - NF) & 1) : 0) + (lane >> 5);
        if (slab >= slabs) o -= (u32)(slab - slabs + 1) * (stride[i] / (F::kStep / 32));
      }
      load_to_lds(f < NF ? wbase : xbase, o, to + (u32)f * 1024u);
    }
    if constexpr (F::k4) {
      if (wave < PARAMS) {
        const u32 o = poff + (u32)(s >> 2) * (wave / (NF / 4) < F::kS || !F::kZ4 ? F::kRow : F::kRow / 4);
        const u32 in_block = wave / (NF / 4) < F::kS || !F::kZ4 ? F::scale_at(s & 3) : F::zero_at(s & 3);
        load4_to_lds(pbase, o + in_block, to + FRAGS * 1024 + wave * 256);
      }
    }
  };
  typename F::Acc acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = typename F::Acc{};
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < steps) fetch(s);
  for (int s = 0; s < steps; ++s) {
    if (s + STAGES - 2 >= steps) wait_loads<0>();
    else if (PARAMS > 0 && wave < PARAMS) wait_loads<(LOADS + 1) * (STAGES - 2)>();
    else wait_loads<LOADS * (STAGES - 2)>();
    barrier();
    if (s + STAGES - 1 < steps) fetch(s + STAGES - 1);
    const char* at = lds + (s % STAGES) * STAGE + lane * 16;
    if constexpr (!F::k4) {
      u32x4 x[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) x[i] = *reinterpret_cast<const u32x4*>(at + (NF + wm * TM + i) * 1024);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(at + (wn * TN + j) * 1024);
#pragma unroll
        for (int i = 0; i < TM; ++i) acc[i][j] = mfma(w, x[i], acc[i][j]);
      }
    } else {
      const char* par = lds + (s % STAGES) * STAGE + FRAGS * 1024;
      u32x4 x[TM][2];
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) x[i][h] = *reinterpret_cast<const u32x4*>(at + (NF + (wm * TM + i) * 2 + h) * 1024);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const u32x4 raw = *reinterpret_cast<const u32x4*>(at + (wn * TN + j) * 1024);
        u32 word[F::kParams];
#pragma unroll
        for (int p = 0; p < F::kParams; ++p)
          word[p] = *reinterpret_cast<const u32*>(par + p * (NF / 4 * 256) + (wn * TN + j) * 64 + (lane & 15) * 4);
        u32x4 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32 z = F::zero(word + F::kS, s & 3, h, lane) * 0x01010101u;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            w[h][2 * q] = less(raw[2 * h + q], z);
            w[h][2 * q + 1] = less(raw[2 * h + q] >> 4, z);
          }
        }
        F::product(x, w, word, s & 3, lane, acc, j);
      }
    }
  }
  if constexpr (F::k4) {
    // lane: column n0 + .. + lane % 16, rows m0 + .. + 4 (lane / 16) + 0 .. 3
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m0 + (wm * TM + i) * 16 + 4 * (lane >> 4);
      float sx[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sx[e] = m + e < a.M ? a.x_scale[m + e] : 0.f;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = n0 + (wn * TN + j) * 16 + (lane & 15);
        if (n >= a.N) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (m + e >= a.M) continue;
          const float v = acc[i][j][e] * sx[e];
          const size_t to = (size_t)(m + e) * a.N + n;
          if (a.y_type == SVG_F32) static_cast<float*>(a.y)[to] = v;
          else static_cast<uint16_t*>(a.y)[to] = (uint16_t)round_to(a.y_type, v);
        }
      }
    }
    return;
  } else {
  // lane: row m0 + .. + lane % 16, columns n0 + .. + 4 (lane / 16) + 0 .. 3
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    const int n = n0 + (wn * TN + j) * 16 + 4 * (lane >> 4);
    float sw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) sw[e] = n + e < a.N ? half_bits_to_float(a.w_scale[n + e]) : 0.f;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m0 + (wm * TM + i) * 16 + (lane & 15);
      if (m >= a.M || n >= a.N) continue;
      const float sx = a.x_scale[m];
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][e] * (sx * sw[e]);
      const size_t at = (size_t)m * a.N + n;
      if (a.y_type == SVG_F32) {
        float* p = static_cast<float*>(a.y) + at;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) p[e] = v[e];
      } else {
        uint16_t* p = static_cast<uint16_t*>(a.y) + at;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < a.N) p[e] = (uint16_t)round_to(a.y_type, v[e]);
      }
    }
  }
  }
}

template <class F, int WM, int WN, int TM, int TN, int STAGES>
hipError_t launch(Args a, hipStream_t stream) {
  constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + BN - 1) / BN;
  const auto fn = k_prompt_linear<F, WM, WN, TM, TN, STAGES>;
  hipLaunchKernelGGL(fn, dim3((u32)a.tiles_m * (u32)a.tiles_n), dim3(64 * WM * WN), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t svg_launch_prompt_w8(const int8_t* xq, const float* x_scale, int M, int K, const int8_t* wq, const uint16_t* w_scale, int N,
                                void* y, int y_type, hipStream_t stream) {
  const Args a{xq, x_scale, reinterpret_cast<const char*>(wq), w_scale, nullptr, y, M, N, K, y_type, 0, 0};
  if (M <= 128) return launch<W8, 2, 4, 4, 2, 4>(a, stream);
  return launch<W8, 2, 4, 8, 4, 4>(a, stream);
}

template <int G, bool Z4>
static hipError_t launch_w4(const Args& a, hipStream_t stream) {
  return launch<W4<G, Z4>, 2, 4, 4, 2, 4>(a, stream);
}

hipError_t svg_launch_prompt_w4(const int8_t* xq, const float* x_scale, int M, int K, const uint8_t* wq, const uint16_t* w_scale,
                                const void* w_zero, bool z4, int group, int N, void* y, int y_type, hipStream_t stream) {
  const Args a{xq, x_scale, reinterpret_cast<const char*>(wq), w_scale, static_cast<const char*>(w_zero), y, M, N, K, y_type, 0, 0};
  if (z4) return group == 32 ? launch_w4<32, true>(a, stream) : (group == 64 ? launch_w4<64, true>(a, stream) : launch_w4<128, true>(a, stream));
  return group == 32 ? launch_w4<32, false>(a, stream) : (group == 64 ? launch_w4<64, false>(a, stream) : launch_w4<128, false>(a, stream));
}
