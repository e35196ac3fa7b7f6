// y = x . W^T of many int8 activation rows against the tiled int8 or 4-bit weights, gfx950.
//
//   W8: y[m][n] = sx[m] s[n] S[m][n],  W4: y[m][n] = sx[m] sum_g s[n][g] S_g[m][n],
// S an int32 sum of products of codes (exact: at most 127^2 K, 127 * 15 * group), from v_mfma_i32_16x16x64_i8; the rest fp32.
//
// Four ways, one rule between them (choose):
//  big   256 x 256 outputs, one workgroup of 8 waves a compute unit (W8): a step of 64 values of K brings 32 KiB for 2 x 256 x
//        256 x 64 operations, so that loads, LDS reads and products each take about the same time.  8192^3: 425 us, 2580 TOP/s.
//  mid   128 x 128 outputs, two workgroups a compute unit: for fewer tiles, and for 4-bit weights.
//  small 64 x 64 outputs, four workgroups a compute unit: for fewer tiles than compute units.
//  few   16 columns and up to 128 rows, 8 waves that share K and add their sums up in LDS: bound by the weights' bytes.
// big, mid and small go from tile to tile (k_prompt_linear): loads go straight into a ring in LDS, a stage is waited for by the count of
// loads behind it, and neither the ring nor the products stop between tiles.  W8's stores, four values each, are counted too, so
// that whole tiles' are not waited for; W4's lane has one value of a row, so that it stores four times as often as is counted and the next
// tile's first step waits for most of them.  A tile that is not whole, or whose rows of y cannot take four values at once, waits for all.
//
// What bounds them.  W8 at 4099 x 24576 x 4096: 380 us a call, 17 of them in few for the last 3 rows (4096 rows: 369, a library product
// 367); the loads alone and the products alone each take about nine tenths of it, matrix units busy 52 %.  W8 at 512 x 4096 x 4096: 18 us
// of 6.9 that its operations take at the library's rate: 64 steps of 64 values, each 0.27 us of wait, barrier and the chain through LDS
// whatever the work.  W4 at 1001 x 4096 x 12288: 108 us, 0.94 POP/s: the chain within a wave (read, unpack, product, conversion, sum,
// barrier), since 256 tiles leave a compute unit one workgroup and a SIMD two waves.  No part of it alone is the bound: vector units are busy
// 64 %, matrix units 17 %; without the sums, three quarters of the vector instructions, it takes 97 us, without the unpacking (45
// instructions a step) 107, without loads 100.  Converting by adding 1.5 * 2^23 in the matrix unit instead takes as many instructions
// and the same time.
//
// Registers.  few with eight row tiles (97 rows and more) spills where weights have 4 bits: vector registers | bytes of scratch a lane
// 40 | 148 for groups of 32 with fp16 zeros, 20 | 84 with 4-bit ones, 9 | 40 for 64 with fp16 zeros, 3 to 4 | 16 to 20 for 128; small 3 | 12 for
// groups of 32 with fp16 zeros; big has 20 bytes of scratch for scalar registers.  The waits by counts allow for it: what a spill adds
// behind a load only makes them stricter.
#include <limits.h>

#include <type_traits>

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
  int whole;  // four values of a row of y can be stored together
};

SVG_DEV u32 round_to(int type, float v) { return type == SVG_F16 ? kv_round<false>(v) : kv_round<true>(v); }
SVG_DEV u32 round2(int type, float x, float y) { return round_to(type, x) | (round_to(type, y) << 16); }
SVG_DEV void put(const Args& a, size_t at, float v) {
  if (a.y_type == SVG_F32) static_cast<float*>(a.y)[at] = v;
  else static_cast<uint16_t*>(a.y)[at] = (uint16_t)round_to(a.y_type, v);
}

// Four values of a row together (Args::whole).
SVG_DEV void put4(const Args& a, size_t at, const float (&v)[4]) {
  if (a.y_type == SVG_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) = make_uint2(round2(a.y_type, v[0], v[1]), round2(a.y_type, v[2], v[3]));
}

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

SVG_DEV v4i mfma(u32x4 a, u32x4 b, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
}

// Weight formats: kStep values of K a step; kX fragments of 16 x 64 activation codes in one.
struct W8 {
  static constexpr int kStep = 64, kX = 1, kParams = 0, kStages = 4, kAhead = 3, kRing = 4;
  static constexpr bool k4 = false;
  typedef v4i Acc;
  template <int TN>
  struct Operands {
    u32x4 w[TN];
    SVG_DEV void take(const u32x4 (&raw)[TN], const u32 (&)[TN][1], int, int) {
#pragma unroll
      for (int j = 0; j < TN; ++j) w[j] = raw[j];
    }
    template <int TM>
    SVG_DEV void multiply(const u32x4 (&x)[1], int i, v4i (&acc)[TM][TN]) const {
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = mfma(w[j], x[0], acc[i][j]);
    }
  };
  // 16 rows and columns, scales from memory
  SVG_DEV static void store_one(const Args& a, v4i sum, int m0, int n0, int lane) {
    const int m = m0 + (lane & 15), n = n0 + 4 * (lane >> 4);
    if (m >= a.M) return;
    const float sx = a.x_scale[m];
    const size_t at = (size_t)m * a.N + n;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = n + e < a.N ? (float)sum[e] * (sx * half_bits_to_float(a.w_scale[n + e])) : 0.f;
    if (a.whole && n < a.N) {
      put4(a, at, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) put(a, at + e, v[e]);
    }
  }
  // lane: row 16 (tm + i) + lane % 16 of the tile, columns 16 (tn + j) + 4 (lane / 16) + 0 .. 3
  template <int TM, int TN>
  SVG_DEV static void store(const Args& a, const Acc (&acc)[TM][TN], const char* scales, int columns, int m0, int n0, int tm, int tn,
                            int lane, bool full) {
    float sx[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) sx[i] = *reinterpret_cast<const float*>(scales + ((tm + i) * 16 + (lane & 15)) * 4);
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      const u32x4 h = *reinterpret_cast<const u32x4*>(scales + columns + ((tn + j) * 16 + 4 * (lane >> 4)) * 4);
      const int n = n0 + (tn + j) * 16 + 4 * (lane >> 4);
      float sw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) sw[e] = half_bits_to_float((uint16_t)h[e]);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int m = m0 + (tm + i) * 16 + (lane & 15);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][e] * (sx[i] * sw[e]);
        const size_t at = (size_t)m * a.N + n;
        if (full) {
          put4(a, at, v);
        } else if (m < a.M) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < a.N) put(a, at + e, v[e]);
        }
      }
    }
  }
};
// Codes 0 .. 15 of the low nibbles less their zero points (the same in every byte of z), as int8: no byte borrows.
SVG_DEV u32 less(u32 codes, u32 z) { return (((codes & 0x0F0F0F0Fu) | 0x80808080u) - z) ^ 0x80808080u; }

template <int G, bool Z4_>
struct W4 {
  static constexpr int kStep = 128, kX = 2, kGroup = G, kStages = 3, kAhead = 1, kRing = 2;
  static constexpr bool k4 = true, kZ4 = Z4_;
  // dwords of scales and of zeros that a row has in a step
  static constexpr int kS = G == 32 ? 2 : 1, kZ = G == 32 && !Z4_ ? 2 : 1, kParams = kS + kZ;
  static constexpr u32 kRow = 16 * (512 / G) * 2;  // bytes of scales of 16 rows and 512 values of K
  // first byte of a step's dword in a row's 512 values (4-bit zeros: of the row's dword; two rows of groups of 128 share one)
  SVG_DEV static u32 scale_at(int s) { return G == 32 ? s * 8u : (G == 64 ? s * 4u : (s >> 1) * 4u); }
  SVG_DEV static u32 zero_at(int s) { return G == 32 ? (s >> 1) * 4u : 0u; }
  typedef f32x4 Acc;
  // the zero point of the 16 values that a lane holds of half h of step s (of four in 512 values), in every byte; fp16
  // zeros: added to 1024 they are the low bits of the sum
  SVG_DEV static u32 zero(const u32* word, int s, int h, int lane) {
    const int b = lane >> 5;  // which half of 64 values
    if constexpr (Z4_) {
      const int at = G == 64 ? 2 * s + h : (G == 128 ? 4 * (lane & 1) + s : 4 * (s & 1) + 2 * h + b);
      return __builtin_amdgcn_perm(0u, (word[0] >> (4 * at)) & 15u, 0u);
    } else {
      const u32 w = __builtin_bit_cast(u32, __builtin_bit_cast(f16x2, G == 32 ? word[h] : word[0]) + f16x2{1024, 1024});
      const int hi = G == 64 ? h : (G == 128 ? s & 1 : b);
      return __builtin_amdgcn_perm(0u, w & 0x00FF00FFu, hi ? 0x02020202u : 0u);
    }
  }
  // A step's weights: codes less zero points, and the scales of its groups.
  template <int TN>
  struct Operands {
    static constexpr int GROUPS = 128 / G;
    u32x4 w[TN][2];
    float scale[TN][GROUPS];
    bool high;
    SVG_DEV void take(const u32x4 (&raw)[TN], const u32 (&word)[TN][kParams + 1], int s, int lane) {
      high = lane >= 32;
#pragma unroll
      for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32 z = zero(word[j] + kS, s, h, lane);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            w[j][h][2 * q] = less(raw[j][2 * h + q], z);
            w[j][h][2 * q + 1] = less(raw[j][2 * h + q] >> 4, z);
          }
        }
#pragma unroll
        for (int q = 0; q < GROUPS; ++q)
          scale[j][q] = G == 128 ? half_bits_to_float((uint16_t)(s & 1 ? word[j][0] >> 16 : word[j][0] & 0xFFFFu)) : half_at(word[j], q);
      }
    }
    // the products of row tile i, and what those of the one before add to its sums
    v4i sum[2][TN][GROUPS];
    template <int TM>
    SVG_DEV void multiply(const u32x4 (&x)[2], int i, f32x4 (&acc)[TM][TN]) {
      const v4i none{};
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        v4i (&to)[GROUPS] = sum[i & 1][j];
        if constexpr (G == 128) {
          to[0] = mfma(x[1], w[j][1], mfma(x[0], w[j][0], none));
        } else if constexpr (G == 64) {
#pragma unroll
          for (int h = 0; h < 2; ++h) to[h] = mfma(x[h], w[j][h], none);
        } else {
          // groups of 32: half the lanes' weights at a time
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            u32x4 part = w[j][q >> 1];
            if (high != (q & 1)) part = u32x4{};
            to[q] = mfma(x[q >> 1], part, none);
          }
        }
      }
      if (i > 0) add(i - 1, acc);
      if (i == TM - 1) add(i, acc);
    }
    template <int TM>
    SVG_DEV void add(int i, f32x4 (&acc)[TM][TN]) {
#pragma unroll
      for (int j = 0; j < TN; ++j) {
#pragma unroll
        for (int q = 0; q < GROUPS; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf((float)sum[i & 1][j][q][e], scale[j][q], acc[i][j][e]);
        asm volatile("" : "+v"(acc[i][j]));  // here, not at the step's end: the products' registers are needed again
      }
    }
  };
  SVG_DEV static void store_one(const Args& a, f32x4 sum, int m0, int n0, int lane) {
    const int m = m0 + 4 * (lane >> 4), n = n0 + (lane & 15);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n < a.N && m + e < a.M) put(a, (size_t)(m + e) * a.N + n, sum[e] * a.x_scale[m + e]);
  }
  // lane: column 16 (tn + j) + lane % 16 of the tile, rows 16 (tm + i) + 4 (lane / 16) + 0 .. 3
  template <int TM, int TN>
  SVG_DEV static void store(const Args& a, const Acc (&acc)[TM][TN], const char* scales, int, int m0, int n0, int tm, int tn, int lane,
                            bool) {
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int m = m0 + (tm + i) * 16 + 4 * (lane >> 4);
      const f32x4 sx = *reinterpret_cast<const f32x4*>(scales + ((tm + i) * 16 + 4 * (lane >> 4)) * 4);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        const int n = n0 + (tn + j) * 16 + (lane & 15);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n < a.N && m + e < a.M) put(a, (size_t)(m + e) * a.N + n, acc[i][j][e] * sx[e]);
      }
    }
  }
};

// 4 bytes a lane from global memory straight into LDS (256 bytes from `to` on), as load_to_lds.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
SVG_DEV void load4_to_lds(const char* from, u32 lane4, u32 to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               ::"s"(__builtin_amdgcn_readfirstlane((int)to)), "v"(lane4), "s"(from) : "memory", "m0");
}
// 2 bytes a lane, each to a dword of its own.
SVG_DEV void load2_to_lds(const char* from, u32 lane2, u32 to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ushort %1, %2"
               ::"s"(__builtin_amdgcn_readfirstlane((int)to)), "v"(lane2), "s"(from) : "memory", "m0");
}
#pragma clang diagnostic pop
// A pointer that is the same for the wave, in scalar registers.
SVG_DEV const char* uniform(const char* p) {
  const unsigned long long v = reinterpret_cast<unsigned long long>(p);
  const u32 lo = (u32)__builtin_amdgcn_readfirstlane((int)(u32)v), hi = (u32)__builtin_amdgcn_readfirstlane((int)(u32)(v >> 32));
  return reinterpret_cast<const char*>((unsigned long long)hi << 32 | lo);
}
// All but the last N loads of this wave have arrived.
template <int N>
SVG_DEV void wait_vm() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));  // vmcnt(N)
  asm volatile("" ::: "memory");
}

// One workgroup a compute unit, which goes from tile to tile: the next tile's first stages are requested during a
// tile's last steps and its results are on their way out while the next one is computed.
template <class F, int WM, int WN, int TM, int TN, int WGS>
__global__ __launch_bounds__(64 * WM * WN, WGS * WM * WN / 4) void k_prompt_linear(Args a) {
  constexpr int WAVES = WM * WN, MF = WM * TM, NF = WN * TN, STAGES = F::kStages;  // fragments of 16 rows, of 16 columns
  constexpr int FRAGS = NF + MF * F::kX;                              // KiB of a stage
  constexpr int PARAMS = F::k4 ? NF / 4 * F::kParams : 0;             // 256-byte loads of parameters
  constexpr int STAGE = FRAGS * 1024 + PARAMS * 256;
  constexpr int XI = MF / 4, WI = F::k4 ? 0 : NF / 4;                 // 64 row scales, 64 column scales a load
  static_assert(FRAGS % WAVES == 0 && PARAMS <= WAVES && MF % 4 == 0 && NF % 4 == 0 && XI + WI <= WAVES, "loads of a wave");
  static_assert(TM % F::kRing == 0, "the places of the activations' fragments are the same in every step");
  constexpr int LOADS = FRAGS / WAVES, STORES = TM * TN;              // (STORES: at least so many for each wave's part of a whole tile)
  static_assert(STORES + LOADS < 64, "the largest count that is waited for");
  __shared__ __attribute__((aligned(1024))) char lds[STAGES * STAGE + (XI + WI) * 256];
  char* const scales = lds + STAGES * STAGE;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
  const u32 base = lds_at(lds);
  const int steps = (a.K + F::kStep - 1) / F::kStep, slabs = a.K >> 5;
  const int last_tile = ((a.N + 15) >> 4) - 1;
  // Tiles: round after round of one for each workgroup; in a round every XCD takes a stretch of them, by columns inside
  // groups of 8 tile rows.
  const u32 total = (u32)a.tiles_m * (u32)a.tiles_n, grid = gridDim.x;
  auto tile_of = [&](u32 round, int& m0, int& n0) {
    const u32 first = round * grid, left = total - first < grid ? total - first : grid, per = left >> 3, more = left & 7u;
    const u32 xcd = blockIdx.x & 7u, at = blockIdx.x >> 3;
    if (first >= total || at >= per + (xcd < more ? 1u : 0u)) return false;
    const u32 t = first + xcd * per + (xcd < more ? xcd : more) + at;
    const u32 group = t / (8u * a.tiles_n), in = t % (8u * a.tiles_n);
    const u32 rows_in = (u32)a.tiles_m - group * 8 < 8 ? (u32)a.tiles_m - group * 8 : 8;
    m0 = (int)(group * 8 + in % rows_in) * MF * 16;
    n0 = (int)(in / rows_in) * NF * 16;
    return true;
  };

  // This wave's loads of a stage: fragment wave + i * WAVES, first the weights', then the activations'.  The addresses are
  // the same for the wave but for a lane's place, and rise by the same number each stage.
  const char* src[LOADS];
  u32 lane_at[LOADS], stride[LOADS];
  // parameters: load number p brings one dword of 64 rows, of kind p / (NF / 4); waves below PARAMS have one each
  const char* pbase = nullptr;
  u32 poff = 0;
  auto aim = [&](int m0, int n0) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int f = wave + i * WAVES;
      if (f < NF) {
        const int tile = (n0 >> 4) + f;
        src[i] = a.wq + (size_t)(tile < last_tile ? tile : last_tile) * steps * 1024;
        lane_at[i] = lane * 16u;
        stride[i] = 1024u;
      } else {
        // rows past the last one: that one's codes, whose products are not stored
        const int j = (f - NF) / F::kX, h = (f - NF) % F::kX, kb = lane >> 4, m = m0 + 16 * j;
        const int buf = (m < a.M ? m : a.M - 1) & ~31, R = a.M - buf < 32 ? a.M - buf : 32;
        const int row = 16 * (j & 1) + (lane & 15);
        src[i] = reinterpret_cast<const char*>(a.xq) + (size_t)buf * a.K;
        lane_at[i] = ((u32)((2 * h + (kb >> 1)) * R) + (u32)(row < R ? row : R - 1)) * 32u + (kb & 1) * 16u;
        stride[i] = (u32)R * F::kStep;
      }
    }
    if constexpr (F::k4) {
      const int kind = wave / (NF / 4), tile = (n0 >> 4) + wave % (NF / 4) * 4 + (lane >> 4);
      const u32 blocks = (u32)(a.K + 511) >> 9, row = (u32)((tile < last_tile ? tile : last_tile) - (n0 >> 4)) * blocks * 16u + (lane & 15);
      if (kind < F::kS) {
        pbase = reinterpret_cast<const char*>(a.w_scale) + (size_t)(n0 >> 4) * blocks * F::kRow;
        poff = row * (F::kRow / 16) + 4u * kind;
      } else {
        constexpr u32 zrow = F::kZ4 ? F::kRow / 64 : F::kRow / 16;
        pbase = a.w_zero + (size_t)(n0 >> 4) * blocks * (zrow * 16u);
        poff = (row * zrow & ~3u) + 4u * (kind - F::kS);
      }
    }
  };
  auto fetch_piece = [&](int s, int slot, int i, bool last) {
    const int f = wave + i * WAVES;
    u32 o = lane_at[i];
    if (last && f >= NF) {
      // K's last slabs may be missing: the last one's codes, the weights there are zero
      const int slab = s * (F::kStep / 32) + (F::kX == 2 ? 2 * ((f - NF) & 1) : 0) + (lane >> 5);
      if (slab >= slabs) o -= (u32)(slab - slabs + 1) * (stride[i] / (F::kStep / 32));
    }
    load_to_lds(uniform(src[i]), o, base + (u32)slot * STAGE + (u32)f * 1024u);
    src[i] += stride[i];
  };
  auto fetch_params = [&](int s, int slot) {
    if constexpr (F::k4) {
      if (wave < PARAMS) {
        const bool scale = wave / (NF / 4) < F::kS || !F::kZ4;
        const u32 o = poff + (u32)(s >> 2) * (scale ? F::kRow : F::kRow / 4) + (scale ? F::scale_at(s & 3) : F::zero_at(s & 3));
        load4_to_lds(uniform(pbase), o, base + (u32)slot * STAGE + FRAGS * 1024 + wave * 256);
      }
    }
  };
  // Waits until this wave's loads of a stage have arrived, behind which those of N more stages were requested (and EXTRA others).
  auto arrived = [&](auto n, auto extra) {
    constexpr int N = decltype(n)::value, X = decltype(extra)::value;
    if constexpr (PARAMS == 0) {
      wait_vm<LOADS * N + X>();
    } else {
      if (wave < PARAMS) wait_vm<(LOADS + 1) * N + X>();
      else wait_vm<LOADS * N + X>();
    }
  };
  using std::integral_constant;
  using Zero = integral_constant<int, 0>;
  using One = integral_constant<int, 1>;

  int m0 = 0, n0 = 0;
  if (!tile_of(0, m0, n0)) return;
  u32 tiles = 1, round = 0;          // of this workgroup; the round whose tile is being requested
  for (int x, y; tile_of(tiles, x, y);) ++tiles;
  const u32 all = tiles * (u32)steps;
  int fs = 0;                        // the stage of that tile that is requested next
  bool feeding = true;
  auto fed = [&] {                   // a stage has been requested
    if (++fs < steps) return;
    fs = 0;
    int x = 0, y = 0;
    feeding = tile_of(++round, x, y);
    if (feeding) aim(x, y);
  };

  typename F::Acc acc[TM][TN];
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = typename F::Acc{};
  };
  clear();
  aim(m0, n0);
#pragma unroll 1
  for (int s = 0; s < STAGES - 1; ++s) {
    if (!feeding) break;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) fetch_piece(fs, s, i, fs == steps - 1);
    fetch_params(fs, s);
    fed();
  }
  if (all > STAGES - 2) arrived(integral_constant<int, STAGES - 2>{}, Zero{});
  else wait_vm<0>();
  barrier();

  // The weights' fragments of a step are read while the step before is computed, from the next stage, which has arrived
  // before the step begins; the activations' a few groups of products ahead.
  constexpr int AHEAD = F::kAhead, RING = F::kRing;
  u32x4 x[RING][F::kX], w[2][TN];
  u32 word[2][TN][F::kParams + 1];
  const char* mine = lds + lane * 16;
  const char* params = lds + FRAGS * 1024 + wn * TN * 64 + (lane & 15) * 4;
  auto read_w = [&](int slot, int j, int to) {
    w[to][j] = *reinterpret_cast<const u32x4*>(mine + slot * STAGE + (wn * TN + j) * 1024);
#pragma unroll
    for (int p = 0; p < F::kParams; ++p) word[to][j][p] = *reinterpret_cast<const u32*>(params + slot * STAGE + p * (NF / 4 * 256) + j * 64);
  };
  auto read_x = [&](int slot, int i) {
#pragma unroll
    for (int h = 0; h < F::kX; ++h)
      x[i % RING][h] = *reinterpret_cast<const u32x4*>(mine + slot * STAGE + (NF + (wm * TM + i) * F::kX + h) * 1024);
  };
#pragma unroll
  for (int j = 0; j < TN; ++j) read_w(0, j, 0);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) read_x(0, i);

  int s = 0, slot = 0;               // step of the tile, its place
  u32 g = 0;                         // steps done
  u32 round_done = 0;
  bool stored = false;               // whether stores are on their way (STORES of every wave)
  // One step (parity: of its fragments).  FAST: in the middle of a tile.
  auto step = [&](auto parity, auto fast) {
    constexpr int P = decltype(parity)::value;
    constexpr bool FAST = decltype(fast)::value;
    constexpr int NEWER = STAGES - 3;  // stages that were requested behind the one that is needed
    const int next = slot + 1 == STAGES ? 0 : slot + 1, into = slot == 0 ? STAGES - 1 : slot - 1;
    __builtin_amdgcn_sched_barrier(0);
    if (FAST) arrived(integral_constant<int, NEWER>{}, Zero{});
    else if (g + 1 + NEWER >= all) wait_vm<0>();
    else if (stored && s < STAGES - 2) arrived(integral_constant<int, NEWER>{}, integral_constant<int, STORES>{});
    else arrived(integral_constant<int, NEWER>{}, Zero{});
    barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (!FAST && s == 0 && wave < XI + WI) {
      // the tile's scales, read behind its last step
      const bool rows = wave < XI;
      const int at = rows ? m0 + wave * 64 + lane : n0 + (wave - XI) * 64 + lane, most = rows ? a.M : a.N;
      const u32 clamped = (u32)(at < most ? at : most - 1);
      const u32 to = base + STAGES * STAGE + wave * 256;
      if (rows) load4_to_lds(reinterpret_cast<const char*>(a.x_scale), clamped * 4u, to);
      else load2_to_lds(reinterpret_cast<const char*>(a.w_scale), clamped * 2u, to);
    }
    typename F::template Operands<TN> op;
    op.take(w[P], word[P], s & 3, lane);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if (i + AHEAD < TM) read_x(slot, i + AHEAD);
      else read_x(next, i + AHEAD - TM);
#pragma unroll
      for (int j = i * TN / TM; j < (i + 1) * TN / TM; ++j) read_w(next, j, P ^ 1);
      if (FAST || feeding) {
#pragma unroll
        for (int l = i * LOADS / TM; l < (i + 1) * LOADS / TM; ++l) fetch_piece(fs, into, l, !FAST && fs == steps - 1);
        if (i == TM - 1) fetch_params(fs, into);
      }
      op.multiply(x[i % RING], i, acc);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (FAST) ++fs;
    else if (feeding) fed();
    ++s;
    ++g;
    slot = next;
  };
  auto finish = [&] {
    if (steps < STAGES) {            // (the scales have had no step to arrive in)
      wait_vm<0>();
      barrier();
    }
    stored = a.whole && m0 + MF * 16 <= a.M && n0 + NF * 16 <= a.N;
    F::template store<TM, TN>(a, acc, scales, XI * 256, m0, n0, wm * TM, wn * TN, lane, stored);
    if (!stored) wait_vm<0>();
    clear();
    s = 0;
    ++round_done;
    tile_of(round_done, m0, n0);
  };
  while (g < all) {
    while (s >= 2 && s + 6 <= steps) {
      step(Zero{}, std::true_type{});
      step(One{}, std::true_type{});
    }
    step(Zero{}, std::false_type{});
    if (s == steps) finish();
    if (g >= all) break;
    step(One{}, std::false_type{});
    if (s == steps) finish();
  }
}

// Few rows: bound by the weights' bytes, and by the way to them.  A workgroup takes 16 columns and up to 16 TM rows; its waves
// take the steps of K in turn, weights and codes straight into registers, and their sums are added up in LDS.
constexpr int kShortWaves = 8;
template <class F, int TM>
__global__ __launch_bounds__(64 * kShortWaves) void k_prompt_linear_short(Args a) {
  typedef typename F::Acc Acc;
  __shared__ __attribute__((aligned(1024))) char lds[kShortWaves * TM * 1024];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16, m0 = blockIdx.y * TM * 16;
  const int steps = (a.K + F::kStep - 1) / F::kStep, slabs = a.K >> 5;
  const char* wp = a.wq + (size_t)blockIdx.x * steps * 1024 + lane * 16;
  const char* xp[TM];
  u32 stride[TM];
  int slab_bytes[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int m = m0 + 16 * i + (lane & 15), row = m < a.M ? m : a.M - 1, buf = row & ~31, R = a.M - buf < 32 ? a.M - buf : 32;
    xp[i] = reinterpret_cast<const char*>(a.xq) + (size_t)buf * a.K + (u32)((lane >> 5) * R + (row & 31)) * 32u + ((lane >> 4) & 1) * 16u;
    slab_bytes[i] = R * 32;
    stride[i] = (u32)R * F::kStep;
  }
  struct Regs {
    u32x4 w[1], x[TM][F::kX];
    u32 word[1][F::kParams + 1];
  };
  auto load = [&](int s, Regs& r) {
    r.w[0] = *reinterpret_cast<const u32x4*>(wp + (size_t)s * 1024);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int h = 0; h < F::kX; ++h) {
        // K's last slabs may be missing: the last one's codes, the weights there are zero
        const int slab = s * (F::kStep / 32) + 2 * h + (lane >> 5), over = slab < slabs ? 0 : slab - slabs + 1;
        r.x[i][h] = *reinterpret_cast<const u32x4*>(xp[i] + (size_t)((u32)s * stride[i]) + (2 * h - over) * slab_bytes[i]);
      }
    if constexpr (F::k4) {
      const u32 blocks = (u32)(a.K + 511) >> 9, row = ((u32)blockIdx.x * blocks + (u32)(s >> 2)) * 16u + (lane & 15);
      const char* sp = reinterpret_cast<const char*>(a.w_scale) + (size_t)row * (F::kRow / 16) + F::scale_at(s & 3);
#pragma unroll
      for (int p = 0; p < F::kS; ++p) r.word[0][p] = *reinterpret_cast<const u32*>(sp + 4 * p);
      constexpr u32 zrow = F::kZ4 ? F::kRow / 64 : F::kRow / 16;
      const char* zp = a.w_zero + ((size_t)row * zrow & ~(size_t)3) + (F::kZ4 ? F::zero_at(s & 3) : F::scale_at(s & 3));
#pragma unroll
      for (int p = 0; p < F::kZ; ++p) r.word[0][F::kS + p] = *reinterpret_cast<const u32*>(zp + 4 * p);
    }
  };
  Acc acc[TM][1];
#pragma unroll
  for (int i = 0; i < TM; ++i) acc[i][0] = Acc{};
  auto compute = [&](int s, const Regs& r) {
    typename F::template Operands<1> op;
    op.take(r.w, r.word, s & 3, lane);
#pragma unroll
    for (int i = 0; i < TM; ++i) op.multiply(r.x[i], i, acc);
  };
  Regs r[2];
  if (wave < steps) load(wave, r[0]);
  int s = wave;
#pragma unroll 1
  for (; s + kShortWaves < steps; s += 2 * kShortWaves) {
    load(s + kShortWaves, r[1]);
    compute(s, r[0]);
    if (s + 2 * kShortWaves < steps) load(s + 2 * kShortWaves, r[0]);
    compute(s + kShortWaves, r[1]);
  }
  if (s < steps) compute(s, r[0]);
#pragma unroll
  for (int i = 0; i < TM; ++i) *reinterpret_cast<Acc*>(lds + (wave * TM + i) * 1024 + lane * 16) = acc[i][0];
  __syncthreads();
  if (wave >= TM) return;
  Acc sum{};
#pragma unroll
  for (int w = 0; w < kShortWaves; ++w) sum += *reinterpret_cast<const Acc*>(lds + (w * TM + wave) * 1024 + lane * 16);
  F::store_one(a, sum, m0 + wave * 16, n0, lane);
}

template <class F, int WM, int WN, int TM, int TN, int WGS>
hipError_t launch(Args a, hipStream_t stream) {
  constexpr int BM = WM * TM * 16, BN = WN * TN * 16;
  a.tiles_m = (a.M + BM - 1) / BM;
  a.tiles_n = (a.N + BN - 1) / BN;
  a.whole = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
  const auto fn = k_prompt_linear<F, WM, WN, TM, TN, WGS>;
  const u32 tiles = (u32)a.tiles_m * (u32)a.tiles_n, cus = WGS * (u32)svg_cu_count() & ~7u;
  hipLaunchKernelGGL(fn, dim3(tiles < cus ? (tiles + 7) / 8 * 8 : cus), dim3(64 * WM * WN), 0, stream, a);
  return hipGetLastError();
}

template <class F, int TM>
hipError_t launch_short(Args a, hipStream_t stream) {
  a.whole = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 15) == 0;
  hipLaunchKernelGGL((k_prompt_linear_short<F, TM>), dim3((a.N + 15) / 16, (a.M + 16 * TM - 1) / (16 * TM)), dim3(64 * kShortWaves), 0,
                     stream, a);
  return hipGetLastError();
}
template <class F>
hipError_t launch_few(const Args& a, hipStream_t stream) {
  switch ((a.M + 15) / 16) {
    case 1: return launch_short<F, 1>(a, stream);
    case 2: return launch_short<F, 2>(a, stream);
    case 3: return launch_short<F, 3>(a, stream);
    case 4: return launch_short<F, 4>(a, stream);
    case 5: case 6: return launch_short<F, 6>(a, stream);
    default: return launch_short<F, 8>(a, stream);
  }
}

// Which of them: the one that is expected to take the least time, in 1/100 us, from the rounds of workgroups that its tiles
// take and what a round takes for a step of K.  Measured, us (kernel alone; rows x columns x K):
//   W8   few | mid    128 x 24576 x 4096: 46 | 33    256 x 4096 x 4096: 16.5 | 20.2    512 x 4096 x 4096: 31 | 21
//        mid | big    512 x 4096 x 4096: 21 | 44     512 x 24576 x 4096: 56 | 53       2048 x 12288 x 4096: 113 | 109
//                     4096 x 24576 x 4096: 448 | 369
//        small | mid  512 x 4096 x 4096: 18 | 21      768 x 4096 x 4096: 23.5 | 21        small | few  128 x 12288 x 4096: 18 | 21
//   W4   few | mid    256 x 4096 x 4096: 21 | 36      128 x 24576 x 4096: 55 | 37          (groups of 64)
//        small | mid  512 x 4096 x 4096: 26.5 | 39    1024 x 4096 x 4096: 41 | 40          4096 x 24576 x 4096: 932 | 729
//                     512 x 4096 x 4096 in groups of 32: 38 | 60, of 128: 24 | 34
enum { kNone = -1, kFew, kSmall, kMid, kBig };
// A launch has no more workgroups in y.  (In x it has fewer than 2^32 threads, 2^27 columns of few: so wide a product always costs less
// in small, where a workgroup takes tile after tile.)
constexpr long kMaxGridY = 65535;
// A step's cost: few, in a round of one workgroup a compute unit, for a workgroup and each 16 of its rows (1 / 10000 us); small
// and mid, for 1, 2, .. workgroups on a compute unit.
struct Cost {
  long few, few_rows;
  long small[4];
  int mids;
  long mid[2];
};
constexpr Cost kCostW8{250, 120, {23, 27, 35, 44}, 2, {33, 58}};
constexpr Cost kCostW4[3] = {{950, 570, {84, 108, 143, 179}, 1, {177, 0}},   // groups of 32
                             {500, 300, {64, 72, 93, 118}, 2, {114, 190}},   // 64
                             {425, 255, {59, 65, 82, 102}, 2, {97, 164}}};   // 128
template <class F>
constexpr const Cost& costs() {
  if constexpr (F::k4) return kCostW4[F::kGroup / 64];
  else return kCostW8;
}
template <class F>
long cost_of(int way, int M, int N, int K, long cus) {
  constexpr const Cost& c = costs<F>();
  const long steps = (K + F::kStep - 1) / F::kStep;
  const auto up = [](long x, long y) { return (x + y - 1) / y; };
  const auto rounds = [&](long tiles, const long* each, long n) {
    const long rest = up(tiles % (n * cus), cus);
    return steps * (tiles / (n * cus) * each[n - 1] + (rest > 0 ? each[rest - 1] : 0));
  };
  if (M == 0) return 0;
  if (way == kFew) {
    if (up(M, 128) > kMaxGridY) return LONG_MAX;
    const long tm = up(M < 128 ? M : 128, 16);
    return up(up(N, 16) * up(M, 128), cus) * steps * (c.few + c.few_rows * tm) / 100;
  }
  if (way == kSmall) return rounds(up(M, 64) * up(N, 64), c.small, 4);
  if (way == kMid) return rounds(up(M, 128) * up(N, 128), c.mid, c.mids);
  return steps * 86 * up(up(M, 256) * up(N, 256), cus);
}
template <class F>
hipError_t launch_way(int way, const Args& a, hipStream_t stream) {
  if (way == kFew) return launch_few<F>(a, stream);
  if (way == kSmall) return launch<F, 1, 4, 4, 1, 4>(a, stream);
  if constexpr (F::k4) {
    return launch<F, 1, 8, 8, 1, costs<F>().mids>(a, stream);
  } else {
    if (way == kMid) return launch<F, 2, 4, 4, 2, 2>(a, stream);
    return launch<F, 2, 4, 8, 4, 1>(a, stream);
  }
}
// The ways of a product: the first rows one way, and the others (if any) another, in a launch of its own.
struct Choice {
  int way, rows, then;
};
template <class F>
Choice choose(int M, int N, int K, int cus) {
  Choice best{kFew, M, kNone};
  long least = cost_of<F>(kFew, M, N, K, cus);
  const auto look = [&](int way) {
    const long c = cost_of<F>(way, M, N, K, cus);
    if (c < least) least = c, best.way = way;
  };
  look(kSmall);
  look(kMid);
  if constexpr (!F::k4) {
    look(kBig);
    // the rows of whole large tiles, and the rest another way (3 us)
    const int main = M & ~255, rest = M - main;
    if (main > 0 && rest > 0) {
      int then = kFew;
      for (const int w : {kSmall, kMid})
        if (cost_of<F>(w, rest, N, K, cus) < cost_of<F>(then, rest, N, K, cus)) then = w;
      if (cost_of<F>(kBig, main, N, K, cus) + cost_of<F>(then, rest, N, K, cus) + 300 < least) best = {kBig, main, then};
    }
  }
  return best;
}
template <class F>
hipError_t launch_best(const Args& a, hipStream_t stream) {
  const Choice c = choose<F>(a.M, a.N, a.K, svg_cu_count());
  Args first = a;
  first.M = c.rows;
  const hipError_t e = launch_way<F>(c.way, first, stream);
  if (e != hipSuccess || c.then == kNone) return e;
  Args second = a;
  second.M = a.M - c.rows;
  second.xq += (size_t)c.rows * a.K;
  second.x_scale += c.rows;
  second.y = static_cast<char*>(a.y) + (size_t)c.rows * a.N * (a.y_type == SVG_F32 ? 4 : 2);
  return launch_way<F>(c.then, second, stream);
}

// The weights' format, as a type, for f.
template <class Fn>
auto of_format(bool w8, bool z4, int group, const Fn& f) {
  if (w8) return f(W8{});
  if (z4) return group == 32 ? f(W4<32, true>{}) : (group == 64 ? f(W4<64, true>{}) : f(W4<128, true>{}));
  return group == 32 ? f(W4<32, false>{}) : (group == 64 ? f(W4<64, false>{}) : f(W4<128, false>{}));
}

}  // namespace

hipError_t svg_launch_prompt_w8(const int8_t* xq, const float* x_scale, int M, int K, const int8_t* wq, const uint16_t* w_scale, int N,
                                void* y, int y_type, hipStream_t stream) {
  return launch_best<W8>({xq, x_scale, reinterpret_cast<const char*>(wq), w_scale, nullptr, y, M, N, K, y_type, 0, 0, 0}, stream);
}

hipError_t svg_launch_prompt_w4(const int8_t* xq, const float* x_scale, int M, int K, const uint8_t* wq, const uint16_t* w_scale,
                                const void* w_zero, bool z4, int group, int N, void* y, int y_type, hipStream_t stream) {
  const Args a{xq, x_scale, reinterpret_cast<const char*>(wq), w_scale, static_cast<const char*>(w_zero), y, M, N, K, y_type, 0, 0, 0};
  return of_format(false, z4, group, [&](auto f) { return launch_best<decltype(f)>(a, stream); });
}

void svg_prompt_linear_choice(int fmt, int group, int M, int N, int K, int cus, int32_t* choice) {
  const Choice c = of_format(fmt == SVG_W8_SYM, fmt == SVG_W4_ASYM_Z4, group, [&](auto f) { return choose<decltype(f)>(M, N, K, cus); });
  choice[0] = c.way;
  choice[1] = c.rows;
  choice[2] = c.then;
}
