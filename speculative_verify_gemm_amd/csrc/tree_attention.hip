// Attention of draft trees over a paged cache, gfx950.
//
// Row (slot s, node i, query head a) attends to the slot's committed tokens and
// to the tree tokens on node i's root path:
//   o = sum_t p_t v_t / sum_t p_t,   p_t = 2^(f (q . k_t) - M),  f = scale log2(e),
// computed in one pass over the tokens with a running maximum M per row, split over
// the whole device along the tokens and joined by a second, small launch.
//
// Work.  All rows that read the same keys form one item: for a token prefix that the
// slots share, every row of every slot of a key/value head; for a slot's own
// tokens, the rows of its tree (nodes x query heads of the group).  An item's tokens
// are counted in tiles of 32; all tiles of all items, in order, are dealt out
// evenly over the workgroups (one a CU), so unequal lengths and few rows both fill the
// device.  A workgroup writes one partial (O, M, sum) for each item it meets.  The lengths are read
// on the device: the same launch serves any lengths, also from a captured graph.
//
// Layout.  A page is laid out in the lane order of v_mfma_f32_16x16x32: S^T = K Q^T
// leaves a row's scores in one lane column, four consecutive tokens in each lane,
// which is the order the values are stored in, so the probabilities go from the
// first product's result registers into the second's operand registers with no
// exchange: O^T += V^T P^T.  A wave reads a tile as contiguous KiB.
//
// Ways over an item's tiles, by the rows that the launch's largest item may have:
//  * thin (up to 32 rows, 16 of dim 256: plain decoding, small trees): bound by the cache's
//    bytes.  Each of the eight waves takes every eighth tile for all the rows,
//    keys and values straight into registers, the next tile's requested as
//    soon as the registers are free; the waves' results are joined in LDS.
//  * alone (many slots of few tokens): a thin item is one wave's, with no barrier and
//    nothing to join; the eight waves of a workgroup work on eight items at once.
//  * thick (more rows: large trees, shared prefixes): every tile is used by up to eight
//    waves.  It is brought into LDS once, by loads that go there
//    directly and run STEPS - 1 steps ahead, one barrier a step.  Bound by the matrix unit.
// A shared prefix that is walked the thick way and slots that are walked the thin way are one launch.
//
// Measured (kernel + join in a kernel trace, us; bytes and the matrix units' busy share by counters):
//   1 token, 1001 seen, 8 heads of 128 for 32 query heads, fp16        9 to 10 + 4     a chain of dependent loads
//   16 nodes, 8206 seen, 32 heads of 128, fp16                               26 + 4.5   bytes: 139 MB, 5.3 TB/s
//   32 nodes, 131033 seen, 8 heads of 128 for 32, bf16     180 to 200 on average + 8.5 products: 172 GFLOP in five parts, 0.9
//                           (155 to 215 as the clock goes)                              PFLOP/s, units busy 46 % (a library
//                                                                                       product of 8192^3: 67 %); 562 MB
//   32 slots of up to 2000 tokens behind 32768, 8 heads for 32, fp16         70 + 6     bytes and products side by side: 289 MB,
//                                                                                       39 GFLOP in four parts, units busy 21 %
//   6 trees of 7 nodes, 301 tokens behind 4992, 2 heads of 256 for 16      25.5 + 6.4   a few tiles a workgroup: its start, and
//                                                                                       27 MB of partials for 22 MB read
//
// Precision.  q is fp32 and the keys 16-bit: q is normalised per row by a power of
// two and split into 16-bit parts (two of fp16: 22 bits; three of bf16: 24 bits), one
// product each; the probabilities into two parts.  fp16 parts end at 2^-24 whatever they belong to, so
// a row's largest q is brought to 2^13 and more: what is small beside it is off by 2^-38 of it at most (brought to 1, by 2^-25:
// one channel 2^13 above the others would put 2e-4 into the output).  Sums, maxima and accumulators
// are fp32.  One product with everything rounded to 16 bits would be off by
// 2^-9 (bf16), which the fp32 consumers of the output would see.
//
// The running maximum is raised only when a score passes it by more than
// 2^kSlack: until then probabilities above 1 are kept as they are, which takes the
// exchange between lanes and the rescaling of O out of almost every tile.  Probabilities are lifted by 2^kLift; fp16 has
// room for 2^(kLift + kSlack) < 2^16.  Their low part ends at 2^-24, so each loses up to 2^-(24 + kLift) of the largest
// that its wave has seen for the row (the sum keeps it): 2^-36 for each token of the wave's.  A wider slack is faster and loses
// more: 32 branches behind 32768, kLift 9 and slack 6 67.7 us (2^-33), 12 and 3.9 68.4 us, 13 and 2.9 69.5 us, 14 and 1.9 71.4 us.
#include "svg_cache.h"
#include "svg_internal.h"

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512, kWaves = 8;
constexpr int kMaxGroups = SVG_ATTN_MAX_GROUPS;
constexpr int kMaxSlots = 1024;
constexpr float kLow = -3e38f;       // the maximum before any token
constexpr float kLowest = -3.402823466e38f;
// A probability is 2^(f s + bias), bias = kLift - f m: one operation, off by half a step of f m.  Beyond
// kFar that step would be felt as a factor, and far beyond it would overflow: 2^(f (s - m) + kLift) then.
constexpr float kFar = 65536.f;
// A unit of work is a tile; an item counts as kItemThin / kItemThick tiles more, the time that starting and ending it
// takes (thin, 8 heads of 128: 32 slots of 2000 tokens 33.0 us, with 8: 37.2, with 4: 43.2, with 24: 33.0; 8 slots of
// 3000 with 4 nodes 22.1, 22.9, 24.8, 21.6.  Thick: 2 to 8 are alike).  A workgroup gets kMinThin / kMinThick units at
// least: fewer workgroups have fewer partials to join (1000 tokens of 8 heads 12.5 us, with 7: 12.9, with 16: 14.5, with
// 2: 12.3; 7656 tokens of 2 heads of 256 16.6, 20.7, 20.4, 17.7; thick, 500 tokens of 32 heads 17.7 us, with 8: 24.4).
constexpr int kItemThin = 12, kItemThick = 4, kMinThin = 4, kMinThick = 2;

// Slot items are worked on alone where that is expected to take less time (in tiles of a wave): kAloneItem and the
// longest slot's tiles against the joins that are saved, kAloneGain for each item of a workgroup, and the item's
// tiles over the whole device.  8 heads of 128, one token, alone / not: 64 slots of 100 tokens 14.3 / 23.2 us, 128 of
// 400 31.8 / 48, 32 of 300 17.3 / 19.3, 64 of 600 29.6 / 32, 64 of 1000 40.3 / 39.  Kernels that can do it are only taken
// from kAloneFrom items on: below, the few calls that gained (16.5 -> 15.0 us) did not outweigh 1 us that all others lost.
constexpr int kAloneFrom = 256, kAloneItem = 5, kAloneGain = 15, kAloneRow = 2048;

constexpr int item_cost(bool thin) { return thin ? kItemThin : kItemThick; }

// Row tiles of an item that is walked the thin way (dim 256: the accumulators of two do not fit).  32 rows of 8 heads of
// 128, thin / thick: 32768 tokens 36.9 / 46.8 us, 8000 tokens 22.6 / 24.8 us.
template <int D>
constexpr int kThinTiles = D < 256 ? 2 : 1;

// What the second launch has to know of an item: the workgroups that wrote partials of it.
struct Span {
  int first, count;
};

// Rows of an item block and the workspace's parts: a header (the prefix that was used), a Span for each item, (M, sum) and
// O of every row of partials.
constexpr int kBlock = 16 * kWaves;  // rows of an item at most
struct Shape {
  int block_p, block_s;     // rows of a prefix item, of a slot item: kBlock where there are several row blocks
  int rb_p, rb_s;           // row blocks
  int items_p, items_s;
  Shape(int S, int T, int G, int heads) {
    const int rows_p = S * T * G, rows_s = T * G;
    block_p = rows_p < kBlock ? (rows_p + 15) / 16 * 16 : kBlock;
    block_s = rows_s < kBlock ? (rows_s + 15) / 16 * 16 : kBlock;
    rb_p = (rows_p + block_p - 1) / block_p;
    rb_s = (rows_s + block_s - 1) / block_s;
    items_p = heads * rb_p;
    items_s = heads * rb_s * S;
  }
  // first row of partials of workgroup w in item j (prefix items, then slot items): either number rising by one
  // is another place, and the pairs that occur rise in both
  __host__ __device__ long slot_p(int w, int j) const { return (long)(w + j) * block_p; }
  __host__ __device__ long slot_s(int w, int j) const { return (long)(kMaxGroups + items_p) * block_p + (long)(w + j) * block_s; }
  long rows() const { return (long)(kMaxGroups + items_p) * block_p + (long)(kMaxGroups + items_s) * block_s; }
  size_t stats_at() const { return (256 + (size_t)(items_p + items_s) * sizeof(Span) + 255) / 256 * 256; }
  size_t parts_at() const { return (stats_at() + (size_t)rows() * 8 + 255) / 256 * 256; }
  size_t bytes(int dim) const { return parts_at() + (size_t)rows() * dim * 4; }
};

struct AttnArgs {
  svg_kv_cache c;
  const float* q;
  const int32_t* parent;
  const int32_t* n_nodes;
  const int32_t* shared;
  float* out;
  int* header;        // the workspace, see Shape
  Span* spans;
  float* stats;
  float* parts;
  long ld_q;
  int layer, T, G, groups;
  u32 over_g;         // 2^32 / G, rounded up (0: G = 1)
  Shape sh;
  float scale;

  // row / G
  SVG_DEV int node_of(int row) const {
    if (over_g == 0) return row;
    const int n = (int)__umulhi((u32)row, over_g);  // the quotient or one more
    return n * G > row ? n - 1 : n;
  }
};

// How the launch's work is dealt out; the same in every workgroup.
struct Plan {
  int cum[kMaxSlots + 1];   // units of an item of each slot before s (own tokens), added up
  int len[kMaxSlots];       // committed tokens; -1: not a valid slot
  int nodes[kMaxSlots];
  int red[5][kWaves];
};
// The part of it that every wave keeps in scalar registers.  (Units are below 2^31: the host has seen to that.)
struct Deal {
  int prefix, first;        // shared tokens (a multiple of 32), a slot whose row names their pages
  u32 total, units_p;       // units of the launch, of the prefix items
  u32 groups;               // workgroups that take part: w has the units from start(w) on
  u32 quot, rest;           // total / groups
  u32 alone;                // units of a slot item that one wave works on alone (0: a workgroup does)
  SVG_DEV u32 start(u32 w) const { return w * quot + (w < rest ? w : rest); }
};

SVG_DEV int node_count(const AttnArgs& a, int s) {
  if (a.n_nodes == nullptr) return a.T;
  const int n = a.n_nodes[s];
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}
// Committed tokens of a slot, -1 where its pages do not cover them and its nodes.
SVG_DEV int valid_len(const AttnArgs& a, int s, int nodes) {
  const int held = a.c.pages[s], len = a.c.len[s];
  return len < 0 || held < 0 || held > a.c.width || (long)len + nodes > (long)held * a.c.page ? -1 : len;
}

SVG_DEV u32 uniform(u32 v) { return (u32)__builtin_amdgcn_readfirstlane((int)v); }

// Minimum and sum over the wave, the same in every lane; the sum of the lanes up to this one.
template <int CTRL>
SVG_DEV int dpp(int v) { return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, false); }
SVG_DEV int min_i(int a, int b) { return a < b ? a : b; }
SVG_DEV int wave_min(int v) {
  v = min_i(v, dpp<0xB1>(v));
  v = min_i(v, dpp<0x4E>(v));
  v = min_i(v, dpp<0x124>(v));
  v = min_i(v, dpp<0x128>(v));
  return min_i(min_i(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
               min_i(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}
SVG_DEV int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) {
    const int y = off == 1 ? dpp<0x111>(v) : (off == 2 ? dpp<0x112>(v) : (off == 4 ? dpp<0x114>(v) : dpp<0x118>(v)));
    if ((lane & 15) >= off) v += y;
  }
  const int a = __builtin_amdgcn_readlane(v, 15), b = a + __builtin_amdgcn_readlane(v, 31),
            c = b + __builtin_amdgcn_readlane(v, 47);
  return v + (lane < 16 ? 0 : (lane < 32 ? a : (lane < 48 ? b : c)));
}

// What the wave's lanes have written to LDS is there for its other lanes, and what they have read is read.
SVG_DEV void wave_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

template <int RTHIN, bool ALONE, bool BOTH>
SVG_DEV Deal make_plan(const AttnArgs& a, Plan& p, int& wg) {
  constexpr int cost = item_cost(RTHIN > 0), cost_p = BOTH ? kItemThick : cost;
  constexpr u32 least = RTHIN > 0 ? kMinThin : kMinThick, least_p = kMinThick;
  const int S = a.c.n_slots, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int said = a.shared != nullptr ? a.shared[0] : 0;
  // A slot with nodes whose tokens lie inside its pages is active; the others take no part.  Two slots a thread; up to
  // 128 slots every wave makes the whole plan by itself, and waits for no other.
  const bool few = S <= 128;
  const int who = few ? lane : tid;
  int n[2], len[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 2 * who + i;
    n[i] = len[i] = 0;
    if (s < S) {
      n[i] = node_count(a, s);
      len[i] = valid_len(a, s, n[i]);
      p.nodes[s] = n[i];
      p.len[s] = len[i];
      if (len[i] < 0) n[i] = 0;
    }
  }
  Deal d;
  d.prefix = 0;
  d.first = 0;
  if (a.shared != nullptr) {
    int low = 0x7FFFFFFF, first = S;
#pragma unroll
    for (int i = 1; i >= 0; --i)
      if (n[i] > 0) {
        low = min_i(low, len[i]);
        first = 2 * who + i;
      }
    int active = __builtin_popcountll(__ballot(n[0] > 0)) + __builtin_popcountll(__ballot(n[1] > 0));
    low = wave_min(low);
    first = wave_min(first);
    if (!few) {
      if (lane == 0) {
        p.red[0][wave] = low;
        p.red[1][wave] = first;
        p.red[2][wave] = active;
      }
      __syncthreads();
      active = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        low = min_i(low, p.red[0][w]);
        first = min_i(first, p.red[1][w]);
        active += p.red[2][w];
      }
    }
    if (active > 1) d.prefix = __builtin_amdgcn_readfirstlane((said < 0 ? 0 : min_i(said, low)) & ~31);
    d.first = __builtin_amdgcn_readfirstlane(first < S ? first : 0);
  }
  // units before each slot
  const int t0 = n[0] > 0 ? ((len[0] + n[0] - d.prefix + 31) >> 5) + cost : 0;
  const int t1 = n[1] > 0 ? ((len[1] + n[1] - d.prefix + 31) >> 5) + cost : 0;
  const int upto = wave_scan(t0 + t1);
  int before = upto - t0 - t1, all = __builtin_amdgcn_readlane(upto, 63), longest = 0;
  if constexpr (ALONE) longest = -wave_min(t0 > t1 ? -t0 : -t1);
  if (!few) {
    if (lane == 0) {
      p.red[3][wave] = all;
      p.red[4][wave] = longest;
    }
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int t = p.red[3][w];
      if (w < wave) before += t;
      all += t;
      if constexpr (ALONE) longest = longest > p.red[4][w] ? longest : p.red[4][w];
    }
  }
  if (2 * who < S) p.cum[2 * who] = before;
  if (2 * who + 1 < S) p.cum[2 * who + 1] = before + t0;
  if (who == 0) p.cum[S] = all;
  d.units_p = uniform(d.prefix > 0 ? (u32)(a.sh.items_p * ((d.prefix >> 5) + cost_p)) : 0u);
  u32 own = uniform((u32)(all * a.c.heads * a.sh.rb_s));
  d.alone = 0;
  if constexpr (ALONE) {
    const int items = S * a.c.heads;
    if (own > 0 && kAloneItem * ((items + kAloneRow - 1) / kAloneRow) + longest - cost <=
                       items * kAloneGain / 256 + all * a.c.heads / kAloneRow) {
      const int each = (all + S - 1) / S - cost + kAloneItem;
      d.alone = uniform(each > 1 ? (u32)each : 1u);
      own = (u32)items * d.alone;
    }
  }
  u32 groups = (u32)a.groups, at_least = least;
  if constexpr (BOTH) {
    // The device is shared out between the prefix and the slots' own tokens by what either takes; a thick tile counts
    // as 2.5 thin ones where one row tile of up to 128 dims is thin, as 1.8 of dim 256, as 1.5 of two row tiles.  (32 slots
    // of one token: 32 heads, 200 tokens behind 1024 36.3 us, with 2: 38.8, with 3: 34.7; 8 heads, 2000 behind 32768
    // 68.8, 67.7, 74.1; 19 slots of 3 nodes, 32 heads, 862 behind 10496 95, 88, 116.  Two row tiles: 24 slots of 8 nodes,
    // 300 behind 2048 45.5 us, with 3: 54)
    u32 front = 0;
    if (d.units_p > 0) {
      const float w = (float)d.units_p * (RTHIN == 1 ? (a.c.dim < 256 ? 2.5f : 1.8f) : 1.5f);
      front = (u32)((float)groups * w * __builtin_amdgcn_rcpf(w + (float)own) + 0.5f);
      const u32 most = (d.units_p + least_p - 1) / least_p, room = own > 0 ? groups - 1 : groups;
      front = front < most ? front : most;
      front = front < room ? front : room;
      front = uniform(front > 0 ? front : 1u);
    }
    if ((u32)wg < front) {
      groups = front;
      at_least = least_p;
      own = 0;
      d.alone = 0;
    } else {
      wg -= (int)front;
      groups -= front;
      d.units_p = 0;
    }
  }
  d.total = uniform(d.units_p + own);
  const u32 want = (d.total + at_least - 1) / at_least;
  d.groups = uniform(want < 1 ? 1 : (want < groups ? want : groups));
  d.quot = uniform(d.total / d.groups);
  d.rest = d.total - d.quot * d.groups;
  if (few) wave_sync();
  else __syncthreads();
  return d;
}
static_assert(2 * kThreads >= kMaxSlots, "two slots a thread");

// The workgroup that holds unit u: the first `rest` have a unit more.
SVG_DEV int group_of(u32 u, const Deal& p) {
  const u32 more = p.rest * (p.quot + 1);
  return (int)(u < more ? u / (p.quot + 1) : p.rest + (u - more) / p.quot);
}


// ------------------------------------------------------------ 16-bit operands
template <bool BF>
struct Ops;
template <>
struct Ops<false> {
  static constexpr int kQ = 2;     // parts of q
  static constexpr int kTop = 13;  // the power of two of a row's largest q
  static constexpr float kLift = 12.f, kSlack = 3.875f;
  SVG_DEV static f32x4 mfma(u32x4 x, u32x4 y, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
  }
  // bits 15 and 31: the halves that are not finite (their exponent, all ones, plus one)
  SVG_DEV static u32 odd(u32 w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }
  static constexpr u32 kOne = 0x3C00u;
};
template <>
struct Ops<true> {
  static constexpr int kQ = 3;
  static constexpr int kTop = 0;
  static constexpr float kLift = 9.f, kSlack = 6.f;
  SVG_DEV static f32x4 mfma(u32x4 x, u32x4 y, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  }
  SVG_DEV static u32 odd(u32 w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
  static constexpr u32 kOne = 0x3F80u;
};

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two probabilities in two parts, packed: fp16 parts are cut off (what the first leaves, the second takes; the rest
// is below 2^-21 of it or 2^-24, see above), bf16 parts are rounded.
template <bool BF>
SVG_DEV void split_pair(float x, float y, u32& hi, u32& lo) {
  if constexpr (BF) {
    hi = __builtin_bit_cast(u32, __builtin_convertvector(f32x2{x, y}, bf16x2));
    lo = __builtin_bit_cast(u32, __builtin_convertvector(
                                     f32x2{x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u)}, bf16x2));
  } else {
    const auto h = __builtin_amdgcn_cvt_pkrtz(x, y);
    hi = __builtin_bit_cast(u32, h);
    lo = __builtin_bit_cast(u32, __builtin_amdgcn_cvt_pkrtz(__builtin_fmaf((float)h[0], -1.f, x), __builtin_fmaf((float)h[1], -1.f, y)));
  }
}

// A pair of fp32 values split into N 16-bit parts each (part n: the rounding of what the parts
// before left over), packed two to a word.
template <bool BF, int N>
SVG_DEV void split2(float x, float y, u32 (&w)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    if constexpr (BF) {
      w[n] = __builtin_bit_cast(u32, __builtin_convertvector(f32x2{x, y}, bf16x2));
      x -= __uint_as_float(w[n] << 16);
      y -= __uint_as_float(w[n] & 0xFFFF0000u);
    } else {
      const f16x2 h = __builtin_convertvector(f32x2{x, y}, f16x2);
      w[n] = __builtin_bit_cast(u32, h);
      x -= (float)h[0];
      y -= (float)h[1];
    }
  }
}

// ----------------------------------------------------------------- the kernel
// All but the last N loads of this wave have arrived, and everything it has read from LDS.
template <int N>
SVG_DEV void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));  // vmcnt(N) lgkmcnt(0)
  asm volatile("" ::: "memory");
}
SVG_DEV void barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// 1 KiB from global memory at `from` (lane16: this lane's 16 bytes) straight into LDS at byte `to`; both the same for the
// wave.  In asm: the compiler would wait for all of them before it reads any LDS; here wait_loads() and the
// barrier say what has arrived.
SVG_DEV void load_to_lds(const char* from, u32 lane16, u32 to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               ::"s"(__builtin_amdgcn_readfirstlane((int)to)), "v"(lane16), "s"(from) : "memory");
}
// Bytes of LDS before p.
SVG_DEV u32 lds_at(const char* p) { return (u32)(uintptr_t)(const __attribute__((address_space(3))) char*)p; }

// This item: one head of one layer, the pages of one table row.
struct Item {
  const char *k, *v;         // page 0 of the head
  const int32_t* table;
  size_t stride;             // bytes of a page of all heads
  int log_tp;                // log2(tiles of a page)
  int n_pages;
  int len, total;            // tree tokens begin at len; tokens in all (a prefix item: beyond every tile)
  SVG_DEV bool bad(int page) const { return (u32)page >= (u32)n_pages; }
};

// The page numbers of a run of tiles: 64 of them at a time in the lanes of a register, so that a tile's costs no
// memory access (which the loads behind it would have to wait for).
struct Pages {
  int base, last, v;  // table entry of lane 0; the last entry of the run
  SVG_DEV void look(const Item& it, int entry) {
    base = entry;
    const int e = entry + (int)(threadIdx.x & 63u);
    v = it.table[e < last ? e : last];
  }
  SVG_DEV void start(const Item& it, int tile, int last_tile) {
    last = last_tile >> it.log_tp;
    look(it, tile >> it.log_tp);
  }
  // tiles in rising order
  SVG_DEV int at(const Item& it, int tile) {
    const int entry = tile >> it.log_tp;
    if (entry - base >= 64) look(it, entry);
    return __builtin_amdgcn_readlane(v, entry - base);
  }
};

template <int D, bool BF, int RT>
struct Attn {
  using O = Ops<BF>;
  static constexpr float kLift = O::kLift, kSlack = O::kSlack;
  static constexpr int NQ = O::kQ, NC = D / 32, ND = D / 16;
  static constexpr int TILE = 128 * D;               // bytes of a tile: 32 keys, 32 values
  static constexpr int QBYTES = RT * NC * NQ * 1024;  // thin: q's parts in LDS
  static constexpr int JOIN = RT * ND * 1024;         // O of a wave in LDS
  // thick: TW waves for each share of the rows, tiles of a step; RW shares of RT row tiles; STEPS steps in LDS
  static constexpr int TW = D < 256 ? 2 : 1, RW = kWaves / TW, STEPS = 3;
  static constexpr int RING = STEPS * TW * TILE;
  static_assert(RT * NC <= kWaves, "a wave splits one chunk of q");
  static constexpr int SOLO = QBYTES * kWaves <= 128 * 1024 ? kWaves : 128 * 1024 / QBYTES;  // thin: waves that work alone
  static_assert(RW * JOIN <= RING || TW == 1, "the join of the token waves takes the ring's place");

  struct Row {                 // per lane: row n = lane % 16 of a row tile
    f32x4 o[ND];
    float m, bias, l, f;       // maximum (in units of q . k), exponent's offset, sum, factor
    int far;                   // (the same for the wave) maxima beyond kFar: the offset is not used
    SVG_DEV void start(float factor) {
      f = factor;
      m = kLow;
      bias = kLift - kLow * f;
      l = 0.f;
      far = 0;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // the maximum in powers of two that o and l are relative to
    SVG_DEV float top() const { return fmaxf(far ? m * f : kLift - bias, kLowest); }
  };

  // Bytes before a tile's keys (and values); a page number outside the cache gives page 0 (and NaN rows).
  SVG_DEV static size_t tile_at(const Item& it, int tile, int page) {
    const u32 in = (u32)tile & ((1u << it.log_tp) - 1u);
    return (size_t)(it.bad(page) ? 0u : (u32)page) * it.stride + (size_t)in * (32 * D * 2);
  }

  // Raise the running maximum of a row tile to the largest score seen.
  SVG_DEV static void raise(Row& r, float top) {
    top = fmaxf(top, lane_xorf<16>(top));
    top = fmaxf(top, lane_xorf<32>(top));
    const float m = fmaxf(r.m, top);
    const float bias = kLift - m * r.f;
    r.far = __any(fabsf(bias) > kFar);
    const float w = m == r.m ? 1.f : __builtin_amdgcn_exp2f(r.far ? (r.m - m) * r.f : bias - r.bias);
    r.m = m;
    r.bias = bias;
    r.l *= w;
#pragma unroll
    for (int d = 0; d < ND; ++d) r.o[d] *= w;
  }

  // Scores to probabilities, split in two parts in the order of the second product's operand.  TREE: the
  // tile holds tree tokens, of which the row sees those of `seen`; its root path being broken makes it NaN.
  template <bool TREE>
  SVG_DEV static void soften(const Item& it, int tile, const f32x4 (&s)[2], Row& r, u32 seen, bool broken,
                             u32x4 (&p)[2]) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = s[j >> 2][j & 3];
    u32 ok = 0xFFu;
    if constexpr (TREE) {
      const int first = tile * 32 + 4 * (int)((threadIdx.x & 63) >> 4) - it.len;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int node = first + 16 * (j >> 2) + (j & 3);
        if (!(node < 0 || (node < 32 && ((seen >> node) & 1u)))) {
          ok &= ~(1u << j);
          x[j] = kLow;
        }
      }
    }
    // exponents; if one passes the slack the maximum is raised, and they are taken again
    float y[8];
    auto exponents = [&] {
      float more = r.bias;
      if (r.far) {
        more = kLift;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j] - r.m;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __builtin_fmaf(y[j], r.f, more);
    };
    exponents();
    const float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(y[4], y[5]), fmaxf(y[6], y[7])));
    if (__any(top > kLift + kSlack)) {
      raise(r, fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))));
      exponents();
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __builtin_amdgcn_exp2f(y[j]);
    if constexpr (TREE) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!((ok >> j) & 1u)) x[j] = 0.f;
        if (broken) x[j] = __builtin_nanf("");
      }
    }
    r.l += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      u32 hi, lo;
      split_pair<BF>(x[2 * w], x[2 * w + 1], hi, lo);
      p[0][w] = hi;
      p[1][w] = lo;
    }
  }

  // Which halves of a lane's words are tokens of the item: those behind the last token are whatever the page held.
  SVG_DEV static u32x4 token_mask(const Item& it, int tile) {
    const int first = tile * 32 + 4 * (int)((threadIdx.x & 63) >> 4);
    u32x4 keep;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int tok = first + 2 * (w & 1) + 16 * (w >> 1);
      keep[w] = (tok < it.total ? 0xFFFFu : 0u) | (tok + 1 < it.total ? 0xFFFF0000u : 0u);
    }
    return keep;
  }
  // O += V^T P^T for a tile with tree tokens, val(d) the values of columns 16 d ..  Values that are not finite are left
  // out of the product (0 times them
  // would be NaN in every row) and make NaN where a row has a share of them.
  template <class F>
  SVG_DEV static void gather_tree(F val, const u32x4 keep, const u32x4 (&p)[2], Row& r) {
    u32 odd = 0;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      u32x4 v = val(d) & keep;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const u32 b = O::odd(v[w]) >> 15;  // 1 in each half
        odd |= b;
        v[w] &= ~(b * 0xFFFFu);
      }
      r.o[d] = O::mfma(v, p[0], r.o[d]);
      r.o[d] = O::mfma(v, p[1], r.o[d]);
      __builtin_amdgcn_sched_barrier(0);  // one block at a time: this path must not set the kernel's registers
    }
    if (__any(odd != 0)) {
      u32x4 some;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        some[w] = ((p[0][w] & 0xFFFFu) ? O::kOne : 0u) | ((p[0][w] >> 16) ? O::kOne << 16 : 0u);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        u32x4 y = val(d) & keep;
#pragma unroll
        for (int w = 0; w < 4; ++w) y[w] = (O::odd(y[w]) >> 15) * O::kOne;
        const f32x4 hit = O::mfma(y, some, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
        for (int i = 0; i < 4; ++i) r.o[d][i] = hit[i] == 0.f ? r.o[d][i] : __builtin_nanf("");
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // ------------------------------------------------------------------- thin
  // Where registers do not last for both (dim 256, two row tiles of 128), one set serves: values are requested as the
  // keys are used, keys as the values are (8192 tokens of 32 heads of 256: 54.6 us, with both and spills 72).
  static constexpr bool kOne = D * RT >= 256;
  struct Regs {
    u32x4 k[2][NC], v[ND];
  };
  SVG_DEV static u32x4 piece(const char* base, size_t off, int i) {
    return *reinterpret_cast<const u32x4*>(base + off + (threadIdx.x & 63u) * 16u + 1024 * i);
  }
  SVG_DEV static void load_k(const Item& it, size_t off, Regs& g) {
#pragma unroll
    for (int i = 0; i < 2 * NC; ++i) g.k[i & 1][i >> 1] = piece(it.k, off, (i & 1) * NC + (i >> 1));
  }
  SVG_DEV static void load_v(const Item& it, size_t off, Regs& g) {
#pragma unroll
    for (int i = 0; i < ND; ++i) g.v[i] = piece(it.v, off, i);
  }
  // Tile t for all row tiles (nrt of them): its keys are in g or on their way (kOne: the values are not), and the next tile
  // (t2, on `page2`) follows: its keys are requested as soon as this one's are used, its values likewise: one
  // set of registers of each, always a request in flight.
  template <bool TREE>
  SVG_DEV static void thin_tile(const Item& it, int t, int t2, Regs& g, int page, int page2, const char* ql, Row (&row)[RT], int nrt,
                                const u32 (&seen)[RT], u32 broken) {
    asm volatile("" : "+v"(ql));  // q is read again for every tile, not kept
    const size_t at = tile_at(it, t, page), at2 = tile_at(it, t2, page2);
    f32x4 s[RT][2];
    auto scores = [&](int rt, int c) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        const u32x4 q = *reinterpret_cast<const u32x4*>(ql + ((rt * NC + c) * NQ + n) * 1024);
        s[rt][0] = O::mfma(g.k[0][c], q, s[rt][0]);
        s[rt][1] = O::mfma(g.k[1][c], q, s[rt][1]);
        if constexpr (kOne) __builtin_amdgcn_sched_barrier(0);
      }
    };
    u32x4 p[RT][2];
    auto weights = [&](int rt) {
      if (it.bad(page)) row[rt].l = __builtin_nanf("");
      soften<TREE>(it, t, s[rt], row[rt], seen[rt], (broken >> rt) & 1u, p[rt]);
    };
    auto sum = [&](int rt, int d) {
      row[rt].o[d] = O::mfma(g.v[d], p[rt][0], row[rt].o[d]);
      row[rt].o[d] = O::mfma(g.v[d], p[rt][1], row[rt].o[d]);
    };
    auto sum_tree = [&](int rt) { gather_tree([&](int d) { return g.v[d]; }, token_mask(it, t), p[rt], row[rt]); };
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (kOne) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) scores(rt, c);
        g.v[2 * c] = piece(it.v, at, 2 * c);
        g.v[2 * c + 1] = piece(it.v, at, 2 * c + 1);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        weights(rt);
        if constexpr (TREE) sum_tree(rt);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (TREE) {
        load_k(it, at2, g);
        return;
      }
#pragma unroll
      for (int d = 0; d < ND; ++d) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) sum(rt, d);
        __builtin_amdgcn_sched_barrier(0);
        if (d & 1) {
          g.k[0][d >> 1] = piece(it.k, at2, d >> 1);
          g.k[1][d >> 1] = piece(it.k, at2, NC + (d >> 1));
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (rt < nrt) {
#pragma unroll
          for (int c = 0; c < NC; ++c) scores(rt, c);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      load_k(it, at2, g);  // (these keys' registers, not others)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (rt < nrt) {
          weights(rt);
          if constexpr (TREE) {
            sum_tree(rt);
          } else {
#pragma unroll
            for (int d = 0; d < ND; ++d) sum(rt, d);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      load_v(it, at2, g);
    }
  }
  // Tiles t, t + step, ... up to `last`: the committed tokens' tiles, then those with tree tokens.
  SVG_DEV static void walk_thin(const Item& it, int t, int step, int last, Regs& g, Pages& pages, int page, const char* qs, Row (&row)[RT],
                                int nrt, const u32 (&seen)[RT], u32 broken) {
    const char* ql = qs + (threadIdx.x & 63u) * 16u;
    for (; t <= last && t * 32 + 32 <= it.len; t += step) {
      const int t2 = t + step <= last ? t + step : last, page2 = pages.at(it, t2);
      thin_tile<false>(it, t, t2, g, page, page2, ql, row, nrt, seen, broken);
      page = page2;
    }
    for (; t <= last; t += step) {
      const int t2 = t + step <= last ? t + step : last, page2 = pages.at(it, t2);
      thin_tile<true>(it, t, t2, g, page, page2, ql, row, nrt, seen, broken);
      page = page2;
    }
  }

  // ------------------------------------------------------------------ thick
  // This wave's share of a step on its way into the step's place at byte `to` of LDS: a run of KiB of the keys or of the
  // values of the tile that it will work on (RW waves bring a tile).  Returns 1 for a page number outside the cache.
  static constexpr int SHARE = TILE / 1024 / RW;
  SVG_DEV static u32 fetch(const Item& it, Pages& pages, int tile, int last, u32 to, int wave) {
    const int t = tile + wave / RW, mine = t <= last ? t : last, page = pages.at(it, mine);
    const int part = wave % RW;
    const size_t off = tile_at(it, mine, page) + (size_t)(part % (RW / 2) * SHARE) * 1024;
    const char* from = (part < RW / 2 ? it.k : it.v) + off;
    to += (u32)(wave / RW * TILE + part * SHARE * 1024);
#pragma unroll
    for (int i = 0; i < SHARE; ++i) load_to_lds(from + 1024 * i, (threadIdx.x & 63u) * 16u, to + 1024 * i);
    return it.bad(page) ? 1u : 0u;
  }
  // Tile t, whose keys and values begin at kt (this lane's 16 bytes) in LDS, for this wave's row tiles (nrt of them).
  template <bool TREE>
  SVG_DEV static void thick_tile(const Item& it, int t, const char* kt, bool bad, const u32x4 (&q)[RT][NC][NQ], Row (&row)[RT],
                                 const u32 (&seen)[RT], u32 broken) {
    f32x4 s[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
    // (fragments are read one ahead of the products that use them)
    auto key = [&](int i) { return *reinterpret_cast<const u32x4*>(kt + (i & 1 ? NC + i / 2 : i / 2) * 1024); };
    u32x4 k0 = key(0), k1 = key(1);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      u32x4 n0 = k0, n1 = k1;
      if (c + 1 < NC) {
        n0 = key(2 * c + 2);
        n1 = key(2 * c + 3);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          s[rt][0] = O::mfma(k0, q[rt][c][n], s[rt][0]);
          s[rt][1] = O::mfma(k1, q[rt][c][n], s[rt][1]);
        }
      __builtin_amdgcn_sched_barrier(0);
      k0 = n0;
      k1 = n1;
    }
    if (bad) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) row[rt].l = __builtin_nanf("");
    }
    const char* vt = kt + 2 * NC * 1024;
    auto val = [&](int d) { return *reinterpret_cast<const u32x4*>(vt + d * 1024); };
    const u32x4 first = val(0);
    u32x4 p[RT][2];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) soften<TREE>(it, t, s[rt], row[rt], seen[rt], (broken >> rt) & 1u, p[rt]);
    if constexpr (TREE) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) gather_tree(val, token_mask(it, t), p[rt], row[rt]);
    } else {
      u32x4 v = first;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        u32x4 ahead = v;
        if (d + 1 < ND) ahead = val(d + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) row[rt].o[d] = O::mfma(v, p[rt][i], row[rt].o[d]);
        __builtin_amdgcn_sched_barrier(0);
        v = ahead;
      }
    }
  }
  // Tiles t .. last, of each step the one that is this wave's; the first STEPS - 1 steps are on their way, bad: fetch()'s
  // answers for them, a bit a step.  live: the wave has rows.
  SVG_DEV static void walk_thick(const Item& it, int t, int last, const char* ring, Pages& pages, u32 bad, int wave, bool live,
                                 const u32x4 (&q)[RT][NC][NQ], Row (&row)[RT], const u32 (&seen)[RT], u32 broken) {
    const char* mine = ring + wave / RW * TILE + (threadIdx.x & 63u) * 16u;
    const u32 ring_at = lds_at(ring);
    const int tw = wave / RW;
    int here = 0;
    if (wave < kWaves / 2) __builtin_amdgcn_s_setprio(2);
    auto next = [&] {
      const int stale = here == 0 ? STEPS - 1 : here - 1;
      wait_loads<SHARE * (STEPS - 2)>();  // this wave's share of the step has arrived; after the barrier all of it has,
      barrier();                          // and nobody reads the place of the step before any more
      bad |= fetch(it, pages, t + TW * (STEPS - 1), last, ring_at + stale * (TW * TILE), wave) << (STEPS - 1);
    };
    auto done = [&] {
      t += TW;
      bad >>= 1;
      here = here == STEPS - 1 ? 0 : here + 1;
    };
    while (t <= last && (t + TW) * 32 <= it.len) {
      next();
      if (live && t + tw <= last)
        thick_tile<false>(it, t + tw, mine + here * (TW * TILE), bad & 1u, q, row, seen, broken);
      done();
    }
    while (t <= last) {
      next();
      if (live && t + tw <= last)
        thick_tile<true>(it, t + tw, mine + here * (TW * TILE), bad & 1u, q, row, seen, broken);
      done();
    }
    __builtin_amdgcn_s_setprio(0);
    wait_loads<0>();  // what was requested behind the last tile has landed before the ring is anything else
    barrier();
  }

  // The exponent of the power of two that a row is divided by, so that its largest q lies in [2^kTop, 2^(kTop + 1)) (0 and
  // what is not finite: none).
  SVG_DEV static int exponent_of(float top) {
    const int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
    return top == 0.f || e == 128 ? 0 : (e - O::kTop > 126 ? 126 : (e - O::kTop < -126 ? -126 : e - O::kTop));
  }
  SVG_DEV static float two_to(int e) { return __uint_as_float((u32)(127 + e) << 23); }
  // Eight values of q times a power of two, in parts.
  SVG_DEV static void split8(const f32x4 a, const f32x4 b, float by, u32x4 (&q)[NQ]) {
    u32 w[4][NQ];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      split2<BF, NQ>(a[2 * i] * by, a[2 * i + 1] * by, w[i]);
      split2<BF, NQ>(b[2 * i] * by, b[2 * i + 1] * by, w[2 + i]);
    }
#pragma unroll
    for (int n = 0; n < NQ; ++n) q[n] = u32x4{w[0][n], w[1][n], w[2][n], w[3][n]};
  }
};

template <bool X>
struct Is {
  static constexpr bool value = X;
};

// LDS of either way: thin: q's parts, then the waves' O; thick: the ring of tiles.
template <int D, bool BF, int RTHIN>
constexpr int lds_bytes() {
  using A = Attn<D, BF, RTHIN ? RTHIN : (D < 256 ? 2 : 1)>;
  return RTHIN == 0 ? A::RING : (A::SOLO * A::QBYTES > kWaves * A::JOIN ? A::SOLO * A::QBYTES : kWaves * A::JOIN);
}

// The items of workgroup wg.  RTHIN: row tiles of the thin way, 0: the thick way.  ALONE: slot items may be worked on by
// single waves.
template <int D, bool BF, int RTHIN, bool ALONE>
SVG_DEV void walk_items(const AttnArgs& a, const Plan& plan, const Deal& deal, const int wg, char* const lds) {
  constexpr bool THIN = RTHIN > 0;
  constexpr int RT = THIN ? RTHIN : (D < 256 ? 2 : 1);
  using A = Attn<D, BF, RT>;
  constexpr int NC = A::NC, ND = A::ND, NQ = A::NQ;
  __shared__ float stat[kWaves][RT][2][16];
  __shared__ float factor[RT][16];
  const Shape& sh = a.sh;
  float* const stats = a.stats;
  float* const parts = a.parts;
  int cost = item_cost(THIN);
  asm("" : "+s"(cost));  // (as a constant it makes the compiler spill 150 registers in the thick loop of 256 dims)
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float sign = a.scale < 0.f ? -1.f : 1.f;
  const float unit = fabsf(a.scale) * 1.44269504088896341f;
  const u32 till = deal.start(wg + 1), end = ALONE && deal.alone && till > deal.units_p ? deal.units_p : till;
  u32 u = deal.start(wg);
  // the first item: its slot (a prefix item: -1), head, row block and the unit of it that u is
  int s = -1, h = 0, rb = 0, off = 0;
  if (u < end) {
    u32 v = u, j, units = (u32)((deal.prefix >> 5) + cost);
    int blocks = sh.rb_p;
    if (u >= deal.units_p) {
      v -= deal.units_p;
      blocks = sh.rb_s;
      const u32 per = (u32)(a.c.heads * sh.rb_s), at = v / per;
      int lo = 0, hi = a.c.n_slots;  // cum[lo] <= at < cum[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((u32)plan.cum[mid] <= at) lo = mid;
        else hi = mid;
      }
      s = (int)uniform(lo);
      v -= (u32)plan.cum[s] * per;
      units = (u32)(plan.cum[s + 1] - plan.cum[s]);
    }
    j = v / units;
    off = (int)uniform(v - j * units);
    h = (int)uniform(blocks == 1 ? j : j / (u32)blocks);
    rb = (int)uniform(j) - h * blocks;
  }
  // An item, from its unit `off` on: by the workgroup, or (ALONE) a slot's by one wave alone.
  auto work = [&](auto by_one) {
    constexpr bool alone = decltype(by_one)::value;
    const bool prefix = s < 0;
    const int slot = prefix ? deal.first : s;
    const int tiles = __builtin_amdgcn_readfirstlane(prefix ? deal.prefix >> 5 : plan.cum[s + 1] - plan.cum[s] - cost);
    const int units = tiles + cost;
    const int left = (int)(end - u), stop = alone || left >= units - off ? units : off + left;
    const int t0 = off > cost ? off - cost : 0, t1 = stop - cost;
    const u32 item_end = u - off + units;
    if (!alone) u += stop - off;
    if (t1 <= t0) return;  // the units of its start only
    const int j = prefix ? h * sh.rb_p + rb : (s * a.c.heads + h) * sh.rb_s + rb;
    const int who = alone ? 0 : wg;
    const long place = prefix ? sh.slot_p(who, j) : sh.slot_s(who, j);
    if (t0 == 0 && (alone ? lane == 0 : threadIdx.x == 0))
      a.spans[prefix ? j : sh.items_p + j] = Span{who, stop == units ? 1 : group_of(item_end - 1, deal) - wg + 1};

    const int nodes = plan.nodes[slot];
    const int block = prefix ? sh.block_p : sh.block_s;
    const int all_rows = prefix ? a.c.n_slots * a.T * a.G : nodes * a.G;
    const int rows = __builtin_amdgcn_readfirstlane(all_rows - rb * block < block ? all_rows - rb * block : block);
    if (rows <= 0) return;  // a row block behind a small tree's rows
    const int row_tiles = (rows + 15) >> 4;

    Item it;
    const size_t head = (size_t)a.c.page * D * 2;
    it.stride = head * a.c.heads;
    const size_t base = (size_t)a.layer * a.c.n_pages * it.stride + (size_t)h * head;
    it.k = static_cast<const char*>(a.c.k) + base;
    it.v = static_cast<const char*>(a.c.v) + base;
    const int skip = prefix ? 0 : deal.prefix >> 5;  // tiles of the prefix, in front of the slot's own
    it.table = a.c.table + (size_t)slot * a.c.width;
    it.log_tp = a.c.page == 32 ? 0 : (a.c.page == 64 ? 1 : 2);
    it.n_pages = a.c.n_pages;
    it.len = __builtin_amdgcn_readfirstlane(prefix ? 0x7FFFFFFF : plan.len[slot]);
    it.total = __builtin_amdgcn_readfirstlane(prefix ? 0x7FFFFFFF : plan.len[slot] + nodes);
    const int first = t0 + skip, last = t1 - 1 + skip;

    // the tree's root paths: lane j < 32 holds node j's, by doubling
    u32 path = 0, broken = 0;
    const bool tree = !prefix && (last + 1) * 32l > it.len;  // (the workgroup's tiles have tree tokens)
    int up = (lane & 31) - 1, tree_page = -1, held = 0;
    // what is asked for in memory, before the tiles are: parents and pages, then the pages' counts
    auto look_up = [&] {
      const int j = lane & 31;
      if (!tree || j >= nodes) return;
      if (a.c.refs != nullptr) tree_page = it.table[(it.len + j) >> (it.log_tp + 5)];
      if (a.parent != nullptr) up = a.parent[(size_t)s * a.T + j];
    };
    auto count_holders = [&] {
      if (!it.bad(tree_page)) held = a.c.refs[tree_page];
    };
    auto root_paths = [&] {
      if (!tree) return;
      const int j = lane & 31;
      broken = j == 0 ? up != -1 : (up < 0 || up >= j);
      broken |= held > 1;  // other slots hold the node's page too: its rows are not there
      if (j == 0 || broken || j >= nodes) up = j;  // a path ends here
      if (j >= nodes) broken = 0;
      path = 1u << j;
#pragma unroll
      for (int r = 0; r < 5; ++r) {
        path |= (u32)__shfl((int)path, up, 32);
        broken |= (u32)__shfl((int)broken, up, 32);
        up = __shfl(up, up, 32);
      }
      broken |= (u32)__shfl((int)broken, 0, 32);
    };
    // q of row idx of the block (its values 8 g .. of every 32), and its node
    auto node_of = [&](int idx) { return a.node_of(rb * block + (idx < rows ? idx : 0)); };
    auto q_of = [&](int idx) {
      const int all = rb * block + (idx < rows ? idx : 0), node = a.node_of(all);
      return a.q + (size_t)((prefix ? 0 : s * a.T) + node) * a.ld_q + (h * a.G + all - node * a.G) * D + 8 * g;
    };
    auto at4 = [](const float* p) { return *reinterpret_cast<const f32x4*>(p); };
    auto top8 = [&](const float* p, float top) {
      const f32x4 x = at4(p), y = at4(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(x[i]), fabsf(y[i])));
      return top;
    };
    auto row_max = [](float top) {
      top = fmaxf(top, lane_xorf<16>(top));
      return fmaxf(top, lane_xorf<32>(top));
    };

    // The rows' q first, then the first tiles: loads arrive in order, and q is worked on while the tiles come.
    if constexpr (THIN) {
      const int mine = alone ? first : first + wave;  // this wave's first tile
      Pages pages;
      look_up();
      if (mine <= last) pages.start(it, mine, last);
      typename A::Regs regs;
      int my_page = 0;
      auto request = [&] {
        if (mine <= last) {
          my_page = pages.at(it, mine);
          const size_t at = A::tile_at(it, mine, my_page);
          A::load_k(it, at, regs);
          if constexpr (!A::kOne) A::load_v(it, at, regs);
        }
      };
      char* const qs = lds + (alone ? wave * A::QBYTES : 0);
      float scale[RT];
      auto put = [&](int rt, int c, const f32x4 x, const f32x4 y, float by) {
        u32x4 parts_of[NQ];
        A::split8(x, y, by, parts_of);
#pragma unroll
        for (int p = 0; p < NQ; ++p) *reinterpret_cast<u32x4*>(qs + ((rt * NC + c) * NQ + p) * 1024 + lane * 16) = parts_of[p];
      };
      if constexpr (alone) {  // a row tile of q after the other
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const int idx = rt * 16 + n;
          const float* qp = q_of(idx);
          f32x4 raw[2 * NC];
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            raw[2 * i] = at4(qp + 32 * i);
            raw[2 * i + 1] = at4(qp + 32 * i + 4);
          }
          if (rt == RT - 1) {
            count_holders();
            request();
          }
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < 2 * NC; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, fabsf(raw[i][k]));
          const int e = A::exponent_of(row_max(top));
          scale[rt] = unit * A::two_to(e);
          const float by = idx < rows ? A::two_to(-e) * sign : 0.f;
#pragma unroll
          for (int i = 0; i < NC; ++i) put(rt, i, raw[2 * i], raw[2 * i + 1], by);
        }
        root_paths();
        wave_sync();
      } else {
        // each wave splits one chunk of 32 values of one row tile
        const int my_rt = wave / NC, my_c = wave % NC, my_idx = my_rt * 16 + n;
        const bool splits = wave < RT * NC;
        f32x4 x = {0.f, 0.f, 0.f, 0.f}, y = x;
        float largest = 0.f;
        if (splits) {
          const float* qp = q_of(my_idx);
          x = at4(qp + 32 * my_c);
          y = at4(qp + 32 * my_c + 4);
#pragma unroll
          for (int i = 0; i < NC; ++i) largest = top8(qp + 32 * i, largest);
        }
        count_holders();
        request();
        if (splits) {
          const int e = A::exponent_of(row_max(largest));
          put(my_rt, my_c, x, y, my_idx < rows ? A::two_to(-e) * sign : 0.f);
          if (my_c == 0 && g == 0) factor[my_rt][n] = unit * A::two_to(e);
        }
        root_paths();
        __syncthreads();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) scale[rt] = factor[rt][n];
      }
      typename A::Row row[RT];
      u32 seen[RT], bad = 0;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        row[rt].start(scale[rt]);
        const int node = node_of(rt * 16 + n) & 31;
        seen[rt] = (u32)__shfl((int)path, node);
        if (__shfl((int)broken, node)) bad |= 1u << rt;
      }
      if (mine <= last) A::walk_thin(it, mine, alone ? 1 : kWaves, last, regs, pages, my_page, qs, row, row_tiles, seen, bad);
      if constexpr (alone) {  // nothing to join
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          typename A::Row& r = row[rt];
          const int idx = rt * 16 + n;
          r.l += lane_xorf<16>(r.l);
          r.l += lane_xorf<32>(r.l);
          if (idx < rows) {
            float* po = parts + (size_t)(place + idx) * D + 4 * g;
#pragma unroll
            for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(po + 16 * d) = r.o[d];
            if (g == 0) {
              stats[2 * (place + idx)] = r.top();
              stats[2 * (place + idx) + 1] = r.l;
            }
          }
        }
        wave_sync();
        return;
      }

      // join the waves: maxima first, then every thread adds the waves' values of its places
      float top[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        typename A::Row& r = row[rt];
        r.l += lane_xorf<16>(r.l);
        r.l += lane_xorf<32>(r.l);
        top[rt] = r.top();
        if (g == 0) stat[wave][rt][0][n] = top[rt];
      }
      __syncthreads();
      f32x4* join = reinterpret_cast<f32x4*>(lds);  // q is not needed any more
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (rt < row_tiles) {
          typename A::Row& r = row[rt];
          const float own = top[rt];
#pragma unroll
          for (int w = 0; w < kWaves; ++w) top[rt] = fmaxf(top[rt], stat[w][rt][0][n]);
          const float w = __builtin_amdgcn_exp2f(own - top[rt]);
          if (g == 0) stat[wave][rt][1][n] = r.l * w;
#pragma unroll
          for (int d = 0; d < ND; ++d) join[((wave * RT + rt) * ND + d) * 64 + lane] = r.o[d] * w;
        }
      }
      __syncthreads();
      for (int x = wave; x < row_tiles * ND; x += kWaves) {  // the wave's lanes: 16 columns of a row tile
        const int rt = x / ND, d = x - rt * ND, idx = rt * 16 + n;
        f32x4 o = join[x * 64 + lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) o += join[(w * RT * ND + x) * 64 + lane];
        if (idx < rows) {
          *reinterpret_cast<f32x4*>(parts + (size_t)(place + idx) * D + 16 * d + 4 * g) = o;
          if (d == 0 && g == 0) {
            float l = 0.f, t = kLowest;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
              l += stat[w][rt][1][n];
              t = fmaxf(t, stat[w][rt][0][n]);
            }
            stats[2 * (place + idx)] = t;
            stats[2 * (place + idx) + 1] = l;
          }
        }
      }
      __syncthreads();  // LDS is free again
    } else {
      // row tiles of this wave: as even shares as they make
      const int each = (row_tiles + A::RW - 1) / A::RW, rw = wave % A::RW, rt0 = rw * each;
      int nrt = row_tiles - rt0;
      nrt = nrt < 0 ? 0 : (nrt < each ? nrt : each);
      Pages pages;
      look_up();
      pages.start(it, first, last);
      count_holders();
      // q has to be here before the tiles are asked for (the compiler does not see those loads, and would wait for them too)
      f32x4 raw[RT][2 * NC];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float* qp = q_of((rt0 + rt) * 16 + n);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          raw[rt][2 * c] = at4(qp + 32 * c);
          raw[rt][2 * c + 1] = at4(qp + 32 * c + 4);
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i) asm volatile("" : "+v"(raw[rt][i]));
      u32 outside = 0;
#pragma unroll
      for (int i = 0; i < A::STEPS - 1; ++i)
        outside |= A::fetch(it, pages, first + i * A::TW, last, lds_at(lds) + i * (A::TW * A::TILE), wave) << i;
      u32x4 q[RT][NC][NQ];
      typename A::Row row[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * NC; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) top = fmaxf(top, fabsf(raw[rt][i][j]));
        const int e = A::exponent_of(row_max(top));
        const float by = rt < nrt && (rt0 + rt) * 16 + n < rows ? A::two_to(-e) * sign : 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) A::split8(raw[rt][2 * c], raw[rt][2 * c + 1], by, q[rt][c]);
        row[rt].start(unit * A::two_to(e));
        __builtin_amdgcn_sched_barrier(0);
      }
      root_paths();
      u32 seen[RT], bad = 0;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int node = node_of((rt0 + rt) * 16 + n) & 31;
        seen[rt] = (u32)__shfl((int)path, node);
        if (__shfl((int)broken, node)) bad |= 1u << rt;
      }
      A::walk_thick(it, first, last, lds, pages, outside, wave, nrt > 0, q, row, seen, bad);

      // join the token waves, then write
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        row[rt].l += lane_xorf<16>(row[rt].l);
        row[rt].l += lane_xorf<32>(row[rt].l);
      }
      f32x4* join = reinterpret_cast<f32x4*>(lds);
      if constexpr (A::TW > 1) {
        if (wave >= A::RW) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            if (g == 0) {
              stat[rw][rt][0][n] = row[rt].top();
              stat[rw][rt][1][n] = row[rt].l;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) join[((rw * RT + rt) * ND + d) * 64 + lane] = row[rt].o[d];
          }
        }
        __syncthreads();
      }
      if (wave < A::RW) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const int idx = (rt0 + rt) * 16 + n;
          float top = row[rt].top(), l = row[rt].l, w0 = 1.f, w1 = 0.f;
          if constexpr (A::TW > 1) {
            const float own = top, other = stat[rw][rt][0][n];
            top = fmaxf(own, other);
            w0 = __builtin_amdgcn_exp2f(own - top);
            w1 = __builtin_amdgcn_exp2f(other - top);
            l = l * w0 + stat[rw][rt][1][n] * w1;
          }
          if (rt < nrt && idx < rows) {
            float* po = parts + (size_t)(place + idx) * D + 4 * g;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
              f32x4 o = row[rt].o[d];
              if constexpr (A::TW > 1) o = o * w0 + join[((rw * RT + rt) * ND + d) * 64 + lane] * w1;
              *reinterpret_cast<f32x4*>(po + 16 * d) = o;
            }
            if (g == 0) {
              stats[2 * (place + idx)] = top;
              stats[2 * (place + idx) + 1] = l;
            }
          }
        }
      }
      __syncthreads();  // LDS is free again
    }
  };
  for (bool more = false; u < end; more = true) {
    if (more) {  // the next item in order: row blocks, heads, then the next slot that has units
      off = 0;
      if (++rb == (s < 0 ? sh.rb_p : sh.rb_s)) {
        rb = 0;
        if (++h == a.c.heads) {
          h = 0;
          do ++s;
          while (plan.cum[s + 1] == plan.cum[s]);
          s = __builtin_amdgcn_readfirstlane(s);
        }
      }
    }
    work(Is<false>{});
  }
  if constexpr (ALONE) {
    if (deal.alone == 0 || wave >= A::SOLO) return;
    // the items whose first unit is this workgroup's
    const u32 from = deal.start(wg) > deal.units_p ? deal.start(wg) - deal.units_p : 0u, to = till > deal.units_p ? till - deal.units_p : 0u;
    const int behind = (int)uniform((to + deal.alone - 1) / deal.alone);
    rb = off = 0;
    for (int next = (int)uniform((from + deal.alone - 1) / deal.alone) + wave; next < behind; next += A::SOLO) {
      s = (int)uniform((u32)next / (u32)a.c.heads);
      h = next - s * a.c.heads;
      work(Is<true>{});
    }
  }
}

// All items the same way, or (BOTH) the shared prefix the thick way and the slots' own tokens the thin way.
template <int D, bool BF, int RTHIN, bool ALONE, bool BOTH>
__global__ __launch_bounds__(kThreads, 1) void k_tree_attention(AttnArgs a) {
  __shared__ Plan plan;
  constexpr int thin = lds_bytes<D, BF, RTHIN>(), thick = BOTH ? lds_bytes<D, BF, 0>() : 0;
  __shared__ __attribute__((aligned(1024))) char lds[thin > thick ? thin : thick];
  int wg = blockIdx.x;
  const Deal deal = make_plan<RTHIN, ALONE, BOTH>(a, plan, wg);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.header = deal.prefix;
  if ((u32)wg >= deal.groups || deal.total == 0) return;
  if constexpr (BOTH) {
    if (deal.units_p > 0) walk_items<D, BF, 0, false>(a, plan, deal, wg, lds);
    else walk_items<D, BF, RTHIN, ALONE>(a, plan, deal, wg, lds);
  } else {
    walk_items<D, BF, RTHIN, ALONE>(a, plan, deal, wg, lds);
  }
}

// W waves per output row (query head, node y, slot z of the grid) join its partials, in an order that the launch alone
// decides: D / 4 lanes read one partial's O, a wave 256 / D of them at a time.
// From kJoinMany partials of a row on eight waves share them (one head of 256, 56 rows, 256 partials: the call 29.7 us, with
// one wave 59; 30000 tokens of one head of 128 14.0 / 19.4; 4 heads, 32 partials 33.5 / 30.4).
constexpr int kJoinMany = 40;


template <int W>
constexpr int kJoinThreads = W > 1 ? 64 * W : 256;

template <int D, int W>
__global__ __launch_bounds__(kJoinThreads<W>) void k_tree_attention_join(AttnArgs a) {
  const Shape& sh = a.sh;
  constexpr int L = D / 4, NP = 64 / L;  // lanes of a partial, partials at a time
  const int lane = threadIdx.x & 63, i = blockIdx.y, s = blockIdx.z;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int head = W > 1 ? blockIdx.x : blockIdx.x * (kJoinThreads<1> / 64) + wave;
  if (head >= a.c.heads * a.G) return;
  const int h = a.node_of(head), gq = head - h * a.G;
  const int r_p = (s * a.T + i) * a.G + gq, r_s = i * a.G + gq;           // rows of a prefix item, of the slot's
  const int b_p = sh.rb_p == 1 ? 0 : r_p / kBlock, b_s = sh.rb_s == 1 ? 0 : r_s / kBlock;
  const int j_p = h * sh.rb_p + b_p, j_s = (s * a.c.heads + h) * sh.rb_s + b_s;
  const int nodes = node_count(a, s), len = valid_len(a, s, nodes);
  const int prefix = *a.header;
  const Span sp = a.spans[j_p], ss = a.spans[sh.items_p + j_s];
  if (i >= nodes) return;  // no such node: the row stays as it was
  float* out = a.out + ((size_t)(s * a.T + i) * (a.c.heads * a.G) + head) * D + 4 * (lane % L);
  if (len < 0) {
    const float nan = __builtin_nanf("");
    if (lane < L && (W == 1 || wave == 0)) *reinterpret_cast<f32x4*>(out) = f32x4{nan, nan, nan, nan};
    return;
  }
  const int np = prefix > 0 ? sp.count : 0, all = np + ss.count;
  const long at_p = sh.slot_p(sp.first, j_p) + (r_p - b_p * kBlock), at_s = sh.slot_s(ss.first, j_s) + (r_s - b_s * kBlock);
  auto row_of = [&](int k) { return k < np ? at_p + (long)k * sh.block_p : at_s + (long)(k - np) * sh.block_s; };
  const float* const stats = a.stats;
  const float* const parts = a.parts;
  float m = kLowest, l = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  constexpr int U = 8;  // requests in flight a lane
  constexpr int STEP = NP * W;
  for (int k0 = (W > 1 ? wave * NP : 0) + lane / L; k0 < all; k0 += STEP * U) {
    float pm[U], pl[U];
    f32x4 po[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * STEP;
      const long row = row_of(k < all ? k : k0);
      pm[u] = stats[2 * row];
      pl[u] = stats[2 * row + 1];
      po[u] = *reinterpret_cast<const f32x4*>(parts + row * D + 4 * (lane % L));
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * STEP >= all) { pm[u] = kLowest; pl[u] = 0.f; po[u] = f32x4{0.f, 0.f, 0.f, 0.f}; }
      top = fmaxf(top, pm[u]);
    }
    const float w0 = __builtin_amdgcn_exp2f(m - top);
    l *= w0;
    o *= w0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = __builtin_amdgcn_exp2f(pm[u] - top);
      l += pl[u] * w;
      o += po[u] * w;
    }
    m = top;
  }
#pragma unroll
  for (int off = L; off < 64; off <<= 1) {
    const float m2 = __shfl_xor(m, off), l2 = __shfl_xor(l, off), top = fmaxf(m, m2);
    const float w1 = __builtin_amdgcn_exp2f(m - top), w2 = __builtin_amdgcn_exp2f(m2 - top);
    l = l * w1 + l2 * w2;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * w1 + __shfl_xor(o[e], off) * w2;
    m = top;
  }
  if constexpr (W > 1) {
    __shared__ float stat[W][2];
    __shared__ f32x4 part[W][L];
    if (lane < L) part[wave][lane] = o;
    if (lane == 0) {
      stat[wave][0] = m;
      stat[wave][1] = l;
    }
    __syncthreads();
    if (wave > 0 || lane >= L) return;
#pragma unroll
    for (int w = 0; w < W; ++w) m = fmaxf(m, stat[w][0]);
    l = 0.f;
    o = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float by = __builtin_amdgcn_exp2f(stat[w][0] - m);
      l += stat[w][1] * by;
      o += part[w][lane] * by;
    }
  }
  if (lane < L) *reinterpret_cast<f32x4*>(out) = o / l;
}

template <int D, bool BF, bool ALONE>
void launch_items(const AttnArgs& a, long rows_p, long rows_s, hipStream_t stream) {
  const dim3 grid(a.groups), threads(kThreads);
  constexpr int most = kThinTiles<D>;
  if (rows_p <= 16) hipLaunchKernelGGL((k_tree_attention<D, BF, 1, ALONE, false>), grid, threads, 0, stream, a);
  else if (rows_p <= 16 * most) hipLaunchKernelGGL((k_tree_attention<D, BF, most, ALONE, false>), grid, threads, 0, stream, a);
  else if (a.groups < 2 || rows_s > 16 * most) hipLaunchKernelGGL((k_tree_attention<D, BF, 0, false, false>), grid, threads, 0, stream, a);
  else if (rows_s <= 16) hipLaunchKernelGGL((k_tree_attention<D, BF, 1, ALONE, true>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((k_tree_attention<D, BF, most, ALONE, true>), grid, threads, 0, stream, a);
}

template <int D, bool BF>
void launch(const AttnArgs& a, hipStream_t stream) {
  const long rows_s = (long)a.T * a.G, rows_p = a.shared != nullptr ? a.c.n_slots * rows_s : rows_s;
  if (a.c.n_slots * a.c.heads >= kAloneFrom) launch_items<D, BF, true>(a, rows_p, rows_s, stream);
  else launch_items<D, BF, false>(a, rows_p, rows_s, stream);
  // partials that a row of the longest items may have: as many as the device has workgroups for an item, as the table has tiles for
  const int items = a.c.heads * (a.shared != nullptr ? a.sh.rb_p : a.c.n_slots * a.sh.rb_s), q_heads = a.c.heads * a.G;
  const long tiles = (long)a.c.width * a.c.page / 32, few = rows_p <= 16 * kThinTiles<D> ? kMinThin : kMinThick;
  constexpr int per = kJoinThreads<1> / 64;
  if (a.groups >= kJoinMany * items && tiles >= kJoinMany * few)
    hipLaunchKernelGGL((k_tree_attention_join<D, 8>), dim3(q_heads, a.T, a.c.n_slots), dim3(kJoinThreads<8>), 0, stream, a);
  else
    hipLaunchKernelGGL((k_tree_attention_join<D, 1>), dim3((q_heads + per - 1) / per, a.T, a.c.n_slots), dim3(kJoinThreads<1>), 0,
                       stream, a);
}

}  // namespace

bool svg_tree_attention_fits(const svg_kv_cache& c, int T, int G) {
  const Shape sh(c.n_slots, T, G, c.heads);
  const int64_t most = ((int64_t)c.width * c.page + 31) / 32 + 1 + (kItemThin > kItemThick ? kItemThin : kItemThick);
  return most * ((int64_t)sh.items_p + sh.items_s) < (1ll << 31);
}

uint64_t svg_tree_attention_bytes(const svg_kv_cache& c, int T, int G) {
  return Shape(c.n_slots, T, G, c.heads).bytes(c.dim);
}

hipError_t svg_launch_tree_attention(const svg_kv_cache& c, int layer, const float* q, int64_t ld_q, int G,
                                     const int32_t* parent, int T, const int32_t* n_nodes, const int32_t* shared,
                                     float scale, float* out, void* workspace, hipStream_t stream) {
  const int cus = svg_cu_count();
  const Shape sh(c.n_slots, T, G, c.heads);
  char* ws = static_cast<char*>(workspace);
  const AttnArgs a{c, q, parent, n_nodes, shared, out, reinterpret_cast<int*>(ws), reinterpret_cast<Span*>(ws + 256),
                   reinterpret_cast<float*>(ws + sh.stats_at()), reinterpret_cast<float*>(ws + sh.parts_at()), (long)ld_q,
                   layer, T, G, cus < kMaxGroups ? cus : kMaxGroups,
                   G == 1 ? 0u : (u32)(((1ull << 32) + G - 1) / G), sh, scale};
  const bool bf = c.type == SVG_BF16;
  if (c.dim == 64) {
    if (bf) launch<64, true>(a, stream);
    else launch<64, false>(a, stream);
  } else if (c.dim == 128) {
    if (bf) launch<128, true>(a, stream);
    else launch<128, false>(a, stream);
  } else {
    if (bf) launch<256, true>(a, stream);
    else launch<256, false>(a, stream);
  }
  return hipGetLastError();
}
