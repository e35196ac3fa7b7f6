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
// evenly over the workgroups, so unequal lengths and few rows both fill the device.  A workgroup
// writes one partial (O, M, sum) for each item it meets.  The lengths are read
// on the device: the same launch serves any lengths, also from a captured graph.
//
// A workgroup's four waves split an item's rows (16 RT each) as far as it has them,
// and its tiles otherwise.  A page is laid out in the lane order of
// v_mfma_f32_16x16x32: S^T = K Q^T leaves a row's scores in one lane column, four
// consecutive tokens in each lane, which is the order the values are stored in, so
// the probabilities go from the first product's result registers into the second's
// operand registers with no exchange and no LDS: O^T += V^T P^T.
//
// Precision.  q is fp32 and the keys 16-bit: q is normalised per row by a power of
// two and split into 16-bit parts (two of fp16: 22 bits; three of bf16: 24 bits), one
// product each; the probabilities into two parts.  Sums, maxima and accumulators
// are fp32.  One product with everything rounded to 16 bits would be off by
// 2^-9 (bf16), which the fp32 consumers of the output would see.
//
// The running maximum is raised only when a score passes it by more than
// 2^kSlack: until then probabilities above 1 are kept as they are (their scale
// 2^kLift leaves fp16 room: at most 2^(kLift + kSlack) = 2^15), which takes the
// exchange between lanes and the rescaling of O out of almost every tile.
#include "svg_cache.h"
#include "svg_internal.h"

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256, kWaves = 4;
constexpr int kMaxGroups = SVG_ATTN_MAX_GROUPS;
constexpr int kMaxSlots = 1024;
constexpr float kLift = 9.f, kSlack = 6.f;
constexpr float kLow = -1e30f;  // below every score: no token seen yet
// A probability is 2^(f s + bias), bias = kLift - f m: one operation, off by half a step of f m.  Beyond
// kFar that step would be felt as a factor, and far beyond it would overflow: 2^(f (s - m) + kLift) then.
constexpr float kFar = 65536.f;
constexpr int kMinTiles = 4;    // tiles of a workgroup at least

struct AttnArgs {
  svg_kv_cache c;
  const float* q;
  const int32_t* parent;
  const int32_t* n_nodes;
  const int32_t* shared;
  float* out;
  float* part;        // partials: see Shape
  long ld_q;
  int layer, T, G, groups;
  float scale;
};

// Rows of an item block and the places of partials, the same on host and device.
struct Shape {
  int block_p, block_s;   // rows of a prefix item, of a slot item
  int rb_p, rb_s;         // row blocks
  long items_p, items_s;
  __host__ __device__ Shape(int S, int T, int G, int heads, int rt) {
    const int most = 16 * rt * kWaves;
    const long rows_p = (long)S * T * G, rows_s = (long)T * G;
    block_p = (int)(rows_p < most ? (rows_p + 15) / 16 * 16 : most);
    block_s = (int)(rows_s < most ? (rows_s + 15) / 16 * 16 : most);
    rb_p = (int)((rows_p + block_p - 1) / block_p);
    rb_s = (int)((rows_s + block_s - 1) / block_s);
    items_p = (long)heads * rb_p;
    items_s = (long)heads * rb_s * S;
  }
  // first row of partials of workgroup w in item j (prefix items, then slot items)
  __host__ __device__ long slot_p(long w, long j) const { return (w + j) * block_p; }
  __host__ __device__ long slot_s(long w, long j) const {
    return (long)(kMaxGroups + items_p) * block_p + (w + j) * block_s;
  }
  __host__ __device__ long rows() const {
    return (long)(kMaxGroups + items_p) * block_p + (long)(kMaxGroups + items_s) * block_s;
  }
};

// How the launch's work is dealt out; the same in every workgroup.
struct Plan {
  long cum[kMaxSlots + 1];  // tiles of the slots before s (own tokens)
  int len[kMaxSlots];       // committed tokens; -1: not a valid slot
  int nodes[kMaxSlots];
  int prefix, first;        // shared tokens (a multiple of 32), a slot whose row names their pages
  long total, units_p;      // units of the launch, of the prefix items
  int groups;               // workgroups that take part
  long wred[kWaves];
  int ired[3][kWaves];
};

SVG_DEV int node_count(const AttnArgs& a, int s) {
  if (a.n_nodes == nullptr) return a.T;
  const int n = a.n_nodes[s];
  return n < 0 ? 0 : (n > a.T ? a.T : n);
}

SVG_DEV void make_plan(const AttnArgs& a, const Shape& sh, Plan& p) {
  const int S = a.c.n_slots, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // a slot with nodes whose tokens lie inside its pages is active; the others take no part
  int low = 0x7FFFFFFF, active = 0, first = S;
  for (int s = tid; s < S; s += kThreads) {
    const int n = node_count(a, s), held = a.c.pages[s];
    int len = a.c.len[s];
    if (len < 0 || held < 0 || held > a.c.width || (long)len + n > (long)held * a.c.page) len = -1;
    p.len[s] = len;
    p.nodes[s] = n;
    if (n > 0 && len >= 0) {
      low = len < low ? len : low;
      ++active;
      first = s < first ? s : first;
    }
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int l2 = __shfl_xor(low, off), f2 = __shfl_xor(first, off);
    low = l2 < low ? l2 : low;
    first = f2 < first ? f2 : first;
    active += __shfl_xor(active, off);
  }
  if (lane == 0) {
    p.ired[0][wave] = low;
    p.ired[1][wave] = active;
    p.ired[2][wave] = first;
  }
  __syncthreads();
  active = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    low = p.ired[0][w] < low ? p.ired[0][w] : low;
    first = p.ired[2][w] < first ? p.ired[2][w] : first;
    active += p.ired[1][w];
  }
  int prefix = 0;
  if (a.shared != nullptr && active > 1) {
    prefix = a.shared[0];
    prefix = prefix < 0 ? 0 : (prefix < low ? prefix : low);
    prefix &= ~31;
  }
  // tiles before each slot: four consecutive slots a thread
  long t[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = 4 * tid + i;
    t[i] = sum;
    if (s < S && p.nodes[s] > 0 && p.len[s] >= 0) sum += ((long)p.len[s] + p.nodes[s] - prefix + 31) >> 5;
  }
  long x = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const long y = __shfl_up(x, off);
    if (lane >= off) x += y;
  }
  if (lane == 63) p.wred[wave] = x;
  __syncthreads();
  long before = x - sum, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += p.wred[w];
    all += p.wred[w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * tid + i < S) p.cum[4 * tid + i] = before + t[i];
  if (tid == 0) {
    p.cum[S] = all;
    p.prefix = prefix;
    p.first = first;
    p.units_p = sh.items_p * (prefix >> 5);
    p.total = p.units_p + all * (long)a.c.heads * sh.rb_s;
    const long want = (p.total + kMinTiles - 1) / kMinTiles;
    p.groups = want < 1 ? 1 : (want < a.groups ? (int)want : a.groups);
  }
  __syncthreads();
}

// ------------------------------------------------------------ 16-bit operands
template <bool BF>
struct Ops;
template <>
struct Ops<false> {
  static constexpr int kQ = 2;  // parts of q
  SVG_DEV static f32x4 mfma(u32x4 x, u32x4 y, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
  }
  SVG_DEV static float wide(u32 h) { return (float)__builtin_bit_cast(_Float16, (uint16_t)h); }
  // bits 15 and 31: the halves that are not finite (their exponent, all ones, plus one)
  SVG_DEV static u32 odd(u32 w) { return ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u; }
  static constexpr u32 kOne = 0x3C00u;
};
template <>
struct Ops<true> {
  static constexpr int kQ = 3;
  SVG_DEV static f32x4 mfma(u32x4 x, u32x4 y, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  }
  SVG_DEV static float wide(u32 h) { return __uint_as_float(h << 16); }
  SVG_DEV static u32 odd(u32 w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }
  static constexpr u32 kOne = 0x3F80u;
};

// A pair of fp32 values split into N 16-bit parts each (part n: the rounding of what the parts
// before left over), packed two to a word.
template <bool BF, int N>
SVG_DEV void split2(float x, float y, u32 (&w)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const u32 hx = kv_round<BF>(x), hy = kv_round<BF>(y);
    w[n] = hx | (hy << 16);
    x -= Ops<BF>::wide(hx);
    y -= Ops<BF>::wide(hy);
  }
}

// ----------------------------------------------------------------- the kernel
template <int D, bool BF, int RT>
struct Attn {
  using O = Ops<BF>;
  static constexpr int NQ = O::kQ, NC = D / 32, ND = D / 16;

  struct Row {                 // per lane: row n = lane % 16 of a row tile
    f32x4 o[ND];
    float m, thr, bias, l, f;  // maximum (in units of q . k), when to raise it, exponent's offset, sum, factor
    int far;                   // (the same for the wave) maxima beyond kFar: the offset is not used
    // the maximum in powers of two that o and l are relative to
    SVG_DEV float top() const { return m == kLow ? kLow : (far ? m * f : kLift - bias); }
  };

  // This item: one head of one layer, the pages of one table row.
  struct Item {
    const char *k, *v;         // page 0 of the head, this lane's 16 bytes
    const int32_t* table;
    size_t stride;             // bytes of a page of all heads
    int log_tp;                // log2(tiles of a page)
    int n_pages;
    int len, total;            // tree tokens begin at len; tokens in all (a prefix item: beyond every tile)
  };

  SVG_DEV static int page_at(const Item& it, int tile) { return it.table[tile >> it.log_tp]; }
  // Bytes before a tile's keys (and values); a page number outside the cache gives page 0 (and NaN rows).
  SVG_DEV static size_t tile_at(const Item& it, int tile, int page) {
    const u32 in = (u32)tile & ((1u << it.log_tp) - 1u);
    return (size_t)((u32)page < (u32)it.n_pages ? page : 0) * it.stride + (size_t)in * (32 * D * 2);
  }
  SVG_DEV static void load_k(const Item& it, size_t off, u32x4 (&k)[2][NC]) {
#pragma unroll
    for (int i = 0; i < 2 * NC; ++i) k[i / NC][i % NC] = *reinterpret_cast<const u32x4*>(it.k + off + 1024 * i);
  }
  SVG_DEV static void load_v(const Item& it, size_t off, u32x4 (&v)[ND]) {
#pragma unroll
    for (int i = 0; i < ND; ++i) v[i] = *reinterpret_cast<const u32x4*>(it.v + off + 1024 * i);
  }

  // Raise the running maximum of a row tile to the largest score seen.
  SVG_DEV static void raise(Row& r, float top) {
    top = fmaxf(top, lane_xorf<16>(top));
    top = fmaxf(top, lane_xorf<32>(top));
    const float m = fmaxf(r.m, top);
    const float bias = kLift - m * r.f;
    r.far = __any(fabsf(bias) > kFar);
    const float w = __builtin_amdgcn_exp2f(r.far ? (r.m - m) * r.f : bias - r.bias);
    r.m = m;
    r.thr = m + kSlack / r.f;
    r.bias = bias;
    r.l *= w;
#pragma unroll
    for (int d = 0; d < ND; ++d) r.o[d] *= w;
  }

  // Scores to probabilities, split in two parts in the order of the second product's operand.  tree: the
  // tile holds tree tokens, of which the row sees those of `seen`; its root path being broken makes it NaN.
  SVG_DEV static void soften(const Item& it, int tile, bool tree, const f32x4 (&s)[2], Row& r, u32 seen, bool broken,
                             u32x4 (&p)[2]) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = s[j >> 2][j & 3];
    u32 ok = 0xFFu;
    if (tree) {
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
    const float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    if (__any(top > r.thr)) raise(r, top);
    if (r.far) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __builtin_fmaf(x[j] - r.m, r.f, kLift);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __builtin_fmaf(x[j], r.f, r.bias);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __builtin_amdgcn_exp2f(x[j]);
    if (tree) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!((ok >> j) & 1u)) x[j] = 0.f;
        if (broken) x[j] = __builtin_nanf("");
      }
    }
    r.l += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      u32 h[2];
      split2<BF, 2>(x[2 * w], x[2 * w + 1], h);
      p[0][w] = h[0];
      p[1][w] = h[1];
    }
  }

  // Values of a tile with tree tokens: those behind the last token are whatever the page held, and become 0.  True
  // (for the wave) if any other is not finite.
  SVG_DEV static bool clean(const Item& it, int tile, u32x4 (&v)[ND]) {
    const int first = tile * 32 + 4 * (int)((threadIdx.x & 63) >> 4);
    u32 odd = 0, keep[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int tok = first + 2 * (w & 1) + 16 * (w >> 1);
      keep[w] = (tok < it.total ? 0xFFFFu : 0u) | (tok + 1 < it.total ? 0xFFFF0000u : 0u);
    }
#pragma unroll
    for (int d = 0; d < ND; ++d) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        v[d][w] &= keep[w];
        odd |= O::odd(v[d][w]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    return __any(odd != 0);
  }

  // O += V^T P^T.
  SVG_DEV static void gather(const u32x4 (&v)[ND], const u32x4 (&p)[2], Row& r) {
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      r.o[d] = O::mfma(v[d], p[0], r.o[d]);
      r.o[d] = O::mfma(v[d], p[1], r.o[d]);
    }
  }
  // The same with values that are not finite: they are left out of the product (0 times them would be NaN in
  // every row) and make NaN where a row has a share of them.
  SVG_DEV static void gather_odd(const u32x4 (&v)[ND], const u32x4 (&p)[2], Row& r) {
    u32x4 some;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      some[w] = ((p[0][w] & 0xFFFFu) ? O::kOne : 0u) | ((p[0][w] >> 16) ? O::kOne << 16 : 0u);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      u32x4 x = v[d], y;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const u32 b = O::odd(x[w]) >> 15;  // 1 in each half
        y[w] = b * O::kOne;
        x[w] &= ~(b * 0xFFFFu);
      }
      r.o[d] = O::mfma(x, p[0], r.o[d]);
      r.o[d] = O::mfma(x, p[1], r.o[d]);
      const f32x4 hit = O::mfma(y, some, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(hit[i] == 0.f)) r.o[d][i] = __builtin_nanf("");
      __builtin_amdgcn_sched_barrier(0);  // one block at a time: a rare path must not set the kernel's registers
    }
  }

  // Tiles t, t + tw, ... up to `last` of an item for a wave's row tiles.  Keys of the next tile are
  // requested as soon as this one's are used, values likewise: one set of registers
  // of each, always a request in flight.
  SVG_DEV static void walk(const Item& it, int t, int tw, int last, const u32x4 (&q)[RT][NC][NQ], Row (&row)[RT], int nrt,
                           const u32 (&seen)[RT], u32 broken) {
    u32x4 k[2][NC], v[ND];
    int page = page_at(it, t);
    int t2 = t + tw <= last ? t + tw : last, page2 = page_at(it, t2);
    size_t at = tile_at(it, t, page);
    load_k(it, at, k);
    load_v(it, at, v);
    for (;;) {
      const int t3 = t2 + tw <= last ? t2 + tw : last, page3 = page_at(it, t3);
      const bool tree = t * 32 + 32 > it.len;
      f32x4 s[RT][2];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        s[rt][0] = s[rt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (rt < nrt) {
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              s[rt][0] = O::mfma(k[0][c], q[rt][c][n], s[rt][0]);
              s[rt][1] = O::mfma(k[1][c], q[rt][c][n], s[rt][1]);
            }
        }
      }
      const size_t at2 = tile_at(it, t2, page2);
      __builtin_amdgcn_sched_barrier(0);  // the next keys take these keys' registers, not others
      load_k(it, at2, k);
      if ((u32)page >= (u32)it.n_pages) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) row[rt].l = __builtin_nanf("");
      }
      bool odd = false;
      if (tree) odd = clean(it, t, v);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (rt < nrt) {
          u32x4 p[2];
          soften(it, t, tree, s[rt], row[rt], seen[rt], (broken >> rt) & 1u, p);
          if (odd) gather_odd(v, p, row[rt]);
          else gather(v, p, row[rt]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      load_v(it, at2, v);
      t += tw;
      if (t > last) break;
      page = page2;
      page2 = page3;
      t2 = t3;
    }
  }

  // LDS: one buffer of O for each row wave while the token waves are joined.
  static constexpr int kJoin = 2 * RT * ND * 64;  // float4s
};

template <int D, bool BF, int RT>
__global__ __launch_bounds__(kThreads, (D * RT <= 128 ? 2 : 1)) void k_tree_attention(AttnArgs a) {
  using A = Attn<D, BF, RT>;
  constexpr int NC = A::NC, ND = A::ND, NQ = A::NQ;
  __shared__ Plan plan;
  __shared__ f32x4 join[A::kJoin];
  __shared__ float stat[kWaves][RT][2][16];
  const Shape sh(a.c.n_slots, a.T, a.G, a.c.heads, RT);
  make_plan(a, sh, plan);
  const long wg = blockIdx.x;
  if (wg >= plan.groups || plan.total == 0) return;
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const long end = (wg + 1) * plan.total / plan.groups;
  for (long u = wg * plan.total / plan.groups; u < end;) {
    // the item at unit u, and the tiles of it that are this workgroup's
    int s, h, rb, t0, tiles;
    long place;
    const bool prefix = u < plan.units_p;
    if (prefix) {
      tiles = plan.prefix >> 5;
      const long j = u / tiles;
      t0 = (int)(u - j * tiles);
      rb = (int)(j % sh.rb_p);
      h = (int)(j / sh.rb_p);
      s = plan.first;
      place = sh.slot_p(wg, j);
    } else {
      const long per = (long)a.c.heads * sh.rb_s, v = u - plan.units_p;
      int lo = 0, hi = a.c.n_slots;  // the slot: cum[lo] * per <= v < cum[hi] * per
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (plan.cum[mid] * per <= v) lo = mid;
        else hi = mid;
      }
      s = lo;
      tiles = (int)(plan.cum[s + 1] - plan.cum[s]);
      const long rest = v - plan.cum[s] * per, j = rest / tiles;
      t0 = (int)(rest - j * tiles);
      rb = (int)(j % sh.rb_s);
      h = (int)(j / sh.rb_s);
      place = sh.slot_s(wg, s * per + j);
    }
    s = __builtin_amdgcn_readfirstlane(s);
    h = __builtin_amdgcn_readfirstlane(h);
    rb = __builtin_amdgcn_readfirstlane(rb);
    t0 = __builtin_amdgcn_readfirstlane(t0);
    tiles = __builtin_amdgcn_readfirstlane(tiles);
    const int t1 = __builtin_amdgcn_readfirstlane((int)(t0 + (end - u) < tiles ? t0 + (end - u) : tiles));
    u += t1 - t0;

    const int nodes = plan.nodes[s];
    const int block = prefix ? sh.block_p : sh.block_s;
    const int all_rows = prefix ? a.c.n_slots * a.T * a.G : nodes * a.G;
    const int rows = __builtin_amdgcn_readfirstlane(all_rows - rb * block < block ? all_rows - rb * block : block);
    if (rows <= 0) continue;  // a row block behind a small tree's rows
    const int row_tiles = (rows + 15) >> 4;
    const int rw = row_tiles <= RT ? 1 : (row_tiles <= 2 * RT ? 2 : 4), tw = kWaves / rw;
    const int my_r = wave % rw, my_t = wave / rw;
    int nrt = row_tiles - my_r * RT;
    nrt = nrt < 0 ? 0 : (nrt < RT ? nrt : RT);

    typename A::Item it;
    const size_t head = (size_t)a.c.page * D * 2;
    it.stride = head * a.c.heads;
    const size_t base = (size_t)a.layer * a.c.n_pages * it.stride + (size_t)h * head;
    it.k = static_cast<const char*>(a.c.k) + base + lane * 16;
    it.v = static_cast<const char*>(a.c.v) + base + lane * 16;
    const int log_tp = a.c.page == 32 ? 0 : (a.c.page == 64 ? 1 : 2);
    const int skip = prefix ? 0 : plan.prefix >> 5;  // tiles of the prefix, in front of the slot's own
    it.table = a.c.table + (size_t)s * a.c.width;
    it.log_tp = log_tp;
    it.n_pages = a.c.n_pages;
    it.len = prefix ? 0x7FFFFFFF : plan.len[s];
    it.total = prefix ? 0x7FFFFFFF : plan.len[s] + nodes;
    it.len = __builtin_amdgcn_readfirstlane(it.len);
    it.total = __builtin_amdgcn_readfirstlane(it.total);

    // the tree's root paths: lane j < 32 holds node j's, by doubling
    u32 path = 0, broken = 0;
    if (!prefix && (t1 + skip) * 32l > it.len) {
      const int j = lane & 31;
      int up = j - 1;
      if (a.parent != nullptr && j < nodes) up = a.parent[(size_t)s * a.T + j];
      broken = j == 0 ? up != -1 : (up < 0 || up >= j);
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
    }

    // the rows: q split into 16-bit parts in the order of the matrix operand
    u32x4 q[RT][NC][NQ];
    typename A::Row row[RT];
    u32 seen[RT], bad = 0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int idx = (my_r * RT + rt) * 16 + n;
      const bool live = idx < rows;
      const int all = rb * block + (live ? idx : 0);
      const int node = all / a.G;  // of the slot, or of all slots
      const float* qp = a.q + ((size_t)(prefix ? 0 : s) * a.T + node) * a.ld_q + (size_t)(h * a.G + all % a.G) * D + 8 * g;
      float x[NC][8], top = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(qp + 32 * c), hi = *reinterpret_cast<const f32x4*>(qp + 32 * c + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[c][i] = live ? (i < 4 ? lo[i] : hi[i - 4]) : 0.f;
          top = fmaxf(top, fabsf(x[c][i]));
        }
      }
      top = fmaxf(top, lane_xorf<16>(top));
      top = fmaxf(top, lane_xorf<32>(top));
      // |q| < 2 in the parts; the power of two goes into the factor (0 and what is not finite: none)
      int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
      if (top == 0.f || e == 128) e = 0;
      const float down = __uint_as_float((u32)(127 - (e > 126 ? 126 : e)) << 23);
      const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        u32 w[4][NQ];
#pragma unroll
        for (int i = 0; i < 4; ++i) split2<BF, NQ>(x[c][2 * i] * down * sign, x[c][2 * i + 1] * down * sign, w[i]);
#pragma unroll
        for (int p = 0; p < NQ; ++p) q[rt][c][p] = u32x4{w[0][p], w[1][p], w[2][p], w[3][p]};
      }
      typename A::Row& r = row[rt];
      r.f = fabsf(a.scale) * 1.44269504088896341f / down;
      r.m = kLow;
      r.thr = kLow;
      r.bias = kLift - kLow * r.f;
      r.l = 0.f;
      r.far = 0;
#pragma unroll
      for (int d = 0; d < ND; ++d) r.o[d] = f32x4{0.f, 0.f, 0.f, 0.f};
      seen[rt] = (u32)__shfl((int)path, node & 31);
      if (__shfl((int)broken, node & 31)) bad |= 1u << rt;
      __builtin_amdgcn_sched_barrier(0);
    }

    const int last = t1 - 1 + skip, t = t0 + my_t + skip;
    if (nrt > 0 && t <= last) A::walk(it, t, tw, last, q, row, nrt, seen, bad);

    // sums over the lanes of a row; maxima in powers of two from here on
    float top[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      typename A::Row& r = row[rt];
      r.l += lane_xorf<16>(r.l);
      r.l += lane_xorf<32>(r.l);
      top[rt] = r.m = r.top();
    }
    // join the token waves of a row wave
    if (tw > 1) {
      if (g == 0) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) stat[wave][rt][0][n] = row[rt].m;
      }
      __syncthreads();
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        for (int i = 0; i < tw; ++i) top[rt] = fmaxf(top[rt], stat[i * rw + my_r][rt][0][n]);
        const float w = __builtin_amdgcn_exp2f(row[rt].m - top[rt]);
        row[rt].l *= w;
#pragma unroll
        for (int d = 0; d < ND; ++d) row[rt].o[d] *= w;
        if (g == 0) stat[wave][rt][1][n] = row[rt].l;
      }
      for (int i = 1; i < tw; ++i) {
        __syncthreads();
        if (my_t == i) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int d = 0; d < ND; ++d) join[((my_r * RT + rt) * ND + d) * 64 + lane] = row[rt].o[d];
        }
        __syncthreads();
        if (my_t == 0) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            row[rt].l += stat[i * rw + my_r][rt][1][n];
#pragma unroll
            for (int d = 0; d < ND; ++d) row[rt].o[d] += join[((my_r * RT + rt) * ND + d) * 64 + lane];
          }
        }
      }
      __syncthreads();  // stat and join are free again
    }
    if (my_t == 0) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int idx = (my_r * RT + rt) * 16 + n;
        if (idx < rows) {
          float* po = a.part + 2 * sh.rows() + (size_t)(place + idx) * D + 4 * g;
#pragma unroll
          for (int d = 0; d < ND; ++d) *reinterpret_cast<f32x4*>(po + 16 * d) = row[rt].o[d];
          if (g == 0) {
            float* ps = a.part + 2 * (size_t)(place + idx);
            ps[0] = top[rt];
            ps[1] = row[rt].l;
          }
        }
      }
    }
  }
}

// The workgroup that holds unit u of `total` dealt over `groups`.
SVG_DEV long group_of(long u, long total, int groups) { return ((u + 1) * groups - 1) / total; }

// One wave per output row (slot, node, query head): its partials, joined in the
// order of the workgroups.
template <int D>
__global__ __launch_bounds__(kThreads) void k_tree_attention_join(AttnArgs a, int rt) {
  __shared__ Plan plan;
  const Shape sh(a.c.n_slots, a.T, a.G, a.c.heads, rt);
  make_plan(a, sh, plan);
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int heads = a.c.heads * a.G;
  const long x = (long)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (x >= (long)a.c.n_slots * a.T * heads) return;
  const int head = (int)(x % heads), i = (int)(x / heads) % a.T, s = (int)(x / heads / a.T);
  if (i >= plan.nodes[s]) return;  // no such node: the row stays as it was
  float* out = a.out + x * D + lane * E;
  const int h = head / a.G, gq = head % a.G;
  if (plan.len[s] < 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = __builtin_nanf("");
    return;
  }
  float m = kLow, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const float* stats = a.part;
  const float* parts = a.part + 2 * sh.rows();
  auto take = [&](long row) {
    const float pm = stats[2 * row], pl = stats[2 * row + 1];
    const float top = fmaxf(m, pm);
    const float w0 = __builtin_amdgcn_exp2f(m - top), w1 = __builtin_amdgcn_exp2f(pm - top);
    m = top;
    l = l * w0 + pl * w1;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * w0 + parts[row * D + lane * E + e] * w1;
  };
  if (plan.prefix > 0) {
    const long r = ((long)s * a.T + i) * a.G + gq;
    const long tiles = plan.prefix >> 5, j = (long)h * sh.rb_p + r / sh.block_p;
    const long w1 = group_of((j + 1) * tiles - 1, plan.total, plan.groups);
    for (long w = group_of(j * tiles, plan.total, plan.groups); w <= w1; ++w) take(sh.slot_p(w, j) + r % sh.block_p);
  }
  const long r = (long)i * a.G + gq, tiles = plan.cum[s + 1] - plan.cum[s], per = (long)a.c.heads * sh.rb_s;
  const long jj = (long)h * sh.rb_s + r / sh.block_s, u = plan.units_p + plan.cum[s] * per + jj * tiles;
  const long w1 = group_of(u + tiles - 1, plan.total, plan.groups);
  for (long w = group_of(u, plan.total, plan.groups); w <= w1; ++w) take(sh.slot_s(w, s * per + jj) + r % sh.block_s);
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = o[e] / l;
}

// Row tiles of a wave: two where an item has more than one and the registers hold them (dim 256: one).
int row_tiles(const svg_kv_cache& c, int T, int G) { return c.dim < 256 && (long)c.n_slots * T * G > 16 ? 2 : 1; }

template <int D, bool BF>
void launch(const AttnArgs& a, hipStream_t stream) {
  const int rt = row_tiles(a.c, a.T, a.G);
  if (D < 256 && rt == 2) hipLaunchKernelGGL((k_tree_attention<D, BF, (D < 256 ? 2 : 1)>), dim3(a.groups), dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((k_tree_attention<D, BF, 1>), dim3(a.groups), dim3(kThreads), 0, stream, a);
  const long rows = (long)a.c.n_slots * a.T * a.c.heads * a.G;
  hipLaunchKernelGGL((k_tree_attention_join<D>), dim3((unsigned)((rows + kWaves - 1) / kWaves)), dim3(kThreads), 0, stream, a,
                     rt);
}

}  // namespace

uint64_t svg_tree_attention_bytes(const svg_kv_cache& c, int T, int G) {
  const Shape sh(c.n_slots, T, G, c.heads, row_tiles(c, T, G));
  return (uint64_t)sh.rows() * (c.dim + 2) * 4;
}

hipError_t svg_launch_tree_attention(const svg_kv_cache& c, int layer, const float* q, int64_t ld_q, int G,
                                     const int32_t* parent, int T, const int32_t* n_nodes, const int32_t* shared,
                                     float scale, float* out, void* workspace, hipStream_t stream) {
  const int cus = svg_cu_count();
  const AttnArgs a{c, q, parent, n_nodes, shared, out, static_cast<float*>(workspace), (long)ld_q, layer, T, G,
                   cus < kMaxGroups ? cus : kMaxGroups, scale};
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
