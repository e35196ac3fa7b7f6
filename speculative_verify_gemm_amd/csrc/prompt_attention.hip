// Causal attention of prompt rows over a paged cache, gfx950.
//
// Row i of slot s attends to the positions 0 .. len[s] + i:
//   o = sum_t p_t v_t / sum_t p_t,   p_t = 2^(f (q . k_t) - m),  f = scale log2(e),
// in one pass over the tokens with a running maximum m per row.
//
// Work.  The rows of a slot and a key/value head (tokens x query heads of the group) are cut into tiles of kTile; a tile and
// the tokens that it sees form an item.  Items are counted by the tokens that they see and all of them, in order, are
// dealt out evenly over the workgroups, so that one long row fills the device as well as many prompts do.  A workgroup that does
// not have all of an item writes a partial (O, m, sum); a second launch joins those.  Lengths are read on the device.
//
// Layout.  A page is laid out in the lane order of v_mfma_f32_16x16x32: S^T = K Q^T leaves a row's scores in one
// lane column, four consecutive tokens in each lane, which is the order the values are stored in, so the probabilities
// go from the first product's result registers into the second's operand registers: O^T += V^T P^T.
// The sum of the probabilities is a product as well, with ones: it adds up what the second product sees.
//
// Tiles.  32 tokens' keys and values go straight into a ring of four places in LDS.  While every row sees a whole tile, a wave
// computes the next tile's scores beside this one's probabilities (v_mfma and v_exp from one wave side by side), reads fragments
// ahead of their products, and does not touch masks; the tiles of the rows' own tokens go one by one.  A running maximum is
// raised only when a score passes it by 2^kSlack.
//
// Precision.  Scores, maxima, sums and accumulators are fp32.  The probabilities enter the second product rounded to the cache's type,
// as the values are held in it, and their sum is that of the rounded ones: a second part of them would be half as many
// products again.  Distance from the 64-bit result over the result's size (rms), here | all in fp32 but the output: bf16 2.0e-3 | 1.7e-3,
// fp16 2.5e-4 | 2.1e-4.
//
// Bound by the matrix units and the vector instructions of the exponential together.  1000 rows behind 30001 tokens, 8 heads of 128
// for 32, bf16: 500 us, 1.0 PFLOP/s (a library product of 8192^3: 1.46), matrix units and vector units each busy 46 to 47 % of the
// cycles (in how many neither is has not been counted); heads of 256 1.05 PFLOP/s; heads of 64 0.80, where the exponentials weigh
// twice as much.  Shorter items pay for their starts, the rows' own tokens and the partials: a prompt of 4099 tokens, 32 heads of 128:
// 200 us, 0.69 PFLOP/s, 15 of them the join.
// Heads of 256 have 16 rows a wave: 32 rows fill the registers with one wave a SIMD and take as long (step 148 | 144 us).
#include <math.h>

#include <type_traits>

#include "../../include/svgemm_prompt.h"
#include "svg_cache.h"
#include "svg_internal.h"
#include "svg_lds.h"

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

constexpr int kTile = 128;                   // rows of an item
constexpr int kMaxSlots = 1024;
// Token tiles that starting and ending an item counts as: finding it, the wait for its first tile, the tiles of the rows' own
// tokens, which take half as long again, and the results' way out were 7 to 8 tiles of 1900 cycles (counted as 4 | 8: a prompt of
// 4099 tokens, 32 heads of 128, 214 | 203 us, 24 slots of a step 140 | 137 us).
constexpr int kItem = 8;
constexpr int kLeast = 4;                    // token tiles of a workgroup at least

template <bool BF>
SVG_DEV f32x4 mfma(u32x4 x, u32x4 y, f32x4 c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, y), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x), __builtin_bit_cast(f16x8, y), c, 0, 0, 0);
}
// Two values rounded to nearest, packed.
template <bool BF>
SVG_DEV u32 pack2(float x, float y) {
  if constexpr (BF) return __builtin_bit_cast(u32, __builtin_convertvector(f32x2{x, y}, bf16x2));
  else return __builtin_bit_cast(u32, __builtin_convertvector(f32x2{x, y}, f16x2));
}
template <bool BF>
constexpr u32 kOnes = BF ? 0x3F803F80u : 0x3C003C00u;
// Bits 15 and 31: the halves that are not finite (their exponent, all ones, plus one).
template <bool BF>
SVG_DEV u32 odd_halves(u32 w) {
  return BF ? ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u : ((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
}

// A probability is at most 2^kTop: the running maximum is raised when a score passes it by kSlack, and everything is lifted by
// kTop - kSlack.  fp16: up, so that small ones stay above the type's smallest number.  bf16, whose values reach fp32's largest number: down,
// so that those of 2^25 tokens (a table row's most) add up to less than 1 and O stays below the largest value; a product of O is
// rounded to fp32's smallest number, 2^-149, which is 2^-116 in an output.
constexpr float kSlack = 7.f;
template <bool BF>
constexpr float kTop = BF ? -26.f : 15.f;
template <bool BF>
constexpr float kLift = kTop<BF> - kSlack;
// A probability is 2^(f s + bias), bias = kLift - m: one operation.  What rounds kLift - m is the same for all of a row's
// probabilities since then, and goes out with their sum; the largest is a power of two and loses nothing to 16 bits.  Beyond kFar the product
// inside that operation and the rounded one that m came from would differ by 2^-11 and more (from 2^24 on by whole numbers, and kLift - m
// loses kLift), which fp16 has no room for: there it is 2^((f s - m) + kLift) with each step rounded, 2^kLift where s is the maximum,
// whatever its size.  Such rows cost the others a branch in the step that raises maxima (a prompt of 4099 tokens 201 -> 204 us, 1000
// rows behind 30001 504 either way; a clamp of every probability costs those 4 %).
constexpr float kFar = 16384.f;

// What the second launch has to know of an item that begins in a workgroup's share and does not end there.
struct Join {
  u32 last;               // the last workgroup that has some of it (the workgroup itself: there is no such item)
  int first, rows, row0, head;
};

struct Args {
  svg_kv_cache c;
  const uint16_t* q;
  uint16_t* out;
  const int32_t *start, *count;
  float* stats;   // [groups][2][kTile] (kLift less the maximum, sum): infinite where no token was seen
  float* parts;   // [groups][2][kTile][dim]
  Join* joins;    // [groups + 1]: the last one's `last` is the number of workgroups that took part
  long ld_q;
  int layer, G, n_rows, groups;
  float scale;
};

// ---------------------------------------------------------------------- plan
// Cost of the items of a slot, in 1 / G of a token tile of 32: item j of a head counts G * (tiles of the committed tokens +
// kItem) + per * (j + 1), where per = kTile / 32 covers the rows' own tokens; the cost of the first j is a polynomial.  It
// decides only how the work is shared out.
struct Slot {
  int first, n, len;    // its rows in q and out, committed tokens
  bool valid;
  u32 items;            // of a head
  unsigned long long base;
  SVG_DEV unsigned long long before(unsigned long long j) const { return base * j + (kTile / 64) * j * (j + 1); }
  SVG_DEV unsigned long long cost(u32 j) const { return base + (kTile / 32) * (unsigned long long)(j + 1); }
};
// Values that are the same for the wave, in scalar registers.
SVG_DEV int uniform_i(int v) { return __builtin_amdgcn_readfirstlane(v); }
SVG_DEV unsigned long long uniform_l(unsigned long long v) {
  return (unsigned long long)(u32)uniform_i((int)(u32)(v >> 32)) << 32 | (u32)uniform_i((int)(u32)v);
}

template <bool UNIFORM>
SVG_DEV Slot slot_of(const Args& a, int s) {
  Slot x;
  const int first = a.start[s], held = a.c.pages[s];
  int n = a.count[s];
  x.len = a.c.len[s];
  if (first < 0 || first >= a.n_rows || n < 0) n = 0;
  else if (n > a.n_rows - first) n = a.n_rows - first;
  x.first = first;
  x.n = n;
  x.valid = x.len >= 0 && held >= 0 && held <= a.c.width && (long)x.len + n <= (long)held * a.c.page;
  if (UNIFORM) {
    x.first = uniform_i(x.first);
    x.n = uniform_i(x.n);
    x.len = uniform_i(x.len);
    x.valid = uniform_i(x.valid) != 0;
  }
  x.items = (u32)(((long)x.n * a.G + kTile - 1) / kTile);
  x.base = (unsigned long long)a.G * ((x.valid ? (u32)x.len >> 5 : 0u) + kItem);
  return x;
}

struct Plan {
  unsigned long long cum[kMaxSlots + 1];  // cost of the slots before s
  unsigned long long red[8];
};

SVG_DEV unsigned long long shfl_up64(unsigned long long v, int off) {
  const u32 lo = (u32)__shfl_up((int)(u32)v, off), hi = (u32)__shfl_up((int)(u32)(v >> 32), off);
  return (unsigned long long)hi << 32 | lo;
}

template <int WAVES>
SVG_DEV void make_plan(const Args& a, Plan& p) {
  const int S = a.c.n_slots, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int EACH = kMaxSlots / (64 * WAVES);
  unsigned long long c[EACH], sum = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int s = tid * EACH + i;
    c[i] = 0;
    if (s < S) {
      const Slot x = slot_of<false>(a, s);
      c[i] = x.before(x.items) * (unsigned long long)a.c.heads;
    }
    sum += c[i];
  }
  unsigned long long upto = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const unsigned long long y = shfl_up64(upto, off);
    if (lane >= off) upto += y;
  }
  if (lane == 63) p.red[wave] = upto;
  __syncthreads();
  unsigned long long at = upto - sum;
#pragma unroll
  for (int w = 0; w < WAVES; ++w)
    if (w < wave) at += p.red[w];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int s = tid * EACH + i;
    if (s < S) p.cum[s] = at;
    at += c[i];
  }
  if (tid == 64 * WAVES - 1) p.cum[S] = at;
  __syncthreads();
}

struct Deal {
  unsigned long long total;
  unsigned long long quot, rest;
  u32 groups;  // workgroups that take part: w has the costs from start(w) on
  SVG_DEV unsigned long long start(u32 w) const { return w * quot + (w < rest ? w : rest); }
};
SVG_DEV Deal deal_of(const Args& a, const Plan& p) {
  Deal d;
  d.total = uniform_l(p.cum[a.c.n_slots]);
  const unsigned long long want = d.total / ((unsigned long long)a.G * (kItem + kLeast)) + 1;
  d.groups = (u32)(want < (unsigned long long)a.groups ? want : (unsigned long long)a.groups);
  d.quot = uniform_l(d.total / d.groups);
  d.rest = d.total - d.quot * d.groups;
  return d;
}

// The item at cost `at`.
struct Item {
  int s;
  u32 h, j;
  unsigned long long from, cost;  // of the whole launch; its own
};
SVG_DEV Item item_at(const Args& a, const Plan& p, unsigned long long at, Slot& x) {
  int s = 0;
  for (int step = kMaxSlots / 2; step > 0; step >>= 1)
    if (s + step <= a.c.n_slots - 1 && p.cum[s + step] <= at) s += step;  // the last slot that begins at or before
  s = uniform_i(s);
  x = slot_of<true>(a, s);
  const unsigned long long first = uniform_l(p.cum[s]), head = x.before(x.items), in = at - first;
  Item it;
  it.s = s;
  it.h = (u32)uniform_i((int)(u32)(in / head));
  const unsigned long long rest = in - it.h * head;
  u32 lo = 0, hi = x.items;  // the last j with before(j) <= rest
  while (hi - lo > 1) {
    const u32 mid = (lo + hi) >> 1;
    if (x.before(mid) <= rest) lo = mid;
    else hi = mid;
  }
  lo = (u32)uniform_i((int)lo);
  it.j = lo;
  it.from = first + it.h * head + x.before(lo);
  it.cost = x.cost(lo);
  return it;
}
// The item behind it, which begins at cost `at`.
SVG_DEV void next_item(const Args& a, const Plan& p, unsigned long long at, Item& it, Slot& x) {
  if (it.j + 1 < x.items) {
    ++it.j;
  } else if (it.h + 1 < (u32)a.c.heads) {
    ++it.h;
    it.j = 0;
  } else {
    it = item_at(a, p, at, x);
    return;
  }
  it.from = at;
  it.cost = x.cost(it.j);
}
// Tokens of an item: what its last row sees; tiles of 32.
SVG_DEV int tokens_of(const Args& a, const Slot& x, u32 j) {
  const int rows = x.n * a.G, end = (int)(j + 1) * kTile < rows ? (int)(j + 1) * kTile : rows;
  return x.len + (end - 1) / a.G + 1;
}
// The token tile where a share that begins at cost c of the item begins.
SVG_DEV int tile_at(unsigned long long c, const Item& it, int tiles) { return (int)(c * (u32)tiles / it.cost); }

// ---------------------------------------------------------------------- kernel
template <int D, bool BF, int STAGES, int RT>
struct Kernel {
  static constexpr int WAVES = kTile / 16 / RT;         // RT row tiles of 16 each
  static constexpr int NC = D / 32, ND = D / 16;     // fragments of a token tile's half, of its values
  static constexpr int HALF = D * 64;                // bytes of a tile's keys, of its values
  static constexpr int STAGE = 2 * HALF, LOADS = STAGE / 1024 / WAVES;

  struct Row {
    f32x4 o[ND];
    f32x4 l;
    float limit;     // the score from which the maximum m is raised: m + kSlack; -infinity without a token, and beyond kFar
    float bias;      // what is added to the exponents: kLift - m; kLift beyond kFar, where m is kept in LDS (`far`)
    SVG_DEV bool beyond() const { return limit == -INFINITY && bias != 0.f; }
    SVG_DEV float m(const float* far) const { return limit != -INFINITY ? limit - kSlack : (bias != 0.f ? *far : -INFINITY); }
    // kLift less the maximum that o and l are relative to
    SVG_DEV float offset(const float* far) const { return limit != -INFINITY ? bias : (bias != 0.f ? kLift<BF> - *far : INFINITY); }
  };

  // The pages of a slot's table row, 64 entries at a time: entry base + l in lane l (reading them one by one would wait for
  // the tiles that are on their way).  Numbers outside the cache and pages that other slots hold too are marked.
  static constexpr u32 kOutside = 1u << 31, kShared = 1u << 30;
  static constexpr int kNone = 0x7FFFFFFF;
  struct Pages {
    const int32_t *table, *refs;
    int first_own, n_pages, last, base;   // the entry of the first of the step's own positions; the last entry
    u32 v, first;                         // first: entries 0 .. 63, kept for the slot's next item
    SVG_DEV void look(int entry) {
      base = entry;
      const int e = entry + (int)(threadIdx.x & 63u);
      v = kOutside;
      if (e <= last) {
        const u32 page = (u32)table[e];
        if (page < (u32)n_pages) {
          v = page;
          if (refs != nullptr && e >= first_own && refs[page] > 1) v |= kShared;
        }
      }
    }
    SVG_DEV void rewind() {
      base = 0;
      v = first;
    }
    SVG_DEV u32 at(int entry) {
      if (entry - base >= 64) look(entry);
      return (u32)__builtin_amdgcn_readlane((int)v, entry - base);
    }
  };

  // Value that is not finite in a tile that not all rows see whole: taken out of the product, and put into the sums of the
  // rows that see it as NaN.
  SVG_DEV static void odd_values(const char* v, int lane, const u32x4 (&p)[RT], const u32x4 (&sees)[RT], Row (&row)[RT]) {
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      u32x4 x = *reinterpret_cast<const u32x4*>(v + d * 1024 + lane * 16), is;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const u32 mask = (odd_halves<BF>(x[w]) >> 15) * 0xFFFFu;  // (bits 0 and 16 times all ones: no carry)
        is[w] = mask & kOnes<BF>;
        x[w] &= ~mask;
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const f32x4 hits = mfma<BF>(is, sees[rt], f32x4{});
        row[rt].o[d] = mfma<BF>(x, p[rt], row[rt].o[d]);
#pragma unroll
        for (int e = 0; e < 4; ++e) row[rt].o[d][e] = hits[e] > 0.f ? __builtin_nanf("") : row[rt].o[d][e];
      }
      __builtin_amdgcn_sched_barrier(0);  // one at a time: this path must not set the kernel's registers
    }
  }

  SVG_DEV static void run(const Args& a, char* lds, Plan& plan, float* far_all) {
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform_i(tid >> 6), col = lane & 15, quad = lane >> 4;
    make_plan<WAVES>(a, plan);
    const Deal deal = deal_of(a, plan);
    // XCDs take stretches of neighbouring workgroups, which read the same keys
    const u32 per = deal.groups >> 3, more = deal.groups & 7u, xcd = blockIdx.x & 7u;
    if ((blockIdx.x >> 3) >= per + (xcd < more ? 1u : 0u)) return;
    const u32 wg = xcd * per + (xcd < more ? xcd : more) + (blockIdx.x >> 3);
    if (tid == 0) {
      a.joins[wg].last = wg;
      if (wg == 0) a.joins[a.groups].last = deal.groups;
    }
    unsigned long long at = deal.start(wg);
    const unsigned long long end = deal.start(wg + 1);
    const u32 base = lds_at(lds);
    const float f = a.scale * 1.4426950408889634f;
    float* const far = far_all + tid % 64 + wave * (64 * RT);
    const int shift = __builtin_ctz(a.c.page);
    const size_t page_bytes = (size_t)a.c.heads * a.c.page * D * 2;
    const int G = a.G;
    static_assert(LOADS % 2 == 0 && HALF / 1024 == LOADS / 2 * WAVES, "a wave's pieces of the keys, then of the values");
    const u32 piece_at = (u32)wave * 1024u + (u32)lane * 16u;
    Slot x;
    Item it;
    Pages pages;
    pages.refs = a.c.refs;
    pages.n_pages = a.c.n_pages;
    int pages_of = -1;  // the slot that `pages` is of
    for (bool more = false; at < end; more = true) {
      if (more) next_item(a, plan, at, it, x);
      else it = item_at(a, plan, at, x);
      const unsigned long long stop = it.from + it.cost < end ? it.from + it.cost : end;
      const bool whole = at == it.from && stop == it.from + it.cost;
      const int which = at == it.from ? 1 : 0;  // the partial's place: an item's first share, or a later one
      const int slot_no = it.s, head = (int)it.h, len = x.len, first = x.first;
      const int row0 = (int)it.j * kTile, all_rows = x.n * G, rows = all_rows - row0 < kTile ? all_rows - row0 : kTile;
      const bool valid = x.valid;
      const int tokens = uniform_i(valid ? tokens_of(a, x, it.j) : 0), tiles = (tokens + 31) >> 5;
      const int t0 = uniform_i(at == it.from ? 0 : tile_at(at - it.from, it, tiles));
      const int t1 = uniform_i(stop == it.from + it.cost ? tiles : tile_at(stop - it.from, it, tiles));
      at = stop;
      // this lane's rows (those past the item's: its last one, not stored), and the last position that each sees
      const int mine = wave * 16 * RT;
      const bool live = mine < rows;
      int seen[RT];
      size_t q_at[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        int r = mine + 16 * rt + col;
        r = row0 + (r < rows ? r : rows - 1);
        const int tok = r / G;
        seen[rt] = len + tok;
        q_at[rt] = (size_t)(first + tok) * (size_t)a.ld_q + (size_t)(head * G + (r - tok * G)) * D;
      }
      const int low = len + (row0 + (mine < rows ? mine : rows - 1)) / G;                                      // of the wave's rows
      const int high = len + (row0 + (mine + 16 * RT < rows ? mine + 16 * RT : rows) - 1) / G;
      u32x4 q[RT][NC];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int c = 0; c < NC; ++c) q[rt][c] = *reinterpret_cast<const u32x4*>(a.q + q_at[rt] + 32 * c + 8 * quad);
      Row row[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
        for (int d = 0; d < ND; ++d) row[rt].o[d] = f32x4{};
        row[rt].l = f32x4{};
        row[rt].limit = -INFINITY;
        row[rt].bias = 0.f;
      }
      // pages: position p lies in entry p >> shift of the slot's table row
      if (slot_no != pages_of) {
        pages_of = slot_no;
        pages.table = a.c.table + (size_t)slot_no * a.c.width;
        pages.first_own = len >> shift;
        pages.last = valid ? (len + x.n - 1) >> shift : -1;
        pages.look(0);
        pages.first = pages.v;
      } else {
        pages.rewind();
      }
      const char* kl = static_cast<const char*>(a.c.k) + (size_t)a.layer * a.c.n_pages * page_bytes + (size_t)head * a.c.page * D * 2;
      const char* vl = static_cast<const char*>(a.c.v) + (size_t)a.layer * a.c.n_pages * page_bytes + (size_t)head * a.c.page * D * 2;
      // Requests a tile; the first of its positions that makes the rows which see it NaN (no page of the cache: all; the
      // step's own positions in a page that other slots hold: those).
      const char *kp = nullptr, *vp = nullptr;  // the tile that was requested last
      int from = kNone;
      auto fetch = [&](int t, int slot) {
        const int p = t * 32;
        if (t == t0 || (p & (a.c.page - 1)) == 0) {
          const u32 mark = pages.at(p >> shift), page = mark & kOutside ? 0u : mark & ~kShared;
          const size_t off = (size_t)page * page_bytes + (size_t)(p & (a.c.page - 1)) * D * 2;
          kp = kl + off;
          vp = vl + off;
          from = mark & kOutside ? 0 : (mark & kShared ? len : kNone);
        } else {
          kp += 64 * D;
          vp += 64 * D;
        }
        const u32 to = base + (u32)slot * STAGE + wave * 1024u;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
          load_to_lds(i < LOADS / 2 ? kp : vp, piece_at + (u32)(i % (LOADS / 2)) * (WAVES * 1024u), to + (u32)i * (WAVES * 1024u));
        return from;
      };
      barrier();  // (the places of the item before are free: its loads have arrived, and nobody reads them any more)
      int odd_from[STAGES];
#pragma unroll
      for (int i = 0; i < STAGES - 1; ++i) odd_from[i] = t0 + i < t1 ? fetch(t0 + i, i) : kNone;
      int slot = 0, t = t0;
      // What the loops' tops share: tile t + AHEAD has arrived for the whole workgroup, and tile t + STAGES - 1 is requested into the
      // place of tile t - 1, which nobody reads any more.
      int nan_from = kNone;
      auto arrive = [&](auto ahead, auto more) {
        constexpr int LEFT = STAGES - 2 - decltype(ahead)::value;
        if (decltype(more)::value || t + STAGES - 2 < t1) wait_loads<LOADS * LEFT>();
        else wait_loads<0>();
        barrier();
      };
      auto request = [&](auto more) {
        nan_from = odd_from[0];
#pragma unroll
        for (int i = 0; i + 1 < STAGES - 1; ++i) odd_from[i] = odd_from[i + 1];
        if (decltype(more)::value || t + STAGES - 1 < t1) odd_from[STAGES - 2] = fetch(t + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
      };
      // Fragments are read AHEAD of the products that need them.
      constexpr int AHEAD = 3;
      auto scores = [&](const char* k, f32x4 (&s)[RT][2]) {
        u32x4 kf[2][2];
        auto read_k = [&](int c) {
          kf[c & 1][0] = *reinterpret_cast<const u32x4*>(k + c * 1024 + lane * 16);
          kf[c & 1][1] = *reinterpret_cast<const u32x4*>(k + (NC + c) * 1024 + lane * 16);
        };
        read_k(0);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if (c + 1 < NC) read_k(c + 1);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 2; ++i) s[rt][i] = mfma<BF>(kf[c & 1][i], q[rt][c], c == 0 ? f32x4{} : s[rt][i]);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      auto highest = [&](const f32x4 (&s)[2]) {
        float top = fmaxf(s[0][0], s[0][1]);
        top = fmaxf(fmaxf(top, s[0][2]), s[0][3]);
        top = fmaxf(fmaxf(top, s[1][0]), s[1][1]);
        return fmaxf(fmaxf(top, s[1][2]), s[1][3]);
      };
      // Raises a row's maximum to `top` (for the whole row: its four lanes agree).
      auto raise = [&](Row& r, float top, float* far) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        float before = r.limit - kSlack;
        if (__builtin_expect(__any(r.beyond()), false)) before = r.m(far);
        if (top - before > kSlack) {
          const bool beyond = fabsf(top) > kFar;
          float bias = kLift<BF> - top, by = __builtin_amdgcn_exp2f(bias - r.bias), limit = top + kSlack;
          if (__builtin_expect(__any(beyond || r.beyond()), false)) {
            by = beyond || r.beyond() ? __builtin_amdgcn_exp2f(before - top) : by;
            limit = beyond ? -INFINITY : limit;
            bias = beyond ? kLift<BF> : bias;
            if (beyond) *far = top;
          }
          by = before == -INFINITY ? 0.f : by;
          r.limit = limit;
          r.bias = bias;
#pragma unroll
          for (int d = 0; d < ND; ++d) r.o[d] *= by;
          r.l *= by;
        }
      };
      // Scores s of a row beyond kFar less its maximum, in the unit that they come in (s * unit are the exponents).
      auto nearer = [&](const Row& r, f32x4 (&s)[2], float unit, float back, const float* far) {
        if (!r.beyond()) return;
        const float m = *far;
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e >> 2][e & 3] = (s[e >> 2][e & 3] * unit - m) * back;
      };
      auto weights = [&](const f32x4 (&s)[2], float scale, float bias) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[e >> 2][e & 3], scale, bias));
        return u32x4{pack2<BF>(w[0], w[1]), pack2<BF>(w[2], w[3]), pack2<BF>(w[4], w[5]), pack2<BF>(w[6], w[7])};
      };
      const u32x4 ones{kOnes<BF>, kOnes<BF>, kOnes<BF>, kOnes<BF>};
      auto values = [&](const char* v, const u32x4 (&p)[RT]) {
        u32x4 y[AHEAD + 1];
        auto read_v = [&](int d) { y[d % (AHEAD + 1)] = *reinterpret_cast<const u32x4*>(v + d * 1024 + lane * 16); };
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) read_v(d);
#pragma unroll
        for (int d = 0; d < ND; ++d) {
          if (d + AHEAD < ND) read_v(d + AHEAD);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            if (d == 0) row[rt].l = mfma<BF>(ones, p[rt], row[rt].l);
            row[rt].o[d] = mfma<BF>(y[d % (AHEAD + 1)], p[rt], row[rt].o[d]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      // Tiles that every row of the item sees whole: the next tile's scores are computed beside this one's probabilities.
      int whole_tiles = (len + row0 / G + 1) >> 5;
      whole_tiles = f > 0.f && whole_tiles < t1 ? whole_tiles : (f > 0.f ? t1 : t0);
      if (t < whole_tiles) {
        f32x4 s[RT][2], ahead[RT][2];
        bool poisoned = false;
        if (t + STAGES - 2 < t1) wait_loads<LOADS * (STAGES - 2)>();
        else wait_loads<0>();
        barrier();
        scores(lds, s);
        float top[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) top[rt] = highest(s[rt]) * f;
        auto tile = [&](auto more) {
          arrive(std::integral_constant<int, 1>{}, more);
          const char* v = lds + slot * STAGE + HALF;
          const int next = slot + 1 == STAGES ? 0 : slot + 1;
          // the values' first fragments before all else
          u32x4 y[AHEAD + 1], kf[2][2];
          auto read_v = [&](int d) { y[d % (AHEAD + 1)] = *reinterpret_cast<const u32x4*>(v + d * 1024 + lane * 16); };
          const char* k = lds + next * STAGE + lane * 16;
          auto read_k = [&](int c) {
            kf[c & 1][0] = *reinterpret_cast<const u32x4*>(k + c * 1024);
            kf[c & 1][1] = *reinterpret_cast<const u32x4*>(k + (NC + c) * 1024);
          };
          read_k(0);
#pragma unroll
          for (int d = 0; d < AHEAD; ++d) read_v(d);
          __builtin_amdgcn_sched_barrier(0);
          request(more);
          poisoned = poisoned || nan_from != kNone;
          slot = next;
          ++t;
          if (!live) return;
          bool raised = false;
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) raised = raised || top[rt] > row[rt].limit;
          if (__any(raised)) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              raise(row[rt], top[rt], far + 64 * rt);
              if (__builtin_expect(__any(row[rt].beyond()), false)) nearer(row[rt], s[rt], f, 1.f / f, far + 64 * rt);
            }
          }
          u32x4 p[RT];
          __builtin_amdgcn_s_setprio(1);
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            if (c + 1 < NC) read_k(c + 1);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
#pragma unroll
              for (int i = 0; i < 2; ++i) ahead[rt][i] = mfma<BF>(kf[c & 1][i], q[rt][c], c == 0 ? f32x4{} : ahead[rt][i]);
            // this share of the probabilities, pairs of scores
#pragma unroll
            for (int n = c * 4 * RT / NC; n < (c + 1) * 4 * RT / NC; ++n) {
              const int rt = n / 4, e = n % 4;
              p[rt][e] = pack2<BF>(__builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][e >> 1][2 * (e & 1)], f, row[rt].bias)),
                                   __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][e >> 1][2 * (e & 1) + 1], f, row[rt].bias)));
            }
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            if (d + AHEAD < ND) read_v(d + AHEAD);
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
              if (d == 0) row[rt].l = mfma<BF>(ones, p[rt], row[rt].l);
              row[rt].o[d] = mfma<BF>(y[d % (AHEAD + 1)], p[rt], row[rt].o[d]);
            }
            if (d >= 1 && d <= RT) top[d - 1] = highest(ahead[d - 1]) * f;
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            s[rt][0] = ahead[rt][0];
            s[rt][1] = ahead[rt][1];
          }
          __builtin_amdgcn_s_setprio(0);
        };
        while (t < whole_tiles && t + STAGES - 1 < t1) tile(std::true_type{});
        while (t < whole_tiles) tile(std::false_type{});
        if (poisoned) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) row[rt].l = f32x4{} + __builtin_nanf("");
        }
      }
      for (; t < t1; ++t) {
        arrive(std::integral_constant<int, 0>{}, std::false_type{});
        request(std::false_type{});
        const char* k = lds + slot * STAGE;
        const char* v = k + HALF;
        slot = slot + 1 == STAGES ? 0 : slot + 1;
        const int p0 = t * 32;
        if (!live || p0 > high) continue;
        f32x4 s[RT][2];
        scores(k, s);
        // scaled here, so that what a row does not see can be left out whatever the scale
        const bool part = p0 + 31 > low;  // (not all of the wave's rows see all of the tile)
        u32x4 p[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
          for (int i = 0; i < 2; ++i) s[rt][i] *= f;
          if (part || nan_from != kNone) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tok = p0 + 16 * i + 4 * quad + e;
                if (tok >= nan_from) s[rt][i][e] = __builtin_nanf("");
                if (tok > seen[rt]) s[rt][i][e] = -INFINITY;
              }
          }
          const float top = highest(s[rt]);
          if (__any(top > row[rt].limit)) {
            raise(row[rt], top, far + 64 * rt);
            if (__builtin_expect(__any(row[rt].beyond()), false)) nearer(row[rt], s[rt], 1.f, 1.f, far + 64 * rt);
          }
          p[rt] = weights(s[rt], 1.f, row[rt].bias);
        }
        bool odd = false;
        if (part) {
          u16x2 largest{0, 0};  // of the values' patterns without their signs
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            const u32x4 y = *reinterpret_cast<const u32x4*>(v + d * 1024 + lane * 16);
#pragma unroll
            for (int w = 0; w < 4; ++w)
              largest = __builtin_elementwise_max(largest, __builtin_bit_cast(u16x2, y[w] & 0x7FFF7FFFu));
            if (d % 4 == 3) __builtin_amdgcn_sched_barrier(0);
          }
          constexpr unsigned short kInf = BF ? 0x7F80 : 0x7C00;
          odd = largest[0] >= kInf || largest[1] >= kInf;
        }
        if (__any(odd)) {
          u32x4 sees[RT];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tok = p0 + 16 * (e >> 1) + 4 * quad + 2 * (e & 1);
              sees[rt][e] = (tok <= seen[rt] ? kOnes<BF> & 0xFFFFu : 0u) | (tok + 1 <= seen[rt] ? kOnes<BF> & 0xFFFF0000u : 0u);
            }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) row[rt].l = mfma<BF>(ones, p[rt], row[rt].l);
          odd_values(v, lane, p, sees, row);
        } else {
          values(v, p);
        }
      }
      if (stop < it.from + it.cost && which == 1 && tid == 0) {
        // the item goes on in the next workgroups' shares
        u32 last = wg + 1;
        while (deal.start(last + 1) < it.from + it.cost) ++last;
        a.joins[wg] = Join{last, first, rows, row0, head};
      }
      if (!live) continue;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int r = mine + 16 * rt + col;
        if (r >= rows) continue;
        Row& w = row[rt];
        if (whole) {
          const float inv = valid ? 1.f / w.l[0] : __builtin_nanf("");
          const int tok = (row0 + r) / G, qh = head * G + (row0 + r - tok * G);
          uint16_t* to = a.out + ((size_t)(first + tok) * a.c.heads * G + qh) * D + 4 * quad;
#pragma unroll
          for (int d = 0; d < ND; ++d)
            *reinterpret_cast<uint2*>(to + 16 * d) = make_uint2(pack2<BF>(w.o[d][0] * inv, w.o[d][1] * inv),
                                                                pack2<BF>(w.o[d][2] * inv, w.o[d][3] * inv));
        } else {
          const size_t at_part = ((size_t)wg * 2 + which) * kTile + r;
          float* to = a.parts + at_part * D + 4 * quad;
#pragma unroll
          for (int d = 0; d < ND; ++d)
            *reinterpret_cast<float4*>(to + 16 * d) = make_float4(w.o[d][0], w.o[d][1], w.o[d][2], w.o[d][3]);
          if (quad == 0) {
            a.stats[at_part * 2] = w.offset(far + 64 * rt);
            a.stats[at_part * 2 + 1] = valid ? w.l[0] : __builtin_nanf("");
          }
        }
      }
    }
  }
};

template <int D, bool BF, int STAGES, int RT>
__global__ __launch_bounds__(kTile / 16 / RT * 64, D == 64 ? 3 : 2) void k_prompt_attention(Args a) {
  __shared__ __attribute__((aligned(1024))) char lds[STAGES * Kernel<D, BF, STAGES, RT>::STAGE];
  __shared__ Plan plan;
  __shared__ float far[kTile / 16 * 64];
  Kernel<D, BF, STAGES, RT>::run(a, lds, plan, far);
}

// Joins the partials of the item that begins in workgroup blockIdx.x's share and goes on behind it: its first share's partial
// lies at place 1 of that workgroup, the others' at place 0 of the next ones.
// Bound by the partials' bytes: 512 workgroups' of 128 rows of 128 values, 77 MB, 15 us; 256 of 256 values, 61 MB, 12 us (one partial after the
// other, 16 rows a workgroup: 16 us each).
constexpr int kJoinRows = 8, kJoinWaves = 4;
template <int D, bool BF>
__global__ __launch_bounds__(64 * kJoinWaves) void k_prompt_attention_join(Args a) {
  const u32 wg = blockIdx.x, took_part = a.joins[a.groups].last;
  const Join j = a.joins[wg];
  if (wg >= took_part || j.last <= wg) return;
  const int H = a.c.heads;
  for (int u = threadIdx.x; u < kJoinRows * (D / 4); u += 64 * kJoinWaves) {
    const int r = blockIdx.y * kJoinRows + u / (D / 4), d = 4 * (u % (D / 4));
    if (r >= j.rows) continue;
    // the weights go by the smallest offset (the largest maximum) so far; two partials on their way at once
    float low = INFINITY, sum = 0.f;
    f32x4 o{};
    for (u32 w = wg; w <= j.last; w += 2) {
      const bool two = w < j.last;
      const size_t at0 = ((size_t)w * 2 + (w == wg)) * kTile + r, at1 = two ? (size_t)(w + 1) * 2 * kTile + r : at0;
      const float2 s0 = *reinterpret_cast<const float2*>(a.stats + at0 * 2), s1 = *reinterpret_cast<const float2*>(a.stats + at1 * 2);
      const float4 y0 = *reinterpret_cast<const float4*>(a.parts + at0 * D + d), y1 = *reinterpret_cast<const float4*>(a.parts + at1 * D + d);
      const float bias1 = two ? s1.x : INFINITY, next = fminf(low, fminf(s0.x, bias1));
      const float by = low == INFINITY ? 0.f : __builtin_amdgcn_exp2f(next - low);
      const float by0 = s0.x == INFINITY ? 0.f : __builtin_amdgcn_exp2f(next - s0.x), by1 = bias1 == INFINITY ? 0.f : __builtin_amdgcn_exp2f(next - bias1);
      low = next;
      sum = __builtin_fmaf(s0.y, by0, sum * by);
      o[0] = __builtin_fmaf(y0.x, by0, o[0] * by);
      o[1] = __builtin_fmaf(y0.y, by0, o[1] * by);
      o[2] = __builtin_fmaf(y0.z, by0, o[2] * by);
      o[3] = __builtin_fmaf(y0.w, by0, o[3] * by);
      if (two) {
        sum = __builtin_fmaf(s1.y, by1, sum);
        o[0] = __builtin_fmaf(y1.x, by1, o[0]);
        o[1] = __builtin_fmaf(y1.y, by1, o[1]);
        o[2] = __builtin_fmaf(y1.z, by1, o[2]);
        o[3] = __builtin_fmaf(y1.w, by1, o[3]);
      }
    }
    const float inv = 1.f / sum;
    const int tok = (j.row0 + r) / a.G, head = j.head * a.G + (j.row0 + r - tok * a.G);
    *reinterpret_cast<uint2*>(a.out + ((size_t)(j.first + tok) * H * a.G + head) * D + d) =
        make_uint2(pack2<BF>(o[0] * inv, o[1] * inv), pack2<BF>(o[2] * inv, o[3] * inv));
  }
}

template <int D, bool BF, int STAGES, int RT>
void launch(const Args& a, hipStream_t stream) {
  hipLaunchKernelGGL((k_prompt_attention<D, BF, STAGES, RT>), dim3(a.groups), dim3(kTile / 16 / RT * 64), 0, stream, a);
  hipLaunchKernelGGL((k_prompt_attention_join<D, BF>), dim3(a.groups, kTile / kJoinRows), dim3(64 * kJoinWaves), 0, stream, a);
}

// Workgroups of a launch: as many as a compute unit holds at once, the same number on each XCD.
constexpr int kMaxCus = 256;
constexpr int per_cu(int dim) { return dim == 64 ? 3 : (dim == 128 ? 2 : 1); }
int groups_of(int dim) {
  const int cus = svg_cu_count(), n = (cus < kMaxCus ? cus : kMaxCus) * per_cu(dim) / 8 * 8;
  return n < 8 ? 8 : n;
}
size_t stats_at(int groups) { return ((size_t)(groups + 1) * sizeof(Join) + 255) / 256 * 256; }
size_t parts_at(int groups) { return stats_at(groups) + ((size_t)groups * 2 * kTile * 8 + 255) / 256 * 256; }

}  // namespace

uint64_t svg_prompt_attention_bytes(const svg_kv_cache& c) {
  const int groups = kMaxCus * per_cu(c.dim);
  return parts_at(groups) + (size_t)groups * 2 * kTile * c.dim * 4;
}

hipError_t svg_launch_prompt_attention(const svg_kv_cache& c, int layer, const void* q, int64_t ld_q, int G, int n_rows,
                                       const int32_t* start, const int32_t* count, float scale, void* out, void* workspace,
                                       hipStream_t stream) {
  const int groups = groups_of(c.dim);
  char* ws = static_cast<char*>(workspace);
  const Args a{c, static_cast<const uint16_t*>(q), static_cast<uint16_t*>(out), start, count, reinterpret_cast<float*>(ws + stats_at(groups)),
               reinterpret_cast<float*>(ws + parts_at(groups)), reinterpret_cast<Join*>(ws), ld_q, layer, G, n_rows, groups, scale};
  const bool bf = c.type == SVG_BF16;
  if (c.dim == 64) bf ? launch<64, true, 4, 2>(a, stream) : launch<64, false, 4, 2>(a, stream);
  else if (c.dim == 128) bf ? launch<128, true, 4, 2>(a, stream) : launch<128, false, 4, 2>(a, stream);
  else bf ? launch<256, true, 4, 1>(a, stream) : launch<256, false, 4, 1>(a, stream);
  return hipGetLastError();
}
