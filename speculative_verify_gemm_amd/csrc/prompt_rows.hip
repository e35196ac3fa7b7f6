// The rows of a step on gfx950: which slot, position and place in the pages each belongs to, and the rotation
// of their queries and keys by those positions, with keys and values written into the pages.
//
// Row map.  Bound by a launch and two to three dependent round trips of memory: lengths, table entry, count of the page.  128 rows of
// 8 trees 2.2 us; 230754 rows of 512 slots 4.9 us (3.7 MB).  The sums over the slots are made by every workgroup for itself: one
// launch instead of two.
//
// Rotation.  (a, b) -> (a c - b s, b c + a s) with c, s the cosine and sine of pos * freq.  Bound by bytes where there are many rows
// (3334 rows of 32 + 8 + 8 heads of 128, half of each rotated, bf16: 82 MB at least, 24.5 us), else by a launch and a chain of
// position, angle, row (32 rows: 5.8 us).  The angles are fp64, 35 instructions a pair: a workgroup computes those of its 32 rows
// once into LDS and turns eight heads with them.  A unit is 16 values of one head and row, both values of each pair, two 16-byte
// pieces; two (fp32) or four units are on their way at once (one after the other: 29.4 us).
#include "../../include/svgemm_prompt.h"
#include "svg_cache.h"
#include "svg_internal.h"

#pragma clang fp contract(off)

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlots = 1024;

// ------------------------------------------------------------------ row map
// Sums stop at the number of rows: min(a + b, R) is associative for numbers from 0 to R < 2^31.
SVG_DEV u32 add_upto(u32 a, u32 b, u32 most) {
  const u32 s = a + b;
  return s < most ? s : most;
}

struct MapArgs {
  svg_kv_cache c;
  const int32_t* n_new;
  const int32_t* parent;
  int32_t *start, *count, *slot, *pos, *place;
  int T, n_rows;
};

SVG_DEV void write_row(const MapArgs& a, int r, int s, int i, int depth) {
  int pos = -1, place = -1;
  if (s >= 0 && depth >= 0) {
    const int len = a.c.len[s];
    if (len >= 0 && (long)len + depth <= 0x7FFFFFFFl) {
      const u32 p = (u32)len + (u32)i;
      int page;
      pos = len + depth;
      if (own_page_of(a.c, s, p / (u32)a.c.page, page)) place = page * a.c.page + (int)(p % (u32)a.c.page);
    }
  }
  if (a.slot != nullptr) a.slot[r] = s;
  a.pos[r] = pos;
  a.place[r] = place;
}

// Packed rows.  Every workgroup adds the slots' numbers up by itself (four slots a thread) and looks its rows up in
// the sums; the first one writes the slots' starts and counts.
__global__ __launch_bounds__(kThreads) void k_row_map_packed(MapArgs a) {
  __shared__ u32 end[kMaxSlots];
  __shared__ u32 red[kThreads / 64];
  const int S = a.c.n_slots, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const u32 R = (u32)a.n_rows;
  u32 n[4], sum = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int s = 4 * tid + j, x = s < S ? a.n_new[s] : 0;
    n[j] = x < 0 ? 0u : ((u32)x < R ? (u32)x : R);
    sum = add_upto(sum, n[j], R);
  }
  u32 upto = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const u32 y = (u32)__shfl_up((int)upto, off);
    if (lane >= off) upto = add_upto(upto, y, R);
  }
  u32 before = (u32)__shfl_up((int)upto, 1);
  if (lane == 0) before = 0;
  if (lane == 63) red[wave] = upto;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w)
    if (w < wave) before = add_upto(before, red[w], R);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int s = 4 * tid + j;
    const u32 first = before;
    before = add_upto(before, n[j], R);
    end[s] = before;
    if (blockIdx.x == 0 && s < S) {
      a.start[s] = (int)first;
      a.count[s] = (int)(before - first);
    }
  }
  __syncthreads();
  for (long r = (long)blockIdx.x * kThreads + tid; r < a.n_rows; r += (long)gridDim.x * kThreads) {
    int s = 0;  // slots whose rows end at r or before
#pragma unroll
    for (int step = kMaxSlots / 2; step > 0; step >>= 1)
      if (end[s + step - 1] <= (u32)r) s += step;
    const bool none = s >= S || end[s] <= (u32)r;  // (behind the last slot's: all sums are at most r)
    const int i = none ? 0 : (int)((u32)r - (s > 0 ? end[s - 1] : 0u));
    write_row(a, (int)r, none ? -1 : s, i, i);
  }
}

// T rows a slot, as chains.
__global__ __launch_bounds__(kThreads) void k_row_map_dense(MapArgs a) {
  const int T = a.T;
  for (long r = (long)blockIdx.x * kThreads + threadIdx.x; r < a.n_rows; r += (long)gridDim.x * kThreads) {
    const int s = (int)(r / T), i = (int)(r % T);
    int n = a.n_new[s];
    n = n < 0 ? 0 : (n > T ? T : n);
    if (i == 0) {
      a.start[s] = (int)r;
      a.count[s] = n;
    }
    write_row(a, (int)r, i < n ? s : -1, i, i);
  }
}

// T rows a slot, as trees: 32 lanes a slot.  A lane holds an ancestor of its node and the steps to it; each turn both become
// the ancestor's, so the paths' lengths double and five turns reach the root of any of 32 nodes.
__global__ __launch_bounds__(kThreads) void k_row_map_tree(MapArgs a) {
  static_assert(SVG_TREE_MAX_NODES == 32, "lanes of a slot, turns");
  const int T = a.T, i = threadIdx.x & 31, s = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const bool slot = s < a.c.n_slots, node = slot && i < T;
  const int p = node ? a.parent[(size_t)s * T + i] : -1;
  const bool bad = i == 0 ? p != -1 : (p < 0 || p >= i);
  u32 v = (bad || i == 0 ? 0u : (u32)p | 0x100u) | (bad ? 0x10000u : 0u);  // ancestor, steps, whether the rule is broken
#pragma unroll
  for (int turn = 0; turn < 5; ++turn) {
    const u32 up = (u32)__shfl((int)v, (threadIdx.x & 32) + (int)(v & 0xFFu));
    v = (up & 0xFFu) | ((v & 0xFF00u) + (up & 0xFF00u)) | ((v | up) & 0x10000u);
  }
  if (!slot) return;
  int n = a.n_new[s];
  n = n < 0 ? 0 : (n > T ? T : n);
  if (i == 0) {
    a.start[s] = s * T;
    a.count[s] = n;
  }
  if (node) write_row(a, s * T + i, i < n ? s : -1, i, (v & 0x10000u) ? -1 : (int)((v >> 8) & 0xFFu));
}

// --------------------------------------------------------------------- rope
constexpr int kRows = 32;  // rows of a workgroup

struct RopeArgs {
  svg_kv_cache c;
  const void *q, *k, *v;
  void* q_out;
  const double* freq;
  const int32_t *pos, *place;
  long ld_q, ld_k, ld_v;
  int layer, q_heads, n_rows, x_type, q_f32, rot, interleaved, heads_each;
  float amplitude;
};

// N consecutive values (4 or 8) of a row as they lie in memory, and as fp32.
template <int XT, int N>
struct Raw {
  static constexpr int WORDS = XT == SVG_F32 ? N : N / 2;
  u32 w[WORDS];
  SVG_DEV void load(const void* base, size_t at) {
    const char* p = static_cast<const char*>(base) + at * (XT == SVG_F32 ? 4 : 2);
    if constexpr (WORDS == 2) {
      const uint2 t = *reinterpret_cast<const uint2*>(p);
      w[0] = t.x;
      w[1] = t.y;
    } else {
#pragma unroll
      for (int i = 0; i < WORDS / 4; ++i) {
        const uint4 t = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = t.x;
        w[4 * i + 1] = t.y;
        w[4 * i + 2] = t.z;
        w[4 * i + 3] = t.w;
      }
    }
  }
  SVG_DEV float at(int i) const {
    if constexpr (XT == SVG_F32) return __uint_as_float(w[i]);
    else if constexpr (XT == SVG_F16) return half_at(w, i);
    else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
};

template <bool BF>
SVG_DEV uint4 pack8(const float (&v)[8]) {
  return make_uint4(kv_round<BF>(v[0]) | (kv_round<BF>(v[1]) << 16), kv_round<BF>(v[2]) | (kv_round<BF>(v[3]) << 16),
                    kv_round<BF>(v[4]) | (kv_round<BF>(v[5]) << 16), kv_round<BF>(v[6]) | (kv_round<BF>(v[7]) << 16));
}

// Cosine and sine of an angle (radians): the quarter turns taken off in fp64 (pi/2 in two parts, 2^-85 of it left), the
// rest within pi/4 by the Taylor series to the 11th and 10th power (left out: 7e-12 and 1.1e-10).
SVG_DEV float2 cos_sin(double angle, double amplitude) {
  const double quarter = rint(angle * 0.63661977236758134308);
  const double r = __builtin_fma(-quarter, 6.1232339957367658e-17, __builtin_fma(-quarter, 1.5707963267948966, angle));
  const double z = r * r;
  double s = -1.0 / 39916800, c = -1.0 / 3628800;
  s = __builtin_fma(s, z, 1.0 / 362880);
  c = __builtin_fma(c, z, 1.0 / 40320);
  s = __builtin_fma(s, z, -1.0 / 5040);
  c = __builtin_fma(c, z, -1.0 / 720);
  s = __builtin_fma(s, z, 1.0 / 120);
  c = __builtin_fma(c, z, 1.0 / 24);
  s = __builtin_fma(s, z, -1.0 / 6);
  c = __builtin_fma(c, z, -0.5);
  s = __builtin_fma(s * z, r, r) * amplitude;
  c = __builtin_fma(c, z, 1.0) * amplitude;
  const int turn = (int)((long)quarter & 3);
  const float fs = (float)s, fc = (float)c;
  const float co = turn & 1 ? fs : fc, si = turn & 1 ? fc : fs;
  return make_float2(turn == 1 || turn == 2 ? -co : co, turn >= 2 ? -si : si);
}

// A workgroup takes 32 rows and `heads_each` of the q_heads + 2 heads; the angles of its rows are computed once into LDS.
template <bool BF, int XT>
__global__ __launch_bounds__(kThreads) void k_rope_append(RopeArgs a) {
  extern __shared__ float2 turns[];  // [kRows][rot / 2]
  __shared__ int pos[kRows], place[kRows], quads[kRows], n_quads;
  const int tid = threadIdx.x, dim = a.c.dim, pairs = a.rot >> 1, per_row = dim >> 4;
  const int H = a.c.heads, first = blockIdx.y * a.heads_each, all = a.q_heads + 2 * H;
  const int last = first + a.heads_each < all ? first + a.heads_each : all;
  const size_t head_size = (size_t)a.c.page * dim;
  const long places = (long)a.c.n_pages * a.c.page;
  const int page_bits = __builtin_ctz(a.c.page);
  uint16_t* kl = static_cast<uint16_t*>(a.c.k) + (size_t)a.layer * a.c.n_pages * H * head_size;
  uint16_t* vl = static_cast<uint16_t*>(a.c.v) + (size_t)a.layer * a.c.n_pages * H * head_size;
  for (long r0 = (long)blockIdx.x * kRows; r0 < a.n_rows; r0 += (long)gridDim.x * kRows) {
    __syncthreads();
    if (tid < 64) {  // (the first wave; lanes from kRows on have no row)
      const long r = r0 + tid;
      int p = -1, at = -1;
      if (tid < kRows && r < a.n_rows) {
        p = a.pos[r];
        at = a.place[r];
        if (p < 0 || at < 0 || at >= places) at = -1;
      }
      // rows at consecutive places are stored up to four together, those whose values share 8 bytes
      const int prev = __shfl_up(at, 1);
      const bool leads = at >= 0 && (tid == 0 || (at & 3) == 0 || prev != at - 1);
      const unsigned long long who = __ballot(leads);
      if (tid < kRows) {
        pos[tid] = p;
        place[tid] = at;
        if (leads) quads[__popcll(who & ((1ull << tid) - 1))] = tid;
        if (tid == 0) n_quads = __popcll(who);
      }
    }
    __syncthreads();
    if (first < a.q_heads + H) {
      for (int x = tid; x < kRows * pairs; x += kThreads) {
        const int p = pos[x / pairs];
        if (p >= 0) turns[x] = cos_sin((double)p * a.freq[x % pairs], a.amplitude);
      }
      __syncthreads();
    }
    // queries and keys: 16 values of a head at a time, with both values of each pair; several on their way at once
    constexpr int U = XT == SVG_F32 ? 2 : 4;
    const int rotating = (last < a.q_heads + H ? last : a.q_heads + H) - first, units = kRows * per_row;
    for (int x0 = tid; x0 < rotating * units; x0 += U * kThreads) {
      Raw<XT, 8> raw[U][2];
      int h[U], row[U], d0[U], d1[U];
      bool live[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int x = x0 + i * kThreads, u = x % units, c = u % per_row;
        h[i] = first + x / units;
        row[i] = u / per_row;
        const bool key = h[i] >= a.q_heads;
        live[i] = x < rotating * units && (key ? place[row[i]] >= 0 : pos[row[i]] >= 0);
        const bool halves = 16 * c < a.rot && !a.interleaved;
        d0[i] = halves ? 8 * c : 16 * c;
        d1[i] = halves ? d0[i] + pairs : d0[i] + 8;
        if (!live[i]) continue;
        const size_t r = (size_t)(r0 + row[i]);
        const void* base = key ? a.k : a.q;
        const size_t from = key ? r * (size_t)a.ld_k + (size_t)(h[i] - a.q_heads) * dim : r * (size_t)a.ld_q + (size_t)h[i] * dim;
        raw[i][0].load(base, from + d0[i]);
        raw[i][1].load(base, from + d1[i]);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (!live[i]) continue;
        float lo[8], hi[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          lo[e] = raw[i][0].at(e);
          hi[e] = raw[i][1].at(e);
        }
        if (!a.interleaved && d0[i] < pairs) {
          const float2* t = turns + row[i] * pairs + d0[i];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x0 = lo[e], x1 = hi[e];
            lo[e] = __builtin_fmaf(x0, t[e].x, -(x1 * t[e].y));
            hi[e] = __builtin_fmaf(x1, t[e].x, x0 * t[e].y);
          }
        } else if (d0[i] < a.rot) {
          const float2* t = turns + row[i] * pairs + d0[i] / 2;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float x0 = lo[2 * e], x1 = lo[2 * e + 1], y0 = hi[2 * e], y1 = hi[2 * e + 1];
            lo[2 * e] = __builtin_fmaf(x0, t[e].x, -(x1 * t[e].y));
            lo[2 * e + 1] = __builtin_fmaf(x1, t[e].x, x0 * t[e].y);
            hi[2 * e] = __builtin_fmaf(y0, t[e + 4].x, -(y1 * t[e + 4].y));
            hi[2 * e + 1] = __builtin_fmaf(y1, t[e + 4].x, y0 * t[e + 4].y);
          }
        }
        if (h[i] >= a.q_heads) {
          const int at = place[row[i]], page = at >> page_bits, t = at & (a.c.page - 1);
          uint16_t* to = kl + ((size_t)page * H + (h[i] - a.q_heads)) * head_size;
          *reinterpret_cast<uint4*>(to + kv_key_at(t, d0[i], dim)) = pack8<BF>(lo);
          *reinterpret_cast<uint4*>(to + kv_key_at(t, d1[i], dim)) = pack8<BF>(hi);
        } else {
          const size_t to = ((size_t)(r0 + row[i]) * a.q_heads + h[i]) * dim;
          if (a.q_f32) {
            float4* p0 = reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + to + d0[i]);
            float4* p1 = reinterpret_cast<float4*>(static_cast<float*>(a.q_out) + to + d1[i]);
            p0[0] = make_float4(lo[0], lo[1], lo[2], lo[3]);
            p0[1] = make_float4(lo[4], lo[5], lo[6], lo[7]);
            p1[0] = make_float4(hi[0], hi[1], hi[2], hi[3]);
            p1[1] = make_float4(hi[4], hi[5], hi[6], hi[7]);
          } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + to + d0[i]) = pack8<BF>(lo);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.q_out) + to + d1[i]) = pack8<BF>(hi);
          }
        }
      }
    }
    // values: up to four rows that share 8-byte pieces, four values of a head at a time
    const int from_v = first > a.q_heads + H ? first : a.q_heads + H, vheads = last - from_v, quarter = dim >> 2;
    const int vunits = n_quads * quarter;
    for (int x = tid; x < vheads * vunits; x += kThreads) {
      const int h = from_v - a.q_heads - H + x / vunits, u = x % vunits, row = quads[u / quarter], d = 4 * (u % quarter);
      const int at = place[row], page = at >> page_bits, t = at & (a.c.page - 1);
      Raw<XT, 4> w[4];
      int n = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (n == j && (t & 3) + j < 4 && row + j < kRows && place[row + j] == at + j) {
          w[j].load(a.v, (size_t)(r0 + row + j) * (size_t)a.ld_v + (size_t)h * dim + d);
          n = j + 1;
        }
      }
      uint16_t* to = vl + ((size_t)page * H + h) * head_size;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint16_t* p = to + kv_value_at(t, d + e, dim);
        if (n == 4) {
          *reinterpret_cast<uint2*>(p) = make_uint2(kv_round<BF>(w[0].at(e)) | (kv_round<BF>(w[1].at(e)) << 16),
                                                    kv_round<BF>(w[2].at(e)) | (kv_round<BF>(w[3].at(e)) << 16));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < n) p[j] = (uint16_t)kv_round<BF>(w[j].at(e));
        }
      }
    }
  }
}

int blocks_of(long n, long most) { return (int)(n < most ? n : most); }

}  // namespace

hipError_t svg_launch_kv_row_map(const svg_kv_cache& c, const int32_t* n_new, const int32_t* parent, int T, int n_rows,
                                 int32_t* start, int32_t* count, int32_t* slot, int32_t* pos, int32_t* place, hipStream_t stream) {
  const MapArgs a{c, n_new, parent, start, count, slot, pos, place, T, n_rows};
  const int blocks = blocks_of(((long)n_rows + kThreads - 1) / kThreads, 4096);
  if (parent != nullptr)
    hipLaunchKernelGGL(k_row_map_tree, dim3((c.n_slots + kThreads / 32 - 1) / (kThreads / 32)), dim3(kThreads), 0, stream, a);
  else if (T > 0) hipLaunchKernelGGL(k_row_map_dense, dim3(blocks), dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL(k_row_map_packed, dim3(blocks > 0 ? blocks : 1), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

hipError_t svg_launch_rope_append(const svg_kv_cache& c, int layer, const svg_rope& rope, const void* q, int64_t ld_q, int q_heads,
                                  const void* k, int64_t ld_k, const void* v, int64_t ld_v, int x_type, int n_rows,
                                  const int32_t* pos, const int32_t* place, void* q_out, int q_type, hipStream_t stream) {
  const int heads = q_heads + 2 * c.heads, cus = svg_cu_count();
  const int rows = blocks_of(((long)n_rows + kRows - 1) / kRows, 1 << 16);
  int groups = (2 * cus + rows - 1) / rows;  // of heads: two workgroups a compute unit, and eight heads a workgroup at most
  if (groups < (heads + 7) / 8) groups = (heads + 7) / 8;
  const int each = groups >= heads ? 1 : (heads + groups - 1) / groups;
  const RopeArgs a{c, q, k, v, q_out, rope.freq, pos, place, ld_q, ld_k, ld_v, layer, q_heads, n_rows, x_type, q_type == SVG_F32,
                   rope.rot, rope.interleaved, each, rope.amplitude};
  const dim3 grid(rows, (heads + each - 1) / each);
  const u32 lds = kRows * (u32)(rope.rot / 2) * sizeof(float2);
#define SVG_ROPE(BF)                                                                                             \
  if (x_type == SVG_F32) hipLaunchKernelGGL((k_rope_append<BF, SVG_F32>), grid, dim3(kThreads), lds, stream, a); \
  else if (x_type == SVG_F16) hipLaunchKernelGGL((k_rope_append<BF, SVG_F16>), grid, dim3(kThreads), lds, stream, a); \
  else hipLaunchKernelGGL((k_rope_append<BF, SVG_BF16>), grid, dim3(kThreads), lds, stream, a)
  if (c.type == SVG_BF16) {
    SVG_ROPE(true);
  } else {
    SVG_ROPE(false);
  }
#undef SVG_ROPE
  return hipGetLastError();
}
