// The pages of a key/value cache on gfx950: writing new tokens, keeping the
// accepted path of a draft tree, forking and freeing slots, making room with
// copies of shared pages, copying pages.  Pure data movement (kv_append rounds
// once) and whole numbers: results do not depend on the order of threads.
//
// The state is the tables and one count per page; a page is free where its
// count is 0, and free pages are always taken lowest number first, so nothing
// but the counts has to be kept and a captured graph needs no host list.
#include "svg_cache.h"
#include "svg_internal.h"

namespace {

constexpr int kThreads = 256;

// Whether slot s's table row names a page of the cache for page number i.
SVG_DEV bool page_of(const svg_kv_cache& c, int s, long i, int& page) {
  const int held = c.pages[s];
  if (i < 0 || i >= held || held > c.width) return false;
  page = c.table[(size_t)s * c.width + i];
  return (u32)page < (u32)c.n_pages;
}

// Whether that page may be written: no other slot holds it.  (A slot that kv_reserve refused still has the page that it
// shares.)
SVG_DEV bool own_page_of(const svg_kv_cache& c, int s, long i, int& page) {
  return page_of(c, s, i, page) && (c.refs == nullptr || c.refs[page] <= 1);
}

// ------------------------------------------------------------------- append
// One wave per (four consecutive positions, head, slot): four tokens share the
// eight-byte halves of the values' 16-byte pieces, so they are written whole.
// Bound by its launch and two dependent loads (4 slots of 8 tokens, 32 heads of 128: 1.6 MB in 3.9 us).
template <bool BF>
__global__ __launch_bounds__(64) void k_kv_append(svg_kv_cache c, int layer, const float* __restrict__ k, long ld_k,
                                                 const float* __restrict__ v, long ld_v, int T,
                                                 const int32_t* __restrict__ n_rows) {
  const int h = blockIdx.y, s = blockIdx.z, dim = c.dim;
  int n = n_rows ? n_rows[s] : T;
  n = n < 0 ? 0 : (n > T ? T : n);
  const int len = c.len[s];
  if (len < 0 || n == 0) return;
  const long p0 = (len & ~3) + 4l * blockIdx.x;  // first of the four positions
  if (p0 >= (long)len + n) return;
  int page;
  if (!own_page_of(c, s, p0 / c.page, page)) return;
  const u32 t0 = (u32)(p0 % c.page);
  const size_t base = (((size_t)layer * c.n_pages + page) * c.heads + h) * ((size_t)c.page * dim);
  uint16_t* kp = static_cast<uint16_t*>(c.k) + base;
  uint16_t* vp = static_cast<uint16_t*>(c.v) + base;
  const long i0 = p0 - len;  // node of the first position (may be -3 .. n - 1)
  const int npiece = dim >> 3;
  for (int x = threadIdx.x; x < 4 * npiece; x += 64) {
    const int q = x / npiece, d = 8 * (x % npiece);
    const long i = i0 + q;
    if (i < 0 || i >= n) continue;
    const float* row = k + ((long)s * T + i) * ld_k + (long)h * dim + d;
    const float4 a = *reinterpret_cast<const float4*>(row), b = *reinterpret_cast<const float4*>(row + 4);
    uint4 o;
    o.x = kv_round<BF>(a.x) | (kv_round<BF>(a.y) << 16);
    o.y = kv_round<BF>(a.z) | (kv_round<BF>(a.w) << 16);
    o.z = kv_round<BF>(b.x) | (kv_round<BF>(b.y) << 16);
    o.w = kv_round<BF>(b.z) | (kv_round<BF>(b.w) << 16);
    *reinterpret_cast<uint4*>(kp + kv_key_at(t0 + q, d, dim)) = o;
  }
  for (int d = threadIdx.x; d < dim; d += 64) {
    u32 w[4];
    bool ok[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const long i = i0 + q;
      ok[q] = i >= 0 && i < n;
      w[q] = ok[q] ? kv_round<BF>(v[((long)s * T + i) * ld_v + (long)h * dim + d]) : 0u;
    }
    uint16_t* at = vp + kv_value_at(t0, d, dim);
    if (ok[0] && ok[3]) {  // i rises over the four: the ends being rows, all are
      *reinterpret_cast<uint2*>(at) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (ok[q]) at[q] = (uint16_t)w[q];
    }
  }
}

// ------------------------------------------------------------------- commit
// What slot s commits: `kept` tokens, the root's and the accepted nodes' (0: the path is not valid, or its tokens are not
// inside the slot's pages, or in one that others hold too), the same in every lane of the wave; in lane j the node that
// moves to len + 1 + j.
struct Moves {
  int kept, len, node;
};
SVG_DEV Moves moves_of(const svg_kv_cache& c, int s, int T, const int32_t* path, const int32_t* n_emit) {
  const int lane = threadIdx.x & 63;
  const int n = n_emit[s], len = c.len[s], held = c.pages[s];
  const int p = lane < T ? path[(size_t)s * T + lane] : -1;
  int before = __shfl_up(p, 1);
  if (lane == 0) before = 0;
  const bool mine = lane < n - 1;
  bool ok = n >= 1 && n <= T && len >= 0 && held >= 0 && held <= c.width;
  ok = ok && !__any(mine && !(p > before && p < T));
  // every position from len on that is read or written lies between the root's and the last node's: two pages at most
  if (ok) {
    const int last = n > 1 ? __shfl(p, n - 2) : 0;
    int page;
    ok = !__any(!own_page_of(c, s, ((long)len + (lane & 1 ? last : 0)) / c.page, page));  // (both pages at once)
  }
  return {ok ? n : 0, len, p};
}

// One workgroup per (head, layer, slot): all rows are read before any is written (a row's place may be another's source).
// The two pages and the places in them are looked up once, by one wave, while nothing else waits.
// Bound by latency, a chain of the path, the table and the rows, and by the lines that the values touch: a token's lie in
// 2-byte pieces 16 bytes apart (8 slots of 16 nodes, 32 layers of 8 heads of 128: 8.4 MB moved, 23.4 MB read and 16.3 MB written
// by the counters, 12 to 13 us; every thread looking its places up by itself: 18.4 us).
template <int DIM>
__global__ __launch_bounds__(kThreads) void k_kv_commit(svg_kv_cache c, int T, const int32_t* __restrict__ path,
                                                       const int32_t* __restrict__ n_emit, int32_t* len_out) {
  __shared__ uint4 kb[(SVG_TREE_MAX_NODES - 1) * DIM / 8];
  __shared__ uint16_t vb[(SVG_TREE_MAX_NODES - 1) * DIM];
  __shared__ int place[SVG_TREE_MAX_NODES][2];  // of each move: the source's (page << 7) + token, the destination's
  const int h = blockIdx.x, l = blockIdx.y, s = blockIdx.z;
  const Moves m = moves_of(c, s, T, path, n_emit);
  if (len_out != nullptr && h == 0 && l == 0 && threadIdx.x == 0) len_out[s] = m.len + m.kept;
  const int rows = m.kept - 1;
  if (rows <= 0) return;
  if ((int)threadIdx.x < rows) {
    const int32_t* tab = c.table + (size_t)s * c.width;
    const int from = m.len + m.node, to = m.len + 1 + (int)threadIdx.x;
    place[threadIdx.x][0] = (tab[from / c.page] << 7) + from % c.page;
    place[threadIdx.x][1] = (tab[to / c.page] << 7) + to % c.page;
  }
  __syncthreads();
  const size_t stride = (size_t)c.heads * c.page * DIM;  // of a page
  const size_t at = (size_t)l * c.n_pages * stride + (size_t)h * c.page * DIM;
  uint16_t* kl = static_cast<uint16_t*>(c.k) + at;
  uint16_t* vl = static_cast<uint16_t*>(c.v) + at;
  for (int x = threadIdx.x; x < rows * (DIM / 8); x += kThreads) {
    const int p = place[x / (DIM / 8)][0];
    kb[x] = *reinterpret_cast<const uint4*>(kl + (size_t)(p >> 7) * stride + kv_key_at(p & 127, 8 * (x % (DIM / 8)), DIM));
  }
#pragma unroll 4
  for (int x = threadIdx.x; x < rows * DIM; x += kThreads) {
    const int p = place[x / DIM][0];
    vb[x] = vl[(size_t)(p >> 7) * stride + kv_value_at(p & 127, x % DIM, DIM)];
  }
  __syncthreads();
  for (int x = threadIdx.x; x < rows * (DIM / 8); x += kThreads) {
    const int p = place[x / (DIM / 8)][1];
    *reinterpret_cast<uint4*>(kl + (size_t)(p >> 7) * stride + kv_key_at(p & 127, 8 * (x % (DIM / 8)), DIM)) = kb[x];
  }
  for (int x = threadIdx.x; x < rows * DIM; x += kThreads) {
    const int p = place[x / DIM][1];
    vl[(size_t)(p >> 7) * stride + kv_value_at(p & 127, x % DIM, DIM)] = vb[x];
  }
}

// The new lengths in place, after every reader of the old ones: a wave a slot.
__global__ __launch_bounds__(kThreads) void k_kv_commit_len(svg_kv_cache c, int T, const int32_t* __restrict__ path,
                                                           const int32_t* __restrict__ n_emit) {
  const int s = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (s >= c.n_slots) return;
  const Moves m = moves_of(c, s, T, path, n_emit);
  if ((threadIdx.x & 63) == 0) c.len[s] = m.len + m.kept;
}

// --------------------------------------------------------------------- fork
// A workgroup per slot.  Bound by its launch and the chain of src, pages and table (16 slots: 4.8 us).
SVG_DEV int clampi(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

__global__ __launch_bounds__(kThreads) void k_kv_fork(svg_kv_cache c, const int32_t* __restrict__ src,
                                                     int32_t* __restrict__ table_out, int32_t* __restrict__ pages_out,
                                                     int32_t* __restrict__ len_out) {
  const int s = blockIdx.x;
  int from = src[s];
  if (from < -1 || from >= c.n_slots) from = s;
  const bool keep = from == s;
  const int had = clampi(c.pages[s], 0, c.width);
  int len = 0, has = 0;
  if (from >= 0) {
    len = c.len[from];
    const int held = clampi(c.pages[from], 0, c.width);
    const int full = len <= 0 ? 0 : (len - 1) / c.page + 1;
    has = keep ? held : (full < held ? full : held);
  }
  const int32_t* old_row = c.table + (size_t)s * c.width;
  const int32_t* new_row = c.table + (size_t)(from < 0 ? 0 : from) * c.width;
  int32_t* out = table_out + (size_t)s * c.width;
  for (int i = threadIdx.x; i < has; i += kThreads) {
    const int p = new_row[i];
    out[i] = p;
    if (!keep && (u32)p < (u32)c.n_pages) atomicAdd(c.refs + p, 1);
  }
  if (!keep) {
    for (int i = threadIdx.x; i < had; i += kThreads) {
      const int p = old_row[i];
      if ((u32)p < (u32)c.n_pages) atomicSub(c.refs + p, 1);
    }
  }
  if (threadIdx.x == 0) {
    pages_out[s] = has;
    len_out[s] = len;
  }
}

// ------------------------------------------------------------------ reserve
constexpr int kPlan = 1024;  // threads of the planning workgroup: one slot each

// Sum of v over the threads before this one, and over all (`total`); one
// barrier pair.  wsum: 16 ints of LDS.
SVG_DEV int scan_before(int v, int* wsum, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();  // wsum may still be read by the call before
  if (lane == 63) wsum[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kPlan / 64; ++w) {
    const int t = wsum[w];
    if (w < wave) before += t;
    all += t;
  }
  total = all;
  return before + x - v;
}

// ws: [0] number of copies, then (from, to) pairs from ws + 4.
//
// One workgroup: thread s plans slot s.  Without a shortage of pages every slot's demand
// is known at once (the k-th holder of a page, in slot order, copies it while
// more than one of its counts is left: k < refs - 1), one scan gives each its
// share of the free pages, and the pass over refs hands them out.  With a
// shortage the slots are taken one after another, as the order then decides.
// Bound by the chain of loads and barriers of one workgroup (16 slots, 20 to 24 copies: 6.9 us).
__global__ __launch_bounds__(kPlan) void k_kv_reserve(svg_kv_cache c, const int32_t* __restrict__ need,
                                                     int32_t* __restrict__ status, int32_t* __restrict__ ws) {
  __shared__ int wsum[kPlan / 64];
  __shared__ int part[kPlan];      // the partly filled page a slot writes to, -1: none
  __shared__ int first[kPlan + 1]; // pages handed out before slot s
  __shared__ int copies[kPlan], at[kPlan];
  __shared__ int left;
  const int s = threadIdx.x, S = c.n_slots;
  int state = 0, more = 0, held = 0, refs = 0, copy = 0, idx = 0;
  part[s] = -1;
  if (s < S && need[s] > 0) {
    const int len = c.len[s];
    held = c.pages[s];
    const long last = (long)len + need[s];  // tokens after the call
    if (len < 0 || held < 0 || held > c.width || (long)len > (long)held * c.page ||
        last > (long)c.width * c.page) {
      state = 2;
    } else {
      const int total = (int)((last - 1) / c.page + 1);
      more = total > held ? total - held : 0;
      if (more > c.n_pages) more = c.n_pages + 1;  // a shortage whatever the others do
      if (len % c.page) {
        idx = len / c.page;
        const int p = c.table[(size_t)s * c.width + idx];
        if ((u32)p >= (u32)c.n_pages) {
          state = 2;
          more = 0;
        } else {
          part[s] = p;
          refs = c.refs[p];
        }
      }
    }
  }
  // free pages, a count a thread and turn
  int found = 0;
  for (int i = s; i < c.n_pages; i += kPlan) found += c.refs[i] == 0;
  int n_free;
  scan_before(found, wsum, n_free);  // (also the barrier before part[] is read)
  const int mine = part[s];
  if (mine >= 0) {
    int rank = 0;
    for (int t = 0; t < s; ++t) rank += part[t] == mine;
    copy = rank < refs - 1;
  }
  int want = more + copy, all;
  int before = scan_before(want, wsum, all);
  if (all > n_free) {
    // a shortage: in order, each slot takes all it wants or nothing
    copies[s] = 0;
    if (s == 0) left = n_free;
    __syncthreads();
    for (int t = 0; t < S; ++t) {
      // copies made of t's page by slots before it
      const int made = __syncthreads_count(s < t && copies[s] && part[s] == part[t]);
      if (s == t) {
        copy = mine >= 0 && refs - made > 1;
        want = more + copy;
        if (want > left) {
          state = 1;
          want = more = copy = 0;
        } else {
          left -= want;
          copies[s] = copy;
        }
      }
      __syncthreads();
    }
    before = scan_before(want, wsum, all);
  }
  first[s] = before;
  if (s == 0) first[kPlan] = all;
  copies[s] = copy;
  at[s] = copy ? idx : held;  // row entry of the slot's first page
  int n_copy;
  const int c_before = scan_before(copy, wsum, n_copy);
  // (the barriers of that scan also publish first[], copies[] and at[])
  __shared__ int c_first[kPlan], held_of[kPlan];
  c_first[s] = c_before;
  held_of[s] = held;
  __syncthreads();
  int given = 0;
  for (int i0 = 0; i0 < c.n_pages && given < all; i0 += kPlan) {
    const int i = i0 + s;
    const bool is_free = i < c.n_pages && c.refs[i] == 0;
    int now;
    const int r = given + scan_before(is_free ? 1 : 0, wsum, now);
    if (is_free && r < all) {
      // the slot whose share holds r: the last one with first <= r and a share
      int lo = 0, hi = kPlan;  // first[lo] <= r < first[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= r) lo = mid;
        else hi = mid;
      }
      const int j = r - first[lo];
      const int entry = j == 0 ? at[lo] : held_of[lo] + j - copies[lo];
      c.table[(size_t)lo * c.width + entry] = i;
      c.refs[i] = 1;
      if (j == 0 && copies[lo]) {
        ws[4 + 2 * c_first[lo]] = part[lo];
        ws[5 + 2 * c_first[lo]] = i;
      }
    }
    given += now;
  }
  if (copy) atomicSub(c.refs + mine, 1);
  if (s < S) {
    status[s] = state;
    if (more) c.pages[s] = held + more;
  }
  if (s == 0) ws[0] = n_copy;
}

// -------------------------------------------------------------------- copies
// Pages copied in every layer, keys and values: (pair, layer, k or v) blocks of kChunk 16-byte pieces, spread over the
// grid.  COUNTED: the pairs and their number as kv_reserve's plan left them.  Bound by memory: 407 MB of pages in 162 us
// (5.0 TB/s read and written; 166 us through the caches).  One piece of a thread at a time: with four on their way the same copy
// took 169 us, 24 pages of forks 37 us instead of 30 us.
constexpr int kChunk = 4096;  // pieces of a workgroup's turn (64 KiB)

template <bool COUNTED>
__global__ __launch_bounds__(kThreads) void k_kv_copy(svg_kv_cache c, const int32_t* __restrict__ src,
                                                     const int32_t* __restrict__ dst, int n) {
  if constexpr (COUNTED) n = src[0];
  const long pieces = (long)c.heads * c.page * c.dim / 8;  // of a page
  const long chunks = (pieces + kChunk - 1) / kChunk;
  const long turns = (long)n * 2 * c.n_layers * chunks;
  for (long t = blockIdx.x; t < turns; t += gridDim.x) {
    const long ch = t % chunks, plane = t / chunks;
    const int kv = (int)(plane & 1);
    const long rest = plane >> 1;
    const int l = (int)(rest % c.n_layers), i = (int)(rest / c.n_layers);
    int a, b;
    if constexpr (COUNTED) {
      a = src[4 + 2 * i];
      b = src[5 + 2 * i];
    } else {
      a = src[i];
      b = dst[i];
    }
    if ((u32)a >= (u32)c.n_pages || (u32)b >= (u32)c.n_pages) continue;
    uint4* base = static_cast<uint4*>(kv ? c.v : c.k) + (size_t)l * c.n_pages * pieces;
    const uint4* from = base + (size_t)a * pieces;
    uint4* to = base + (size_t)b * pieces;
    const long end = (ch + 1) * kChunk < pieces ? (ch + 1) * kChunk : pieces;
#pragma unroll 1
    for (long x = ch * kChunk + threadIdx.x; x < end; x += kThreads) {
      if constexpr (COUNTED) {
        to[x] = from[x];  // one source for several forks, and what is written is read next
      } else {
        const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + x));
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(to + x));
      }
    }
  }
}

}  // namespace

hipError_t svg_launch_kv_append(const svg_kv_cache& c, int layer, const float* k, int64_t ld_k, const float* v,
                                int64_t ld_v, int T, const int32_t* n_rows, hipStream_t stream) {
  // no more positions than a table row has (a dimension of the grid holds fewer than 2^32 work-items; T may be 2^31 - 1)
  const long most = (long)c.width * c.page, rows = T < most ? T : most;
  const dim3 grid((unsigned)((rows + 3) / 4 + 1), c.heads, c.n_slots);
  if (c.type == SVG_BF16)
    hipLaunchKernelGGL(k_kv_append<true>, grid, dim3(64), 0, stream, c, layer, k, (long)ld_k, v, (long)ld_v, T, n_rows);
  else
    hipLaunchKernelGGL(k_kv_append<false>, grid, dim3(64), 0, stream, c, layer, k, (long)ld_k, v, (long)ld_v, T, n_rows);
  return hipGetLastError();
}

hipError_t svg_launch_kv_commit(const svg_kv_cache& c, int T, const int32_t* path, const int32_t* n_emit,
                                int32_t* len_out, hipStream_t stream) {
  const dim3 grid(c.heads, c.n_layers, c.n_slots);
  int32_t* out = len_out == c.len ? nullptr : len_out;
  if (c.dim == 64)
    hipLaunchKernelGGL(k_kv_commit<64>, grid, dim3(kThreads), 0, stream, c, T, path, n_emit, out);
  else if (c.dim == 128)
    hipLaunchKernelGGL(k_kv_commit<128>, grid, dim3(kThreads), 0, stream, c, T, path, n_emit, out);
  else
    hipLaunchKernelGGL(k_kv_commit<256>, grid, dim3(kThreads), 0, stream, c, T, path, n_emit, out);
  if (out == nullptr)
    hipLaunchKernelGGL(k_kv_commit_len, dim3((c.n_slots + kThreads / 64 - 1) / (kThreads / 64)), dim3(kThreads), 0, stream, c, T,
                       path, n_emit);
  return hipGetLastError();
}

hipError_t svg_launch_kv_fork(const svg_kv_cache& c, const int32_t* src, int32_t* table_out, int32_t* pages_out,
                              int32_t* len_out, hipStream_t stream) {
  hipLaunchKernelGGL(k_kv_fork, dim3(c.n_slots), dim3(kThreads), 0, stream, c, src, table_out, pages_out, len_out);
  return hipGetLastError();
}

hipError_t svg_launch_kv_reserve(const svg_kv_cache& c, const int32_t* need, int32_t* status, void* workspace,
                                 hipStream_t stream) {
  int32_t* ws = static_cast<int32_t*>(workspace);
  hipLaunchKernelGGL(k_kv_reserve, dim3(1), dim3(kPlan), 0, stream, c, need, status, ws);
  hipLaunchKernelGGL(k_kv_copy<true>, dim3(2048), dim3(kThreads), 0, stream, c, ws, nullptr, 0);
  return hipGetLastError();
}

hipError_t svg_launch_kv_copy(const svg_kv_cache& c, const int32_t* src, const int32_t* dst, int n,
                              hipStream_t stream) {
  hipLaunchKernelGGL(k_kv_copy<false>, dim3(4096), dim3(kThreads), 0, stream, c, src, dst, n);
  return hipGetLastError();
}
