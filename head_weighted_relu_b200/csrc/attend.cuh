// attend.cuh -- what the attention kernels over the 8-bit cache share: the
// tiles of query rows, their division among the CTAs, and the table that
// translates a tile's keys to cache tokens.
//
// Mathematics.  With codes K, V, a token's scales ks, vs, and a row's query q:
//   t_j = scale * log2(e) * ks_j * (q . K_j)         (base-2 logarithms)
//   o   = sum_j 2^{t_j} vs_j V_j / sum_j 2^{t_j}.
// The value scale is a power of two (or any positive number) per token, so it
// goes into the exponent: with u_j = t_j + log2 vs_j and a running reference
// m >= max u_j - slack,
//   acc = sum_j 2^{u_j - m + kHead} V_j,   l = sum_j 2^{u_j - m + kHead - kSum} / vs_j,
//   o = 2^{-kSum} acc / l,   log sum_j e^{...} = ln2 * (m - kHead + kSum + log2 l).
// The weights 2^{u_j - m + kHead} lie below 2^{kHead + slack} <= 2^15 and are
// rounded to FP16 for the matrix instruction: 11 bits, and a weight vanishes
// only below 2^{-25-kHead} of the largest.  V_j are the bare codes, exact in FP16.
// The sum's terms span the value scales: a block of zeros has 2^-100, so that terms
// reach 2^{15+100}, and a scale of 2^120 makes a row's largest 2^{7-120}.  kSum
// brings both ends inside FP32: 2^24 tokens of zeros at the slack, 2^32 at the
// reference, stay finite, and the other end stays normal.
#pragma once

#include "cache.h"

namespace hwr {

constexpr float kHead = 7.f;    // weights are 2^kHead at the reference
constexpr float kSum = 12.f;    // bits that the row's sum is held lower by
constexpr float kSumUnit = 0x1p-12f;  // 2^-kSum
constexpr float kSlack = 8.f;   // a row's reference rises once it is exceeded by this much
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The (tile, head) that begins in a CTA's share and goes on in the next: its
// parts are `first`, then the first part of each CTA that follows.
struct JoinJob {
  int64_t last, units;   // its last unit, of so many; last -1 for no such one
  int32_t first;
  int32_t rows, q0, pair, h;
};

struct AttendParams {
  CacheView c;
  SeqView s;
  const uint8_t* q;
  int64_t q_stride;        // bytes
  uint8_t* out;
  float* lse;
  const int32_t* sel_idx;
  const int32_t* sel_len;
  int32_t sel_width;
  int32_t causal;
  int32_t Hq, G;           // query heads, and query heads per key/value head
  float scale_log2;        // scale * log2(e)
  int32_t max_keys;        // positions that the page table can hold
  int32_t n_tiles;         // tile slots
  int32_t sel_tiles;       // tiles of one query (selection)
  int32_t n_ctas;          // CTAs that share the units, or 0: one CTA per (tile, head)
  int32_t lanes;           // CTAs side by side on the same keys, one a head; or 1
  JoinJob* jobs;           // [n_ctas] (workspace)
  float* part_o;           // [2 n_ctas][rows][D]
  float2* part_ml;         // [2 n_ctas][rows]: reference and sum
  uint32_t* status;
  int32_t test_wait;       // test hook: the tile kernel's look-ups do not come
};

// A tile: up to R consecutive rows of one sequence's (query, head in group)
// pairs, query-major; with a selection, rows of one query.
struct Tile {
  int b;         // sequence
  int q0;        // first activation row of the sequence
  int first;     // first (query, head) pair, counted from the sequence's first
  int rows;      // pairs
  int n_q;       // queries of the sequence
  int len;       // its length
  int n_keys;    // entries to go over: positions, or entries of the selection
  int row;       // the query's activation row (selection)
};

__device__ __forceinline__ Tile tile_at(const AttendParams& p, int t, int R) {
  Tile x;
  x.rows = 0;
  x.n_keys = 0;
  x.row = 0;
  if (p.sel_width) {
    const int r = t / p.sel_tiles, part = t - r * p.sel_tiles;
    if (r >= seq_row(p.s, p.s.B)) return x;
    x.b = slot_owner(p.s, r, 1, 1, 0);
    x.q0 = seq_row(p.s, x.b);
    x.n_q = seq_row(p.s, x.b + 1) - x.q0;
    x.len = __ldg(p.s.kv_len + x.b);
    x.row = r;
    x.first = (r - x.q0) * p.G + part * R;
    x.rows = min(R, p.G - part * R);
    if (r < x.q0) x.rows = 0;
    x.n_keys = min(max(__ldg(p.sel_len + r), 0), p.sel_width);
    return x;
  }
  x.b = slot_owner(p.s, t, p.G, R, 1);
  x.q0 = seq_row(p.s, x.b);
  x.n_q = seq_row(p.s, x.b + 1) - x.q0;
  x.len = __ldg(p.s.kv_len + x.b);
  const int64_t i = t - slot_base(p.s, x.b, p.G, R, 1);
  const int64_t left = static_cast<int64_t>(x.n_q) * p.G - i * R;
  if (i < 0 || left <= 0) return x;
  x.first = static_cast<int>(i * R);
  x.rows = static_cast<int>(min(left, static_cast<int64_t>(R)));
  int n = x.len;
  if (p.causal) n = x.len - x.n_q + (x.first + x.rows - 1) / p.G + 1;
  x.n_keys = min(max(n, 0), p.max_keys);
  if (n > p.max_keys && p.status) atomicOr(p.status, kStatusToken);
  return x;
}

// Units of UNIT keys of a tile: at least one where it has rows, so that a row
// that sees nothing is written too.
template <int UNIT>
__device__ __forceinline__ int tile_units(const Tile& x) {
  return x.rows <= 0 ? 0 : max(1, (x.n_keys + UNIT - 1) / UNIT);
}

// Number of positions that (query, head) pair `pair` of the tile's sequence sees.
__device__ __forceinline__ int row_limit(const AttendParams& p, const Tile& x, int pair) {
  return p.causal ? x.len - x.n_q + pair / p.G + 1 : x.len;
}

// prefix[t]: the units of the tiles before t, for one head; prefix[n_tiles]: of
// all, which is returned.  For CTAs of THREADS threads that share a launch's
// units; all take part.
template <int UNIT, int THREADS>
__device__ __forceinline__ int tile_prefix(const AttendParams& p, int R, int* prefix, int* warp_sums);

// How CTAs share units.  With lanes = 1, those of all heads in a row, head by
// head.  With lanes = heads, CTAs c, c + 1, .. stand for heads 0, 1, .. of the
// same keys, and `lanes` shares of the units of one head: heads lie beside one
// another in the cache, and read together they are read in longer pieces.
struct Share {
  int64_t units, n, start, end;  // of these units, n shares; this CTA's
  int heads, h;                  // heads among the units, and the head they begin with
};
__device__ __forceinline__ int64_t share_start(int64_t c, int64_t u, int64_t n);
__device__ __forceinline__ Share share_of(const AttendParams& p, int total) {
  Share s;
  s.heads = p.lanes > 1 ? 1 : p.c.heads;
  s.h = blockIdx.x % p.lanes;
  s.units = static_cast<int64_t>(total) * s.heads;
  s.n = min(s.units, static_cast<int64_t>(p.n_ctas / p.lanes));
  const int64_t c = blockIdx.x / p.lanes;
  s.start = c < s.n ? share_start(c, s.units, s.n) : 0;
  s.end = c < s.n ? share_start(c + 1, s.units, s.n) : 0;
  return s;
}

// Share c of n <= u is units [start(c), start(c+1)) of u: one or more each.
__device__ __forceinline__ int64_t share_start(int64_t c, int64_t u, int64_t n) { return c * u / n; }
__device__ __forceinline__ int64_t share_owner(int64_t unit, int64_t u, int64_t n) {
  return ((unit + 1) * n - 1) / u;
}

// The piece of a CTA's share that starts at unit u: units [u0, u1) of (tile, h).
struct Piece {
  int tile, h, u0, u1;
  bool whole;  // all of the (tile, head)'s units
};
__device__ __forceinline__ int tile_of(const AttendParams& p, const int* prefix, int heads, int64_t u) {
  int lo = 0, hi = p.n_tiles - 1;  // the last tile that starts at or before u (empty ones start with the next)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(prefix[mid]) * heads <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ Piece piece_at(const AttendParams& p, const int* prefix, const Share& sh, int64_t u, int64_t end) {
  const int lo = tile_of(p, prefix, sh.heads, u);
  const int tu = prefix[lo + 1] - prefix[lo];
  const int64_t in = u - static_cast<int64_t>(prefix[lo]) * sh.heads;
  Piece r;
  r.tile = lo;
  r.h = sh.h + static_cast<int>(in / tu);
  r.u0 = static_cast<int>(in % tu);
  r.u1 = static_cast<int>(min(static_cast<int64_t>(tu), r.u0 + (end - u)));
  r.whole = r.u0 == 0 && r.u1 == tu;
  return r;
}

// The token that key entry `e` of a tile stands for, as the kernels read it.
struct TokenEntry {
  uint32_t off16;  // offset of the token in the cache, in units of 16 bytes, without the head (0 for none)
  int32_t pos;     // its position; INT_MAX where nothing is to be seen
  float ks;        // key scale
  float lvs;       // log2 of the value scale
};

// Translation of a key entry of (tile, head) to its token in three dependent
// loads, so that a caller can issue each well before its value is used.  An
// entry at or beyond `end`, or that stands for nothing, is pos INT_MAX throughout.
struct Translate {
  const AttendParams& p;
  const Tile& x;
  int h, end, seen;
  const int32_t* sel;
  const int32_t* pages;

  struct Index { int pos; };                              // position, or INT_MAX
  struct Page { int pos; int off; int page; };            // page: as loaded
  struct Place { int pos; uint32_t off16; int64_t scale; };  // scale: index of its scales
  struct Scale { int pos; uint32_t off16; float ks, vs; };

  __device__ __forceinline__ Translate(const AttendParams& p_, const Tile& x_, int h_, int end_)
      : p(p_), x(x_), h(h_), end(end_) {
    sel = p.sel_width ? p.sel_idx + static_cast<int64_t>(x.row) * p.sel_width : nullptr;
    pages = p.s.pages + x.b * p.s.page_stride;
    seen = p.sel_width ? min(x.len, row_limit(p, x, x.first)) : 0;
  }
  __device__ __forceinline__ Index index(int e) const {
    if (e >= end || e < 0) return Index{INT32_MAX};
    return Index{sel ? __ldg(sel + e) : e};
  }
  __device__ __forceinline__ Page page(const Index& i) const {
    Page r{INT32_MAX, 0, 0};
    if (i.pos == INT32_MAX || (sel && (i.pos < 0 || i.pos >= seen))) return r;
    const int pi = i.pos / p.c.page_size;
    r.pos = i.pos;
    r.off = i.pos - pi * p.c.page_size;
    r.page = pi < p.s.table_pages ? __ldg(pages + pi) : -1;
    return r;
  }
  __device__ __forceinline__ Place place(const Page& g) const {
    Place r{INT32_MAX, 0, 0};
    if (g.pos == INT32_MAX) return r;
    if (g.page < 0 || g.page >= p.c.n_pages) {
      if (p.status) atomicOr(p.status, kStatusToken);
      return r;
    }
    r.pos = g.pos;
    r.off16 = static_cast<uint32_t>(g.page * p.c.page16 + g.off * p.c.token16);
    r.scale = (static_cast<int64_t>(g.page) * p.c.page_blocks + (g.off >> p.c.block_shift)) * p.c.heads + h;
    return r;
  }
  __device__ __forceinline__ Scale scale(const Page& g) const {
    const Place a = place(g);
    Scale r{a.pos, a.off16, 0.f, 1.f};
    if (a.pos != INT32_MAX) {
      r.ks = __ldg(p.c.ks + a.scale);
      r.vs = __ldg(p.c.vs + a.scale);
    }
    return r;
  }
  __device__ __forceinline__ TokenEntry entry(const Scale& s) const {
    return TokenEntry{s.off16, s.pos, s.ks, __log2f(fmaxf(s.vs, kMinBlockScale))};
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^-kSum / vs, of log2 vs (2^-132 for the largest scale: not flushed).
__device__ __forceinline__ float inverse_scale(float lvs) { return ex2(-lvs) * kSumUnit; }
// The square root of 2^{m - to}, the factor from reference m to reference `to` >= m:
// sums are multiplied by it twice, since the factor alone may be flushed where a
// sum of tiny value scales still counts.  0 where nothing was seen (m = -inf < to).
__device__ __forceinline__ float root_factor(float m, float to) { return m == to ? 1.f : ex2((m - to) * 0.5f); }
// A row's log-sum-exp.
__device__ __forceinline__ float row_lse(float m, float l) {
  return m == -INFINITY ? -INFINITY : kLn2 * (m - kHead + kSum + log2f(l));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;  // 0: the 16 bytes become zero, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// FP16 operands hold a query row scaled by a power of two to a largest
// magnitude in [1, 2): exact for BF16 values down to 2^-14 of the largest, and
// within 2^-25 of it below.  The exponent of the row's scale:
__device__ __forceinline__ float row_pow2(float amax) {
  int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
  if (!(amax < INFINITY)) e = 0;
  e = min(max(e, -100), 120);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

template <int UNIT, int THREADS>
__device__ __forceinline__ int tile_prefix(const AttendParams& p, int R, int* prefix, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int total = 0;
  for (int t0 = 0; t0 < p.n_tiles; t0 += THREADS) {
    const int t = t0 + threadIdx.x;
    const int v = t < p.n_tiles ? tile_units<UNIT>(tile_at(p, t, R)) : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFullMask, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      const int n = warp_sums[w];
      before += w < warp ? n : 0;
      all += n;
    }
    if (t < p.n_tiles) prefix[t] = total + before + inc - v;
    total += all;
  }
  if (threadIdx.x == 0) prefix[p.n_tiles] = total;
  __syncthreads();
  return total;
}

// Notes this CTA's job for the join.  One thread.
__device__ __forceinline__ void note_job(const AttendParams& p, int R, const int* prefix, const Share& sh) {
  JoinJob j = {};
  j.last = -1;
  if (sh.start < sh.end) {
    const int t = tile_of(p, prefix, sh.heads, sh.end - 1), tu = prefix[t + 1] - prefix[t];
    int64_t u0 = static_cast<int64_t>(prefix[t]) * sh.heads;
    int h = sh.h;
    while (u0 + tu < sh.end) u0 += tu, ++h;  // (a head at a time: no division, which would be a function)
    if (u0 + tu > sh.end && u0 >= sh.start) {
      const Tile x = tile_at(p, t, R);
      j = JoinJob{u0 + tu - 1, sh.units, static_cast<int>(2 * blockIdx.x) + (u0 == sh.start ? 0 : 1), x.rows, x.q0, x.first, h};
    }
  }
  p.jobs[blockIdx.x] = j;
}

// rows: of a tile; 8 or 16 (stream), 128 or 256 (tile)
cudaError_t launch_attend_stream(const AttendParams& p, int D, int rows, bool f16, int grid, cudaStream_t stream);
// u16: every 16 positions from a multiple of 16 on share their scales
cudaError_t launch_attend_tile(const AttendParams& p, int D, int rows, bool u16, bool f16, int grid,
                               cudaStream_t stream);
cudaError_t launch_attend_join(const AttendParams& p, int D, int rows, bool f16, cudaStream_t stream);
int attend_stream_ctas_per_sm(int rows);

constexpr int kMaxSplitTiles = 255;   // tiles of a launch whose CTAs share units: stream
constexpr int kMaxSplitTiles2 = 2047; // tile

}  // namespace hwr
