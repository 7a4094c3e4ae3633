// cache_write.cu -- what writes 8-bit rows before the indexer and the
// attention read them: rotated FP8 rows with a scale each, and the append of
// rotated keys and of values to a paged cache with a scale per block of tokens
// and head.
//
// Both only move bytes.  A lane holds 8 dimensions, so a row of D takes D/8
// lanes and a warp step 256/D rows: two groups of four, which in the rotated
// part of the half-split layout are four dimensions and their partners (so no
// lane needs another's values), elsewhere eight in a row.
//
// Measured: FP8 rows of 16,384 tokens x 64 heads x 128, 64 dimensions rotated:
// 99 us for 407 MB, 4.1 TB/s; the integer pipe is busy 67% of the time (16-bit
// values unpacked, row maxima, codes packed: half-rate instructions), the issue
// slots 70%.  The append of 8,192 tokens (64 heads of q, 8 of k and v): 68 us,
// of which q 42 for 268 MB, 6.4 TB/s, as a copy; keys and values, 50 MB, the rest,
// bound by latency (16 warps an SM at 128 registers).
#include "cache.h"

namespace hwr {
namespace {

template <int D>
constexpr int kLanes = D / 8;      // lanes of a row
template <int D>
constexpr int kRows = 256 / D;     // rows of a warp step

// First dimensions of the two groups of four of lane `sub` of a row.
struct Dims {
  int lo, hi;
};
__device__ __forceinline__ Dims lane_dims(const RotView& r, int sub) {
  if (!r.inter && 8 * sub < r.rot) return Dims{4 * sub, (r.rot >> 1) + 4 * sub};
  return Dims{8 * sub, 8 * sub + 4};
}

// Cosines and sines of a lane's four pairs at one position.
struct Angles {
  float2 c[2], s[2];
};
__device__ __forceinline__ void load_angles(const RotView& r, int64_t pos, int sub, Angles& a) {
  if (8 * sub >= r.rot) return;
  const float* row = r.table + pos * r.rot + 4 * sub;
  const float4 c = __ldg(reinterpret_cast<const float4*>(row));
  const float4 s = __ldg(reinterpret_cast<const float4*>(row + (r.rot >> 1)));
  a.c[0] = make_float2(c.x, c.y), a.c[1] = make_float2(c.z, c.w);
  a.s[0] = make_float2(s.x, s.y), a.s[1] = make_float2(s.z, s.w);
}

struct Raw {
  uint2 lo, hi;
};
__device__ __forceinline__ Raw no_row() { return Raw{make_uint2(0, 0), make_uint2(0, 0)}; }
__device__ __forceinline__ Raw load_row(const uint8_t* row, const Dims& d) {
  return Raw{__ldcs(reinterpret_cast<const uint2*>(row + 2 * d.lo)), __ldcs(reinterpret_cast<const uint2*>(row + 2 * d.hi))};
}

// The lane's values in FP32, rotated: y[0, 4) of the first group, y[4, 8) of the
// second.  Every product and sum is rounded on its own (no contraction), so the
// result is that of the formula in FP32.  PACKED: products two at a time (16,384
// x 64 rows 100 us, 107 without; the append 74 us, 70 without).
template <bool F16, bool PACKED>
__device__ __forceinline__ void rotate(const RotView& r, const Raw& raw, int sub, const Angles& a, float (&y)[8]) {
  float2 p[2] = {unpack_act<F16>(raw.lo.x), unpack_act<F16>(raw.lo.y)};
  float2 q[2] = {unpack_act<F16>(raw.hi.x), unpack_act<F16>(raw.hi.y)};
  if (8 * sub < r.rot) {
    if (r.inter) {  // pairs (x, y) of each float2
      float2* v[4] = {&p[0], &p[1], &q[0], &q[1]};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float c = i & 1 ? a.c[i / 2].y : a.c[i / 2].x, s = i & 1 ? a.s[i / 2].y : a.s[i / 2].x, x = v[i]->x, z = v[i]->y;
        *v[i] = make_float2(__fsub_rn(__fmul_rn(x, c), __fmul_rn(z, s)), __fadd_rn(__fmul_rn(z, c), __fmul_rn(x, s)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // (the sums not in pairs: a packed sum of packed products becomes one FMA)
        auto times = [](float2 a, float2 b) {
          return PACKED ? mul2(a, b) : make_float2(__fmul_rn(a.x, b.x), __fmul_rn(a.y, b.y));
        };
        const float2 pc = times(p[i], a.c[i]), qs = times(q[i], a.s[i]), qc = times(q[i], a.c[i]), ps = times(p[i], a.s[i]);
        p[i] = make_float2(__fsub_rn(pc.x, qs.x), __fsub_rn(pc.y, qs.y));
        q[i] = make_float2(__fadd_rn(qc.x, ps.x), __fadd_rn(qc.y, ps.y));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    y[2 * i] = p[i].x, y[2 * i + 1] = p[i].y;
    y[4 + 2 * i] = q[i].x, y[5 + 2 * i] = q[i].y;
  }
}

// max that is NaN where either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (of the two groups)
__device__ __forceinline__ uint2 pack_codes(const float (&y)[8]) {
  uint2 r;
  r.x = f32x2_to_e4m3x2(y[0], y[1]) | (f32x2_to_e4m3x2(y[2], y[3]) << 16);
  r.y = f32x2_to_e4m3x2(y[4], y[5]) | (f32x2_to_e4m3x2(y[6], y[7]) << 16);
  return r;
}

// ------------------------------------------------------- rotated FP8 rows --
// A warp takes 256/D tokens and a share of the heads, so a lane's cosines and
// sines are loaded once for all of them.
template <int D, bool F16>
__global__ void __launch_bounds__(256) rotate_quantise_kernel(const uint8_t* __restrict__ x, int64_t S, int H,
                                                              int64_t x_stride, const int32_t* __restrict__ positions,
                                                              RotView rot, int parts, int heads_per, uint8_t* __restrict__ codes,
                                                              float* __restrict__ scale, uint32_t* status) {
  const int lane = threadIdx.x & 31, sub = lane % kLanes<D>;
  const int64_t t = (blockIdx.x / parts * int64_t(8) + (threadIdx.x >> 5)) * kRows<D> + lane / kLanes<D>;
  const bool live = t < S;
  const int h0 = blockIdx.x % parts * heads_per, h1 = min(H, h0 + heads_per);
  Angles a;
  bool ok = live;
  if (rot.rot && live) {
    const int64_t pos = positions ? __ldg(positions + t) : t;
    ok = pos >= 0 && pos < rot.rows;
    if (ok) load_angles(rot, pos, sub, a);
    if (!ok && sub == 0 && h0 == 0 && status) atomicOr(status, kStatusToken);
  }
  const Dims d = lane_dims(rot, sub);
  const uint8_t* row = x + t * x_stride;
  constexpr int U = 4;
  for (int h = h0; h < h1; h += U) {
    Raw raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = ok && h + u < h1 ? load_row(row + (h + u) * (2 * D), d) : no_row();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[8];
      rotate<F16, true>(rot, raw[u], sub, a, y);
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(y[i]));
#pragma unroll
      for (int o = kLanes<D> / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(kFullMask, m, o));
      if (!ok || !(m < INFINITY)) m = NAN;  // the whole row becomes NaN codes
      // scale = m / 448 and code = RNE_e4m3(y / scale), both quotients rounded to
      // nearest by a residual step (Markstein, 1990): with r the correctly rounded
      // reciprocal of b and q = a r, the quotient is q - r (q b - a), unless b's
      // fraction is all ones or something leaves the normal range.  Such rows
      // take the division itself.
      constexpr float k448 = 1.f / 448.f;
      const float q0 = m * k448;
      float sc = fmaf(fmaf(-q0, 448.f, m), k448, q0);
      const bool plain = sc > 0x1p-60f && sc < 0x1p60f && (__float_as_uint(sc) & 0x7FFFFFu) != 0x7FFFFFu;
      float z[8];
      if (__all_sync(kFullMask, plain)) {
        const float inv = __frcp_rn(sc);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          // (q b - a, not a - q b: an exact quotient then keeps the sign of a zero)
          const float2 q = mul2(make_float2(y[i], y[i + 1]), make_float2(inv, inv));
          const float2 r = make_float2(fmaf(q.x, sc, -y[i]), fmaf(q.y, sc, -y[i + 1]));
          const float2 w = fma2(r, make_float2(-inv, -inv), q);
          z[i] = w.x, z[i + 1] = w.y;
        }
      } else {
        sc = m == 0.f ? 1.f : __fdiv_rn(m, 448.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = __fdiv_rn(y[i], sc);
      }
      const uint2 code = pack_codes(z);
      if (live && h + u < h1) {
        const int64_t o = t * H + h + u;
        *reinterpret_cast<uint32_t*>(codes + o * D + d.lo) = code.x;
        *reinterpret_cast<uint32_t*>(codes + o * D + d.hi) = code.y;
        if (sub == 0) scale[o] = ok ? sc : 1.f;
      }
    }
  }
}

// ----------------------------------------------------------- cache append --
// log2 of the least power of two s with amax <= 448 s = 1.75 * 2^8 s, at least
// -100: the exponent of amax less 8, or less 7 where its fraction is above 1.75.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  if (e < -100) e = -100;  // zero and tiny blocks
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Keys and values.  CTAs [0, kv_slots * kv_split): slot = one block of tokens
// (floor(rows/block) + 2 slots a sequence), split over the 2*heads key and
// value heads.  A (block, head) is taken by a team of warps, 4 or 8 warp steps of
// rows each, whose rotated values stay in registers between the maximum and the
// quantisation: every row is read once.  Then q, or in a
// kernel of its own: 8 warps x 256/D rows x a share of the query heads per CTA.
constexpr int kAppendWarps = 8;
constexpr int kAppendCtas = 2;  // of an SM

// Rotates the rows r of q and its share of the heads; i: the CTA's number among those for q.
template <int D, bool F16, int U>
__device__ __forceinline__ void rotate_q(const AppendParams& p, int i) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes<D>, rsub = lane / kLanes<D>;
  const int parts = (p.Hq + p.q_heads - 1) / p.q_heads;  // of a row, side by side
  const int r = (i / parts * kAppendWarps + warp) * kRows<D> + rsub;
  const int h0 = i % parts * p.q_heads, h1 = min(p.Hq, h0 + p.q_heads);
  Angles a;
  bool ok = r < p.s.S && r < seq_row(p.s, p.s.B);
  if (ok) {
    const int b = slot_owner(p.s, r, 1, 1, 0);
    const int pos = __ldg(p.s.kv_len + b) - (seq_row(p.s, b + 1) - r);
    ok = pos >= 0 && (p.r.rot == 0 || pos < p.r.rows);
    if (ok && p.r.rot) load_angles(p.r, pos, sub, a);
    if (!ok && sub == 0 && h0 == 0 && p.status) atomicOr(p.status, kStatusToken);
  }
  const Dims d = lane_dims(p.r, sub);
  const uint8_t* in = p.q + r * p.q_stride;
  uint8_t* out = p.q_out + (static_cast<int64_t>(r) * p.Hq) * (2 * D);
  for (int h = h0; h < h1; h += U) {
    Raw raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = ok && h + u < h1 ? load_row(in + (h + u) * (2 * D), d) : no_row();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[8];
      rotate<F16, false>(p.r, raw[u], sub, a, y);
      if (ok && h + u < h1) {
        uint8_t* to = out + (h + u) * (2 * D);
        *reinterpret_cast<uint2*>(to + 2 * d.lo) = make_uint2(pack_act<F16>(y[0], y[1]), pack_act<F16>(y[2], y[3]));
        *reinterpret_cast<uint2*>(to + 2 * d.hi) = make_uint2(pack_act<F16>(y[4], y[5]), pack_act<F16>(y[6], y[7]));
      }
    }
  }
}

// q of many rows, beside the kernel for keys and values: with its registers (two
// CTAs an SM) the copy would wait for memory.
template <int D, bool F16>
__global__ void __launch_bounds__(kAppendWarps * 32, 4) cache_q_kernel(const __grid_constant__ AppendParams p) {
  rotate_q<D, F16, 4>(p, blockIdx.x);
  // complete no earlier than the kernel that this one did not wait for
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// kSteps: warp steps of rows that a warp holds
template <int D, bool F16, int kSteps>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendCtas) cache_append_kernel(const __grid_constant__ AppendParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % kLanes<D>, rsub = lane / kLanes<D>;
  const int kv_ctas = p.kv_slots * p.kv_split;
  if (p.q_apart) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (static_cast<int>(blockIdx.x) >= kv_ctas) {
    rotate_q<D, F16, 4>(p, blockIdx.x - kv_ctas);
    return;
  }

  const int slot = blockIdx.x / p.kv_split, part = blockIdx.x % p.kv_split;
  const int blk = p.c.block;
  const int b = slot_owner(p.s, slot, 1, blk, 2);
  const int row0 = seq_row(p.s, b), row1 = seq_row(p.s, b + 1);
  const int n_new = row1 - row0;
  if (n_new <= 0) return;
  const int len = __ldg(p.s.kv_len + b);
  const int past = len - n_new;  // position of the first new token
  // block number j of the sequence's touched blocks; its tokens [t0, t0 + blk)
  const int j = static_cast<int>(slot - slot_base(p.s, b, 1, blk, 2));
  const int64_t t0 = (static_cast<int64_t>(past >> p.c.block_shift) + j) * blk;  // floor for negative positions too
  if (t0 >= len) return;
  const int lo = static_cast<int>(max(t0, static_cast<int64_t>(past)) - t0);            // first new token in the block
  const int hi = static_cast<int>(min(t0 + blk, static_cast<int64_t>(len)) - t0);       // end of the new tokens
  int off = 0;
  const int64_t page = t0 >= 0 ? page_of(p.s, p.c, b, static_cast<int>(t0), &off) : -1;
  const bool bad_tail = p.r.rot && t0 + hi > p.r.rows;
  if ((page < 0 || bad_tail) && threadIdx.x == 0 && part == 0 && p.status) atomicOr(p.status, kStatusToken);
  if (page < 0) return;
  const int hi_ok = bad_tail ? static_cast<int>(max(p.r.rows - t0, int64_t(lo))) : hi;
  if (hi_ok <= lo) return;

  constexpr int kTeamRows = kSteps * kRows<D>;  // rows of a warp
  const int team = blk <= kTeamRows ? 1 : blk / kTeamRows;
  const int teams = kAppendWarps / team, in_team = warp % team;
  const int jobs = 2 * p.c.heads, jobs_per = (jobs + p.kv_split - 1) / p.kv_split;
  const int j0 = part * jobs_per, j1 = min(jobs, j0 + jobs_per);
  __shared__ float part_max[kAppendWarps];
  const int64_t sc0 = (page * p.c.page_blocks + (off >> p.c.block_shift)) * p.c.heads;
  const int64_t tok0 = page * p.c.page16 + off * p.c.token16;
  const int tw = in_team * kTeamRows + rsub;  // the lane's row of warp step i: tw + i * kRows
  uint32_t in = 0;  // bit i: the lane's row of warp step i is new
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int t = tw + i * kRows<D>;
    if (t >= lo && t < hi_ok) in |= 1u << i;
  }
  const Dims d = lane_dims(p.r, sub);
  Raw raw[kSteps];
  auto load = [&](int job) {
    const bool v = job >= p.c.heads;
    const uint8_t* src = (v ? p.v : p.k) + (v ? job - p.c.heads : job) * (2 * D) +
                         (row0 + (t0 - past) + tw) * p.kv_stride;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      raw[i] = job < j1 && (in >> i & 1) ? load_row(src + i * kRows<D> * p.kv_stride, d) : no_row();
  };
  load(j0 + warp / team);
  for (int jb = j0; jb < j1; jb += teams) {
    const int job = jb + warp / team;
    const bool on = job < j1;
    const bool is_v = on && job >= p.c.heads;
    const int h = on ? (is_v ? job - p.c.heads : job) : 0;
    float* sp = (is_v ? p.c.vs : p.c.ks) + sc0 + h;
    const float old = on && lo > 0 ? *sp : 0.f;
    RotView r = p.r;
    if (is_v) r.rot = 0;
    float m = 0.f, y[kSteps][8];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      Angles a;
      if ((in >> i & 1) && r.rot) load_angles(r, t0 + tw + i * kRows<D>, sub, a);
      rotate<F16, false>(r, raw[i], sub, a, y[i]);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[i][e]));  // (NaN passes by)
      if (top == INFINITY) {  // infinite values become NaN, and do not count
        top = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (fabsf(y[i][e]) == INFINITY) y[i][e] = NAN;
          top = fmaxf(top, fabsf(y[i][e]));
        }
      }
      if (in >> i & 1) m = fmaxf(m, top);
    }
    load(job + teams);  // the next job's rows are on the way meanwhile
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
    if (team > 1) {
      if (lane == 0) part_max[warp] = m;
      __syncthreads();
      for (int w = 0; w < team; ++w) m = fmaxf(m, part_max[warp - in_team + w]);
    }
    const float need = block_scale(m);
    const float sc = lo > 0 ? fmaxf(need, fmaxf(old, kMinBlockScale)) : need;
    // the old scale and the maxima are read before they are overwritten
    if (team > 1)
      __syncthreads();
    else
      __syncwarp();
    uint8_t* dst = (is_v ? p.c.v : p.c.k) + (tok0 + h * p.c.head16 + tw * p.c.token16) * 16;
    // sc = frac * 2^e.  A block's own scales have frac = 1, and dividing by them is
    // exact; a scale that another writer chose and that is kept may have any: then
    // the quotient by frac, correctly rounded by a residual step as above.
    const uint32_t bits = __float_as_uint(sc);
    const float inv = bits < 254u << 23 ? __uint_as_float((254u << 23) - (bits & 0x7F800000u)) : 0x1p-127f;  // 2^-e
    const bool pow2 = (bits & 0x7FFFFFu) == 0;
    const float frac = __uint_as_float(bits & 0x7FFFFFu | 127u << 23), rfrac = __frcp_rn(frac);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      uint8_t* to = dst + i * kRows<D> * p.c.token16 * 16;
      uint32_t* lo4 = reinterpret_cast<uint32_t*>(to + d.lo);
      uint32_t* hi4 = reinterpret_cast<uint32_t*>(to + d.hi);
      if (in >> i & 1) {
        if (on) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] *= inv;
          if (!pow2) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float q = y[i][e] * rfrac;
              y[i][e] = fmaf(fmaf(q, frac, -y[i][e]), -rfrac, q);
            }
          }
          const uint2 code = pack_codes(y[i]);
          *lo4 = code.x, *hi4 = code.y;
        }
      } else if (on && tw + i * kRows<D> < lo && sc != old) {
        // an earlier token of a block whose scale rises (to a power of two)
        const float f = old * inv;
        const uint32_t ww[2] = {*lo4, *hi4};
        float z[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t hh = e4m3x2_to_f16x2(static_cast<uint16_t>(ww[e >> 1] >> (16 * (e & 1))));
          const float2 v = unpack_act<true>(hh);
          z[2 * e] = v.x * f, z[2 * e + 1] = v.y * f;
        }
        const uint2 code = pack_codes(z);
        *lo4 = code.x, *hi4 = code.y;
      }
    }
    if (on && lane == 0 && in_team == 0) *sp = sc;
  }
}

}  // namespace

cudaError_t launch_rotate_quantise(const void* x, int64_t S, int H, int D, bool f16, int64_t x_stride,
                                   const int32_t* positions, const RotView& rot, uint8_t* codes, float* scale,
                                   uint32_t* status, int sms, cudaStream_t stream) {
  if (S == 0 || H == 0) return cudaSuccess;
  const int64_t bx = (S + 8 * (256 / D) - 1) / (8 * (256 / D));
  // the heads are split over CTAs until there are many for each place on the SMs
  // (16,384 tokens: 119 us with 1,024 CTAs, 117 with 4,096)
  int split = 1;
  while (bx * split < 16 * sms && split * 8 <= H) split *= 2;
  const int per = (H + split - 1) / split;
  const int parts = (H + per - 1) / per;  // of a row, side by side
  const unsigned grid = static_cast<unsigned>(bx * parts);
  const uint8_t* xb = static_cast<const uint8_t*>(x);
#define HWR_GO(DD, FF)                                                                                            \
  rotate_quantise_kernel<DD, FF><<<grid, 256, 0, stream>>>(xb, S, H, x_stride * 2, positions, rot, parts, per, codes,    \
                                                           scale, status)
  if (D == 128) {
    if (f16) HWR_GO(128, true); else HWR_GO(128, false);
  } else {
    if (f16) HWR_GO(64, true); else HWR_GO(64, false);
  }
#undef HWR_GO
  return cudaGetLastError();
}

cudaError_t launch_cache_append(AppendParams p, int D, bool f16, int sms, cudaStream_t stream) {
  if (p.s.S == 0 || p.s.B == 0) return cudaSuccess;
  p.kv_slots = static_cast<int32_t>(p.s.S / p.c.block + 2 * static_cast<int64_t>(p.s.B));
  const int steps = D == 128 && p.c.block == 128 ? 8 : 4;  // (a block of tokens is at most a CTA's)
  const int team_rows = steps * (256 / D), team = p.c.block <= team_rows ? 1 : p.c.block / team_rows;
  const int teams = kAppendWarps / team;
  p.kv_split = 1;
  while (static_cast<int64_t>(p.kv_slots) * p.kv_split < 4 * sms && p.kv_split * teams < 2 * p.c.heads) p.kv_split *= 2;
  p.q_slots = p.q_heads = 0;
  int64_t q_ctas = 0;
  if (p.q) {
    const int cta_rows = kAppendWarps * (256 / D);
    p.q_slots = static_cast<int32_t>((p.s.S + cta_rows - 1) / cta_rows);
    int split = 1;
    while (static_cast<int64_t>(p.q_slots) * split < 16 * sms && split * 8 <= p.Hq) split *= 2;
    p.q_heads = (p.Hq + split - 1) / split;
    q_ctas = static_cast<int64_t>(p.q_slots) * ((p.Hq + p.q_heads - 1) / p.q_heads);
  }
  // q in a launch of its own where it is large: 8,192 rows x 64 heads x 128 (2^26
  // values) take 95 us in one launch and 92 in two, 2,450 x 16 x 64 (2^21) 8.3
  // and 10.3 us.
  p.q_apart = p.q && p.s.S * p.Hq * D >= (int64_t(1) << 24);
  const int64_t grid = static_cast<int64_t>(p.kv_slots) * p.kv_split + (p.q_apart ? 0 : q_ctas);
  if (grid > INT32_MAX || q_ctas > INT32_MAX) return cudaErrorInvalidValue;
#define HWR_GO(DD, FF, SS) \
  cache_append_kernel<DD, FF, SS><<<static_cast<unsigned>(grid), kAppendWarps * 32, 0, stream>>>(p)
  if (D == 64) {
    if (f16) HWR_GO(64, true, 4); else HWR_GO(64, false, 4);
  } else if (steps == 4) {
    if (f16) HWR_GO(128, true, 4); else HWR_GO(128, false, 4);
  } else {
    if (f16) HWR_GO(128, true, 8); else HWR_GO(128, false, 8);
  }
#undef HWR_GO
  if (!p.q_apart) return cudaGetLastError();
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(q_ctas));
  cfg.blockDim = dim3(kAppendWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (D == 64)
    return f16 ? cudaLaunchKernelEx(&cfg, cache_q_kernel<64, true>, p) : cudaLaunchKernelEx(&cfg, cache_q_kernel<64, false>, p);
  return f16 ? cudaLaunchKernelEx(&cfg, cache_q_kernel<128, true>, p) : cudaLaunchKernelEx(&cfg, cache_q_kernel<128, false>, p);
}

}  // namespace hwr
