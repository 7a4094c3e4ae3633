// attend_stream.cu -- attention over the 8-bit cache for few query rows per
// key/value head (decode steps, selected positions): up to 8 or 16 rows share
// one pass over the keys, which is bound by reading them.
//
// A warp works alone: it copies 16 tokens' codes (2 D bytes each) at a time
// into a ring of its own in shared memory (cp.async, kDepth - 1 steps ahead),
// and translates key entries to cache tokens two steps at a time, each of the
// dependent loads (selected index -> page -> scales) issued one pair of steps
// before its value is used; no barrier stands in the key loop.  A CTA's four
// warps take every fourth 16 tokens of its keys and join at the end.
//
// Both products are taken transposed, tokens or value columns on the 16 rows of
// mma.m16n8k16 and query rows on its 8 columns, so that 8 rows (one query of 8
// heads) waste nothing.  Codes become FP16 in registers (exact) in fragment
// order without a shuffle: the order of the head dimension inside a product is
// free, so lane group c takes dimensions (D/4)c .. of a key row as 16-byte
// reads; and which columns a tile of the second product holds is free, so lane
// group g takes columns (D/8)g .. of four value rows as 16-byte reads,
// interleaved by byte permutes.  The weights pass to the second product
// through a register transpose (movmatrix).
//
// What bounds it: reading the keys and values.  16 sequences of 16,384 to 65,536
// tokens, 8 heads: 216 us for 1.34 GB, 6.2 TB/s, 95% of what a copy reaches.  That
// took the heads of a token to be read side by side (CTAs c, c + 1, .. on the same
// keys): a head alone is 128 bytes of every 1,024, 258 us.  One entry for 16
// tokens that share their scales, instead of one each, changed nothing.  1,024
// rows over 2,048 selected tokens each of 16,384 (the cache in L2): 587 us, 7.3
// TB/s out of L2, a third of what L2 gives: issue slots 62% busy and the integer pipe
// 54%, with four warps an SM quarter.
#include "attend.cuh"

namespace hwr {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;                  // tokens of a warp step
constexpr int kUnit = kWarps * kStep;      // keys of a unit
constexpr int kDepth = 3;                  // ring entries per warp
constexpr int kTableSteps = 4;             // steps whose translation is kept

template <int D, int NT>
struct Smem {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStepBytes = 2 * kStep * D;
  static constexpr int kRing = kWarps * kDepth * kStepBytes;
  static constexpr int kJoin = kWarps * kRows * (D + 4) * 4;   // reuses the ring
  static constexpr int kData = kRing > kJoin ? kRing : kJoin;
  static constexpr int kTable = kWarps * kTableSteps * kStep * 16;
  static constexpr int kBytes = kData + kTable + kWarps * kRows * 8;
};

// Offset of 16-byte chunk `ch` of token row `r` in a step's K or V image: rows
// of D bytes, the chunks of a 128-byte line permuted so that the reads of the
// fragments (rows r, r+1 of chunk pairs; rows r, r+2, r+4, r+6 of one chunk)
// touch every bank once.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int ch) {
  if (D == 128) return r * 128 + ((ch ^ (r & 7)) << 4);
  const int line = r >> 1, c8 = ((r & 1) << 2) + ch;
  return line * 128 + ((c8 ^ ((line & 3) << 1)) << 4);
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8x8 transpose of 16-bit values held as a lane's row lane/4, columns 2(lane%4), +1.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16)); }

// Query fragments: row g of each 8, the lane's own D/4 consecutive dimensions,
// 4 per product step.  factor: what the accumulated product of rows 2c, 2c+1 is
// multiplied by.
template <int D, int NT, bool F16>
__device__ __forceinline__ void load_q(const AttendParams& p, const Tile& x, int h, uint32_t (&qf)[D / 16][NT][2],
                                       float (&factor)[NT][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int i = g + 8 * nt;
    const bool on = i < x.rows;
    const int pair = x.first + (on ? i : 0);
    const uint8_t* src = p.q + (x.q0 + pair / p.G) * p.q_stride + (h * p.G + pair % p.G) * (2 * D) + c * (D / 2);
    uint32_t w[D / 8];
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const uint4 v = on ? __ldg(reinterpret_cast<const uint4*>(src) + k) : make_uint4(0, 0, 0, 0);
      w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
    }
    float s = 1.f;
    if (!F16) {
      float m = 0.f;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const float2 f = unpack_act<false>(w[k]);
        m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 1));
      m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 2));
      s = row_pow2(m);
      const float inv = 1.f / s;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const float2 f = unpack_act<false>(w[k]);
        w[k] = half2_of(f.x * inv, f.y * inv);
      }
    }
    s *= p.scale_log2;
#pragma unroll
    for (int j = 0; j < 2; ++j) factor[nt][j] = __shfl_sync(kFullMask, s, (2 * c + j) * 4);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[k][nt][0] = w[2 * k];      // dimensions 4k, 4k+1 of the lane's
      qf[k][nt][1] = w[2 * k + 1];  // 4k+2, 4k+3
    }
  }
}

// Copies one step: 16 rows of D/16 chunks, of K and of V.  kbase, vbase: the
// lane's chunk of token 0.
template <int D>
__device__ __forceinline__ void issue_step(const TokenEntry* table, const uint8_t* kbase, const uint8_t* vbase,
                                           uint32_t ring) {
  const int lane = threadIdx.x & 31;
  constexpr int kCh = D / 16, kPer = kCh * kStep / 32;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = i * (32 / kCh) + lane / kCh;
    const uint2 e = *reinterpret_cast<const uint2*>(table + r);
    const bool on = e.y != INT32_MAX;
    const int64_t at = static_cast<int64_t>(e.x) << 4;
    const uint32_t dst = ring + chunk_at<D>(r, lane % kCh);
    cp_async16(dst, kbase + at, on);
    cp_async16(dst + kStep * D, vbase + at, on);
  }
  cp_async_commit();
}

// 0xFF in each byte of w that is a NaN code (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// Takes the NaN codes out of a step's values, and makes NaN the outputs of the
// rows that do see them: the columns where (code is NaN) x (row sees token),
// again a matrix product, is not zero.  sc: the masked scores.
template <int D, int NT>
__device__ __forceinline__ void poison(const float (&sc)[NT][4], uint32_t (&vw)[4][D / 32],
                                       float (&acc)[D / 16][NT][4]) {
  uint32_t sees[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int t = 0; t < 2; ++t)
      sees[nt][t] = transpose8x8((sc[nt][2 * t] == -INFINITY ? 0u : 0x3C00u) |
                                 (sc[nt][2 * t + 1] == -INFINITY ? 0u : 0x3C000000u));
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    uint32_t nb[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      nb[t] = nan_bytes(vw[t][k]);
      vw[t][k] &= ~nb[t];
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t a[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int sh = 16 * half + 8 * (e & 1), t = e & 2;
        a[e] = ((nb[t] >> sh) & 1u) * 0x3C00u | ((nb[t + 1] >> sh) & 1u) * 0x3C000000u;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float hit[4] = {};
        mma16816(hit, a, sees[nt][0], sees[nt][1]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (hit[e] > 0.f) acc[2 * k + half][nt][e] = NAN;
      }
    }
  }
}

// Writes the joined rows of a segment: whole ones as outputs, others as parts.
template <int D, int NT, bool F16>
__device__ __forceinline__ void store_rows(const AttendParams& p, const Tile& x, int h, bool whole, int64_t part,
                                           const float* acc, const float2* ml) {
  // acc [kWarps][rows][D+4] (columns in order), ml [kWarps][rows]
  constexpr int R = 8 * NT, kPer = D / 8;  // threads of a row
  const int d = (threadIdx.x % kPer) * 8;
  for (int i = threadIdx.x / kPer; i < x.rows; i += kWarps * 32 / kPer) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w * R + i].x);
    float l = 0.f, o[8] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 v = ml[w * R + i];
      const float h = root_factor(v.x, m), f = h * h;
      l += v.y * h * h;
      if (v.x != -INFINITY) {  // (a part of a vanishing factor counts, for its NaN)
        const float* a = acc + (w * R + i) * (D + 4) + d;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += f * a[e];
      }
    }
    if (whole) {
      const int pair = x.first + i;
      const int64_t at = (x.q0 + pair / p.G) * static_cast<int64_t>(p.Hq) + h * p.G + pair % p.G;
      const float inv = m == -INFINITY ? 0.f : 1.f / l;
      uint4 v;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= kSumUnit;
      v.x = pack_act<F16>(o[0] * inv, o[1] * inv), v.y = pack_act<F16>(o[2] * inv, o[3] * inv);
      v.z = pack_act<F16>(o[4] * inv, o[5] * inv), v.w = pack_act<F16>(o[6] * inv, o[7] * inv);
      *reinterpret_cast<uint4*>(p.out + (at * D + d) * 2) = v;
      if (p.lse && d == 0) p.lse[at] = row_lse(m, l);
    } else {
      float* dst = p.part_o + (part * R + i) * D + d;
      *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
      if (d == 0) p.part_ml[part * R + i] = make_float2(m, l);
    }
  }
}

// Keys [64 u0, 64 u1) of (tile, head).
template <int D, int NT, bool F16>
__device__ void segment(const AttendParams& p, const Tile& x, int h, int u0, int u1, bool whole, int64_t part,
                        uint8_t* smem) {
  using L = Smem<D, NT>;
  constexpr int R = L::kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  TokenEntry* table = reinterpret_cast<TokenEntry*>(smem + L::kData) + warp * (kTableSteps * kStep);
  float2* ml = reinterpret_cast<float2*>(smem + L::kData + L::kTable);
  const uint32_t ring = smem_u32(smem) + warp * (kDepth * L::kStepBytes);
  const int64_t chunk = (h * p.c.head16 + lane % (D / 16)) * 16;
  const uint8_t* kbase = p.c.k + chunk;
  const uint8_t* vbase = p.c.v + chunk;
  const int n = u1 - u0;  // steps of this warp

  __syncthreads();  // the previous segment's buffers are free

  // The lane's entry of a pair of steps: token lane%16 of step 2*pair + lane/16.
  const int e0 = u0 * kUnit + (lane >> 4) * kUnit + warp * kStep + (lane & 15);
  auto entry = [&](int pair) { return e0 + pair * 2 * kUnit; };
  const int end = min(x.n_keys, u1 * kUnit);
  Translate tr(p, x, h, end);
  Translate::Index i0 = tr.index(entry(0)), i1 = tr.index(entry(1)), i2 = tr.index(entry(2)), i3 = tr.index(entry(3));
  Translate::Page g0 = tr.page(i0), g1 = tr.page(i1), g2 = tr.page(i2);
  Translate::Scale s0 = tr.scale(g0), s1 = tr.scale(g1);
  uint32_t qf[D / 16][NT][2];
  float factor[NT][2];
  load_q<D, NT, F16>(p, x, h, qf, factor);
  int limit[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = 8 * nt + 2 * c + j;
      limit[nt][j] = i < x.rows ? row_limit(p, x, x.first + i) : 0;
    }
  // the least number of positions that a row of the tile sees
  const int first_limit = p.sel_width ? 0 : row_limit(p, x, x.first);
  float acc[D / 16][NT][4] = {};
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) m[nt][0] = m[nt][1] = -INFINITY, l[nt][0] = l[nt][1] = 0.f;

  table[lane] = tr.entry(s0);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) {
    if (i < n)
      issue_step<D>(table + i * kStep, kbase, vbase, ring + i * L::kStepBytes);
    else
      cp_async_commit();
  }
  static_assert(kDepth - 1 == 2, "a pair of steps is in flight ahead of the one that is computed");

  int slot = 0;
#pragma unroll 1
  for (int s = 0; s < n; ++s) {
    if ((s & 1) == 0) {
      // pair s/2 + 1 into the table; each later pair one load further
      table[((s + 2) & 3) * kStep + lane] = tr.entry(s1);
      s1 = tr.scale(g2);
      g2 = tr.page(i3);
      i3 = tr.index(entry((s >> 1) + 4));
      __syncwarp();
    }
    const int next = slot >= 1 ? slot - 1 : kDepth - 1;  // the entry of step s - 1, free now: (s + 2) % 3
    if (s + 2 < n)
      issue_step<D>(table + ((s + 2) & 3) * kStep, kbase, vbase, ring + next * L::kStepBytes);
    else
      cp_async_commit();
    cp_async_wait<kDepth - 1>();
    __syncwarp();
    const uint32_t kb = ring + slot * L::kStepBytes, vb = kb + kStep * D;
    slot = slot + 1 == kDepth ? 0 : slot + 1;

    // Scores of tokens g, g+8 (rows) and query rows 2c, 2c+1 (columns), in two
    // chains of products to halve their latency.
    float sc[NT][4] = {}, sd[NT][4] = {};
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const uint4 v0 = lds128(kb + chunk_at<D>(g, D == 128 ? 2 * c + i : c));
      const uint4 v1 = lds128(kb + chunk_at<D>(g + 8, D == 128 ? 2 * c + i : c));
      const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a[4] = {cvt_lo(w0[j]), cvt_lo(w1[j]), cvt_hi(w0[j]), cvt_hi(w1[j])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816((j & 1) ? sd[nt] : sc[nt], a, qf[i * 4 + j][nt][0], qf[i * 4 + j][nt][1]);
      }
    }
    const TokenEntry* te = table + (s & 3) * kStep;
    const int4 ea = *reinterpret_cast<const int4*>(te + g), eb = *reinterpret_cast<const int4*>(te + g + 8);
    const float ks[2] = {__int_as_float(ea.z), __int_as_float(eb.z)};
    const float lvs[2] = {__int_as_float(ea.w), __int_as_float(eb.w)};
    const float ivs[2] = {inverse_scale(lvs[0]), inverse_scale(lvs[1])};
    const int pos[2] = {ea.y, eb.y};
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float u = fmaf((sc[nt][2 * t + j] + sd[nt][2 * t + j]) * ks[t], factor[nt][j], lvs[t]);
          u = pos[t] < limit[nt][j] ? u : -INFINITY;
          sc[nt][2 * t + j] = u;
          up = up || u > m[nt][j] + kSlack;
        }
    // A row's reference rises to its largest score when that exceeds it by the slack
    // (a row's own affair: its results do not depend on its neighbours).
    if (__any_sync(kFullMask, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float top = fmaxf(sc[nt][j], sc[nt][2 + j]);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
          if (!(top > m[nt][j] + kSlack)) top = m[nt][j];
          const float h = root_factor(m[nt][j], top), f = h * h;
          m[nt][j] = top;
          l[nt][j] *= h, l[nt][j] *= h;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) acc[i][nt][j] *= f, acc[i][nt][2 + j] *= f;
        }
    }
    uint32_t pf[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float r0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kHead;
      const float r1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kHead;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float p0 = ex2(sc[nt][2 * t] - r0), p1 = ex2(sc[nt][2 * t + 1] - r1);
        l[nt][0] = fmaf(p0, ivs[t], l[nt][0]);
        l[nt][1] = fmaf(p1, ivs[t], l[nt][1]);
        pf[nt][t] = transpose8x8(half2_of(p0, p1));
      }
    }
    // values: tokens 2c, 2c+1, 2c+8, 2c+9; lane group g's D/8 columns
    uint32_t vw[4][D / 32];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = 2 * c + (t & 1) + (t >> 1) * 8;
      if (D == 128) {
        const uint4 v = lds128(vb + chunk_at<D>(r, g));
        vw[t][0] = v.x, vw[t][1] = v.y, vw[t][D / 32 - 2] = v.z, vw[t][D / 32 - 1] = v.w;
      } else {
        const uint2 v = lds64(vb + chunk_at<D>(r, g >> 1) + (g & 1) * 8);
        vw[t][0] = v.x, vw[t][1] = v.y;
      }
    }
    // Tokens that some rows of the tile see and others do not: a NaN code among
    // their values must not reach the latter as 0 * NaN.
    if (!p.sel_width && (u0 + s + 1) * kUnit > first_limit) {
      bool nan_code = false;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int k = 0; k < D / 32; ++k) nan_code = nan_code || nan_bytes(vw[t][k]) != 0;
      if (__any_sync(kFullMask, nan_code)) poison<D, NT>(sc, vw, acc);
    }
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t sel = half ? 0x7362 : 0x5140;
        const uint32_t w01 = __byte_perm(vw[0][k], vw[1][k], sel), w23 = __byte_perm(vw[2][k], vw[3][k], sel);
        const uint32_t a[4] = {cvt_lo(w01), cvt_hi(w01), cvt_lo(w23), cvt_hi(w23)};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(acc[2 * k + half][nt], a, pf[nt][0], pf[nt][1]);
      }
    }
    __syncwarp();  // every lane has read what the next copies and translations overwrite
  }

  // join the four warps
  cp_async_wait<0>();
  __syncthreads();
  float* jo = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[nt][j] += __shfl_xor_sync(kFullMask, l[nt][j], o);
      if (isnan(l[nt][j])) m[nt][j] = 0.f;  // a row of NaN scores counts in the join
      const int i = 8 * nt + 2 * c + j;
      float* row = jo + (warp * R + i) * (D + 4) + g * (D / 8);
#pragma unroll
      for (int k = 0; k < D / 16; k += 2)
        *reinterpret_cast<float4*>(row + 2 * k) =
            make_float4(acc[k][nt][j], acc[k][nt][2 + j], acc[k + 1][nt][j], acc[k + 1][nt][2 + j]);
      if (g == 0) ml[warp * R + i] = make_float2(m[nt][j], l[nt][j]);
    }
  __syncthreads();
  store_rows<D, NT, F16>(p, x, h, whole, part, jo, ml);
}

template <int D, int NT>
constexpr int kCtasPerSm = NT == 1 ? 4 : 3;

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm<D, NT>)
    attend_stream_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int R = 8 * NT;
  if (p.n_ctas == 0) {
    // one CTA per (tile, head); the last tiles of a causal sequence, which see most, first
    const int t = p.n_tiles - 1 - blockIdx.x / p.c.heads, h = blockIdx.x % p.c.heads;
    const Tile x = tile_at(p, t, R);
    if (x.rows <= 0) return;
    segment<D, NT, F16>(p, x, h, 0, tile_units<kUnit>(x), true, 0, smem);
    return;
  }
  // Equal shares of all units, tile by tile and head by head.
  __shared__ int prefix[kMaxSplitTiles + 1];
  __shared__ int warp_sums[kWarps];
  const int total = tile_prefix<kUnit, kWarps * 32>(p, R, prefix, warp_sums);
  const Share sh = share_of(p, total);
  int64_t u = sh.start;
  const int64_t end = sh.end;
  if (threadIdx.x == 0) note_job(p, R, prefix, sh);
  bool first = true;
  while (u < end) {
    const Piece g = piece_at(p, prefix, sh, u, end);
    segment<D, NT, F16>(p, tile_at(p, g.tile, R), g.h, g.u0, g.u1, g.whole,
                        2 * static_cast<int64_t>(blockIdx.x) + (first ? 0 : 1), smem);
    first = false;
    u += g.u1 - g.u0;
  }
}

// Joins the parts of the (tile, head)s that several CTAs shared, in the order of
// their keys: block x does CTA x's job.  A warp takes a row; of many parts,
// the block's eight warps take a row together, every eighth part each, so that
// it is not one long chain of loads.
template <int D>
__device__ __forceinline__ void add_parts(const AttendParams& p, int first, int parts, int R, int i, int c, int step,
                                          int d, float& m, float& l, float (&o)[D / 32]) {
  auto index = [&](int k) { return (k == 0 ? first : 2 * (static_cast<int64_t>(blockIdx.x) + k * p.lanes)) * R + i; };
  m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int k = c; k < parts; k += step) m = fmaxf(m, __ldcg(&p.part_ml[index(k)]).x);
#pragma unroll 4
  for (int k = c; k < parts; k += step) {
    const int64_t at = index(k);
    const float2 v = __ldcg(&p.part_ml[at]);
    float a[D / 32];
    if (D == 128) {
      const float4 w = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + d));
      a[0] = w.x, a[1] = w.y, a[D / 32 - 2] = w.z, a[D / 32 - 1] = w.w;
    } else {
      const float2 w = __ldcg(reinterpret_cast<const float2*>(p.part_o + at * D + d));
      a[0] = w.x, a[1] = w.y;
    }
    const float h = root_factor(v.x, m), f = h * h;
    l += v.y * h * h;
#pragma unroll
    for (int e = 0; e < D / 32; ++e)
      if (v.x != -INFINITY) o[e] += f * a[e];
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendParams p, int R) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const JoinJob g = p.jobs[blockIdx.x];
  if (g.last < 0) return;
  const int parts = static_cast<int>(share_owner(g.last, g.units, min(g.units, static_cast<int64_t>(p.n_ctas / p.lanes)))) -
                    static_cast<int>(blockIdx.x / p.lanes) + 1;
  constexpr int kN = D / 32, kWarps = 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = lane * kN;
  const bool together = parts > kWarps;
  __shared__ float sum[kWarps][D];
  __shared__ float2 ml[kWarps];
  for (int i = together ? blockIdx.y : blockIdx.y * kWarps + warp; i < g.rows; i += gridDim.y * (together ? 1 : kWarps)) {
    float m, l, o[kN];
    add_parts<D>(p, g.first, parts, R, i, together ? warp : 0, together ? kWarps : 1, d, m, l, o);
    if (together) {  // (all warps have the same i)
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kN; ++e) sum[warp][d + e] = o[e];
      if (lane == 0) ml[warp] = make_float2(m, l);
      __syncthreads();
      if (warp != 0) continue;
#pragma unroll
      for (int k = 1; k < kWarps; ++k) m = fmaxf(m, ml[k].x);
      l = 0.f;
#pragma unroll
      for (int e = 0; e < kN; ++e) o[e] = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float2 v = ml[k];
        const float h = root_factor(v.x, m), f = h * h;
        l += v.y * h * h;
#pragma unroll
        for (int e = 0; e < kN; ++e)
          if (v.x != -INFINITY) o[e] += f * sum[k][d + e];
      }
    }
    const int pair = g.pair + i;
    const int64_t at = (g.q0 + pair / p.G) * static_cast<int64_t>(p.Hq) + g.h * p.G + pair % p.G;
    const float inv = m == -INFINITY ? 0.f : 1.f / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (at * D + d) * 2);
#pragma unroll
    for (int e = 0; e < kN; e += 2) dst[e / 2] = pack_act<F16>(o[e] * kSumUnit * inv, o[e + 1] * kSumUnit * inv);
    if (p.lse && lane == 0) p.lse[at] = row_lse(m, l);
  }
}

template <int D, int NT, bool F16>
cudaError_t go_stream(const AttendParams& p, int grid, cudaStream_t stream) {
  constexpr int kBytes = Smem<D, NT>::kBytes;
  const cudaError_t e =
      cudaFuncSetAttribute(attend_stream_kernel<D, NT, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  attend_stream_kernel<D, NT, F16><<<grid, kWarps * 32, kBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int D, bool F16>
cudaError_t go_join(const AttendParams& p, int R, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_ctas), R <= 16 ? R : 32);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<D, F16>, p, R);
}

}  // namespace

int attend_stream_ctas_per_sm(int rows) { return rows <= 8 ? 4 : 3; }

cudaError_t launch_attend_stream(const AttendParams& p, int D, int rows, bool f16, int grid, cudaStream_t stream) {
#define HWR_GO(DD, NN) return f16 ? go_stream<DD, NN, true>(p, grid, stream) : go_stream<DD, NN, false>(p, grid, stream)
  if (D == 128) {
    if (rows == 8) HWR_GO(128, 1);
    HWR_GO(128, 2);
  }
  if (rows == 8) HWR_GO(64, 1);
  HWR_GO(64, 2);
#undef HWR_GO
}

cudaError_t launch_attend_join(const AttendParams& p, int D, int rows, bool f16, cudaStream_t stream) {
  if (D == 128) return f16 ? go_join<128, true>(p, rows, stream) : go_join<128, false>(p, rows, stream);
  return f16 ? go_join<64, true>(p, rows, stream) : go_join<64, false>(p, rows, stream);
}

}  // namespace hwr
