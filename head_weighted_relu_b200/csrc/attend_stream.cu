// attend_stream.cu -- attention over the 8-bit cache for few query rows per
// key/value head (decode steps, selected positions): up to 16 rows share one
// pass over the keys, which is bound by reading them.
//
// A warp works alone: it copies 16 tokens' codes (2 D bytes each) at a time
// into a ring of its own in shared memory (cp.async, kDepth steps ahead), so
// that nothing but its own copies holds it up.  Codes become FP16 in registers
// (exact) in the fragment layout of mma.m16n8k16 without any shuffle: the order
// of the head dimension inside a product is free, so lane group c takes
// dimensions 32c .. 32c+31 of a key row as two 16-byte reads; and the order of
// an output's columns is free, so lane group g takes columns 16g .. 16g+15 of
// four value rows as four 16-byte reads, interleaved by byte permutes.  The
// score fragment is the weight fragment of the second product.  A CTA's four
// warps take every fourth 16 tokens of its keys and join at the end.
#include "attend.cuh"

namespace hwr {
namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;                  // tokens of a warp step
constexpr int kUnit = kWarps * kStep;      // keys of a unit
constexpr int kChunk = 256;                // keys translated at a time
constexpr int kDepth = 3;                  // ring entries per warp
constexpr int kChunkSteps = kChunk / kUnit;

template <int D>
struct Smem {
  static constexpr int kStepBytes = 2 * kStep * D;
  static constexpr int kRing = kWarps * kDepth * kStepBytes;
  static constexpr int kJoin = kWarps * kStreamRows * (D + 4) * 4;   // reuses the ring
  static constexpr int kTable = 2 * kChunk * 16;
  static constexpr int kBytes = (kRing > kJoin ? kRing : kJoin) + kTable + kWarps * kStreamRows * 8;
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

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The query fragments of rows g and g+8: dimensions 4 steps at a time, of the
// lane's own D/4 consecutive ones.  Returns the two rows' score factors.
template <int D, bool F16>
__device__ __forceinline__ void load_q(const AttendParams& p, const Tile& x, int h, uint32_t (&qf)[D / 16][4],
                                       float (&factor)[2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = g + 8 * half;
    const bool on = i < x.rows;
    const int pair = x.first + (on ? i : 0);
    const uint8_t* src =
        p.q + (x.q0 + pair / p.G) * p.q_stride + (h * p.G + pair % p.G) * (2 * D) + c * (D / 2);
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
    factor[half] = s * p.scale_log2;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qf[k][half] = w[2 * k];          // dimensions 4k, 4k+1 of the lane's
      qf[k][half + 2] = w[2 * k + 1];  // 4k+2, 4k+3
    }
  }
}

template <int D>
__device__ __forceinline__ void issue_step(const AttendParams& p, const TokenEntry* table, int step_in_table,
                                           int64_t head, uint32_t ring) {
  // 16 rows of D/16 chunks, of K and of V
  const int lane = threadIdx.x & 31;
  constexpr int kCh = D / 16, kPer = kCh * kStep / 32;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = (i * 32 + lane) / kCh, ch = lane % kCh;
    const uint32_t off = table[step_in_table * kStep + r].off16;
    const bool on = off != kNoToken;
    const int64_t at = on ? (static_cast<int64_t>(off) + head + ch) * 16 : 0;
    const uint32_t dst = ring + chunk_at<D>(r, ch);
    cp_async16(dst, p.c.k + at, on);
    cp_async16(dst + kStep * D, p.c.v + at, on);
  }
  cp_async_commit();
}

// Writes the joined rows of a segment: whole ones as outputs, others as parts.
template <int D, bool F16>
__device__ __forceinline__ void store_rows(const AttendParams& p, const Tile& x, int h, bool whole, int64_t part,
                                           const float* acc, const float2* ml) {
  // acc [kWarps][16][D+4] (columns in order), ml [kWarps][16]
  constexpr int kPer = D / 8;  // threads of a row
  const int d = (threadIdx.x % kPer) * 8;
  for (int i = threadIdx.x / kPer; i < x.rows; i += kWarps * 32 / kPer) {
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w * kStreamRows + i].x);
    float l = 0.f, o[8] = {};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 v = ml[w * kStreamRows + i];
      const float f = v.x == -INFINITY ? 0.f : ex2(v.x - m);
      l += f * v.y;
      if (f != 0.f) {
        const float* a = acc + (w * kStreamRows + i) * (D + 4) + d;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += f * a[e];
      }
    }
    if (whole) {
      const int pair = x.first + i;
      const int64_t at = (x.q0 + pair / p.G) * static_cast<int64_t>(p.Hq) + h * p.G + pair % p.G;
      const float inv = m == -INFINITY ? 0.f : 1.f / l;
      uint4 v;
      v.x = pack_act<F16>(o[0] * inv, o[1] * inv), v.y = pack_act<F16>(o[2] * inv, o[3] * inv);
      v.z = pack_act<F16>(o[4] * inv, o[5] * inv), v.w = pack_act<F16>(o[6] * inv, o[7] * inv);
      *reinterpret_cast<uint4*>(p.out + (at * D + d) * 2) = v;
      if (p.lse && d == 0) p.lse[at] = m == -INFINITY ? -INFINITY : kLn2 * (m - kHead + log2f(l));
    } else {
      float* dst = p.part_o + (part * kStreamRows + i) * D + d;
      *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<float4*>(dst + 4) = make_float4(o[4], o[5], o[6], o[7]);
      if (d == 0) p.part_ml[part * kStreamRows + i] = make_float2(m, l);
    }
  }
}

// 0xFF in each byte of w that is a NaN code (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// Takes the NaN codes out of a step's values, and makes NaN the outputs of the
// rows that do see them: the columns where (row sees token) x (code is NaN),
// again a matrix product, is not zero.  sc: the masked scores.
template <int D>
__device__ __forceinline__ void poison(const float (&sc)[2][4], uint32_t (&vw)[4][D / 32], float (&acc)[D / 8][4]) {
  uint32_t sees[4];
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int half = 0; half < 2; ++half)
      sees[nt * 2 + half] = (sc[nt][half * 2] == -INFINITY ? 0u : 0x3C00u) |
                            (sc[nt][half * 2 + 1] == -INFINITY ? 0u : 0x3C000000u);
#pragma unroll
  for (int k = 0; k < D / 32; ++k) {
    uint32_t nb[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      nb[t] = nan_bytes(vw[t][k]);
      vw[t][k] &= ~nb[t];
    }
#pragma unroll
    for (int byte = 0; byte < 4; ++byte) {
      const int sh = 8 * byte;
      float hit[4] = {};
      mma16816(hit, sees, ((nb[0] >> sh) & 1u) * 0x3C00u | ((nb[1] >> sh) & 1u) * 0x3C000000u,
               ((nb[2] >> sh) & 1u) * 0x3C00u | ((nb[3] >> sh) & 1u) * 0x3C000000u);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (hit[e] > 0.f) acc[4 * k + byte][e] = NAN;
    }
  }
}

// Keys [64 u0, 64 u1) of (tile, head).
template <int D, bool F16>
__device__ void segment(const AttendParams& p, const Tile& x, int h, int u0, int u1, bool whole, int64_t part,
                        uint8_t* smem) {
  constexpr int kRingBytes = Smem<D>::kRing > Smem<D>::kJoin ? Smem<D>::kRing : Smem<D>::kJoin;
  TokenEntry* table = reinterpret_cast<TokenEntry*>(smem + kRingBytes);
  float2* ml = reinterpret_cast<float2*>(smem + kRingBytes + Smem<D>::kTable);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * (kDepth * Smem<D>::kStepBytes);
  const int64_t head = h * p.c.head16;
  const int n = u1 - u0;

  // translate chunk 0 (and 1 before it is needed)
  auto fill = [&](int chunk) {
    TokenEntry* t = table + (chunk & 1) * kChunk;
#pragma unroll
    for (int i = 0; i < kChunk / (kWarps * 32); ++i) {
      const int k = i * kWarps * 32 + threadIdx.x;
      t[k] = translate(p, x, h, u0 * kUnit + chunk * kChunk + k);
    }
  };
  __syncthreads();  // the previous segment's buffers are free
  fill(0);
  uint32_t qf[D / 16][4];
  float factor[2];
  load_q<D, F16>(p, x, h, qf, factor);
  int limit[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int i = g + 8 * half;
    limit[half] = i < x.rows ? row_limit(p, x, x.first + i) : 0;
  }
  // the least number of positions that a row of the tile sees
  const int first_limit = p.sel_width ? 0 : row_limit(p, x, x.first);
  float acc[D / 8][4] = {};
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  __syncthreads();

  int issued = 0;
  auto step_table = [&](int s) { return ((s / kChunkSteps) & 1) * kChunk + (s % kChunkSteps) * kUnit + warp * kStep; };
#pragma unroll 1
  for (; issued < kDepth - 1; ++issued) {
    if (issued < n && issued < kChunkSteps)
      issue_step<D>(p, table + step_table(issued), 0, head, ring + issued * Smem<D>::kStepBytes);
    else
      cp_async_commit();
  }
  static_assert(kDepth - 1 <= kChunkSteps, "the first chunk covers the first copies");

#pragma unroll 1
  for (int s = 0; s < n; ++s) {
    if (s % kChunkSteps == 0) {
      // the next chunk's table, before a copy of it can be issued; its buffer's
      // last reader was the step before this one
      __syncthreads();
      if (s + kChunkSteps < n) fill(s / kChunkSteps + 1);
      __syncthreads();
    }
    if (issued < n)
      issue_step<D>(p, table + step_table(issued), 0, head, ring + (issued % kDepth) * Smem<D>::kStepBytes);
    else
      cp_async_commit();
    ++issued;
    cp_async_wait<kDepth - 1>();
    __syncwarp();
    const uint32_t kb = ring + (s % kDepth) * Smem<D>::kStepBytes, vb = kb + kStep * D;

    float sc[2][4] = {};
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int r = nt * 8 + g;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint4 v = lds128(kb + chunk_at<D>(r, D == 128 ? 2 * c + i : c));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t b0 = e4m3x2_to_f16x2(static_cast<uint16_t>(w[j]));
          const uint32_t b1 = e4m3x2_to_f16x2(static_cast<uint16_t>(w[j] >> 16));
          mma16816(sc[nt], qf[i * 4 + j], b0, b1);
        }
      }
    }
    // scores of tokens 2c, 2c+1 (nt 0), 8+2c, 8+2c+1 (nt 1), rows g and g+8
    const TokenEntry* te = table + step_table(s);
    float top[2] = {m[0], m[1]};
    float ivs[4], lvs[4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int4 e = *reinterpret_cast<const int4*>(te + nt * 8 + 2 * c + j);
        const float ks = __int_as_float(e.z);
        lvs[nt * 2 + j] = __int_as_float(e.w);
        ivs[nt * 2 + j] = ex2(-lvs[nt * 2 + j]);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float u = fmaf(sc[nt][half * 2 + j] * ks, factor[half], lvs[nt * 2 + j]);
          u = e.y < limit[half] ? u : -INFINITY;
          sc[nt][half * 2 + j] = u;
          top[half] = fmaxf(top[half], u);
        }
      }
    }
    // the reference rises only when it is exceeded by the slack, by the row's
    // maximum over the four lanes that share it
    const bool up = top[0] > m[0] + kSlack || top[1] > m[1] + kSlack;
    if (__any_sync(kFullMask, up)) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        top[half] = fmaxf(top[half], __shfl_xor_sync(kFullMask, top[half], 1));
        top[half] = fmaxf(top[half], __shfl_xor_sync(kFullMask, top[half], 2));
        const float f = top[half] == m[half] || top[half] == -INFINITY ? 1.f : ex2(m[half] - top[half]);
        m[half] = top[half];
        l[half] *= f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) acc[i][half * 2] *= f, acc[i][half * 2 + 1] *= f;
      }
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0] - kHead, m[1] == -INFINITY ? 0.f : m[1] - kHead};
    uint32_t pf[4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float p0 = ex2(sc[nt][half * 2] - ref[half]), p1 = ex2(sc[nt][half * 2 + 1] - ref[half]);
        l[half] = fmaf(p0, ivs[nt * 2], l[half]);
        l[half] = fmaf(p1, ivs[nt * 2 + 1], l[half]);
        pf[nt * 2 + half] = half2_of(p0, p1);
      }
    }
    // values: tokens 2c, 2c+1, 2c+8, 2c+9; lane group g's D/8 columns
    uint32_t vw[4][D / 32];
    bool nan_code = false;
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
    const bool edge = !p.sel_width && u0 * kUnit + (s + 1) * kUnit > first_limit;
    if (edge) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int k = 0; k < D / 32; ++k) nan_code = nan_code || nan_bytes(vw[t][k]) != 0;
      if (__any_sync(kFullMask, nan_code)) poison<D>(sc, vw, acc);
    }
#pragma unroll
    for (int k = 0; k < D / 32; ++k) {
      const uint32_t lo01 = __byte_perm(vw[0][k], vw[1][k], 0x5140), hi01 = __byte_perm(vw[0][k], vw[1][k], 0x7362);
      const uint32_t lo23 = __byte_perm(vw[2][k], vw[3][k], 0x5140), hi23 = __byte_perm(vw[2][k], vw[3][k], 0x7362);
      mma16816(acc[4 * k], pf, e4m3x2_to_f16x2(static_cast<uint16_t>(lo01)),
               e4m3x2_to_f16x2(static_cast<uint16_t>(lo23)));
      mma16816(acc[4 * k + 1], pf, e4m3x2_to_f16x2(static_cast<uint16_t>(lo01 >> 16)),
               e4m3x2_to_f16x2(static_cast<uint16_t>(lo23 >> 16)));
      mma16816(acc[4 * k + 2], pf, e4m3x2_to_f16x2(static_cast<uint16_t>(hi01)),
               e4m3x2_to_f16x2(static_cast<uint16_t>(hi23)));
      mma16816(acc[4 * k + 3], pf, e4m3x2_to_f16x2(static_cast<uint16_t>(hi01 >> 16)),
               e4m3x2_to_f16x2(static_cast<uint16_t>(hi23 >> 16)));
    }
    __syncwarp();  // every lane has read the ring entry that the next copy overwrites
  }

  // join the four warps
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    l[half] += __shfl_xor_sync(kFullMask, l[half], 1);
    l[half] += __shfl_xor_sync(kFullMask, l[half], 2);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half)
    if (isnan(l[half])) m[half] = 0.f;  // a row of NaN scores counts in the join
  cp_async_wait<0>();
  __syncthreads();
  float* jo = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float* row = jo + (warp * kStreamRows + g + 8 * half) * (D + 4);
    // fragment column 2c+j of accumulator i is column (2c+j)*(D/8) + i
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < D / 8; i += 4)
        *reinterpret_cast<float4*>(row + (2 * c + j) * (D / 8) + i) =
            make_float4(acc[i][half * 2 + j], acc[i + 1][half * 2 + j], acc[i + 2][half * 2 + j],
                        acc[i + 3][half * 2 + j]);
    if (c == 0) ml[warp * kStreamRows + g + 8 * half] = make_float2(m[half], l[half]);
  }
  __syncthreads();
  store_rows<D, F16>(p, x, h, whole, part, jo, ml);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kWarps * 32, 3) attend_stream_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  if (p.n_ctas == 0) {
    // one CTA per (tile, head); the last tiles of a causal sequence, which see most, first
    const int t = p.n_tiles - 1 - blockIdx.x / p.c.heads, h = blockIdx.x % p.c.heads;
    const Tile x = tile_at<kStreamRows>(p, t);
    if (x.rows <= 0) return;
    segment<D, F16>(p, x, h, 0, tile_units<kUnit>(x), true, 0, smem);
    return;
  }
  // Equal shares of all units, tile by tile and head by head.
  __shared__ int prefix[kMaxSplitTiles + 1];
  __shared__ int warp_sums[kWarps];
  int total = 0;
  for (int t0 = 0; t0 < p.n_tiles; t0 += kWarps * 32) {
    const int t = t0 + threadIdx.x;
    const int u = t < p.n_tiles ? tile_units<kUnit>(tile_at<kStreamRows>(p, t)) : 0;
    int all;
    const int before = block_scan_tiles<kWarps * 32>(u, &all, warp_sums);
    if (t < p.n_tiles) prefix[t] = total + before;
    total += all;
  }
  if (threadIdx.x == 0) prefix[p.n_tiles] = total;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int t = threadIdx.x; t <= p.n_tiles; t += kWarps * 32) p.prefix[t] = prefix[t];
  const int64_t units = static_cast<int64_t>(total) * p.c.heads;
  const int64_t n = min(units, static_cast<int64_t>(p.n_ctas));
  if (blockIdx.x >= n) return;
  int64_t u = share_start(blockIdx.x, units, n);
  const int64_t end = share_start(blockIdx.x + 1, units, n);
  bool first = true;
  while (u < end) {
    int lo = 0, hi = p.n_tiles - 1;  // the last tile that starts at or before u (empty ones start with the next)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (static_cast<int64_t>(prefix[mid]) * p.c.heads <= u) lo = mid; else hi = mid - 1;
    }
    const int tu = prefix[lo + 1] - prefix[lo];
    const int64_t in = u - static_cast<int64_t>(prefix[lo]) * p.c.heads;
    const int h = static_cast<int>(in / tu), u0 = static_cast<int>(in % tu);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(tu), u0 + (end - u)));
    const Tile x = tile_at<kStreamRows>(p, lo);
    segment<D, F16>(p, x, h, u0, u1, u0 == 0 && u1 == tu, 2 * static_cast<int64_t>(blockIdx.x) + (first ? 0 : 1),
                    smem);
    first = false;
    u += u1 - u0;
  }
}

// Joins the parts of the (tile, head)s that several CTAs shared, in the order
// of their keys.
template <int D, int R, bool F16>
__global__ void __launch_bounds__(128) attend_join_kernel(const __grid_constant__ AttendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = blockIdx.x / p.c.heads, h = blockIdx.x % p.c.heads;
  const int base = p.prefix[t], tu = p.prefix[t + 1] - base;
  if (tu == 0) return;
  const int64_t units = static_cast<int64_t>(p.prefix[p.n_tiles]) * p.c.heads;
  const int64_t u0 = static_cast<int64_t>(base) * p.c.heads + static_cast<int64_t>(h) * tu;
  const int64_t n = min(units, static_cast<int64_t>(p.n_ctas));
  const int64_t c0 = share_owner(u0, units, n), c1 = share_owner(u0 + tu - 1, units, n);
  if (c0 == c1) return;
  const int64_t first = 2 * c0 + (share_start(c0, units, n) == u0 ? 0 : 1);
  const Tile x = tile_at<R>(p, t);
  constexpr int kPer = D / 4;  // threads of a row
  const int d = (threadIdx.x % kPer) * 4;
  for (int i = blockIdx.y * (128 / kPer) + threadIdx.x / kPer; i < x.rows; i += gridDim.y * (128 / kPer)) {
    float m = -INFINITY;
    for (int64_t c = c0; c <= c1; ++c) m = fmaxf(m, p.part_ml[(c == c0 ? first : 2 * c) * R + i].x);
    float l = 0.f, o[4] = {};
#pragma unroll 4
    for (int64_t c = c0; c <= c1; ++c) {
      const int64_t at = (c == c0 ? first : 2 * c) * R + i;
      const float2 v = p.part_ml[at];
      const float4 a = *reinterpret_cast<const float4*>(p.part_o + at * D + d);
      const float f = v.x == -INFINITY ? 0.f : ex2(v.x - m);
      l += f * v.y;
      if (f != 0.f) o[0] += f * a.x, o[1] += f * a.y, o[2] += f * a.z, o[3] += f * a.w;
    }
    const int pair = x.first + i;
    const int64_t at = (x.q0 + pair / p.G) * static_cast<int64_t>(p.Hq) + h * p.G + pair % p.G;
    const float inv = m == -INFINITY ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(p.out + (at * D + d) * 2) =
        make_uint2(pack_act<F16>(o[0] * inv, o[1] * inv), pack_act<F16>(o[2] * inv, o[3] * inv));
    if (p.lse && d == 0) p.lse[at] = m == -INFINITY ? -INFINITY : kLn2 * (m - kHead + log2f(l));
  }
}

template <int D, bool F16>
cudaError_t go_stream(const AttendParams& p, int grid, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(attend_stream_kernel<D, F16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
  if (e != cudaSuccess) return e;
  attend_stream_kernel<D, F16><<<grid, kWarps * 32, Smem<D>::kBytes, stream>>>(p);
  return cudaGetLastError();
}

template <int D, int R, bool F16>
cudaError_t go_join(const AttendParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.n_tiles) * p.c.heads, R / 16);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attend_join_kernel<D, R, F16>, p);
}

}  // namespace

int attend_stream_ctas_per_sm(int D) { return 3; }

cudaError_t launch_attend_stream(const AttendParams& p, int D, bool f16, int grid, cudaStream_t stream) {
  if (D == 128) return f16 ? go_stream<128, true>(p, grid, stream) : go_stream<128, false>(p, grid, stream);
  return f16 ? go_stream<64, true>(p, grid, stream) : go_stream<64, false>(p, grid, stream);
}

cudaError_t launch_attend_join(const AttendParams& p, int D, int R, bool f16, cudaStream_t stream) {
  if (D == 128) return f16 ? go_join<128, 16, true>(p, stream) : go_join<128, 16, false>(p, stream);
  return f16 ? go_join<64, 16, true>(p, stream) : go_join<64, 16, false>(p, stream);
}

}  // namespace hwr
