// attend_tile.cu -- attention over the 8-bit cache for many query rows per
// key/value head (prefill chunks, drafts, one query of a large group): tiles of
// 128 rows x 128 keys on the fifth-generation tensor cores.
//
// Two streams of tiles run side by side in a CTA, so that one's softmax hides
// the other's products: NM = 2, the two halves of 256 rows over the same keys;
// NM = 1, the same 128 rows over alternate key tiles, joined at the end.
//   warps 0-7   softmax, four a stream, a thread a row: scores from TMEM, weights
//               back to TMEM as FP16; outputs at the end of a segment
//   warps 8-15  fill: read codes, keys and values four each, and write them as
//               FP16 (exact) in the swizzled layout of the products' operands,
//               with the tokens' scales
//   warp 16     issues the products, S = Q K^T and O += P V, P from TMEM
//   warps 17-19 look up the tokens of the tiles ahead
// The arithmetic is that of attend.cuh: scales act on the FP32 scores, so the
// operands are bare codes and a row's query scaled by a power of two.  The
// reference of a row's exponentials rises only when a score exceeds it by
// kSlack, which is rare after the first tile; then the row's outputs are
// rescaled in TMEM.
//
// What bounds it (D = 128, two streams).  A tile of 128 keys is 2,048 clocks of
// products for 256 rows (32 of 128x128x16, 64 clocks each), 2,048 of
// exponentials (16 a clock and SM), about 1,000 of the integer pipe (conversions,
// maxima) and 2,000 of shared memory; measured are about 4,700: a stream's
// softmax (2,100 alone, 2,800 beside the other's, 3,000 to 3,400 beside the
// fill) and its products (1,100 and the hand-overs) follow one another, and two
// streams do not cover all of each other.  2,048 rows over 16,384 tokens, 64
// heads on 8: 1.19 ms, 866 TFLOP/s (1.27 ms call after call, at the power limit;
// 41% of the tensor pipe's cycles, 41% of the exponential pipe's).  One stream's
// rows, NM = 1: one query of 64 heads over 1,048,576 tokens 112 us, 2.4 TB/s (33%
// of the tensor pipe's cycles).
// Tried and worse: scores in halves of 64 keys, so that products run during the
// softmax (the halves' products re-read the queries: 1.34 ms); one pass that
// keeps the weights in registers, or takes no maximum until a sum overflows (1.35
// ms: longer code or spilled registers, which meet a small instruction cache and
// the L1 that shared memory leaves); issuing products inside one lane's branch
// (130 clocks each instead of 67).  Beginning the value products after half of the
// weights, and two tiles of codes on the way, changed nothing.
#include "attend.cuh"
#include "internal.h"

namespace hwr {
namespace {

constexpr int kSoftThreads = 256;
constexpr int kFillWarps = 8;
constexpr int kThreads = kSoftThreads + kFillWarps * 32 + 128;
constexpr int kKeys = 128;                     // keys of a tile: a unit
constexpr int kPanel = 128 * 128;              // bytes of 128 rows of 64 FP16
constexpr int kSoftBar = 1, kLookBar = 2;
constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr uint32_t kTmemCols = 512;

// Registers a thread: the block starts with kLaunchRegs (65,536 / 640, in whole
// eights), and the three shares come to no more than that.
constexpr int kLaunchRegs = 96;
template <int NM>
struct Regs {
  static constexpr int kSoft = 128, kFill = 88, kIssue = 48;
  static_assert(kSoftThreads * kSoft + kFillWarps * 32 * kFill + 128 * kIssue <= kThreads * kLaunchRegs, "");
};

template <int N>
__device__ __forceinline__ void regs_to() {  // (down to more than there are, or up to fewer, is no valid instruction)
  if constexpr (N > kLaunchRegs)
    regs_up<N>();
  else
    regs_down<N>();
}

struct Bars {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2];
  uint64_t sfull[2], pfull[2];  // by stream
  uint64_t qfull, ofull, done, left;
  uint64_t tfull[8], tempty[8];
  uint32_t tmem;
  int abort, tries;  // a wait has run out; suspended tries until it does
};

// Dynamic shared memory, from a 1,024-byte boundary.
template <int D, int NM, bool U16>
struct Lay {
  static constexpr int kPanels = D / 64;
  static constexpr int kEntries = U16 ? 8 : 128;  // look-ups of a tile
  static constexpr int kScales = U16 ? 32 : 384;  // their floats: a float4 each, or an array of each
  static constexpr int kRing = U16 || NM == 1 ? 8 : 4;  // tiles whose look-ups are kept
  static constexpr int kKV = kPanels * kPanel;   // a K or V tile
  static constexpr int kQ = 0;                   // [NM][kPanels] panels; then the outputs' stage
  static constexpr int kK = kQ + NM * kKV;       // [2]
  static constexpr int kV = kK + 2 * kKV;        // [2]
  static constexpr int kScale = kV + 2 * kKV;    // [kRing][kScales]: key scales, log2 value scales, 1 / value scales
  static constexpr int kPlace = kScale + kRing * kScales * 4;  // [kRing][entries]: place and number
  static constexpr int kNan = kPlace + kRing * kEntries * 8;  // [2][128][4]: NaN codes of V tokens, a bit a dimension
  static constexpr int kNanAny = kNan + 2 * 128 * 16;             // [2][4]: a word a value warp, not 0 where it has any
  static constexpr int kRowNan = kNanAny + 64;                    // [256][4]: dimensions made NaN, by row
  static constexpr int kFactor = kRowNan + 256 * 16;              // [256]
  static constexpr int kMl = kFactor + 1024;                      // [128] float2
  static constexpr int kSeg = kMl + 1024;                         // [2] the softmax warps' Segment
  static constexpr int kEx = kSeg + 256;                          // NM = 1: [128] rows of 32 columns
  static constexpr int kBars = kEx + (NM == 1 ? 128 * 128 : 0);
  static constexpr int kPrefix = kBars + 320;                     // [kMaxSplitTiles2 + 1] and 17 sums
  static constexpr int kBytes = kPrefix + (kMaxSplitTiles2 + 1) * 4 + 128 + 1024;
};
static_assert(sizeof(Bars) <= 320, "");

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16)); }
// 0xFF in each byte of w that is a NaN code (0x7F or 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); }

// A wait that, once it has run out, makes every further wait of the CTA end at
// once: the loops then run through on what the buffers hold, all within bounds
// (nothing is loaded from a place that no look-up gave), and the rows become NaN.
// A try suspends the thread for up to kTryNs, so that waiting warps take no
// issue slots from the others.
constexpr uint32_t kTryNs = 100000;
constexpr int kWaitTries = 100000, kTestTries = 10;
__device__ __forceinline__ bool try_now(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool try_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kTryNs)
      : "memory");
  return ok != 0;
}
// False when it ran out.
__device__ __forceinline__ bool wait(Bars* b, uint64_t* bar, uint32_t parity) {
  if (try_now(bar, parity)) return true;
#pragma unroll 1
  for (int i = 0; i < *reinterpret_cast<volatile int*>(&b->tries) && !*reinterpret_cast<volatile int*>(&b->abort); ++i)
    if (try_long(bar, parity)) return true;
  *reinterpret_cast<volatile int*>(&b->abort) = 1;
  return false;
}

// What a segment is: keys [128 u0, 128 u1) of (tile, head).
struct Segment {
  Tile x;          // (not for the issuing role)
  int h, u0, n;
  bool whole;
  int64_t part;
};

// -------------------------------------------------------------- look-ups --
// Three warps look up the tokens of the tiles ahead: their places for the fill
// warps, their scales for the softmax.  Where 16 positions share their page and
// scales (U16), an entry stands for 16 tokens: `off` is the place of the first
// and `valid` their number; otherwise for one.
template <int D, int NM, bool U16>
__device__ __forceinline__ void look_up(const AttendParams& p, const Segment& g, uint8_t* smem, uint32_t tiles) {
  using L = Lay<D, NM, U16>;
  constexpr int kEntries = L::kEntries;
  constexpr int kPer = U16 ? 1 : 4;    // of a lane
  constexpr int kTiles = U16 ? 2 : 1;  // that a warp takes at once
  static_assert(3 * kTiles <= L::kRing, "");
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 17;
  const int end = min(g.x.n_keys, (g.u0 + g.n) * kKeys);
  const Translate tr(p, g.x, g.h, end);
  if (p.test_wait) return;  // (test hook: looks up nothing, so that the others' waits run out)
#pragma unroll 1
  for (int j0 = 0; j0 < g.n; j0 += 3 * kTiles) {
    const int j = j0 + warp * kTiles + (U16 ? lane >> 3 & 1 : 0), en = U16 ? lane & 7 : lane;
    const bool on_lane = j < g.n && (!U16 || lane < 16);
    const uint32_t slot = (tiles + j) % L::kRing, parity = ((tiles + j) / L::kRing & 1) ^ 1;
    Translate::Index ix[kPer];
    Translate::Page pg[kPer];
    Translate::Place at[kPer];
    float ks[kPer], vs[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) ix[e] = tr.index(j < g.n ? (g.u0 + j) * kKeys + (U16 ? en * 16 : e * 32 + en) : -1);
#pragma unroll
    for (int e = 0; e < kPer; ++e) pg[e] = tr.page(ix[e]);
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      at[e] = tr.place(pg[e]);
      const bool on = at[e].pos != INT32_MAX;
      ks[e] = on ? __ldg(p.c.ks + at[e].scale) : 0.f;
      vs[e] = on ? __ldg(p.c.vs + at[e].scale) : 1.f;
    }
    if (on_lane) wait(bars, &bars->tempty[slot], parity);
    __syncwarp();
    if (on_lane) {
      float* sc = reinterpret_cast<float*>(smem + L::kScale) + slot * L::kScales;
      uint2* place = reinterpret_cast<uint2*>(smem + L::kPlace) + slot * kEntries;
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int k = e * 32 + en;
        const bool on = at[e].pos != INT32_MAX;
        const float lvs = on ? __log2f(fmaxf(vs[e], kMinBlockScale)) : -INFINITY;
        const float ivs = on ? inverse_scale(lvs) : 0.f;
        if (U16)
          reinterpret_cast<float4*>(sc)[k] = make_float4(ks[e], lvs, ivs, 0.f);
        else
          sc[k] = ks[e], sc[kEntries + k] = lvs, sc[2 * kEntries + k] = ivs;
        place[k] = make_uint2(at[e].off16, on ? (U16 ? min(end - at[e].pos, 16) : 1) : 0);
      }
    }
    __syncwarp();
    if (on_lane && en == 0) mbar_arrive(&bars->tfull[slot]);
    // A round, no longer than the ring, is complete before the next: a barrier's
    // parity would not tell two laps apart.
    named_bar(kLookBar, 96);
  }
}

// ------------------------------------------------------------------- fill --
// Four warps fill the keys' tiles and four the values', 32 tokens of each a warp.
// on: `place` holds a look-up; otherwise nothing is loaded.
template <int D, bool U16>
__device__ __forceinline__ void load_codes(const uint8_t* base, uint32_t row16, const uint2* place, bool on,
                                           uint4 (&r)[D / 16]) {
  constexpr int kCh = D / 16, kRowsPer = 32 / kCh;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint2 w;
    if (U16) w = place[warp * 2 + g];
    const uint8_t* at = base + (static_cast<int64_t>(w.x) << 4);  // (U16: base is of the lane's row)
#pragma unroll
    for (int i = 0; i < kCh / 2; ++i) {
      const uint32_t t = i * kRowsPer + lane / kCh;
      if (!U16) w = place[warp * 32 + g * 16 + t], at = base + (static_cast<int64_t>(w.x) << 4);
      r[g * (kCh / 2) + i] = on && (U16 ? t : 0u) < w.y
                                 ? ldg_stream(U16 ? at + static_cast<int64_t>(i * kRowsPer * 16) * row16 : at)
                                 : make_uint4(0, 0, 0, 0);
    }
  }
}

// Writes 32 tokens' codes as FP16 rows of 64 dimensions, chunks of 16 bytes at
// (chunk ^ row % 8).  The upper half of a row's lanes writes its two chunks in
// the other order, so that eight lanes never meet in a bank.
template <int D>
__device__ __forceinline__ void store_codes(uint32_t dst, const uint4 (&r)[D / 16]) {
  constexpr int kCh = D / 16, kRowsPer = 32 / kCh;
  const int lane = threadIdx.x & 31, ch = lane % kCh, t0 = ((threadIdx.x >> 5) & 3) * 32 + lane / kCh;
  const bool sw = D == 128 && (ch & 4);
  dst += (ch >> 2) * kPanel + t0 * 128;
  const int c0 = (ch & 3) * 2 + (sw ? 1 : 0);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint32_t a0 = sw ? r[i].z : r[i].x, a1 = sw ? r[i].w : r[i].y, b0 = sw ? r[i].x : r[i].z,
                   b1 = sw ? r[i].y : r[i].w;
    const uint32_t at = dst + i * kRowsPer * 128 + ((c0 ^ ((t0 + i * kRowsPer) & 7)) << 4);
    sts128(at, cvt_lo(a0), cvt_hi(a0), cvt_lo(a1), cvt_hi(a1));
    sts128(at ^ 16, cvt_lo(b0), cvt_hi(b0), cvt_lo(b1), cvt_hi(b1));
  }
}

// Takes the NaN codes out of 32 tokens' values and notes them, a bit a dimension.
template <int D>
__device__ __forceinline__ void take_nans(uint4 (&r)[D / 16], uint8_t* nan, uint32_t* nan_any) {
  constexpr int kCh = D / 16, kRowsPer = 32 / kCh;
  const int lane = threadIdx.x & 31, ch = lane % kCh, t0 = ((threadIdx.x >> 5) & 3) * 32 + lane / kCh;
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    uint32_t* w[4] = {&r[i].x, &r[i].y, &r[i].z, &r[i].w};
    uint32_t bits = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t nb = nan_bytes(*w[e]);
      *w[e] &= ~nb;
      bits |= ((nb & 1u) | (nb >> 7 & 2u) | (nb >> 14 & 4u) | (nb >> 21 & 8u)) << (4 * e);
    }
    *reinterpret_cast<uint16_t*>(nan + (t0 + i * kRowsPer) * 16 + ch * 2) = static_cast<uint16_t>(bits);
    any |= bits;
  }
  any = __any_sync(kFullMask, any != 0);
  if (lane == 0) *nan_any = any;
}

// tiles: tiles filled before the segment
template <int D, int NM, bool U16>
__device__ __forceinline__ void fill(const AttendParams& p, const Segment& g, uint8_t* smem, uint32_t tiles) {
  using L = Lay<D, NM, U16>;
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, ch = lane % (D / 16);
  const bool is_v = threadIdx.x >> 7 & 1;
  const uint8_t* base =
      (is_v ? p.c.v : p.c.k) + (g.h * p.c.head16 + ch + (U16 ? lane / (D / 16) * p.c.token16 : 0)) * 16;
  const uint32_t row16 = static_cast<uint32_t>(p.c.token16);
  // tokens from here on are not seen by all rows
  const int partial = p.sel_width || !is_v ? INT32_MAX : row_limit(p, g.x, g.x.first) - g.u0 * kKeys;
  const uint32_t dst = smem_u32(smem) + (is_v ? L::kV : L::kK);
  uint64_t* empty = is_v ? bars->vempty : bars->kempty;
  uint64_t* full = is_v ? bars->vfull : bars->kfull;
  const int n = g.n;
  uint4 c[D / 16];  // codes of the tile ahead
  auto load = [&](int j) {
    if (j >= n) return;
    const uint32_t slot = (tiles + j) % L::kRing;
    const bool on = wait(bars, &bars->tfull[slot], (tiles + j) / L::kRing & 1);
    load_codes<D, U16>(base, row16, reinterpret_cast<const uint2*>(smem + L::kPlace) + slot * L::kEntries, on, c);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->tempty[slot]);
  };
  load(0);
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const uint32_t t = tiles + j, slot = t & 1;
    wait(bars, &empty[slot], (t >> 1 & 1) ^ 1);
    // Tokens that some rows see and others do not: a NaN among their values must
    // not reach the latter as 0 * NaN, so it is noted beside the tile.
    if ((j + 1) * kKeys > partial)
      take_nans<D>(c, smem + L::kNan + slot * (128 * 16),
                   reinterpret_cast<uint32_t*>(smem + L::kNanAny) + slot * 4 + warp);
    store_codes<D>(dst + slot * L::kKV, c);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[slot]);
    load(j + 1);
  }
}

// --------------------------------------------------------------- products --
// One warp.  tiles: as above; phases: bit w, the parity of the tiles that stream
// w has had; one: true for the lane that issues.
template <int D, int NM, bool U16>
__device__ __forceinline__ void products(int n, uint8_t* smem, uint32_t tiles, uint32_t& phases, uint32_t segs,
                                         uint32_t one) {
  using L = Lay<D, NM, U16>;
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const uint32_t tm = bars->tmem, base = smem_u32(smem);
  constexpr uint32_t kScoreDesc = idesc_f16<128, kKeys, false>(), kValueDesc = idesc_f16<128, D, true>();
  // (an address advances its descriptor's low word by a sixteenth of itself)
  const uint64_t qd = sw128_desc(base + L::kQ), kd = sw128_desc(base + L::kK), vd = sw128_mn_desc(base + L::kV, kPanel);
  constexpr uint32_t kHi = (1024 >> 4) | (1u << 14) | (2u << 29);
  const uint32_t q0 = static_cast<uint32_t>(qd), k0 = static_cast<uint32_t>(kd), v0 = static_cast<uint32_t>(vd);
  auto desc = [](uint32_t lo) { return static_cast<uint64_t>(kHi) << 32 | lo; };
  auto score = [&](int w, int i) {
    uint32_t q = q0 + (NM == 2 ? w * (L::kKV >> 4) : 0), k = k0 + ((tiles + i) & 1) * (L::kKV >> 4);
    asm volatile("" : "+r"(q), "+r"(k));  // (or every step's descriptors are kept through the loop)
#pragma unroll 1
    for (int s = 0; s < D / 16; ++s) {
      const uint32_t at = ((s >> 2) * kPanel + (s & 3) * 32) >> 4;
      tc_mma_f16_one(one, tm + w * 128, desc(q + at), desc(k + at), kScoreDesc, s > 0);
    }
    tc_commit_one(one, &bars->sfull[w]);
  };
  auto value = [&](int w, int i, bool first) {
    uint32_t v = v0 + ((tiles + i) & 1) * (L::kKV >> 4);
    asm volatile("" : "+r"(v));
#pragma unroll 1
    for (int s = 0; s < kKeys / 16; ++s)
      tc_mma_f16_ts_one(one, tm + 256 + w * 128, tm + w * 128 + s * 8, desc(v + s * (2048 >> 4)), kValueDesc,
                    !(first && s == 0));
  };
  auto kready = [&](int i) { wait(bars, &bars->kfull[(tiles + i) & 1], (tiles + i) >> 1 & 1); };
  auto vready = [&](int i) { wait(bars, &bars->vfull[(tiles + i) & 1], (tiles + i) >> 1 & 1); };
  auto pready = [&](int w) {
    wait(bars, &bars->pfull[w], phases >> w & 1);
    phases ^= 1u << w;
    tc_fence_after();
  };
  wait(bars, &bars->qfull, segs & 1);
  tc_fence_after();
  if (NM == 2) {
    kready(0);
    score(0, 0);
    score(1, 0);
    tc_commit_one(one, &bars->kempty[tiles & 1]);
    for (int i = 0; i < n; ++i) {
      vready(i);
      if (i + 1 < n) kready(i + 1);
      pready(0);
      value(0, i, i == 0);
      if (i + 1 < n) score(0, i + 1);
      pready(1);
      value(1, i, i == 0);
      tc_commit_one(one, &bars->vempty[(tiles + i) & 1]);
      if (i + 1 < n) {
        score(1, i + 1);
        tc_commit_one(one, &bars->kempty[(tiles + i + 1) & 1]);
      }
    }
  } else {
    for (int i = 0; i < min(n, 2); ++i) {
      kready(i);
      score(i, i);
      tc_commit_one(one, &bars->kempty[(tiles + i) & 1]);
    }
    for (int i = 0; i < n; ++i) {
      const int w = i & 1;
      vready(i);
      if (i + 2 < n) kready(i + 2);
      pready(w);
      value(w, i, i < 2);
      tc_commit_one(one, &bars->vempty[(tiles + i) & 1]);
      if (i + 2 < n) {
        score(w, i + 2);
        tc_commit_one(one, &bars->kempty[(tiles + i) & 1]);
      }
    }
  }
  tc_commit_one(one, &bars->ofull);
}

// ---------------------------------------------------------------- softmax --
// Query rows to shared memory as FP16, scaled by a power of two (and the sign of
// the score scale, so that a larger product is a larger score): copied as they
// are, then each row converted in place by a thread.
template <int D, int NM, bool U16>
__device__ __forceinline__ void load_q(const AttendParams& p, const Segment& g, uint8_t* smem, bool f16) {
  using L = Lay<D, NM, U16>;
  constexpr int kPer = D / 8, kPass = kSoftThreads / kPer;  // 16-byte chunks of a row, rows of a pass
  const int c = threadIdx.x % kPer;
  const uint32_t q = smem_u32(smem) + L::kQ;
  auto place = [&](int r, int ch) {
    return q + (r >> 7) * L::kKV + (ch >> 3) * kPanel + (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4);
  };
#pragma unroll 4
  for (int r = threadIdx.x / kPer; r < g.x.rows; r += kPass) {
    const int pair = g.x.first + r, query = pair / p.G;
    cp_async16(place(r, c), p.q + (g.x.q0 + query) * p.q_stride + (g.h * p.G + pair - query * p.G) * (2 * D) + c * 16,
               true);
  }
  cp_async_commit();
  cp_async_wait<0>();
  named_bar(kSoftBar, kSoftThreads);
  const int r = threadIdx.x;
  if (r >= g.x.rows) return;
  float s = 1.f;
  if (!f16) {
    float m = 0.f;
#pragma unroll 4
    for (int ch = 0; ch < kPer; ++ch) {
      const uint4 v = lds128(place(r, ch));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack_act<false>(w[e]);
        m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
    }
    s = row_pow2(m);
  }
  const float inv = (p.scale_log2 < 0.f ? -1.f : 1.f) / s;
  reinterpret_cast<float*>(smem + L::kFactor)[r] = s * fabsf(p.scale_log2);
  if (f16 && inv > 0.f) return;
#pragma unroll 4
  for (int ch = 0; ch < kPer; ++ch) {
    const uint32_t a = place(r, ch);
    const uint4 v = lds128(a);
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = f16 ? unpack_act<true>(w[e]) : unpack_act<false>(w[e]);
      w[e] = half2_of(f.x * inv, f.y * inv);
    }
    sts128(a, w[0], w[1], w[2], w[3]);
  }
}

struct Row {
  float m, l;      // reference, and the sum
  float factor;
};

// The scales of 16 columns: one entry of each (U16), or sixteen.
template <bool U16>
struct Scales {
  const float* s;  // of the tile
  int col;
  __device__ __forceinline__ float4 all() const { return *reinterpret_cast<const float4*>(s + col / 4); }  // U16
  __device__ __forceinline__ float4 four(int which, int e) const {
    return *reinterpret_cast<const float4*>(s + which * 128 + col + e);
  }
};

// Largest score, in base 2 and with the value's scale, of 16 columns; those from `see` on are not seen.
template <bool U16, bool MASKED>
__device__ __forceinline__ float top_of(const uint32_t* r, const Scales<U16>& sc, const Row& row, int see) {
  float top = -INFINITY;
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    float4 ks, lv;
    if (!U16) ks = sc.four(0, e), lv = sc.four(1, e);
    const float k4[4] = {ks.x, ks.y, ks.z, ks.w}, v4[4] = {lv.x, lv.y, lv.z, lv.w};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      float u[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        u[k] = __uint_as_float(r[e + i + k]);
        if (!U16) u[k] = fmaf(u[k], k4[i + k] * row.factor, v4[i + k]);
        if (MASKED && sc.col + e + i + k >= see) u[k] = -INFINITY;
      }
      top = max3(top, u[0], u[1]);
    }
  }
  if (U16) {
    const float4 a = sc.all();
    top = fmaf(top, a.x * row.factor, a.y);
  }
  return top;
}

// Weights of 16 columns, two a word, and their share of the row's sum.
template <bool U16, bool MASKED>
__device__ __forceinline__ void weights_of(const uint32_t (&r)[16], const Scales<U16>& sc, const Row& row, int see,
                                           float& l, uint32_t* out) {
  const float ref = row.m == -INFINITY ? 0.f : row.m - kHead;
  float2 sum = make_float2(0.f, 0.f), kf, c0;
  float4 a;
  if (U16) {
    a = sc.all();
    kf = make_float2(a.x * row.factor, a.x * row.factor), c0 = make_float2(a.y - ref, a.y - ref);
  }
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    float4 ks, lv, iv;
    if (!U16) ks = sc.four(0, e), lv = sc.four(1, e), iv = sc.four(2, e);
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      if (!U16) {
        kf = mul2(i ? make_float2(ks.z, ks.w) : make_float2(ks.x, ks.y), make_float2(row.factor, row.factor));
        c0 = add2(i ? make_float2(lv.z, lv.w) : make_float2(lv.x, lv.y), make_float2(-ref, -ref));
      }
      const float2 u = fma2(make_float2(__uint_as_float(r[e + i]), __uint_as_float(r[e + i + 1])), kf, c0);
      float2 w = make_float2(ex2(u.x), ex2(u.y));
      if (MASKED) {
        if (sc.col + e + i >= see) w.x = 0.f;
        if (sc.col + e + i + 1 >= see) w.y = 0.f;
      }
      sum = U16 ? add2(sum, w) : fma2(w, i ? make_float2(iv.z, iv.w) : make_float2(iv.x, iv.y), sum);
      out[(e + i) / 2] = half2_of(w.x, w.y);
    }
  }
  l = U16 ? fmaf(sum.x + sum.y, a.z, l) : l + (sum.x + sum.y);
}

// One tile of a stream: the rise of its rows' references, and its weights.  see:
// tokens that the row sees (MASKED; otherwise all).  tm_s, tm_o: the warp's
// lanes of the stream's scores and outputs; fresh: no output yet.  Two passes
// over the scores in TMEM, in loops that are not unrolled further: all roles'
// hot code together has to stay in the instruction cache (with one long pass,
// or both unrolled, every role waited for its own code).
template <int D, bool U16, bool MASKED>
__device__ __forceinline__ void softmax_tile(uint32_t tm_s, uint32_t tm_o, const float* sc, Row& row, int see,
                                             bool fresh) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 128; c += 64) {
    uint32_t a[32], b[32];
    tmem_ld_x32(tm_s + c, a);
    tmem_ld_x32(tm_s + c + 32, b);
    tmem_wait_ld(a);
    tmem_wait_ld(b);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      top = fmaxf(top, top_of<U16, MASKED>((q < 2 ? a : b) + (q & 1) * 16, Scales<U16>{sc, c + q * 16}, row, see));
  }
  uint32_t a[16], b[16], w[8];
  tmem_ld_x16(tm_s, a);
  const bool up = top > row.m + kSlack;  // (a row's own affair: its results do not depend on its neighbours)
  if (__any_sync(kFullMask, up)) {
    const float m = up ? top : row.m, h = root_factor(row.m, m), f = h * h;
    row.m = m;
    row.l *= h, row.l *= h;
    if (!fresh) {
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        tmem_ld_x16(tm_o + c, b);
        tmem_wait_ld(b);
#pragma unroll
        for (int e = 0; e < 16; ++e) b[e] = __float_as_uint(__uint_as_float(b[e]) * f);
        tmem_st_x16(tm_o + c, b);
      }
    }
  }
  // A piece's weights take the place of half its scores, and of no later ones.
  constexpr int kBody = MASKED ? 32 : 64;
#pragma unroll 1
  for (int c0 = 0; c0 < 128; c0 += kBody) {
#pragma unroll
    for (int c = 0; c < kBody; c += 32) {
      const int col = c0 + c;
      tmem_wait_ld(a);
      tmem_ld_x16(tm_s + col + 16, b);
      weights_of<U16, MASKED>(a, Scales<U16>{sc, col}, row, see, row.l, w);
      tmem_st_x8(tm_s + col / 2, w);
      tmem_wait_ld(b);
      if (col + 32 < 128) tmem_ld_x16(tm_s + col + 32, a);
      weights_of<U16, MASKED>(b, Scales<U16>{sc, col + 16}, row, see, row.l, w);
      tmem_st_x8(tm_s + col / 2 + 8, w);
    }
  }
  tmem_wait_st();
}

// A warp's 32 rows, i0 the first: whole ones as outputs, others as parts.  get(c,
// o): columns 32c .. of the lane's row (all lanes take part).  The rows go
// through `stage`, 2 D bytes each, so that they are written in full lines.
template <int D, class Get>
__device__ __forceinline__ void write_rows(const AttendParams& p, const Segment& g, uint32_t stage, int R, int i0,
                                           const Row& row, const uint32_t* nan, bool f16, Get&& get) {
  const int lane = threadIdx.x & 31, i = i0 + lane, count = min(g.x.rows - i0, 32);
  const bool none = row.m == -INFINITY, whole = g.whole;
  int at = 0;  // the row's place among the outputs, or the parts
  if (whole) {
    const int pair = g.x.first + i, query = pair / p.G;
    at = (g.x.q0 + query) * p.Hq + g.h * p.G + pair - query * p.G;
    if (p.lse && lane < count) p.lse[at] = row_lse(row.m, row.l);
  } else {
    at = static_cast<int>(g.part) * R + i;
    if (lane < count) p.part_ml[at] = make_float2(row.m, row.l);
  }
  const float unit = whole ? kSumUnit : 1.f, mul = whole ? 1.f / row.l : 1.f;
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row of the stage
  const uint32_t mine = stage + lane * (2 * D), sw = lane & 7;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    float o[32];
    get(c, o);
    const uint32_t bits = nan[c];
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = bits >> e & 1 ? NAN : none ? 0.f : o[e] * unit * mul;
    if (whole) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[k] = f16 ? pack_act<true>(o[8 * e + 2 * k], o[8 * e + 2 * k + 1])
                     : pack_act<false>(o[8 * e + 2 * k], o[8 * e + 2 * k + 1]);
        sts128(mine + (((c * 4 + e) ^ sw) << 4), w[0], w[1], w[2], w[3]);
      }
      if (c + 1 < D / 32) continue;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        sts128(mine + (((c * 8 + e) % kChunks ^ sw) << 4), __float_as_uint(o[4 * e]), __float_as_uint(o[4 * e + 1]),
               __float_as_uint(o[4 * e + 2]), __float_as_uint(o[4 * e + 3]));
      if ((c + 1) * 8 % kChunks) continue;
    }
    __syncwarp();
#pragma unroll 4
    for (int k = lane; k < 32 * kChunks; k += 32) {
      const int r = k / kChunks, ch = k % kChunks;
      const int to = __shfl_sync(kFullMask, at, r);
      if (r < count) {
        const uint4 v = lds128(stage + r * (2 * D) + ((ch ^ (r & 7)) << 4));
        uint8_t* dst = whole ? p.out + static_cast<int64_t>(to) * (2 * D)
                             : reinterpret_cast<uint8_t*>(p.part_o + static_cast<int64_t>(to) * D + (c + 1) * 32 - D / 2);
        *reinterpret_cast<uint4*>(dst + ch * 16) = v;
      }
    }
    __syncwarp();
  }
}

// Whether row i of the segment's tile sees a token in it.  For rows of NaN alone,
// whose queries may be anything: padding rows too.
__device__ __forceinline__ bool sees_any(const AttendParams& p, const Segment& g, int i) {
  const int end = min(g.x.n_keys, (g.u0 + g.n) * kKeys), limit = row_limit(p, g.x, g.x.first + i);
  const Translate tr(p, g.x, g.h, end);
#pragma unroll 1
  for (int e = g.u0 * kKeys; e < end; ++e)
    if (tr.place(tr.page(tr.index(e))).pos < limit) return true;
  return false;
}

template <int D, int NM, bool U16>
__device__ __forceinline__ void softmax(const AttendParams& p, const Segment& seg, uint8_t* smem, uint32_t tiles,
                                        uint32_t& count, uint32_t segs, bool f16) {
  using L = Lay<D, NM, U16>;
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  const int w = threadIdx.x >> 7, t = threadIdx.x & 127, lane = threadIdx.x & 31, first = t & ~31;
  static_assert(sizeof(Segment) <= 128, "");
  load_q<D, NM, U16>(p, seg, smem, f16);
  // (the key loop has no registers for it)
  const Segment& g = *reinterpret_cast<Segment*>(smem + L::kSeg + (segs & 1) * 128);
  if (threadIdx.x == 0) *reinterpret_cast<Segment*>(smem + L::kSeg + (segs & 1) * 128) = seg;
  uint32_t* row_nan = reinterpret_cast<uint32_t*>(smem + L::kRowNan) + threadIdx.x * 4;
#pragma unroll
  for (int e = 0; e < 4; ++e) row_nan[e] = 0;
  fence_async_smem();
  named_bar(kSoftBar, kSoftThreads);
  if (lane == 0) mbar_arrive(&bars->qfull);

  const int r0 = NM == 2 ? w * 128 : 0;        // the stream's first row of the tile
  const int i = min(r0 + t, g.x.rows - 1);     // (a row beyond the last repeats it; nothing of it is stored)
  const bool busy = r0 + first < g.x.rows;     // of the warp's rows, one at least is one
  Row row;
  row.m = -INFINITY, row.l = 0.f;
  row.factor = reinterpret_cast<const float*>(smem + L::kFactor)[i];
  // Tiles of the segment that all of the warp's rows see whole.
  const int whole_tiles =
      p.sel_width ? g.n : (row_limit(p, g.x, g.x.first + min(r0 + first, g.x.rows - 1)) - g.u0 * kKeys) / kKeys;
  // Tiles that all rows of the tile see whole: from here on fill() takes NaN codes
  // out of the values, for the rows that do see them too.
  const int clean_tiles = p.sel_width ? g.n : max(row_limit(p, g.x, g.x.first) - g.u0 * kKeys, 0) / kKeys;
  const uint32_t lanes = static_cast<uint32_t>(first) << 16, tm = bars->tmem + lanes;
  const uint32_t tm_s = tm + w * 128, tm_o = tm + 256 + w * 128;
  constexpr int kEvery = NM == 2 ? 1 : 2;
  const int n = g.n;
  for (int j = NM == 2 ? 0 : w; j < n; j += kEvery) {
    wait(bars, &bars->sfull[w], count & 1);
    ++count;
    tc_fence_after();
    if (busy) {
      const float* sc = reinterpret_cast<const float*>(smem + L::kScale) + (tiles + j) % L::kRing * L::kScales;
      int see = kKeys;
      if (j < whole_tiles) {
        softmax_tile<D, U16, false>(tm_s, tm_o, sc, row, kKeys, j < kEvery);
      } else {
        see = min(row_limit(p, g.x, g.x.first + min(r0 + t, g.x.rows - 1)) - (g.u0 + j) * kKeys, kKeys);
        softmax_tile<D, U16, true>(tm_s, tm_o, sc, row, see, j < kEvery);
      }
      if (j >= clean_tiles) {
        const uint32_t slot = (tiles + j) & 1;
        wait(bars, &bars->vfull[slot], (tiles + j) >> 1 & 1);
        const uint32_t* any = reinterpret_cast<const uint32_t*>(smem + L::kNanAny) + slot * 4;
        uint32_t nans = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) nans |= any[e];
        if (nans) {
          const uint32_t* bits = reinterpret_cast<const uint32_t*>(smem + L::kNan) + slot * (128 * 4);
          for (int k = 0; k < see; ++k)
#pragma unroll
            for (int e = 0; e < D / 32; ++e) row_nan[e] |= bits[k * 4 + e];
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bars->pfull[w]);
      mbar_arrive(&bars->tempty[(tiles + j) % L::kRing]);
    }
  }

  wait(bars, &bars->ofull, segs & 1);
  tc_fence_after();
  if (*reinterpret_cast<volatile int*>(&bars->abort)) row.l = NAN;
  if (isnan(row.l)) {
    if (row.m == -INFINITY && !sees_any(p, g, i))
      row.l = 0.f;  // (its query times the zeros of tokens that are none)
    else
      row.m = 0.f;  // a row of NaN scores counts in a join
  }
  __syncwarp();  // (the rows' accesses to TMEM are the warp's together)
  const uint32_t stage = smem_u32(smem) + L::kQ + (threadIdx.x >> 5) * (64 * D);  // (all products are done)
  if (NM == 2) {
    if (busy)
      write_rows<D>(p, g, stage, 256, r0 + first, row, row_nan, f16, [&](int c, float (&o)[32]) {
        uint32_t r[32];
        tmem_ld_x32(tm_o + c * 32, r);
        tmem_wait_ld(r);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(r[e]);
      });
    named_bar(kSoftBar, kSoftThreads);  // (a stage may be where another warp's next queries go)
    return;
  }
  // NM = 1: the second stream hands its rows over, 32 columns at a time.
  float2* ml = reinterpret_cast<float2*>(smem + L::kMl);
  const uint32_t ex = smem_u32(smem) + L::kEx + t * 128;
  if (w == 1) ml[t] = make_float2(row.m, row.l);
  named_bar(kSoftBar, kSoftThreads);
  if (w == 1) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t r[32];
      tmem_ld_x32(tm_o + c * 32, r);
      tmem_wait_ld(r);
#pragma unroll
      for (int e = 0; e < 8; ++e) sts128(ex + ((e ^ (t & 7)) << 4), r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
      named_bar(kSoftBar, kSoftThreads);
      named_bar(kSoftBar, kSoftThreads);
    }
  } else {
    const float2 other = ml[t];
    const float m = fmaxf(row.m, other.x);
    // (outputs of a stream that saw nothing may be anything; those of a vanishing
    // factor count, for their NaN)
    const bool on0 = row.m != -INFINITY, on1 = other.x != -INFINITY;
    const float h0 = root_factor(row.m, m), h1 = root_factor(other.x, m), f0 = h0 * h0, f1 = h1 * h1;
    // (NaN where either is, whatever the factors)
    row.l = row.l * h0 * h0 + other.y * h1 * h1;
    row.m = m;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) row_nan[e] |= row_nan[128 * 4 + e];
    write_rows<D>(p, g, stage, 128, first, row, row_nan, f16, [&](int c, float (&o)[32]) {
      uint32_t r[32];
      tmem_ld_x32(tm_o + c * 32, r);
      tmem_wait_ld(r);
      named_bar(kSoftBar, kSoftThreads);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint4 v = lds128(ex + ((e ^ (t & 7)) << 4));
        const uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          o[4 * e + k] = (on0 ? f0 * __uint_as_float(r[4 * e + k]) : 0.f) + (on1 ? f1 * __uint_as_float(b[k]) : 0.f);
      }
      named_bar(kSoftBar, kSoftThreads);
    });
  }
  named_bar(kSoftBar, kSoftThreads);
}

// ----------------------------------------------------------------- kernel --
template <int D, int NM, bool U16>
__global__ void __launch_bounds__(kThreads, 1) attend_tile_kernel(const __grid_constant__ AttendParams p, int f16) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  using L = Lay<D, NM, U16>;
  constexpr int R = NM * 128;
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
  int* prefix = reinterpret_cast<int*>(smem + L::kPrefix);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // The CTA's share of the units, or its one (tile, head): where it starts, and
  // its units.
  int tile, h, u0;
  Share sh = {};
  if (p.n_ctas) {
    sh = share_of(p, tile_prefix<kKeys, kThreads>(p, R, prefix, prefix + kMaxSplitTiles2 + 1));
    if (sh.start == sh.end) {
      if (threadIdx.x == 0) note_job(p, R, prefix, sh);
      return;
    }
    const Piece c = piece_at(p, prefix, sh, sh.start, sh.end);
    tile = c.tile, h = c.h, u0 = c.u0;
  } else {
    tile = p.n_tiles - 1 - blockIdx.x / p.c.heads;  // those of a sequence that see most, first
    h = blockIdx.x % p.c.heads, u0 = 0;
    const Tile x = tile_at(p, tile, R);
    if (x.rows <= 0) return;
    sh.end = tile_units<kKeys>(x), sh.heads = p.c.heads;
    if (threadIdx.x == 0) prefix[tile & 1] = 0, prefix[(tile & 1) + 1] = static_cast<int>(sh.end);
    prefix += (tile & 1) - tile;  // prefix[tile], prefix[tile + 1]
  }
  if (warp == 16) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(&bars->kfull[i], kFillWarps / 2);
        mbar_init(&bars->vfull[i], kFillWarps / 2);
        mbar_init(&bars->kempty[i], 1);
        mbar_init(&bars->vempty[i], 1);
        mbar_init(&bars->sfull[i], 1);
        mbar_init(&bars->pfull[i], 4);
      }
      for (int i = 0; i < L::kRing; ++i) {
        mbar_init(&bars->tfull[i], 1);
        mbar_init(&bars->tempty[i], kFillWarps + (NM == 2 ? 8 : 4));  // and the softmax warps that use the tile
      }
      mbar_init(&bars->qfull, kSoftThreads / 32);
      mbar_init(&bars->ofull, 1);
      mbar_init(&bars->done, 1);
      mbar_init(&bars->left, kSoftThreads / 32);
      bars->abort = 0, bars->tries = p.test_wait ? kTestTries : kWaitTries;
      fence_mbar_init();
    }
    __syncwarp();
    tmem_alloc(&bars->tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  // Each role goes through the segments of the share by itself, and ends by
  // itself: registers are divided among them, so no code but this follows that
  // several of them run, and the two with few call no function (a division of
  // 64 bits is one).
  const int tile_first = tile, h_first = h, u_first = u0;
  auto each = [&](bool with_tile, auto&& role) {
    uint32_t tiles = 0, segs = 0;
    int64_t left = sh.end - sh.start;
    int t = tile_first, hh = h_first, at = u_first;
    while (left > 0) {
      const int units = prefix[t + 1] - prefix[t];
      if (at >= units) {  // the next head, or tile
        at = 0;
        if (units == 0 || ++hh == sh.h + sh.heads) ++t, hh = sh.h;
        continue;
      }
      Segment g;
      if (with_tile) g.x = tile_at(p, t, R);
      g.h = hh, g.u0 = at;
      g.n = static_cast<int>(min(static_cast<int64_t>(units - at), left));
      g.whole = g.n == units;
      g.part = 2 * static_cast<int64_t>(blockIdx.x) + (segs ? 1 : 0);
      role(g, tiles, segs);
      tiles += g.n, at += g.n, left -= g.n;
      ++segs;
    }
  };
  if (warp < 8) {
    regs_to<Regs<NM>::kSoft>();
    uint32_t count = 0;
    each(true, [&](const Segment& g, uint32_t tiles, uint32_t segs) {
      softmax<D, NM, U16>(p, g, smem, tiles, count, segs, f16);
    });
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->left);
    return;
  }
  if (warp < 16) {
    regs_to<Regs<NM>::kFill>();
    each(true, [&](const Segment& g, uint32_t tiles, uint32_t) { fill<D, NM, U16>(p, g, smem, tiles); });
    return;
  }
  regs_to<Regs<NM>::kIssue>();
  if (warp != 16) {
    each(true, [&](const Segment& g, uint32_t tiles, uint32_t) { look_up<D, NM, U16>(p, g, smem, tiles); });
    if (warp == 17 && lane == 0 && p.n_ctas) note_job(p, R, prefix, sh);
    return;
  }
  const uint32_t one = elect_lane();
  uint32_t phases = 0;
  each(false, [&](const Segment& g, uint32_t tiles, uint32_t segs) {
    products<D, NM, U16>(g.n, smem, tiles, phases, segs, one);
  });
  // All products have completed and all softmax warps have left before TMEM is
  // freed: these waits end by a time limit alone, and then it stays allocated.
  tc_commit_one(one, &bars->done);
  const bool gone = mbar_wait(&bars->done, 0u, nullptr, kWaitLimitNs) && mbar_wait(&bars->left, 0u, nullptr, kWaitLimitNs);
  const bool all_gone = __all_sync(kFullMask, gone);
  if (p.status && one && (bars->abort || !all_gone)) atomicOr(p.status, kStatusWaitTimeout);
  tc_fence_after();
  if (all_gone) tmem_dealloc(bars->tmem, kTmemCols);
}

template <int D, int NM, bool U16>
cudaError_t go_tile(const AttendParams& p, bool f16, int grid, cudaStream_t stream) {
  // (at least half of an SM's: one CTA an SM, since each takes all of its TMEM)
  constexpr int kBytes = Lay<D, NM, U16>::kBytes > 118784 ? Lay<D, NM, U16>::kBytes : 118784;
  static_assert(kBytes <= 232448, "");
  // The shares of registers presume those of the launch: with fewer, the waits for
  // more would not end.
  static const bool regs_ok = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, attend_tile_kernel<D, NM, U16>) == cudaSuccess && a.numRegs == kLaunchRegs;
  }();
  if (!regs_ok) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      cudaFuncSetAttribute(attend_tile_kernel<D, NM, U16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  if (e != cudaSuccess) return e;
  attend_tile_kernel<D, NM, U16><<<grid, kThreads, kBytes, stream>>>(p, f16 ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_tile(const AttendParams& p, int D, int rows, bool u16, bool f16, int grid,
                               cudaStream_t stream) {
#define HWR_GO(DD, NN) return u16 ? go_tile<DD, NN, true>(p, f16, grid, stream) : go_tile<DD, NN, false>(p, f16, grid, stream)
  if (D == 128) {
    if (rows == 128) HWR_GO(128, 1);
    HWR_GO(128, 2);
  }
  if (rows == 128) HWR_GO(64, 1);
  HWR_GO(64, 2);
#undef HWR_GO
}

}  // namespace hwr
