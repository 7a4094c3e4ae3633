// cache.h -- what the kernels around the 8-bit key/value cache share: the
// cache and sequence descriptors as the kernels take them, the e4m3 and
// 16-bit conversions, and the launchers (not part of the public C ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx.cuh"

namespace hwr {

constexpr uint32_t kStatusToken = 8u;  // a token's page or position does not exist
constexpr float kMinBlockScale = 0x1p-100f;

struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t n_pages;
  int64_t page16, token16, head16;  // strides in units of 16 bytes
  int32_t page_size;
  int32_t block;
  int32_t block_shift;              // log2(block)
  int32_t page_blocks;              // page_size / block
  int32_t heads;
};

struct SeqView {
  int64_t S;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* pages;
  int64_t page_stride;
  int32_t table_pages;
  int32_t B;
};

struct RotView {
  const float* table;
  int64_t rows;
  int32_t rot;
  int32_t inter;
};

// Row r0 of sequence b and the rows after it: cu_q as given, held inside [0, S].
__device__ __forceinline__ int seq_row(const SeqView& s, int b) {
  const int v = __ldg(s.cu_q + b);
  return min(max(v, 0), static_cast<int>(s.S));
}

// Work slots are laid out by sequence without a scan over the sequences:
// sequence b owns the slots from cu_q[b]*mul/div + extra*b on.  For a rising
// cu_q that leaves it floor(n*mul/div) + extra slots or more, which is
// monotone in b, so the owner of a slot is found by binary search.
__device__ __forceinline__ int64_t slot_base(const SeqView& s, int b, int mul, int div, int extra) {
  return static_cast<int64_t>(seq_row(s, b)) * mul / div + static_cast<int64_t>(extra) * b;
}
__device__ __forceinline__ int slot_owner(const SeqView& s, int64_t slot, int mul, int div, int extra) {
  int lo = 0, hi = s.B - 1;  // the last b whose base is at most slot
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (slot_base(s, mid, mul, div, extra) <= slot)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Page of position pos of sequence b, or -1 when it has none.
__device__ __forceinline__ int64_t page_of(const SeqView& s, const CacheView& c, int b, int pos, int* offset) {
  const int pi = pos / c.page_size;
  *offset = pos - pi * c.page_size;
  if (pos < 0 || pi >= s.table_pages) return -1;
  const int64_t p = __ldg(s.pages + b * s.page_stride + pi);
  return p >= 0 && p < c.n_pages ? p : -1;
}

// Two e4m3 codes (low 16 bits) -> two halves; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
// Two floats -> two e4m3 codes, nearest even; `lo` in the low byte.  NaN -> 0x7F.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool F16>
__device__ __forceinline__ float2 unpack_act(uint32_t v) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack_act(float lo, float hi) {
  if (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

cudaError_t launch_rotate_quantise(const void* x, int64_t S, int H, int D, bool f16, int64_t x_stride,
                                   const int32_t* positions, const RotView& rot, uint8_t* codes, float* scale,
                                   uint32_t* status, int sms, cudaStream_t stream);

struct AppendParams {
  CacheView c;
  SeqView s;
  RotView r;
  const uint8_t* k;
  const uint8_t* v;
  int64_t kv_stride;  // bytes
  const uint8_t* q;
  uint8_t* q_out;
  int64_t q_stride;   // bytes
  int32_t Hq;
  uint32_t* status;
  int32_t kv_slots, kv_split;  // grid layout, set by the launcher
  int32_t q_slots, q_heads;
  int32_t q_apart;             // q is a kernel of its own
};
cudaError_t launch_cache_append(AppendParams p, int D, bool f16, int sms, cudaStream_t stream);

}  // namespace hwr
