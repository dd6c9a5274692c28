// paged8.cuh — the 8-bit paged cache: its view and its numbers.
//
// An entry's dim is an e4m3 code; the entries of a block (`block` neighbouring
// slots of a page), key head and side (keys, values) share a scale, a power of
// two kept as one byte (its exponent + 127).  A code stands for code * 2^e.  With
// powers of two nothing is lost by a scale but range: a 16-bit value divided by
// 2^e is exact, the code is its nearest value, and what it stands for is a number
// of the cache's 16-bit type again, so products of the 16-bit type take it as it
// is.  (e4m3 is a floating type: a scale that fits the largest value exactly would
// win no bit over one that fits its exponent.)
//
// The scale.  e = floor(log2 of the block's largest finite |x|) - 7, so codes
// reach 240 or, rounded up, 256 of the type's 448; at least kLow and at most kHigh:
//   fp16: 2^e * 2^-9, the smallest code, is fp16's smallest number at e = -15;
//         240 * 2^8 is its largest value of four bits that is finite
//   bf16: -100 keeps every product normal; 240 * 2^120 is the largest value
// Values past 240 * 2^kHigh are taken to it; NaN and infinities become the code
// of NaN and do not count in the block's largest value.
#pragma once

#include "paged.cuh"

namespace specv {

struct Paged8View {
  uint8_t* k;
  uint8_t* v;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int64_t page_stride, slot_stride, head_stride;  // of the codes, bytes
  int64_t s_page, s_block, s_head;                // of the scales, bytes
  int64_t n_pages;
  int page_size, n_heads;
  int block_shift;  // log2 of the entries of a block

  __device__ __forceinline__ int64_t scale_at(int64_t page, int slot, int head) const {
    return page * s_page + (slot >> block_shift) * s_block + head * s_head;
  }
};

template <typename T>
struct Scale8;
template <>
struct Scale8<__half> {
  static constexpr int kLow = -15, kHigh = 8;
};
template <>
struct Scale8<__nv_bfloat16> {
  static constexpr int kLow = -100, kHigh = 120;
};

// 2^e, e in [-126, 127]
__device__ __forceinline__ float two_to(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The exponent of a block whose largest finite |x| is `top`.
template <typename T>
__device__ __forceinline__ int block_exponent(float top) {
  const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 7;
  return min(max(e, Scale8<T>::kLow), Scale8<T>::kHigh);
}

// A stored scale's exponent; what no append wrote is taken into the range.
template <typename T>
__device__ __forceinline__ int stored_exponent(uint32_t byte) {
  return min(max(static_cast<int>(byte) - 127, Scale8<T>::kLow), Scale8<T>::kHigh);
}

// what a value counts for in its block's largest
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;
}

// Two codes of x * inv: nearest, ties to even; `most` keeps finite values below
// the code of NaN, infinities become NaN.
__device__ __forceinline__ uint32_t code2(float a, float b, float inv, float most) {
  a = fabsf(a) < INFINITY ? fminf(fmaxf(a, -most), most) * inv : NAN;
  b = fabsf(b) < INFINITY ? fminf(fmaxf(b, -most), most) * inv : NAN;
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));  // the first goes to the high byte
  return d;
}
__device__ __forceinline__ uint2 code8(const float* x, float inv, float most) {
  uint2 w;
  w.x = code2(x[0], x[1], inv, most) | code2(x[2], x[3], inv, most) << 16;
  w.y = code2(x[4], x[5], inv, most) | code2(x[6], x[7], inv, most) << 16;
  return w;
}

// the values of two codes (exact)
__device__ __forceinline__ uint32_t half2_of_codes(uint16_t c) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(c));
  return d;
}
__device__ __forceinline__ float2 values2(uint32_t c) {
  const uint32_t h = half2_of_codes(static_cast<uint16_t>(c));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ void values8(uint2 c, float scale, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = values2((i < 2 ? c.x : c.y) >> (i & 1 ? 16 : 0));
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}

// The sequence whose rows hold n, by one thread (row offsets as they are; -1: none).
__device__ __forceinline__ int find_seq_alone(const PagedBatch& p, int n) {
  const int32_t* const q_indptr = p.q_indptr;
  if (!in_batch(p, n)) return -1;
  int lo = 0, len = p.B;  // the last b of [lo, lo + len) with q_indptr[b] <= n
  while (len > 1) {
    const int half = len >> 1;
    const bool below = q_indptr[lo + half] <= n;
    lo += below ? half : 0;
    len = below ? len - half : half;
  }
  return lo;
}

}  // namespace specv
