// kvappend.cuh — rotary positions and the append to the paged cache, one launch.
//
// New position n of sequence b is entry t = kv_len[b] - q_len[b] + (its place)
// of the sequence.  Pair f of a query or key head turns by the angle
// position * inv_freq[f]; keys and values go to slot t % page_size of page
// block_table[b, t / page_size], queries to q_out.
//
// Angles.  The kernel wants the angle modulo one turn, and positions are whole
// numbers: inv_freq / 2 pi is made a 64-bit binary fraction of a turn once per
// thread, and the product with the position in 64-bit integers drops the whole
// turns by itself.  The fraction is off by at most 2^-53 relative, so position
// 2^20 is off by under 2^-35 turns; the high 32 bits, as a signed fraction of
// half a turn, go to sincospi.  fp64 per angle (a product, a reduction) would
// cost 4 M x 6 operations for 32,768 positions of 256 dims, tens of us at
// GB300's fp64 rate; this is three integer products.
//
// Layout.  A CTA takes a few positions.  Its threads first put the cosines and
// sines of those positions into shared memory, once for all heads; then thread
// i owns the 16-byte vector i % (D/8) of every head it visits, so it reads its
// 8 pairs from shared memory once per position and streams the heads.  The
// other half of a (f, f + rot/2) pair is a second load of the same row, from
// L1.  Bound by the copies: q, k, v read once, written once.
#pragma once

#include "paged.cuh"

namespace specv {

constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTile = 8;   // positions a CTA takes, at most
constexpr int kAppendBatch = 4;     // heads a thread has in flight

struct AppendParams {
  const uint16_t *q, *k, *v;
  int64_t q_ps, q_hs, k_ps, k_hs, v_ps, v_hs;  // strides between positions and heads, elements
  uint16_t* q_out;
  PagedView cache;
  PagedBatch batch;
  const float* inv_freq;
  const int32_t* positions;
  const int32_t* axis;
  int64_t position_base;
  int n_axes, n_q_heads, D, half, tile;  // half = rot_dim / 2
};

template <typename T>
struct Pack16;
template <>
struct Pack16<__nv_bfloat16> {
  __device__ static __forceinline__ float up(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
  __device__ static __forceinline__ void unpack(uint32_t w, float& a, float& b) { bf16x2_unpack(w, a, b); }
  __device__ static __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Pack16<__half> {
  __device__ static __forceinline__ float up(uint16_t x) { return __half2float(__ushort_as_half(x)); }
  __device__ static __forceinline__ void unpack(uint32_t w, float& a, float& b) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    a = f.x;
    b = f.y;
  }
  __device__ static __forceinline__ uint32_t pack(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// cosine and sine of position * (turn64 / 2^64) turns
__device__ __forceinline__ float2 unit_of(int64_t position, uint64_t turn64) {
  const uint64_t turns = static_cast<uint64_t>(position) * turn64;
  const float x = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;  // half turns in [-1, 1)
  float2 cs;
  sincospif(x, &cs.y, &cs.x);
  return cs;
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ float2 ap_units[];  // [tile][half]
  __shared__ int64_t s_dst[kAppendMaxTile];   // element offset of the entry in the pools, -1: not written
  __shared__ int64_t s_entry[kAppendMaxTile];
  __shared__ int s_live[kAppendMaxTile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = static_cast<int>(blockIdx.x) * p.tile;
  const int tile = min(p.tile, p.batch.N - n0);
  grid_dep_launch();
  grid_dep_wait();

  // ---- the entries of the tile's positions ----
  for (int t = warp; t < tile; t += kAppendThreads / 32) {
    const int n = n0 + t;
    const int b = find_seq(p.batch.q_indptr, p.batch.B, n, lane);
    if (lane == 0) {
      int64_t dst = -1, entry = 0;
      bool live = false;
      if (b >= 0) {
        const SeqSpan s = seq_span(p.batch, b);
        live = n >= s.first && n < s.first + s.n;  // not so only where q_indptr is not ascending
        entry = s.kv - s.n + (n - s.first);
        int page = -1;
        if (live && entry >= 0)
          page = p.batch.block_table[static_cast<int64_t>(b) * p.batch.table_width + entry / p.batch.page_size];
        if (page >= 0 && page < p.cache.n_pages)
          dst = page * p.cache.page_stride + (entry % p.batch.page_size) * p.cache.slot_stride;
        else
          atomicOr(p.batch.status, kStatusBadCache);
      }
      s_live[t] = live;
      s_dst[t] = dst;
      s_entry[t] = entry;
    }
  }
  __syncthreads();

  // ---- cosines and sines, one thread per frequency and several positions ----
  if (p.half > 0) {
    const int groups = kAppendThreads / p.half;  // half <= 256
    const int f = tid % p.half, g = tid / p.half;
    if (g < groups) {
      const double turns = static_cast<double>(p.inv_freq[f]) * 0.15915494309189533577;  // 1 / (2 pi)
      const uint64_t turn64 = __double2ull_rn((turns - floor(turns)) * 0x1p63) << 1;
      int a = p.axis != nullptr ? p.axis[f] : 0;
      if (a < 0 || a >= p.n_axes) {
        atomicOr(p.batch.status, kStatusBadCache);
        a = 0;
      }
      for (int t = g; t < tile; t += groups) {
        const int64_t pos = p.positions != nullptr
                                ? static_cast<int64_t>(p.positions[static_cast<int64_t>(a) * p.batch.N + n0 + t])
                                : p.position_base + s_entry[t];
        ap_units[t * p.half + f] = unit_of(pos, turn64);
      }
    }
    __syncthreads();
  }

  // ---- the heads: thread i owns vector i % vpr of each row it visits ----
  const int vpr = p.D >> 3, rpi = kAppendThreads / vpr;
  const int j = tid % vpr, r0 = tid / vpr;
  if (r0 >= rpi) return;
  const int Hq = p.n_q_heads, Hk = p.cache.n_heads, rows = Hq + 2 * Hk;
  const int d0 = 8 * j, rot = 2 * p.half;
  const bool turned = d0 < rot;
  const bool whole = (p.half & 7) == 0;  // the other halves of this vector's pairs are one vector too
  for (int t = 0; t < tile; ++t) {
    if (!s_live[t]) continue;
    const int64_t n = n0 + t, dst0 = s_dst[t];
    // this vector's cosines, and sines with the sign of the other half's term;
    // dims that are not rotated take cos 1, sin 0
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = d0 + e;
      const int f = kInterleaved ? d >> 1 : (d < p.half ? d : d - p.half);
      const bool first = kInterleaved ? (d & 1) == 0 : d < p.half;
      float2 u = make_float2(1.f, 0.f);
      if (d < rot) u = ap_units[t * p.half + f];
      c[e] = u.x;
      s[e] = first ? -u.y : u.y;
    }
    for (int row0 = r0; row0 < rows; row0 += kAppendBatch * rpi) {
      uint4 own[kAppendBatch], other[kAppendBatch];
      const uint16_t* src[kAppendBatch];
#pragma unroll
      for (int i = 0; i < kAppendBatch; ++i) {
        const int row = row0 + i * rpi;
        own[i] = other[i] = make_uint4(0, 0, 0, 0);
        src[i] = nullptr;
        if (row >= rows) continue;
        src[i] = row < Hq        ? p.q + n * p.q_ps + row * p.q_hs
                 : row < Hq + Hk ? p.k + n * p.k_ps + (row - Hq) * p.k_hs
                                 : p.v + n * p.v_ps + (row - Hq - Hk) * p.v_hs;
        own[i] = __ldg(reinterpret_cast<const uint4*>(src[i] + d0));
        if (!kInterleaved && turned && whole && row < Hq + Hk)
          other[i] = __ldg(reinterpret_cast<const uint4*>(src[i] + (d0 < p.half ? d0 + p.half : d0 - p.half)));
      }
#pragma unroll
      for (int i = 0; i < kAppendBatch; ++i) {
        const int row = row0 + i * rpi;
        if (row >= rows) continue;
        uint4 w = own[i];
        if (turned && row < Hq + Hk) {
          float x[8], y[8];
          Pack16<T>::unpack(own[i].x, x[0], x[1]);
          Pack16<T>::unpack(own[i].y, x[2], x[3]);
          Pack16<T>::unpack(own[i].z, x[4], x[5]);
          Pack16<T>::unpack(own[i].w, x[6], x[7]);
          if (kInterleaved) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = x[e ^ 1];
          } else if (whole) {
            Pack16<T>::unpack(other[i].x, y[0], y[1]);
            Pack16<T>::unpack(other[i].y, y[2], y[3]);
            Pack16<T>::unpack(other[i].z, y[4], y[5]);
            Pack16<T>::unpack(other[i].w, y[6], y[7]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int d = d0 + e;
              y[e] = d < rot ? Pack16<T>::up(__ldg(src[i] + (d < p.half ? d + p.half : d - p.half))) : 0.f;
            }
          }
          // a dim past rot_dim keeps its bits: cos 1, sin 0, and its partner
          // (which may be infinite) left out
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = d0 + e < rot ? fmaf(y[e], s[e], x[e] * c[e]) : x[e];
          w.x = Pack16<T>::pack(x[0], x[1]);
          w.y = Pack16<T>::pack(x[2], x[3]);
          w.z = Pack16<T>::pack(x[4], x[5]);
          w.w = Pack16<T>::pack(x[6], x[7]);
        }
        if (row < Hq) {
          *reinterpret_cast<uint4*>(p.q_out + (n * Hq + row) * p.D + d0) = w;
        } else if (dst0 >= 0) {
          const bool is_k = row < Hq + Hk;
          uint16_t* pool = is_k ? p.cache.k : p.cache.v;
          *reinterpret_cast<uint4*>(pool + dst0 + (row - Hq - (is_k ? 0 : Hk)) * p.cache.head_stride + d0) = w;
        }
      }
    }
  }
}

}  // namespace specv
