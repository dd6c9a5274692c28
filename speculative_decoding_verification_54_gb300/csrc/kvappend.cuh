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
// sines of those positions into shared memory, once for all heads; then each
// thread owns two 16-byte vectors of every head it visits, the two that turn
// together where pairs are (f, f + rot/2), so that it reads its 8 pairs'
// cosines from shared memory and every vector once.  The tile's (position,
// head) pairs are one sequence, dealt out in turn: heads that do not fill the
// threads leave none idle (28 + 8 heads of 128, 5,528 positions: 24.0 us against
// 29.4 position by position).  Bound by the copies: q, k, v read once, written
// once (32,768 positions of 256 dims: 188 us, 5.7 TB/s, 0.84 of the measured
// copy bandwidth).
#pragma once

#include "paged.cuh"

namespace specv {

// 256 threads, three CTAs an SM, three heads a thread in flight.  On 32,768
// positions of 256 dims and on 5,528 of 128: two heads 188.2 and 24.6 us, three
// 188.2 and 24.0, four 190.9 and 24.3.
constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTile = 24;   // positions a CTA takes, at most
constexpr int kAppendBatch = 3;      // heads a thread has in flight

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

  // row `row` of position n: query heads, then key heads, then value heads
  __device__ __forceinline__ const uint16_t* row_src(int64_t n, int row) const {
    const int Hk = cache.n_heads, k0 = row - n_q_heads;
    return k0 < 0 ? q + n * q_ps + row * q_hs : k0 < Hk ? k + n * k_ps + k0 * k_hs : v + n * v_ps + (k0 - Hk) * v_hs;
  }
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

// Where angle f stands in a position's table.  A thread reads the 8 angles of
// a vector, its neighbour the next 8: [angle in its vector][vector] puts a
// warp's reads side by side, in all banks (188 us against 228 in order of f, where
// neighbours stand 64 bytes apart).
__device__ __forceinline__ int unit_index(int f, int half) {
  return (half & 7) == 0 ? (f & 7) * (half >> 3) + (f >> 3) : f;
}

// a 16-byte vector that is read once: past L1
__device__ __forceinline__ uint4 ld_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  Pack16<T>::unpack(v.x, x[0], x[1]);
  Pack16<T>::unpack(v.y, x[2], x[3]);
  Pack16<T>::unpack(v.z, x[4], x[5]);
  Pack16<T>::unpack(v.w, x[6], x[7]);
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Pack16<T>::pack(x[0], x[1]), Pack16<T>::pack(x[2], x[3]), Pack16<T>::pack(x[4], x[5]),
                    Pack16<T>::pack(x[6], x[7]));
}

// dims e of x and of y are pair e
template <typename T>
__device__ __forceinline__ void turn_pair(uint4& xv, uint4& yv, const float* c, const float* s) {
  float x[8], y[8], u[8], w[8];
  unpack8<T>(xv, x);
  unpack8<T>(yv, y);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    u[e] = fmaf(y[e], -s[e], x[e] * c[e]);
    w[e] = fmaf(x[e], s[e], y[e] * c[e]);
  }
  xv = pack8<T>(u);
  yv = pack8<T>(w);
}

// dims 2e and 2e + 1 of x are pair e; from dim `end` on x stays
template <typename T>
__device__ __forceinline__ void turn_neighbours(uint4& xv, const float* c, const float* s, int end) {
  float x[8];
  unpack8<T>(xv, x);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (2 * e >= end) continue;
    const float u = fmaf(x[2 * e + 1], -s[e], x[2 * e] * c[e]);
    x[2 * e + 1] = fmaf(x[2 * e], s[e], x[2 * e + 1] * c[e]);
    x[2 * e] = u;
  }
  xv = pack8<T>(x);
}

// dims d and d + half are a pair, `half` no multiple of 8: the others one by
// one.  A dim past rot_dim keeps its bits.
template <typename T>
__device__ __forceinline__ void turn_scattered(uint4& xv, const uint16_t* row, const float2* cs, int d0, int half) {
  float x[8];
  unpack8<T>(xv, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int d = d0 + e;
    if (d >= 2 * half) continue;
    const bool first = d < half;
    const float2 a = cs[first ? d : d - half];
    const float y = Pack16<T>::up(row[first ? d + half : d - half]);
    x[e] = fmaf(y, first ? -a.y : a.y, x[e] * a.x);
  }
  xv = pack8<T>(x);
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads, 3) kv_append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ float2 ap_units[];  // [tile][half]
  __shared__ int64_t s_dst[kAppendMaxTile];   // element offset of the entry in the pools, -1: not written
  __shared__ int64_t s_entry[kAppendMaxTile];
  __shared__ int s_live[kAppendMaxTile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = static_cast<int>(blockIdx.x) * p.tile;
  const int tile = min(p.tile, p.batch.N - n0);
  grid_dep_launch();
  grid_dep_wait();

  // Row offsets that do not begin at 0 or do not ascend: the search below takes
  // them as they are and may not come across them.  (The last warps first: they
  // are the ones without a position to look up.)
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kAppendThreads + kAppendThreads - 1 - tid; i < p.batch.B;
       i += static_cast<int64_t>(gridDim.x) * kAppendThreads) {
    const int b = static_cast<int>(i), at = p.batch.q_indptr[b];
    if (at > p.batch.q_indptr[b + 1] || (b == 0 && at != 0) || (b == p.batch.B - 1 && p.batch.q_indptr[b + 1] > p.batch.N))
      atomicOr(p.batch.status, kStatusBadCache);
  }

  // ---- the entries of the tile's positions ----
  for (int t = warp; t < tile; t += kAppendThreads / 32) {
    const int n = n0 + t;
    const int b = find_seq(p.batch, n, lane);
    if (lane == 0) {
      int64_t dst = -1, entry = 0;
      bool live = false;
      if (b >= 0) {
        const SeqSpan s = seq_span(p.batch, b);
        live = n >= s.first && n < s.first + s.n;  // not so only where q_indptr is not ascending
        // The entry by the lengths as they are, not as seq_span clamps them: a
        // length past the table must not move the new entries over older ones.
        // What has no place in the table is not written.
        entry = n + s.shift;
        int page = -1;
        if (live && entry >= 0 && entry < static_cast<int64_t>(p.batch.table_width) * p.batch.page_size &&
            in_bounds(b < p.batch.B && entry / p.batch.page_size < p.batch.table_width, p.batch.status))
          page = p.batch.block_table[static_cast<int64_t>(b) * p.batch.table_width + entry / p.batch.page_size];
        if (page >= 0 && page < p.cache.n_pages)
          dst = page * p.cache.page_stride + (entry % p.batch.page_size) * p.cache.slot_stride;
        else
          atomicOr(p.batch.status, kStatusBadCache);
      }
      if (in_bounds(t < kAppendMaxTile, p.batch.status)) {
        s_live[t] = live;
        s_dst[t] = dst;
        s_entry[t] = entry;
      }
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
        if (in_bounds(t < p.tile && unit_index(f, p.half) >= 0 && unit_index(f, p.half) < p.half, p.batch.status))
          ap_units[t * p.half + unit_index(f, p.half)] = unit_of(pos, turn64);
      }
    }
    __syncthreads();
  }

  // ---- the heads: thread i owns unit i % upr of each row it visits ----
  const int vpr = p.D >> 3, upr = (vpr + 1) >> 1, rpi = kAppendThreads / upr;
  const int u = tid % upr, r0 = tid / upr;
  if (r0 >= rpi) return;
  const int Hq = p.n_q_heads, Hk = p.cache.n_heads, rows = Hq + 2 * Hk;
  const int hv = p.half >> 3, rot = 2 * p.half;
  // the pairs of a vector are all in one other vector: the unit is the two
  const bool paired = !kInterleaved && (p.half & 7) == 0 && u < hv;
  const int v0 = paired ? u : !kInterleaved && (p.half & 7) == 0 ? 2 * hv + 2 * (u - hv) : 2 * u;
  const int v1 = paired ? u + hv : v0 + 1;
  const bool two = v1 < vpr;
  const int d0 = 8 * v0, d1 = 8 * v1;
  // the tile's (position, row) pairs in one sequence: no thread waits for a
  // position's last rows where their count is no multiple of rpi
  const int t_step = rpi / rows, row_step = rpi - t_step * rows;
  int t_at = r0 / rows, row_at = r0 - t_at * rows;
  while (t_at < tile) {
    uint4 a[kAppendBatch], b[kAppendBatch];
    int ts[kAppendBatch], rs[kAppendBatch];
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      const bool inside =
          t_at < tile && in_bounds(t_at >= 0 && t_at < kAppendMaxTile && row_at >= 0 && row_at < rows && d0 + 8 <= p.D &&
                                       (!two || d1 + 8 <= p.D),
                                   p.batch.status);
      ts[i] = inside && s_live[t_at] ? t_at : -1;
      rs[i] = row_at;
      if (ts[i] >= 0) {
        const uint16_t* src = p.row_src(n0 + t_at, row_at);
        a[i] = ld_once(src + d0);
        if (two) b[i] = ld_once(src + d1);
      }
      t_at += t_step;
      row_at += row_step;
      if (row_at >= rows) {
        row_at -= rows;
        ++t_at;
      }
    }
#pragma unroll
    for (int i = 0; i < kAppendBatch; ++i) {
      if (ts[i] < 0) continue;
      const int row = rs[i];
      const int64_t n = n0 + ts[i], dst0 = s_dst[ts[i]];
      const float2* cs = ap_units + ts[i] * p.half;
      uint4 x = a[i], y = b[i];
      if (row < Hq + Hk) {
        // a pair of vectors turns by its 8 angles; neighbours have 4 each
        float c[8], s[8];
        if (paired || (kInterleaved && d0 < rot)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int f = kInterleaved ? (d0 >> 1) + e : d0 + e;
            const float2 w = f < p.half ? cs[unit_index(f, p.half)] : make_float2(1.f, 0.f);
            c[e] = w.x;
            s[e] = w.y;
          }
        }
        if (paired) {
          turn_pair<T>(x, y, c, s);
        } else if (kInterleaved) {
          if (d0 < rot) turn_neighbours<T>(x, c, s, rot - d0);
          if (two && d1 < rot) turn_neighbours<T>(y, c + 4, s + 4, rot - d1);
        } else if (d0 < rot && (p.half & 7) != 0) {
          turn_scattered<T>(x, p.row_src(n, row), cs, d0, p.half);
          if (two) turn_scattered<T>(y, p.row_src(n, row), cs, d1, p.half);
        }
      }
      uint16_t* dst;
      if (row < Hq) {
        dst = p.q_out + (n * Hq + row) * p.D;
      } else {
        if (dst0 < 0 || !in_bounds(dst0 <= (p.cache.n_pages - 1) * p.cache.page_stride +
                                               (p.batch.page_size - 1) * p.cache.slot_stride,
                                   p.batch.status))
          continue;
        const bool is_k = row < Hq + Hk;
        dst = (is_k ? p.cache.k : p.cache.v) + dst0 + (row - Hq - (is_k ? 0 : Hk)) * p.cache.head_stride;
      }
      *reinterpret_cast<uint4*>(dst + d0) = x;
      if (two) *reinterpret_cast<uint4*>(dst + d1) = y;
    }
  }
}

}  // namespace specv
