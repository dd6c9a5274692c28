// append8.cuh — the append with norms of query and key heads and rotary
// positions in one launch, to a cache of 16 bits or of 8, and the read-back of the
// 8-bit cache.
//
// Norm.  y = x * rsqrt(mean(x^2) + eps) * w over a head's dims, in fp32, before the
// rotation; the result is rounded once, to the cache's type or to its code.
//
// Layout.  As in kvappend.cuh a CTA puts its positions' cosines and sines into
// shared memory; a row (position and head) is held by `lanes` neighbouring lanes
// of a warp, two 16-byte vectors a lane (those that turn together where pairs are
// halves apart), so the norm's sum is a few shuffles and every value is read once.
//
// Blocks of the 8-bit cache.  A block's scale needs all its new rows, so one CTA
// owns each block: the CTA whose tile of positions holds the block's first new
// position (its lead) takes all of it, queries included.  A unit is a block of one
// key head and side; it is held in registers by as many warps as keep four rows'
// steps a lane (block * lanes / 128), so values are rotated and normalised once,
// reduced to their maximum and written.  Where older entries stand in the block
// its scale only rises, and when it does their codes are rewritten (exact but
// for e4m3's subnormals).
//
// What bounds it: q, k, v read once, q (16 bits) and codes written once.  To 16 bits
// 32,768 positions of 256 dims take 186 us, 5.8 TB/s (0.86 of the measured copy
// bandwidth).  To 8 bits some 16,400 positions of 32 + 8 + 8 heads of 128 take 107 us
// for 62: a unit's 64 values a lane leave two CTAs an SM (computed twice instead, for
// three CTAs, they spill: 130 us).  CTAs of whole blocks: 107 us, of 24 positions 118.
#pragma once

#include "kvappend.cuh"
#include "paged8.cuh"

namespace specv {

constexpr int kA8Threads = 256, kA8Warps = kA8Threads / 32;
constexpr int kA8MaxOwn = kAppendMaxTile + 63;  // positions of a CTA: its tile's and the rest of its last block
constexpr int kA8Steps = 4;                     // rows' steps of a unit that a lane holds

struct Append8Params {
  AppendParams a;  // (its cache: the 16-bit pools; with 8 bits only n_heads counts)
  Paged8View c8;
  const float *q_weight, *k_weight;  // [D] or null: no norm
  float eps, inv_dims;  // 1 / D
  int unit_floats; // of a position's cosines and sines
  int lanes;       // lanes of a row: a power of two
  int unit_warps;  // warps of a unit
};

// What a lane holds of a row.
struct RowLane {
  int d0, d1;   // the first dims of its two vectors
  bool live, two, paired;
};

// How a row's pairs stand: a whole number of vectors apart (both of a lane's vectors
// turn together), side by side, or anywhere (the partner dims are read one by one).
// A kernel each: code that a call does not use cost the others 10 to 20 percent.
enum Pairs { kApart8, kNeighbours, kAnywhere };

// two fp32 products at once
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void split2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("{\n\t.reg .f32 x, y;\n\tabs.f32 x, %2;\n\tabs.f32 y, %3;\n\tmax.f32 %0, %1, x, y;\n\t}" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// code8 of values whose finite ones are below the largest code: x * inv, and an
// infinity times 0 makes it NaN.
__device__ __forceinline__ uint2 code8_near(const float* x, float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t z = mul2(pair2(x[2 * i], x[2 * i + 1]), pair2(inv, inv));
    float a, b;
    split2(fma2(z, pair2(0.f, 0.f), z), a, b);
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(b), "f"(a));  // the first goes to the high byte
    w[i] = d;
  }
  return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}

// Where cosine (or sine) of angle f stands in a position's table: kAnywhere in
// order of f, else as the lanes read them, four of a lane's eight angles at a time,
// neighbouring lanes side by side.
template <Pairs kPairs>
__device__ __forceinline__ int table_index(int f, int half, bool sine) {
  if (kPairs == kAnywhere) return 2 * f + (sine ? 1 : 0);
  const int vectors = (half + 7) >> 3, e = f & 7;
  return (((sine ? 2 : 0) + (e >> 2)) * vectors + (f >> 3)) * 4 + (e & 3);
}

// The norms' factors of kRows rows (without weights): their sums of squares go over
// the row's lanes side by side.  All lanes of a warp call it.
template <typename T, int kRows>
__device__ __forceinline__ void row_factors(const Append8Params& p, const uint4 (&a)[kRows], const uint4 (&b)[kRows],
                                            float (&r)[kRows]) {
#pragma unroll
  for (int i = 0; i < kRows; ++i) r[i] = 1.f;
  if (p.q_weight == nullptr && p.k_weight == nullptr) return;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float x[8], y[8];
    unpack8<T>(a[i], x);
    unpack8<T>(b[i], y);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s0 = fmaf(x[e], x[e], s0);
      s1 = fmaf(y[e], y[e], s1);
    }
    r[i] = s0 + s1;
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    if (s >= p.lanes) continue;
#pragma unroll
    for (int i = 0; i < kRows; ++i) r[i] += __shfl_xor_sync(0xffffffffu, r[i], s);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) r[i] = rsqrtf(fmaf(r[i], p.inv_dims, p.eps));
}

// A row's two vectors in fp32, normalised and rotated.  `row`: the row in memory
// (pairs whose other dim is in no vector of the lane are read there).
// `weights`: float4s of w for this side in shared memory (weight_index), or null.
template <typename T, Pairs kPairs>
__device__ __forceinline__ void row_values(const Append8Params& p, const RowLane& u, uint4 av, uint4 bv, bool turn,
                                           const float4* weights, const float* all_weights, const uint16_t* row,
                                           float r, const float* cs, float (&x)[8], float (&y)[8]) {
  const int half = p.a.half, rot = 2 * half;
  unpack8<T>(av, x);
  unpack8<T>(bv, y);
  if (weights != nullptr) {
    const uint64_t r2 = pair2(r, r);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float4 w = weights[v * p.lanes];
      float* const z = v < 2 ? x + 4 * v : y + 4 * (v - 2);
      split2(mul2(mul2(pair2(z[0], z[1]), r2), pair2(w.x, w.y)), z[0], z[1]);
      split2(mul2(mul2(pair2(z[2], z[3]), r2), pair2(w.z, w.w)), z[2], z[3]);
    }
  }
  if (!turn || !u.live || u.d0 >= rot) return;
  if (kPairs != kAnywhere) {
    if (kPairs == kApart8 && !u.paired) return;
    // the lane's eight angles
    const int vectors = (half + 7) >> 3;
    const float4* const at = reinterpret_cast<const float4*>(cs) + (kPairs == kApart8 ? u.d0 >> 3 : u.d0 >> 4);
    float c[8], s[8];
    *reinterpret_cast<float4*>(c) = at[0];
    *reinterpret_cast<float4*>(c + 4) = at[vectors];
    *reinterpret_cast<float4*>(s) = at[2 * vectors];
    *reinterpret_cast<float4*>(s + 4) = at[3 * vectors];
    if (kPairs == kApart8) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const uint64_t x2 = pair2(x[e], x[e + 1]), y2 = pair2(y[e], y[e + 1]), c2 = pair2(c[e], c[e + 1]);
        split2(fma2(y2, pair2(-s[e], -s[e + 1]), mul2(x2, c2)), x[e], x[e + 1]);
        split2(fma2(x2, pair2(s[e], s[e + 1]), mul2(y2, c2)), y[e], y[e + 1]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (u.d0 + 2 * e < rot) {
          const float t = fmaf(x[2 * e + 1], -s[e], x[2 * e] * c[e]);
          x[2 * e + 1] = fmaf(x[2 * e], s[e], x[2 * e + 1] * c[e]);
          x[2 * e] = t;
        }
        if (u.two && u.d1 + 2 * e < rot) {  // d1 = d0 + 8
          const float t = fmaf(y[2 * e + 1], -s[e + 4], y[2 * e] * c[e + 4]);
          y[2 * e + 1] = fmaf(y[2 * e], s[e + 4], y[2 * e + 1] * c[e + 4]);
          y[2 * e] = t;
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int d = e < 8 ? u.d0 + e : u.d1 + e - 8;
      if (d >= rot || (e >= 8 && !u.two)) continue;
      const bool first = d < half;
      const int o = first ? d + half : d - half;
      const float2 w = reinterpret_cast<const float2*>(cs)[first ? d : o];
      float z = Pack16<T>::up(row[o]);
      if (weights != nullptr) z = z * r * all_weights[o];
      float& to = e < 8 ? x[e & 7] : y[e & 7];
      to = fmaf(z, first ? -w.y : w.y, to * w.x);
    }
  }
}

// Three CTAs an SM with a 16-bit cache, two with an 8-bit one, whose units take
// 64 registers.
template <typename T, Pairs kPairs, bool k8>
__global__ void __launch_bounds__(kA8Threads, k8 ? 2 : 3) append_norm_kernel(const __grid_constant__ Append8Params p) {
  extern __shared__ __align__(16) float ap8_units[];  // [positions of the CTA][unit_floats]
  __shared__ int64_t s_dst[kA8MaxOwn];  // element offset of the entry in the pools, -1: not written
  __shared__ int64_t s_entry[kA8MaxOwn];
  __shared__ int s_page[kA8MaxOwn];
  __shared__ int8_t s_live[kA8MaxOwn], s_is_lead[kA8MaxOwn];
  __shared__ int16_t s_lead[kA8MaxOwn + 1];  // places of the leads, then the end
  __shared__ int s_begin, s_end, s_leads;
  __shared__ float s_top[kA8Warps];
  __shared__ float4 s_weights[2][4 * 32];  // [query, key][a lane's fourths of 16 dims][lane of a row]
  const PagedBatch& batch = p.a.batch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = static_cast<int>(blockIdx.x) * p.a.tile;
  const int tile = min(p.a.tile, batch.N - n0);
  const int block = 1 << p.c8.block_shift;
  // positions looked at: the tile's, and with 8 bits those that its last block may reach to
  const int look = k8 ? min(p.a.tile + block - 1, batch.N - n0) : tile;
  const int64_t page_stride = k8 ? p.c8.page_stride : p.a.cache.page_stride;
  const int64_t slot_stride = k8 ? p.c8.slot_stride : p.a.cache.slot_stride;
  const int64_t n_pages = k8 ? p.c8.n_pages : p.a.cache.n_pages;
  // ---- this lane's part of every row it visits ----
  const int vpr = p.a.D >> 3, upr = (vpr + 1) >> 1, rows_at_once = 32 / p.lanes;
  const int u = lane & (p.lanes - 1), row_of_warp = lane / p.lanes;
  const int hv = p.a.half >> 3;
  // the unit u of a row: the first vectors of its two
  auto first_vector = [&](int u) {
    return kPairs != kApart8 ? 2 * u : u < hv ? u : 2 * hv + 2 * (u - hv);
  };
  auto second_vector = [&](int u) { return kPairs == kApart8 && u < hv ? u + hv : first_vector(u) + 1; };
  RowLane my;
  my.live = u < upr;
  my.paired = kPairs == kApart8 && u < hv;
  my.two = second_vector(u) < vpr;
  my.d0 = 8 * first_vector(u);
  my.d1 = 8 * second_vector(u);
  grid_dep_launch();
  grid_dep_wait();

  // row offsets that do not begin at 0 or do not ascend are reported
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kA8Threads + kA8Threads - 1 - tid; i < batch.B;
       i += static_cast<int64_t>(gridDim.x) * kA8Threads) {
    const int b = static_cast<int>(i), at = batch.q_indptr[b];
    if (at > batch.q_indptr[b + 1] || (b == 0 && at != 0) || (b == batch.B - 1 && batch.q_indptr[b + 1] > batch.N))
      atomicOr(batch.status, kStatusBadCache);
  }

  // the norms' weights as the lanes read them: neighbours side by side
  if (p.q_weight != nullptr || p.k_weight != nullptr) {
    const int i = tid & 127, side = tid >> 7, v = i / p.lanes, l = i - v * p.lanes;  // fourth v of lane l's dims
    const float* const from = side == 0 ? p.q_weight : p.k_weight;
    const int d = 8 * (v < 2 ? first_vector(l) : second_vector(l)) + 4 * (v & 1);
    if (v < 4 && from != nullptr)
      s_weights[side][i] = d + 4 <= p.a.D ? make_float4(from[d], from[d + 1], from[d + 2], from[d + 3]) : make_float4(0, 0, 0, 0);
  }
  const float4* const q_weights = p.q_weight != nullptr ? s_weights[0] + u : nullptr;
  const float4* const k_weights = p.k_weight != nullptr ? s_weights[1] + u : nullptr;

  // ---- the entries of the positions, a thread each ----
  for (int t = tid; t < look; t += kA8Threads) {
    const int n = n0 + t;
    const int b = find_seq_alone(batch, n);
    int64_t dst = -1, entry = 0;
    bool live = false, lead = true;
    int page = -1;
    if (b >= 0) {
      const SeqSpan s = seq_span(batch, b);
      live = n >= s.first && n < s.first + s.n;  // not so only where q_indptr is not ascending
      entry = n + s.shift;  // by the lengths as given, not clamped: no length moves an entry over an older one
      lead = !live || n == s.first || (entry & (block - 1)) == 0;
      if (live && entry >= 0 && entry < static_cast<int64_t>(batch.table_width) * batch.page_size &&
          in_bounds(b < batch.B && entry / batch.page_size < batch.table_width, batch.status))
        page = batch.block_table[static_cast<int64_t>(b) * batch.table_width + entry / batch.page_size];
      if (page >= 0 && page < n_pages)
        dst = page * page_stride + (entry % batch.page_size) * slot_stride;
      else
        atomicOr(batch.status, kStatusBadCache);
    }
    if (in_bounds(t < kA8MaxOwn, batch.status)) {
      s_live[t] = live;
      s_dst[t] = dst;
      s_entry[t] = entry;
      s_page[t] = page;
      s_is_lead[t] = lead;
    }
  }
  __syncthreads();
  int begin = 0, end = tile;
  if (k8) {
    // the positions from the tile's first lead to the next tile's
    if (warp == 0) {
      int from = look, to = look, leads = 0;
      for (int t0 = 0; t0 < look; t0 += 32) {
        const int t = t0 + lane;
        const bool lead = t < look && s_is_lead[t];
        const unsigned mine = __ballot_sync(0xffffffffu, lead && t < tile), next = __ballot_sync(0xffffffffu, lead && t >= tile);
        if (from == look && mine != 0u) from = t0 + __ffs(mine) - 1;
        if (to == look && next != 0u) to = t0 + __ffs(next) - 1;
        if (lead && t < tile && in_bounds(leads + __popc(mine & ((1u << lane) - 1)) < kA8MaxOwn, batch.status))
          s_lead[leads + __popc(mine & ((1u << lane) - 1))] = static_cast<int16_t>(t);
        leads += __popc(mine);
      }
      if (lane == 0) {
        if (from == look) to = look;  // no lead: nothing to do
        s_lead[leads] = static_cast<int16_t>(to);
        s_begin = from;
        s_end = to;
        s_leads = leads;
      }
    }
    __syncthreads();
    begin = s_begin;
    end = s_end;
    if (begin >= end) return;
  }

  // ---- cosines and sines, one thread per frequency and several positions ----
  if (p.a.half > 0) {
    const int groups = kA8Threads / p.a.half;  // half <= 256
    const int f = tid % p.a.half, g = tid / p.a.half;
    if (g < groups) {
      const double turns = static_cast<double>(p.a.inv_freq[f]) * 0.15915494309189533577;  // 1 / (2 pi)
      const uint64_t turn64 = __double2ull_rn((turns - floor(turns)) * 0x1p63) << 1;
      int a = p.a.axis != nullptr ? p.a.axis[f] : 0;
      if (a < 0 || a >= p.a.n_axes) {
        atomicOr(batch.status, kStatusBadCache);
        a = 0;
      }
      for (int t = begin + g; t < end; t += groups) {
        const int64_t pos = p.a.positions != nullptr
                                ? static_cast<int64_t>(p.a.positions[static_cast<int64_t>(a) * batch.N + n0 + t])
                                : p.a.position_base + s_entry[t];
        const int c = table_index<kPairs>(f, p.a.half, false), s = table_index<kPairs>(f, p.a.half, true);
        if (in_bounds(t < kA8MaxOwn && c >= 0 && c < p.unit_floats && s >= 0 && s < p.unit_floats, batch.status)) {
          const float2 w = unit_of(pos, turn64);
          ap8_units[(t - begin) * p.unit_floats + c] = w.x;
          ap8_units[(t - begin) * p.unit_floats + s] = w.y;
        }
      }
    }
    __syncthreads();
  }

  const int Hq = p.a.n_q_heads, Hk = p.a.cache.n_heads;

  // ---- queries (and with a 16-bit cache keys and values): (position, row) pairs in one sequence ----
  {
    const int rows = k8 ? Hq : Hq + 2 * Hk, at_once = kA8Warps * rows_at_once;
    const int r0 = warp * rows_at_once + row_of_warp;
    const int t_step = at_once / rows, row_step = at_once - t_step * rows;
    int t_at = begin + r0 / rows, row_at = r0 % rows;
    int t_first = begin + (warp * rows_at_once) / rows;  // of the warp's first row: uniform
    int row_first = (warp * rows_at_once) % rows;
    while (t_first < end) {
      uint4 a[kAppendBatch], b[kAppendBatch];
      int ts[kAppendBatch], rs[kAppendBatch];
#pragma unroll
      for (int i = 0; i < kAppendBatch; ++i) {
        const bool inside = my.live && t_at < end &&
                            in_bounds(t_at >= 0 && t_at < kA8MaxOwn && row_at >= 0 && row_at < rows && my.d0 + 8 <= p.a.D &&
                                          (!my.two || my.d1 + 8 <= p.a.D),
                                      batch.status);
        ts[i] = inside && s_live[t_at] ? t_at : -1;
        rs[i] = row_at;
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        if (ts[i] >= 0) {
          const uint16_t* src = p.a.row_src(n0 + t_at, row_at);
          a[i] = ld_once(src + my.d0);
          if (my.two) b[i] = ld_once(src + my.d1);
        }
        t_at += t_step;
        row_at += row_step;
        if (row_at >= rows) {
          row_at -= rows;
          ++t_at;
        }
        t_first += t_step;
        row_first += row_step;
        if (row_first >= rows) {
          row_first -= rows;
          ++t_first;
        }
      }
      float factors[kAppendBatch];
      row_factors<T>(p, a, b, factors);
#pragma unroll
      for (int i = 0; i < kAppendBatch; ++i) {
        const int t = max(ts[i], begin), row = rs[i];
        const int64_t n = n0 + t;
        const bool is_q = row < Hq, is_v = row >= Hq + Hk;
        float x[8], y[8];
        row_values<T, kPairs>(p, my, a[i], b[i], ts[i] >= 0 && !is_v, is_v ? nullptr : is_q ? q_weights : k_weights,
                              is_q ? p.q_weight : p.k_weight, p.a.row_src(n, row), factors[i],
                              ap8_units + (t - begin) * p.unit_floats, x, y);
        if (ts[i] < 0) continue;
        uint16_t* dst;
        if (is_q) {
          dst = p.a.q_out + (n * Hq + row) * p.a.D;
        } else {
          if (s_dst[t] < 0 || !in_bounds(s_dst[t] <= (n_pages - 1) * page_stride + (batch.page_size - 1) * slot_stride,
                                         batch.status))
            continue;
          dst = (is_v ? p.a.cache.v : p.a.cache.k) + s_dst[t] + (row - Hq - (is_v ? Hk : 0)) * p.a.cache.head_stride;
        }
        *reinterpret_cast<uint4*>(dst + my.d0) = pack8<T>(x);
        if (my.two) *reinterpret_cast<uint4*>(dst + my.d1) = pack8<T>(y);
      }
    }
  }
  if (!k8) return;

  // ---- keys and values of the 8-bit cache, a unit at a time ----
  const int units = s_leads * 2 * Hk, at_once = kA8Warps / p.unit_warps;
  const int unit_of_warp = warp / p.unit_warps, part = warp - unit_of_warp * p.unit_warps;
  const float most = 240.f * two_to(Scale8<T>::kHigh);
  for (int first = 0; first < units; first += at_once) {  // all warps make the same rounds
    const int unit = first + unit_of_warp;
    const bool here = unit < units && unit_of_warp < at_once;
    const int l = here ? unit / (2 * Hk) : 0, h = here ? unit - l * 2 * Hk : 0;
    const bool is_v = h >= Hk;
    const int head = is_v ? h - Hk : h;
    const int t0 = s_lead[l];
    const int64_t dst0 = s_dst[t0];
    const bool writes = here && s_live[t0] && dst0 >= 0;
    const int slot = static_cast<int>(s_entry[t0] % batch.page_size), behind = slot & (block - 1);
    // never more than the block holds, whatever row offsets that do not ascend make of it
    const int rows = min(s_lead[l + 1] - t0, block - behind);
    uint8_t* const pool = is_v ? p.c8.v : p.c8.k;
    uint8_t* const scale = (is_v ? p.c8.v_scales : p.c8.k_scales) + (writes ? p.c8.scale_at(s_page[t0], slot, head) : 0);
    int was = Scale8<T>::kLow;
    if (writes && behind > 0) was = stored_exponent<T>(*scale);
    uint4 a[kA8Steps], b[kA8Steps];
#pragma unroll
    for (int i = 0; i < kA8Steps; ++i) {
      const int r = (i * p.unit_warps + part) * rows_at_once + row_of_warp;
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (writes && my.live && r < rows && in_bounds(t0 + r < end, batch.status)) {
        const uint16_t* src = p.a.row_src(n0 + t0 + r, Hq + h);
        a[i] = ld_once(src + my.d0);
        b[i] = ld_once(src + my.d1);  // D is a multiple of 16: there are always two
      }
    }
    float x[kA8Steps][8], y[kA8Steps][8], factors[kA8Steps], top = 0.f;
    row_factors<T>(p, a, b, factors);
#pragma unroll
    for (int i = 0; i < kA8Steps; ++i) {
      const int r = (i * p.unit_warps + part) * rows_at_once + row_of_warp;
      const bool mine = writes && r < rows;
      const int t = t0 + (mine ? r : 0);
      row_values<T, kPairs>(p, my, a[i], b[i], mine && !is_v, is_v ? nullptr : k_weights, p.k_weight,
                            p.a.row_src(n0 + t, Hq + h), factors[i], ap8_units + (t - begin) * p.unit_floats, x[i], y[i]);
      if (mine && my.live) {  // (a NaN is no maximum)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max3_abs(top, x[i][e], y[i][e]);
      }
    }
    if (__any_sync(0xffffffffu, top == INFINITY)) {  // an infinity does not count
      top = 0.f;
#pragma unroll
      for (int i = 0; i < kA8Steps; ++i) {
        const int r = (i * p.unit_warps + part) * rows_at_once + row_of_warp;
        if (writes && r < rows && my.live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(finite_abs(x[i][e]), finite_abs(y[i][e])));
        }
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    if (p.unit_warps > 1) {
      if (lane == 0) s_top[warp] = top;
      __syncthreads();
      for (int w = 0; w < p.unit_warps; ++w)
        if (unit_of_warp < at_once) top = fmaxf(top, s_top[unit_of_warp * p.unit_warps + w]);
      __syncthreads();
    }
    if (!writes) continue;
    const int now = max(block_exponent<T>(top), was);
    if (lane == 0 && part == 0) *scale = static_cast<uint8_t>(now + 127);
    if (behind > 0 && now > was) {  // older codes to the new scale
      const int64_t block0 = dst0 - behind * p.c8.slot_stride + head * p.c8.head_stride;
      const float less = two_to(max(was - now, -126));
      for (int r = part * rows_at_once + row_of_warp; r < behind; r += p.unit_warps * rows_at_once) {
        if (!my.live) continue;
        uint8_t* const at = pool + block0 + r * p.c8.slot_stride;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          uint2* const c = reinterpret_cast<uint2*>(at + (v == 0 ? my.d0 : my.d1));
          float z[8];
          values8(*c, 1.f, z);
          *c = code8(z, less, INFINITY);
        }
      }
    }
    const float inv = two_to(-now);
    const bool far = now == Scale8<T>::kHigh;  // values may lie past the largest code
#pragma unroll
    for (int i = 0; i < kA8Steps; ++i) {
      const int r = (i * p.unit_warps + part) * rows_at_once + row_of_warp;
      if (r >= rows || !my.live ||
          !in_bounds(dst0 + r * p.c8.slot_stride <=
                         (n_pages - 1) * page_stride + (batch.page_size - 1) * slot_stride && slot + r < batch.page_size,
                     batch.status))
        continue;
      uint8_t* const at = pool + dst0 + r * p.c8.slot_stride + head * p.c8.head_stride;
      *reinterpret_cast<uint2*>(at + my.d0) = far ? code8(x[i], inv, most) : code8_near(x[i], inv);
      *reinterpret_cast<uint2*>(at + my.d1) = far ? code8(y[i], inv, most) : code8_near(y[i], inv);
    }
  }
}

// ---------------------------------------------------------------------------
// read-back: entries of the sequences as rows of 16 bits
// ---------------------------------------------------------------------------
struct Read8Params {
  Paged8View c8;
  PagedBatch batch;      // q_indptr: the rows out; kv_len: not used
  const int32_t* first;  // [B] the entry of each sequence's first row, or null: 0
  uint16_t *k_out, *v_out;  // either may be null
  int64_t k_ps, k_hs, v_ps, v_hs;
  int D, tile;           // positions of a CTA
};

constexpr int kR8Threads = 256, kR8MaxTile = 64, kR8Batch = 4;

// A thread turns 16 codes (16 bytes) into 32 bytes, four in flight; the CTA's
// (row, side, head, 16 dims) in one sequence, so that neighbours write neighbouring
// bytes.  Bound by HBM: one byte read, two written a value.
template <typename T>
__global__ void __launch_bounds__(kR8Threads) read8_kernel(const __grid_constant__ Read8Params p) {
  __shared__ int64_t s_src[kR8MaxTile];  // offset of the entry in the pools, -1: zeros, -2: no row
  __shared__ int s_page[kR8MaxTile], s_slot[kR8MaxTile];
  const PagedBatch& batch = p.batch;
  const int tid = threadIdx.x;
  const int n0 = static_cast<int>(blockIdx.x) * p.tile, tile = min(p.tile, batch.N - n0);
  grid_dep_launch();
  grid_dep_wait();
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kR8Threads + kR8Threads - 1 - tid; i < batch.B;
       i += static_cast<int64_t>(gridDim.x) * kR8Threads) {
    const int b = static_cast<int>(i), at = batch.q_indptr[b];
    if (at > batch.q_indptr[b + 1] || (b == 0 && at != 0) || (b == batch.B - 1 && batch.q_indptr[b + 1] > batch.N))
      atomicOr(batch.status, kStatusBadCache);
  }
  for (int t = tid; t < tile; t += kR8Threads) {
    const int n = n0 + t, b = find_seq_alone(batch, n);
    int64_t src = -2;
    int page = -1, slot = 0;
    if (b >= 0 && n < batch.q_indptr[b + 1]) {
      const int64_t entry = static_cast<int64_t>(p.first != nullptr ? p.first[b] : 0) + (n - batch.q_indptr[b]);
      src = -1;
      if (entry >= 0 && entry < static_cast<int64_t>(batch.table_width) * batch.page_size &&
          in_bounds(b < batch.B, batch.status)) {
        page = batch.block_table[static_cast<int64_t>(b) * batch.table_width + entry / batch.page_size];
        slot = static_cast<int>(entry % batch.page_size);
      }
      if (page >= 0 && page < p.c8.n_pages)
        src = page * p.c8.page_stride + slot * p.c8.slot_stride;
      else
        atomicOr(batch.status, kStatusBadCache);
    }
    if (in_bounds(t < kR8MaxTile, batch.status)) {
      s_src[t] = src;
      s_page[t] = page;
      s_slot[t] = slot;
    }
  }
  __syncthreads();
  const int chunks = p.D >> 4, side = p.c8.n_heads * chunks, per_row = 2 * side, total = tile * per_row;
  for (int i0 = tid; i0 < total; i0 += kR8Threads * kR8Batch) {
    uint4 c[kR8Batch];
    int e[kR8Batch];
    uint16_t* dst[kR8Batch];
#pragma unroll
    for (int k = 0; k < kR8Batch; ++k) {
      const int i = i0 + k * kR8Threads, t = i / per_row, x = i - t * per_row;
      const bool is_v = x >= side;
      const int y = is_v ? x - side : x, head = y / chunks, d = (y - head * chunks) * 16;
      dst[k] = nullptr;
      c[k] = make_uint4(0, 0, 0, 0);
      e[k] = 0;
      if (i >= total || !in_bounds(t < kR8MaxTile, batch.status) || s_src[t] == -2) continue;
      uint16_t* const out = is_v ? p.v_out : p.k_out;
      if (out == nullptr) continue;
      dst[k] = out + static_cast<int64_t>(n0 + t) * (is_v ? p.v_ps : p.k_ps) + head * (is_v ? p.v_hs : p.k_hs) + d;
      if (s_src[t] < 0) continue;
      c[k] = *reinterpret_cast<const uint4*>((is_v ? p.c8.v : p.c8.k) + s_src[t] + head * p.c8.head_stride + d);
      e[k] = stored_exponent<T>((is_v ? p.c8.v_scales : p.c8.k_scales)[p.c8.scale_at(s_page[t], s_slot[t], head)]);
    }
#pragma unroll
    for (int k = 0; k < kR8Batch; ++k) {
      if (dst[k] == nullptr) continue;
      const float scale = two_to(e[k]);
      float x[8], y[8];
      values8(make_uint2(c[k].x, c[k].y), scale, x);
      values8(make_uint2(c[k].z, c[k].w), scale, y);
      reinterpret_cast<uint4*>(dst[k])[0] = pack8<T>(x);
      reinterpret_cast<uint4*>(dst[k])[1] = pack8<T>(y);
    }
  }
}

}  // namespace specv
