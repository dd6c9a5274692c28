// attend8.cuh — attention of the new positions over a cache of 8-bit codes, on the
// tcgen05 tensor cores.
//
// The mathematics, the line of work, the parts and their join are attend.cuh's; the
// products are turned around, because here keys and values have to be converted
// on their way and are half the bytes, so that the work a key costs counts:
//
//   S^T = K Q^T   [128 keys x rows]   K, converted to 16 bits, from TMEM (a lane a
//                                     key), Q from shared memory
//   O^T += V^T P^T [dims x rows]      V, converted, and P from shared memory
//
// The keys are the 128 lanes of a product and the rows its columns: 32, 64 or
// 128 of them, as many as an item has, where the other way around a decode step's few
// rows would take a product's 128 lanes and its softmax those lanes' exponentials.
// A key converted for S^T goes straight to TMEM, not through shared memory.
//
// An item is a row tile (up to 128 rows) against all tiles of 128 keys it sees.
// One CTA per SM, 16 warps:
//   warps 0-3, 4-7   softmax groups 0 and 1: a thread a key, each group half of
//                    the columns.  Weights go to shared memory as P.
//   warps 8-11       converters: a thread a key: its codes from the raw ring, as
//                    16-bit values to TMEM (K) or to a swizzled tile (V; past the
//                    last entry zeros).
//   warp 12          the scheduler, as in attend.cuh; warp 13 issues the products;
//   warps 14, 15     load key and value codes (TMA) and the blocks' scales.
// TMEM: two S^T (128 columns each), O^T (128), two K (D / 2 each).
//
// A row's reference m is shared by the 128 threads of a group: a barrier with a
// vote per tile says whether any score passes it by more than 2^8, and only then
// are the columns' maxima taken and O and the sums multiplied.  The sums are
// kept by key in registers (fp32) and added up over the lanes once a part.
#pragma once

#include "attend.cuh"
#include "paged8.cuh"

namespace specv {

constexpr int kQ8Threads = 512;
// 168 + 168 + 96 + 80 = 4 x 128, the launch's
constexpr int kQ8SoftmaxRegs = 168, kQ8ConvertRegs = 96, kQ8OtherRegs = 80;
constexpr int kQ8Queue = 2;          // parts queued ahead
constexpr float kQ8Unset = 3.0e38f;  // minus the reference of a row that has seen nothing

struct Attend8Params : AttendParams {
  Paged8View c8;
  static constexpr bool kCodes = true;
  __device__ __forceinline__ int64_t head_stride() const { return c8.head_stride; }
  __device__ __forceinline__ int64_t entry_at(int64_t page, int slot) const {
    return page * c8.page_stride + slot * c8.slot_stride;
  }
  template <typename T>
  __device__ __forceinline__ void scales(int64_t page, int slot, int head, float& k, float& v) const {
    const int64_t at = c8.scale_at(page, slot, head);
    k = two_to(stored_exponent<T>(c8.k_scales[at]));
    v = two_to(stored_exponent<T>(c8.v_scales[at]));
  }
  template <typename T>
  __device__ __forceinline__ uint4 keys8(int64_t at, float scale) const {
    float x[8];
    values8(*reinterpret_cast<const uint2*>(c8.k + at), scale, x);
    return pack8<T>(x);
  }
  template <typename T>
  __device__ __forceinline__ uint32_t values2(int64_t at, float scale) const {
    const float2 f = specv::values2(*reinterpret_cast<const uint16_t*>(c8.v + at));
    return Pack16<T>::pack(f.x * scale, f.y * scale);
  }
};

template <int D>
struct Q8Shared {
  static constexpr int kSlots = 32 * 1024 / (kAtTile * D);  // of the key ring and of the value ring
  uint64_t raw_full[2][kSlots], raw_empty[2][kSlots];       // [keys, values]
  uint64_t kc_full[2], kc_empty[2], vc_full[2], vc_empty[2];
  uint64_t s_full[2], p_full, pv_done, o_free, q_full[2], q_empty[2], part_full[kQ8Queue], part_empty[kQ8Queue], done;
  __align__(16) float neg_ref[kAtTile];       // minus the rows' references (log2)
  __align__(16) float cross[2][4][kAtTile / 2];  // per group: its warps' maxima or sums of the columns
  uint8_t scales[2][kSlots][16];              // [keys, values] of 8 keys each
  AtPart parts[kQ8Queue];
  uint32_t tmem;
};

constexpr uint32_t kQ8PBytes = 2 * kAtTile * 128;  // P: two tiles of 64 rows
template <int D>
constexpr uint32_t q8_smem_bytes() {
  // queries x 2, converted values x 2, P, key and value ring
  return 4u * kAtTile * D * 2 + kQ8PBytes + 64 * 1024 + sizeof(Q8Shared<D>);
}
static_assert(q8_smem_bytes<128>() <= 227 * 1024 && q8_smem_bytes<64>() <= 227 * 1024, "one CTA's shared memory");

// Four codes to four 16-bit values (two words) times `scale`, a power of two as
// two values of the type.
template <typename T>
struct Codes;
template <>
struct Codes<__half> {
  uint32_t scale;
  __device__ __forceinline__ explicit Codes(int e) {
    const __half2 s = __float2half2_rn(two_to(e));
    scale = *reinterpret_cast<const uint32_t*>(&s);
  }
  __device__ __forceinline__ uint32_t pair(uint16_t c) const {
    const uint32_t h = half2_of_codes(c);
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(scale));
    return d;
  }
  __device__ __forceinline__ void four(uint32_t w, uint32_t& lo, uint32_t& hi) const {
    lo = pair(static_cast<uint16_t>(w));
    hi = pair(static_cast<uint16_t>(w >> 16));
  }
  __device__ __forceinline__ void sixteen(const uint4& w, uint32_t (&d)[8]) const {
    four(w.x, d[0], d[1]);
    four(w.y, d[2], d[3]);
    four(w.z, d[4], d[5]);
    four(w.w, d[6], d[7]);
  }
};
// A code's exponent and fraction bits, put where bf16's lowest exponent and highest
// fraction bits are, read as the code's value times 2^-120: one exact product
// with 2^(120 + e) gives the value.  (2^(120 + e) passes bf16's range for e > 7:
// two products then.)  The code of NaN would read as 480: looked for apart.
template <>
struct Codes<__nv_bfloat16> {
  uint32_t scale, more;
  __device__ __forceinline__ explicit Codes(int e) {
    const uint32_t a = min(e, 7) + 247, b = max(e - 7, 0) + 127;  // biased exponents of 2^(120 + e) in two factors
    scale = a << 7 | a << 23;
    more = b << 7 | b << 23;
  }
  __device__ static __forceinline__ uint32_t mul(uint32_t x, uint32_t y) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
    return d;
  }
  __device__ __forceinline__ uint32_t pair(uint32_t y) const {  // codes in the high bytes of the halves
    return mul((y >> 4 & 0x07f007f0u) | (y & 0x80008000u), scale);
  }
  __device__ __forceinline__ void sixteen(const uint4& w, uint32_t (&d)[8]) const {
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
    uint32_t nan = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      nan |= (c[i] & 0x7f7f7f7fu) + 0x01010101u;
      d[2 * i] = pair(__byte_perm(c[i], 0, 0x1404));
      d[2 * i + 1] = pair(__byte_perm(c[i], 0, 0x3424));
    }
    if (more != 0x3f803f80u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = mul(d[i], more);
    }
    if (nan & 0x80808080u) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if ((c[i / 4] >> (8 * (i % 4)) & 0x7f) == 0x7f) d[i / 2] |= 0x7fffu << (16 * (i % 2));
    }
  }
};

// whether the condition holds in any of the 128 threads of a softmax group
__device__ __forceinline__ bool group_any(int g, bool c) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.aligned.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(c ? 1u : 0u), "r"(1 + g)
      : "memory");
  return any != 0;
}

// kCount consecutive fp32 columns of this thread's TMEM lane
template <int kCount>
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[kCount]);
template <>
__device__ __forceinline__ void tmem_load<16>(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
template <>
__device__ __forceinline__ void tmem_load<32>(uint32_t taddr, uint32_t (&r)[32]) {
  tmem_ld32_start(taddr, r);
  tmem_ld32_wait(r);
}
template <>
__device__ __forceinline__ void tmem_load<64>(uint32_t taddr, uint32_t (&r)[64]) {
  uint32_t a[32], b[32];
  tmem_ld32_start(taddr, a);
  tmem_ld32_start(taddr + 32, b);
  tmem_ld32_wait(a);
  tmem_ld32_wait(b);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    r[i] = a[i];
    r[i + 32] = b[i];
  }
}

// One value of each of kCount columns a lane, reduced over the warp's 32 lanes in
// halves: log2 steps that each halve what a lane holds, until it holds the
// columns lane * kCount / 32 (kCount 32, 64) or, in lanes 2 c and 2 c + 1, column c
// (kCount 16).
template <int kCount, typename Op>
__device__ __forceinline__ void reduce_columns(float (&v)[kCount], int lane, Op op) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const int half = kCount * s / 32;  // columns a lane keeps in this step (0: all hold one already)
    const bool upper = lane & s;
    if (half > 0) {
#pragma unroll
      for (int i = 0; i < kCount / 2; ++i) {
        if (i >= half) break;
        const float send = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
        v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, s));
      }
    } else {
      v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], s));
    }
  }
}

template <typename T, int D>
struct Q8Softmax {
  const Attend8Params& p;
  Q8Shared<D>& sh;
  uint8_t* pbuf;
  uint32_t tmem;
  int g, quad, lane, key;
  bool ok;

  __device__ __forceinline__ uint32_t tm_s(uint32_t j) const { return tmem + 128 * (j & 1) + (static_cast<uint32_t>(quad * 32) << 16); }
  __device__ __forceinline__ uint32_t tm_o() const { return tmem + 256 + (static_cast<uint32_t>(quad * 32) << 16); }
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.batch.status, kWaitLimitCycles));
  }

  // Scores of the columns in a tile some of whose keys some rows do not see:
  // -inf there.
  template <int C>
  __device__ __forceinline__ void hide(const AtPart& a, int t, uint32_t (&s)[C]) const {
    const int e = t * kAtTile + key;  // the entry
    if (e < a.len && e < a.old) return;
    const int j = e - a.old;  // its place among the new ones
    int tok = (g * C) / p.group, left = (tok + 1) * p.group - g * C;  // of a column's position the columns to come
    bool sees = false;
    auto look = [&]() {
      sees = false;
      if (e >= a.len || tok >= a.n0) return;
      if (p.draft_mask == nullptr) {
        sees = j <= a.first - a.seq_first + tok;
      } else if (j < 64 && in_bounds(a.first >= 0 && a.first + tok < p.batch.N, p.batch.status)) {
        sees = (p.draft_mask[a.first + tok] >> j & 1) != 0;
      }
    };
    look();
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (left == 0) {
        ++tok;
        look();
        left = p.group;
      }
      --left;
      if (!sees) s[c] = 0xff800000u;
    }
  }

  // One column of each kCount / 32 lanes' values (reduce_columns) to the group's place.
  template <int C>
  __device__ __forceinline__ void to_cross(const float (&v)[C]) const {
    float* const at = sh.cross[g][quad];
    if (C == 16) {
      if ((lane & 1) == 0) at[lane / 2] = v[0];
    } else {
#pragma unroll
      for (int c = 0; c < C / 32; ++c) at[lane * (C / 32) + c] = v[c];
    }
  }

  // A part with C columns a group; `base`: tiles before it.
  template <int C>
  __device__ __forceinline__ void part(const AtPart& a, uint32_t base) {
    constexpr float kTop = kAtTop<T>, kOver = kAtTop<T> + kAtRise;
    float* const neg_ref = sh.neg_ref + g * C;
    float(&cross)[4][kAtTile / 2] = sh.cross[g];
    const int mine = quad * 32 + lane;  // this thread's column in what is done once a column
    const int tiles = a.t1 - a.t0, rows = a.n0 * p.group;
    // entries below this one are seen by all rows
    const int open = a.line == 0 ? a.len : p.draft_mask != nullptr ? a.old : a.old + (a.first - a.seq_first) + 1;
    if (mine < C) neg_ref[mine] = kQ8Unset;
    uint64_t l2[C / 2];
#pragma unroll
    for (int c = 0; c < C / 2; ++c) l2[c] = 0;
    group_any(g, false);
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const uint32_t j = base + i;
      const int t = a.t0 + i;
      uint32_t s[C];
      ok = wait(&sh.s_full[j & 1], (j >> 1) & 1) && ok;
      tc_fence_after();
      auto scores = [&]() {
        tmem_load<C>(tm_s(j) + g * C, s);
        if (open - t * kAtTile < kAtTile) hide<C>(a, t, s);
      };
      // scores minus the references, in place; whether one passes its reference by far
      auto against = [&]() {
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2);
#pragma unroll
        for (int c = 0; c < C; c += 4) {
          const ulonglong2 n = *reinterpret_cast<const ulonglong2*>(neg_ref + c);
          float x[4];
          f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, n.x), x[0], x[1]);
          f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), scale2, n.y), x[2], x[3]);
          top[c / 4 % 2 * 2] = max3(top[c / 4 % 2 * 2], x[0], x[1]);
          top[c / 4 % 2 * 2 + 1] = max3(top[c / 4 % 2 * 2 + 1], x[2], x[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) s[c + k] = __float_as_uint(x[k]);
        }
        return fmaxf(max3(top[0], top[1], top[2]), top[3]) > kOver;
      };
      scores();
      const bool rise = against();
      bool waited = false;
      if (group_any(g, rise || !ok)) {
        // (O may be multiplied: the last product into it is complete)
        if (ok && j > 0) ok = wait(&sh.pv_done, (j - 1) & 1);
        waited = true;
        if (group_any(g, !ok)) {
          ok = false;
          return;
        }
        tc_fence_after();
        scores();
        float top[C];
#pragma unroll
        for (int c = 0; c < C; ++c) top[c] = __uint_as_float(s[c]);
        reduce_columns<C>(top, lane, [](float x, float y) { return fmaxf(x, y); });
        to_cross<C>(top);
        group_any(g, false);
        if (mine < C) {
          const float m = fmaxf(max3(cross[0][mine], cross[1][mine], cross[2][mine]), cross[3][mine]) * p.scale_log2;
          const float n = neg_ref[mine];
          const bool up = m + n > kOver;
          cross[0][mine] = up ? ex2(kTop - (m + n)) : 1.f;  // (0 at a row's first keys)
          if (up) neg_ref[mine] = kTop - m;
        }
        group_any(g, false);
#pragma unroll
        for (int c = 0; c < C / 2; ++c) {
          float x, y;
          f32x2_split(l2[c], x, y);
          l2[c] = f32x2(x * cross[0][2 * c], y * cross[0][2 * c + 1]);
        }
        if (i > 0 && (D == 128 || quad < 2)) {
#pragma unroll
          for (int c = 0; c < C; c += 16) {
            uint32_t o[16];
            tmem_load<16>(tm_o() + g * C + c, o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * cross[0][c + x]);
            tmem_st16(tm_o() + g * C + c, o);
          }
          tmem_st_wait();
        }
        scores();
        against();
      }
      // weights: the sums keep them in 32 bits, P in 16 (half a step off at most)
      uint32_t w[C / 2];
#pragma unroll
      for (int c = 0; c < C / 2; ++c) {
        const float e0 = ex2(__uint_as_float(s[2 * c])), e1 = ex2(__uint_as_float(s[2 * c + 1]));
        l2[c] = add_f32x2(l2[c], f32x2(e0, e1));
        w[c] = Pack16<T>::pack(e0, e1);
      }
      if (!waited && j > 0) ok = wait(&sh.pv_done, (j - 1) & 1) && ok;
      // P: [key][64 rows], two tiles, 128-byte swizzle
#pragma unroll
      for (int c = 0; c < C; c += 8) {
        const int col = g * C + c;
        uint8_t* const at = pbuf + (col >> 6) * (kQ8PBytes / 2) + key * 128 + (((col >> 3 & 7) ^ (key & 7)) << 4);
        *reinterpret_cast<uint4*>(at) = make_uint4(w[c / 2], w[c / 2 + 1], w[c / 2 + 2], w[c / 2 + 3]);
      }
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full);
    }

    // ---- the part's results ----
    ok = wait(&sh.pv_done, (base + tiles - 1) & 1) && ok;
    if (group_any(g, !ok)) {
      ok = false;
      return;
    }
    tc_fence_after();
    const int cta = static_cast<int>(blockIdx.x);
    {
      float sum[C];
#pragma unroll
      for (int c = 0; c < C / 2; ++c) f32x2_split(l2[c], sum[2 * c], sum[2 * c + 1]);
      reduce_columns<C>(sum, lane, [](float x, float y) { return x + y; });
      to_cross<C>(sum);
    }
    group_any(g, false);
    const int col0 = g * C + mine;
    if (mine < C && col0 < rows) {
      const float l = (cross[0][mine] + cross[1][mine]) + (cross[2][mine] + cross[3][mine]);
      const float n = neg_ref[mine];
      const float2 ml = make_float2(n == kQ8Unset ? -INFINITY : -n, l);
      const int tok = col0 / p.group;
      if (a.t0 == 0) {
        const int64_t row = p.place(a.line, static_cast<int64_t>(a.first + tok) * p.n_q_heads + a.head * p.group + (col0 - tok * p.group));
        if (in_bounds(a.first >= 0 && a.first + tok < p.batch.N, p.batch.status)) {
          p.part_ml[row] = ml;
          p.part_meta[row] = row_item(a, cta, col0);
        }
      } else if (in_bounds(cta < p.n_ctas && col0 < p.slab_rows, p.batch.status)) {
        p.slab_ml[static_cast<int64_t>(cta) * p.slab_rows + col0] = ml;
      }
    }
    if (D == 128 || quad < 2) {
      const int dim = quad * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < C; c += 16) {
        uint32_t o[16];
        tmem_load<16>(tm_o() + g * C + c, o);
        int col = g * C + c, tok = col / p.group, h = col - tok * p.group;
#pragma unroll
        for (int x = 0; x < 16; ++x, ++col) {
          if (col < rows) {
            if (a.t0 == 0) {
              const int64_t row = p.place(a.line, static_cast<int64_t>(a.first + tok) * p.n_q_heads + a.head * p.group + h);
              if (in_bounds(a.first >= 0 && a.first + tok < p.batch.N, p.batch.status))
                p.part_o[row * D + dim] = __uint_as_float(o[x]);
            } else if (in_bounds(cta < p.n_ctas && col < p.slab_rows, p.batch.status)) {
              p.slab_o[(static_cast<int64_t>(cta) * p.slab_rows + col) * D + dim] = __uint_as_float(o[x]);
            }
          }
          if (++h == p.group) {
            h = 0;
            ++tok;
          }
        }
      }
    }
    tc_fence_before();
    group_any(g, false);  // the sums' places and the references may be written again
    if (lane == 0) mbar_arrive(&sh.o_free);
  }
};

// columns a softmax group has for a part of so many rows
__device__ __forceinline__ int q8_columns(int rows) { return rows <= 32 ? 16 : rows <= 64 ? 32 : 64; }

template <typename T, int D>
__global__ void __launch_bounds__(kQ8Threads, 1) attend8_kernel(const __grid_constant__ Attend8Params p) {
  constexpr int kHalves = D / 64;                 // 64-dim halves of a 16-bit tile
  constexpr uint32_t kHalfBytes = kAtTile * 128;  // 16 KB
  constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  constexpr uint32_t kRawBytes = kAtTile * D;
  constexpr int kSlots = Q8Shared<D>::kSlots;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  // no static shared memory: the swizzled tiles begin at its (1024-byte aligned) start
  extern __shared__ __align__(1024) uint8_t at_smem[];
  uint8_t* const qbuf = at_smem;                    // [2] query tiles
  uint8_t* const vbuf = at_smem + 2 * kTileBytes;   // [2] converted values
  uint8_t* const pbuf = at_smem + 4 * kTileBytes;   // weights
  uint8_t* const ring = pbuf + kQ8PBytes;           // [keys, values][kSlots] codes
  Q8Shared<D>& sh = *reinterpret_cast<Q8Shared<D>*>(ring + 2 * kSlots * kRawBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const status = p.batch.status;
  const int cta = static_cast<int>(blockIdx.x);
  grid_dep_launch();

  if (threadIdx.x == 0) {
    for (int v = 0; v < 2; ++v) {
      for (int i = 0; i < kSlots; ++i) {
        mbar_init(&sh.raw_full[v][i], 2);   // the copies' and the scales'
        mbar_init(&sh.raw_empty[v][i], 4);  // converter warps
      }
      mbar_init(&sh.kc_full[v], 4);
      mbar_init(&sh.kc_empty[v], 1);
      mbar_init(&sh.vc_full[v], 4);
      mbar_init(&sh.vc_empty[v], 1);
      mbar_init(&sh.s_full[v], 1);
      mbar_init(&sh.q_full[v], 1);
      mbar_init(&sh.q_empty[v], 1);
    }
    for (int i = 0; i < kQ8Queue; ++i) {
      mbar_init(&sh.part_full[i], 1);
      mbar_init(&sh.part_empty[i], 15);  // eight softmax warps, four converters, the issuer, the two loaders
    }
    mbar_init(&sh.p_full, 8);
    mbar_init(&sh.pv_done, 1);
    mbar_init(&sh.o_free, 8);
    mbar_init(&sh.done, 1);
    fence_mbar_init();
  }
  if (warp == 13) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  grid_dep_wait();
  if (warp >= 12) {
    regs_down<kQ8OtherRegs>();
    if (warp == 12) {
      // ---------------- scheduler (the whole warp): parts, and their queries ----------------
      const PrefixItems pl = prefix_items(p);
      uint32_t queued = 0;
      bool ok = true;
      // a free place of the queue
      auto queue_place = [&]() {
        const int q = queued % kQ8Queue;
        if (queued >= kQ8Queue)
          ok = ok && mbar_wait(&sh.part_empty[q], ((queued / kQ8Queue) & 1) ^ 1, status, kWaitLimitCycles);
        ok = __all_sync(0xffffffffu, ok);
        return q;
      };
      // the line: the weight of the tiles alone and the number of items side by
      // side, until their sum says which fixed cost counts
      AtPart a;
      SeqWeight first = {0, 0};  // of sequence `lane`
      int64_t own = 0, own_items = 0;
      for (int b = lane; b < p.batch.B; b += 32) {
        const SeqSpan s = seq_span(p.batch, b);
        const SeqWeight w = seq_weight(p, s);
        if (b == lane) first = w;
        own += w.tiles_alone * p.n_heads;
        own_items += static_cast<int64_t>(w.items) * p.n_heads;
        if (cta == 0 && s.kv < s.n) no_tiles(p, s);
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) {
        own += __shfl_xor_sync(0xffffffffu, own, x);
        own_items += __shfl_xor_sync(0xffffffffu, own_items, x);
      }
      a.fixed = fixed_weight(pl.tiles_alone * p.n_heads + own, p.n_ctas);
      const int64_t prefix = pl.per_head(a.fixed) * p.n_heads, total = prefix + own + own_items * a.fixed;
      const int64_t lo = part_begin(total, cta, p.n_ctas), hi = part_begin(total, cta + 1, p.n_ctas);
      // the sequence that this CTA's part of the own pages begins in
      int own_seq = p.batch.B;
      int64_t own_off = prefix;
      if (lo < hi && hi > prefix) {
        const int64_t from = max(lo, prefix);
#pragma unroll 1
        for (int b0 = 0; b0 < p.batch.B; b0 += 32) {
          const int b = b0 + lane;
          int64_t mine = 0;
          if (b < p.batch.B)
            mine = (b0 == 0 ? first : seq_weight(p, seq_span(p.batch, b))).per_head(a.fixed) * p.n_heads;
          int64_t inc = mine;
#pragma unroll
          for (int x = 1; x < 32; x <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, inc, x);
            if (lane >= x) inc += o;
          }
          const int64_t off = own_off + inc - mine;
          const unsigned here = __ballot_sync(0xffffffffu, off <= from && from < off + mine);
          if (here != 0u) {
            own_seq = b0 + __ffs(here) - 1;
            own_off = __shfl_sync(0xffffffffu, off, __ffs(here) - 1);
            break;
          }
          own_off += __shfl_sync(0xffffffffu, inc, 31);
        }
      }
      if (lane == 0 && in_bounds(cta < p.n_ctas, status)) {
        p.begin[cta] = lo;
        if (cta == p.n_ctas - 1) p.begin[cta + 1] = hi;
      }
#pragma unroll 1
      for (a.line = 0; a.line < 2 && ok; ++a.line) {
        // the prefix is like one sequence of all new positions
        if (a.line == 0 ? lo >= prefix : hi <= prefix) continue;
        int64_t off = a.line == 0 ? 0 : own_off;
        a.seq = a.line == 0 ? 0 : own_seq;
#pragma unroll 1
        for (; off < hi && lo < hi && a.seq < p.batch.B && ok; ++a.seq) {
          if (a.line == 0 && a.seq > 0) break;
          SeqSpan s = {0, pl.positions, 0, 0};
          int64_t hw = pl.per_head(a.fixed);
          if (a.line == 1) {
            s = seq_span(p.batch, a.seq);
            hw = seq_weight(p, s).per_head(a.fixed);
          }
          a.len = a.line == 0 ? p.prefix_len : static_cast<int>(s.kv);
          a.old = a.line == 0 ? a.len : a.len - s.n;
          a.seq_first = s.first;
          a.seq_n = s.n;
          a.head = 0;
#pragma unroll 1
          for (; hw > 0 && lo - off >= hw && a.head < p.n_heads; ++a.head) off += hw;
#pragma unroll 1
          for (; a.head < p.n_heads && off < hi && ok; ++a.head) {
#pragma unroll 1
            for (int at = 0; at < s.n && ok; at += p.block) {
              const int rb = at / p.block;
              const int tiles = a.line == 0 ? pl.tiles : block_tiles(p, s, rb), w = block_rows(p, s.n, rb);
              a.off = off;
              a.tiles = tiles;
              a.w = w;
              a.t0 = tiles_before(lo, off, w, a.fixed, tiles);
              a.t1 = tiles_before(hi, off, w, a.fixed, tiles);
              off += item_weight(tiles, w, a.fixed);
              if (a.t0 >= a.t1) continue;
              // the part that the item's last tile begins in
              a.last = cta;
              if (a.t0 == 0 && a.t1 < tiles)
                a.last = static_cast<int>(((off - tile_weight(w) + 1) * p.n_ctas - 1) / total);
              a.first = s.first + at;
              a.n0 = min(p.block, s.n - at);
              a.n1 = 0;
              const int q = queue_place();
              if (!ok) break;
              if (lane == 0) {
                sh.parts[q] = a;
                mbar_arrive(&sh.part_full[q]);
              }
              // its queries: part n's are in buffer n % 2
              const uint32_t qb = queued & 1;
              if (queued >= 2)
                ok = __all_sync(0xffffffffu, mbar_wait(&sh.q_empty[qb], ((queued >> 1) & 1) ^ 1, status, kWaitLimitCycles));
              if (!ok) break;
              if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[qb], kHalves * 128u * p.group * p.tok_tile);
              __syncwarp();
              // (tiled copies stay inside their tensor by themselves: recorded only)
              in_bounds(a.first >= 0 && a.first < p.batch.N && (a.head + 1) * p.group <= p.n_q_heads, status);
              if (lane < kHalves)
                tma_load_3d(smem_u32(qbuf) + qb * kTileBytes + lane * kHalfBytes, &p.tmQ, lane * 64, a.head * p.group, a.first,
                            &sh.q_full[qb]);
              ++queued;
            }
          }
        }
      }
      if (ok) {
        const int q = queue_place();
        if (ok && lane == 0) {
          sh.parts[q].line = -1;
          mbar_arrive(&sh.part_full[q]);
        }
      }
      for (uint32_t n = queued < 2 ? 0 : queued - 2; n < queued; ++n)  // the last copies land before the CTA exits
        mbar_wait(&sh.q_full[n & 1], (n >> 1) & 1, status, kWaitLimitCycles);
    } else if (warp == 13) {
      // ---------------- issuer (the whole warp; one thread issues) ----------------
      const uint32_t utm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = smem_desc_k128(smem_u32(qbuf)), v_desc = smem_desc_mn128(smem_u32(vbuf), kHalfBytes),
                     p_desc = smem_desc_mn128(smem_u32(pbuf), kQ8PBytes / 2);
      uint32_t base = 0;  // tiles before this part
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, status, kWaitLimitCycles));
        return ok;
      };
#pragma unroll 1
      for (uint32_t n = 0; ok; ++n) {
        const int q = n % kQ8Queue;
        if (!wait(&sh.part_full[q], (n / kQ8Queue) & 1)) break;
        const int line = __shfl_sync(0xffffffffu, sh.parts[q].line, 0);
        const int tiles = __shfl_sync(0xffffffffu, sh.parts[q].t1 - sh.parts[q].t0, 0);
        const int columns = 2 * q8_columns(__shfl_sync(0xffffffffu, sh.parts[q].n0, 0) * p.group);
        if (lane == 0) mbar_arrive(&sh.part_empty[q]);
        if (line < 0) break;
        const uint32_t id_qk = idesc_f16_f32(kBf16, false, kAtTile, columns);
        const uint32_t id_pv = idesc_f16_f32(kBf16, true, kAtTile, columns) | 1u << 15;  // A too has K over its rows
        if (!wait(&sh.q_full[n & 1], (n >> 1) & 1)) break;
        // scores of the part's tile i
        auto qk = [&](int i) {
          const uint32_t j = base + i, b = j & 1;
          if (!wait(&sh.kc_full[b], (j >> 1) & 1)) return;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t bd = q_desc + (n & 1) * (kTileBytes >> 4);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              tc_mma_ts(utm + 128 * b, utm + 384 + (D / 2) * b + 8 * k, bd + (k / 4) * (kHalfBytes >> 4) + (k % 4) * 2, id_qk, k > 0);
            tc_commit(&sh.s_full[b]);
            tc_commit(&sh.kc_empty[b]);
            if (i + 1 == tiles) tc_commit(&sh.q_empty[n & 1]);
          }
          __syncwarp();
        };
        qk(0);
        if (tiles > 1) qk(1);
#pragma unroll 1
        for (int i = 0; i < tiles && ok; ++i) {
          const uint32_t j = base + i, b = j & 1;
          if (!wait(&sh.vc_full[b], (j >> 1) & 1)) break;
          if (i == 0 && n > 0 && !wait(&sh.o_free, (n - 1) & 1)) break;
          if (!wait(&sh.p_full, j & 1)) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = v_desc + b * (kTileBytes >> 4);
#pragma unroll
            for (int k = 0; k < kAtTile / 16; ++k)
              tc_mma(utm + 256, ad + k * (2048 >> 4), p_desc + k * (2048 >> 4), id_pv, i > 0 || k > 0);
            tc_commit(&sh.pv_done);
            tc_commit(&sh.vc_empty[b]);
          }
          __syncwarp();
          if (i + 2 < tiles) qk(i + 2);
        }
        base += tiles;
      }
      // nothing is in flight when the TMEM is freed
      if (elect_one()) tc_commit(&sh.done);
      __syncwarp();
      mbar_wait(&sh.done, 0, status, kWaitLimitCycles);
    } else {
      // ---------------- key loads (warp 14) and value loads (warp 15) ----------------
      // A lane (of 16) has 8 keys: their page, ahead of time, and their block's
      // scale; one box a lane where a box (a run of a page's slots) begins.
      const int values = warp == 15 ? 1 : 0;
      const CUtensorMap* const map = values ? &p.tmV : &p.tmK;
      const uint8_t* const scales = values ? p.c8.v_scales : p.c8.k_scales;
      const int my_key = (lane & 15) * 8;
      const bool loads = lane < 16 && my_key % p.box_rows == 0;
      const uint32_t my_dst = smem_u32(ring) + values * kSlots * kRawBytes + my_key * D;
      const uint32_t page_size = p.batch.page_size;
      uint32_t base = 0;
      bool ok = true;
#pragma unroll 1
      for (uint32_t n = 0; ok; ++n) {
        const int q = n % kQ8Queue;
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.part_full[q], (n / kQ8Queue) & 1, status, kWaitLimitCycles));
        if (!ok) break;
        const int line = sh.parts[q].line, head = sh.parts[q].head, t0 = sh.parts[q].t0, tiles = sh.parts[q].t1 - t0,
                  len = sh.parts[q].len, seq = sh.parts[q].seq;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.part_empty[q]);
        if (line < 0) break;
        const int32_t* const table =
            line == 0 ? p.prefix_table : p.batch.block_table + static_cast<int64_t>(seq) * p.batch.table_width;
        const uint32_t table_end = line == 0 ? (p.prefix_len - 1u) / page_size + 1 : p.batch.table_width;
        // the page of this lane's keys in the part's tile i; past the entries, and
        // where the table has none, n_pages: the copy fills zeros
        auto page_at = [&](int i) {
          const uint32_t key = static_cast<uint32_t>(t0 + i) * kAtTile + my_key;
          if (i >= tiles || key >= static_cast<uint32_t>(len) ||
              !in_bounds(key / page_size < table_end && seq >= 0 && seq < p.batch.B, status))
            return p.n_pages;
          const int page = table[key / page_size];
          if (page < 0 || page >= p.n_pages) {
            atomicOr(status, kStatusBadCache);
            return p.n_pages;
          }
          return page;
        };
        auto scale_of = [&](int i, int page) -> uint32_t {
          const uint32_t key = static_cast<uint32_t>(t0 + i) * kAtTile + my_key;
          return page < p.n_pages ? scales[p.c8.scale_at(page, static_cast<int>(key % page_size), head)] : 127;
        };
        // pages three tiles ahead, scales two
        int page0 = page_at(0), page1 = page_at(1), page2 = page_at(2);
        uint32_t scale0 = scale_of(0, page0), scale1 = scale_of(1, page1);
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          const uint32_t j = base + i, slot = j % kSlots, use = j / kSlots;
          const int page = page0, at_slot = static_cast<int>((static_cast<uint32_t>(t0 + i) * kAtTile + my_key) % page_size);
          const uint32_t scale = scale0;
          page0 = page1;
          page1 = page2;
          scale0 = scale1;
          scale1 = scale_of(i + 2, page1);
          page2 = page_at(i + 3);
          if (use > 0)
            ok = __all_sync(0xffffffffu, mbar_wait(&sh.raw_empty[values][slot], (use & 1) ^ 1, status, kWaitLimitCycles));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sh.raw_full[values][slot], kRawBytes);
          __syncwarp();
          if (loads) {
            in_bounds(slot < kSlots && at_slot + p.box_rows <= static_cast<int>(page_size) && head >= 0 && head < p.n_heads, status);
            tma_load_4d(my_dst + slot * kRawBytes, map, 0, at_slot, head, page, &sh.raw_full[values][slot]);
          }
          if (lane < 16) sh.scales[values][slot][lane] = static_cast<uint8_t>(scale);
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.raw_full[values][slot]);
        }
        if (!ok) break;
        base += tiles;
      }
      // copies land before the CTA exits: the converters wait for every tile,
      // unless a wait ran out
      if (!ok) {
        for (uint32_t k = 0; k < kSlots; ++k) mbar_wait(&sh.raw_full[values][k], 0, status, kWaitLimitCycles);
        for (uint32_t k = 0; k < kSlots; ++k) mbar_wait(&sh.raw_full[values][k], 1, status, kWaitLimitCycles);
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    regs_down<kQ8ConvertRegs>();
    // ---------------- converters: a thread a key ----------------
    const int quad = warp - 8, key = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t base = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, status, kWaitLimitCycles));
      return ok;
    };
    // the raw tile's 16 codes c of this thread's key: rows of D bytes, swizzled
    auto codes = [&](const uint8_t* tile, int c) {
      const int at = D == 128 ? c ^ (key & 7) : c ^ (key >> 1 & 3);
      return *reinterpret_cast<const uint4*>(tile + key * D + at * 16);
    };
#pragma unroll 1
    for (uint32_t n = 0; ok; ++n) {
      const int q = n % kQ8Queue;
      if (!wait(&sh.part_full[q], (n / kQ8Queue) & 1)) break;
      const int line = sh.parts[q].line, t0 = sh.parts[q].t0, tiles = sh.parts[q].t1 - t0, len = sh.parts[q].len;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.part_empty[q]);
      if (line < 0) break;
#pragma unroll 1
      for (int i = 0; i < tiles && ok; ++i) {
        const uint32_t j = base + i, b = j & 1, slot = j % kSlots, use = j / kSlots;
        // keys, to TMEM
        if (!wait(&sh.raw_full[0][slot], use & 1)) break;
        if (j >= 2 && !wait(&sh.kc_empty[b], ((j >> 1) & 1) ^ 1)) break;
        tc_fence_after();
        {
          const uint8_t* const tile = ring + slot * kRawBytes;
          const Codes<T> conv(stored_exponent<T>(sh.scales[0][slot][key >> 3]));
#pragma unroll
          for (int c = 0; c < D / 16; c += 4) {
            uint32_t w[32];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              uint32_t d[8];
              conv.sixteen(codes(tile, c + x), d);
#pragma unroll
              for (int y = 0; y < 8; ++y) w[8 * x + y] = d[y];
            }
            tmem_st32(tmem + lanes + 384 + (D / 2) * b + 8 * c, w);
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.kc_full[b]);
          mbar_arrive(&sh.raw_empty[0][slot]);
        }
        // values, to a swizzled tile; past the last entry zeros (zero times what
        // stands there must be zero)
        if (!wait(&sh.raw_full[1][slot], use & 1)) break;
        if (j >= 2 && !wait(&sh.vc_empty[b], ((j >> 1) & 1) ^ 1)) break;
        {
          const uint8_t* const tile = ring + (kSlots + slot) * kRawBytes;
          const Codes<T> conv(stored_exponent<T>(sh.scales[1][slot][key >> 3]));
          const bool live = (t0 + i) * kAtTile + key < len;
          uint8_t* const dst = vbuf + b * kTileBytes + key * 128;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            uint32_t w[8];
            conv.sixteen(codes(tile, c), w);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int at = 2 * c + x;  // 8 dims: one 16-byte vector
              *reinterpret_cast<uint4*>(dst + (at / 8) * kHalfBytes + (((at % 8) ^ (key & 7)) << 4)) =
                  live ? make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]) : make_uint4(0, 0, 0, 0);
            }
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.vc_full[b]);
          mbar_arrive(&sh.raw_empty[1][slot]);
        }
      }
      base += tiles;
    }
  } else {
    regs_up<kQ8SoftmaxRegs>();
    Q8Softmax<T, D> sm = {p, sh, pbuf, tmem, warp >> 2, warp & 3, lane, (warp & 3) * 32 + lane, true};
    uint32_t base = 0;
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
      const int q = n % kQ8Queue;
      sm.ok = sm.wait(&sh.part_full[q], (n / kQ8Queue) & 1) && sm.ok;
      if (group_any(sm.g, !sm.ok)) break;
      const AtPart a = sh.parts[q];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.part_empty[q]);
      if (a.line < 0) break;
      const int columns = q8_columns(a.n0 * p.group);
      if (columns == 16)
        sm.template part<16>(a, base);
      else if (columns == 32)
        sm.template part<32>(a, base);
      else
        sm.template part<64>(a, base);
      if (!sm.ok) break;
      base += a.t1 - a.t0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_dealloc(tmem, 512);
}

}  // namespace specv
