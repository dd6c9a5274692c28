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
// The keys are the 128 lanes of a product and the rows its columns: 16, 32, 64 or
// 128 of them, as many as an item has, where the other way around a decode step's few
// rows would take a product's 128 lanes and its softmax those lanes' exponentials.
// A key converted for S^T goes straight to TMEM, not through shared memory.
//
// Types.  The products are fp16 with a bf16 cache too, wherever that is exact: the
// conversion from e4m3 is one instruction a pair, and to bf16 it is ten.  A key's
// scale counts in its scores, not in its values; queries are multiples of one power
// of two (a part with dims more than 2^31 below its largest, or not finite, keeps bf16
// queries and keys); values are multiples of another (a tile with blocks too small
// for it has bf16 values and weights, and so have all tiles of the part after it, and
// those from which on the unit has risen).
//
// An item is a row tile (up to 128 rows) against all tiles of 128 keys it sees.
// One CTA per SM, 16 warps:
//   warps 0-3, 4-7   softmax groups 0 and 1, a thread a key.  Up to 64 rows they
//                    alternate tiles, each with a reference, sums and an O of its own
//                    that are joined at the end of the part; above, they share each
//                    tile's columns.  Weights go to shared memory as P.
//   warps 8-11       converters, a thread a key: its codes from the raw ring, as
//                    16-bit values to TMEM (K) or to a swizzled tile (V; past the
//                    last entry zeros); at a part's start its queries.
//   warp 12          the scheduler, as in attend.cuh; warp 13 issues the products;
//   warps 14, 15     load key and value codes (TMA) and the blocks' scales.
// TMEM: two S^T (128 columns each), O^T (128), two K (D / 2 each).
//
// A row's reference m is shared by the 128 threads of a group: a barrier with a
// vote per tile says whether any weight passes 2^15, and only then are the columns'
// maxima taken and O and the sums multiplied.  The sums are kept by key in
// registers (fp32) and added up over the lanes once a part.
//
// What bounds it.  16 caches of up to 32,768 entries (472 MB): 125 to 127 us, 3.7 TB/s (the
// 16-bit call 150 us on twice the bytes).  A tile of 128 keys takes 2,400 clocks
// with few rows; HBM would need 1,450.  Two chains are that long: the converters'
// (keys 450, values 950, four waits) and the issuer's (16 products of 50 to 60
// clocks each as issued, and their waits).  With 128 rows it is the softmax warps'
// 3,500.  All of it runs at the rate of instruction fetches (a warp of every
// SM quarter has code of its own): loops that are not unrolled, and code that runs
// once a part kept short, took long caches from 385 to 127 us, long drafts from 2,083 to
// some 700 (666 to 715 on several boxes).  Tried and not kept, against 127 and 670 to
// 705: converters for keys and values apart, 20 warps (160
// registers for the softmax, more code at once: 138 us and 905); an issuer for
// each product besides (180 and 1,059); products unrolled with their operands in
// uniform registers (15 clocks an instruction by itself, no change here); values
// converted four vectors at a time, or one ahead (127 to 133); values converted by
// the softmax groups (129 and 778), and the next scores issued before the output
// besides (128 and 894); bf16 products throughout (207 and 1,091).  Scores past kFar rounded
// within the loop over tiles, instead of in a function of its own that it calls: long
// drafts 725 to 760 beside 710.
#pragma once

#include "attend.cuh"
#include "paged8.cuh"

namespace specv {

constexpr int kQ8Threads = 512;
// 184 + 184 + 80 + 64 = 4 x 128, the launch's
constexpr int kQ8LaunchRegs = 128, kQ8SoftmaxRegs = 184, kQ8ConvertRegs = 80, kQ8OtherRegs = 64;
static_assert(2 * kQ8SoftmaxRegs + kQ8ConvertRegs + kQ8OtherRegs == kQ8Threads / 128 * kQ8LaunchRegs,
              "a share above the launch's registers would be waited for for ever");
constexpr int kQ8Queue = 2;          // parts queued ahead
constexpr float kQ8Unset = 3.0e38f;  // minus the reference of a row that has seen nothing
constexpr float kQ8LeastFactor = 0x1p-126f, kQ8MostFactor = 0x1p127f;  // of a score

struct Attend8Params : AttendParams {
  Paged8View c8;
  // As AttendParams has them: a key tile takes some 3,600 clocks with over 64 rows
  // and 2,300 with fewer, a part's queries, first scores and results 12,000.
  static constexpr int kWide = 10, kNarrow = 6, kFixed = 24;
  static constexpr bool kCodes = true;
  // Scores (log2) from which fp32's step is 2: the difference that a product and sum in
  // one leaves between the score of a row's maximum and its rounded reference.
  static constexpr float kFar = 0x1p24f;
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
  uint64_t kc_full[2], vc_full[2];
  uint64_t s_full[2], pv_done[2];  // the products of tile j (places j % 2) are complete: their operands too are free
  uint64_t p_full[2], meet[2], o_free, q_full[2], q_ready[2], q_empty[2], part_full[kQ8Queue], part_empty[kQ8Queue], done;
  __align__(16) float neg_ref[2][kAtTile / 2];  // per group: minus its columns' references (log2); 0 where far
  float ref[2][kAtTile / 2];                    // the same, far or not
  // Infinite once a reference of the part has passed kFar, else -infinity.  All tiles then take
  // the way of those whose references are set, which puts scores less references into TMEM.
  float far[2];
  int columns[2];                               // of the groups' that are rows
  float unit[2];                                // log2 of the unit of the groups' O
  int8_t scales[2][kSlots][16];                 // [keys, values] exponents of 8 keys each
  int8_t key_exp[4][16];                        // of the keys of tile j % 4
  int16_t raw_unit[kSlots], v_unit[2];          // log2 of the unit that a tile's values have: in the ring, converted
  int8_t raw_wide[kSlots], v_wide[2];           // whether they are converted to bf16 (else fp16)
  int16_t q_exp[2];                             // log2 of the unit of a part's queries
  int8_t q_bf16[2];                             // whether they stay bf16
  uint32_t row_ends[kAtTile];  // of the queries' rows: largest magnitude, smallest that is not 0 less 1 (upper half)
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

// Four codes (a word) to four fp16 values (two words): exact, NaN kept.  3 clocks a
// pair (a warp on its SM quarter); to bf16, which has no such instruction, it takes 8
// clocks of logic a pair and more for NaN (below).  So the products are taken in
// fp16 wherever that is exact.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& a, uint32_t& b) {
  a = half2_of_codes(static_cast<uint16_t>(w));
  b = half2_of_codes(static_cast<uint16_t>(w >> 16));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
// The same to bf16, times 2^e with e in [-227, 7]: a code's exponent and fraction
// bits, put where bf16's lowest exponent and highest fraction bits are, read as its
// value times 2^-120; one product with 2^(120 + e).  The code of NaN would read as 480.
__device__ __forceinline__ void codes_bf16(uint32_t w, int e, uint32_t& a, uint32_t& b) {
  const uint32_t f = static_cast<uint32_t>(e + 247) << 7, scale = f | f << 16;
  auto pair = [&](uint32_t y) {  // codes in the halves' high bytes
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"((y >> 4 & 0x07f007f0u) | (y & 0x80008000u)), "r"(scale));
    const uint32_t nan = (y & 0x7f007f00u) + 0x01000100u;
    return d | (nan & 0x8000u ? 0x7fffu : 0u) | (nan & 0x80000000u ? 0x7fff0000u : 0u);
  };
  a = pair(__byte_perm(w, 0, 0x1404));
  b = pair(__byte_perm(w, 0, 0x3424));
}

// whether the condition holds in any of the 128 threads of softmax group 0 or 1, or
// (2) of the converters
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
__device__ __forceinline__ void tmem_load<8>(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
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
// One value of each of kCount columns a lane, reduced over the warp's 32 lanes in
// halves: log2 steps that each halve what a lane holds, until it holds the
// column `lane` (kCount 32) or, in lanes 2 c and 2 c + 1, column c (kCount 16).
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

// Weights are fp16 (mostly, with a bf16 cache too): log2 of the weight that a maximum
// gets when the reference is set at it, and of the largest one may reach before it is
// set again; small weights count down to 2^-24 minus the first.  bf16 results have
// three bits less, so three more rises are saved.
template <typename T>
constexpr float kQ8Top = std::is_same<T, __half>::value ? 7.f : 4.f;
constexpr float kQ8Most = 15.f;

// Scores in TMEM, rounded, less their references, over the factor (off by 2^-23 of the
// difference): a reference of 0 then gives their weights.
inline __device__ __noinline__ void far_scores(uint32_t tm, int columns, float scale, const float* ref) {
  float less;
  asm("rcp.approx.f32 %0, %1;" : "=f"(less) : "f"(scale));
#pragma unroll 1
  for (int c = 0; c < columns; c += 8) {
    uint32_t s[8];
    tmem_load<8>(tm + c, s);
#pragma unroll
    for (int x = 0; x < 8; ++x)
      s[x] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(s[x]), scale), ref[c + x]) * less);
    tmem_st8(tm + c, s);
  }
  tmem_st_wait();
}

template <typename T, int D>
struct Q8Softmax {
  const Attend8Params& p;
  Q8Shared<D>& sh;
  uint8_t* pbuf;
  uint32_t tmem;
  int g, quad, lane, key;
  bool ok;
  uint32_t next;   // 1 + the last tile that this group had
  uint32_t meets;  // parts in which the groups met
  int q_exp;       // log2 of the unit of the part's queries

  __device__ __forceinline__ uint32_t lanes() const { return static_cast<uint32_t>(quad * 32) << 16; }
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.batch.status, kWaitLimitCycles));
  }

  // The last product of this group's weights is complete.  (Its barrier's next
  // phase needs weights that this group has not written, or follows a part that
  // it has not ended.)
  __device__ __forceinline__ bool products_done() const { return wait(&sh.pv_done[(next - 1) & 1], ((next - 1) >> 1) & 1); }

  // Which of C columns from col0 on see this thread's key of tile t, bit by column.
  // (Loops that are not unrolled here and below: code that runs once a part or
  // less, unrolled, made the kernel 580 KB, and it ran at the rate of its
  // instruction fetches.)
  __device__ __forceinline__ uint64_t seen(const AtPart& a, int t, int col0, int C) const {
    const int e = t * kAtTile + key;  // the entry
    if (e >= a.len) return 0;
    if (e < a.old) return ~0ull;
    const int j = e - a.old;  // its place among the new ones
    uint64_t bits = 0;
    const int last = min(a.n0, (col0 + C - 1) / p.group + 1);
#pragma unroll 1
    for (int tok = col0 / p.group; tok < last; ++tok) {
      bool sees;
      if (p.draft_mask == nullptr)
        sees = j <= a.first - a.seq_first + tok;
      else
        sees = j < 64 && in_bounds(a.first >= 0 && a.first + tok < p.batch.N, p.batch.status) &&
               (p.draft_mask[a.first + tok] >> j & 1) != 0;
      if (!sees) continue;
      const int from = max(tok * p.group - col0, 0), to = min((tok + 1) * p.group - col0, C);  // its columns
      bits |= (to - from == 64 ? ~0ull : (1ull << (to - from)) - 1) << from;
    }
    return bits;
  }

  // A group's place for its warps' maxima and sums of the columns: where its weights
  // are, between the products that read them.
  __device__ __forceinline__ float* cross(int group, int i) const {
    return reinterpret_cast<float*>(pbuf + group * (kQ8PBytes / 2)) + i * (kAtTile / 2);
  }

  // The columns that reduce_columns left in this lane to the group's place.
  template <int C>
  __device__ __forceinline__ void to_cross(int c0, const float (&v)[C]) const {
    float* const at = cross(g, quad) + c0;
    if (C == 32)
      at[lane] = v[0];
    else if ((lane & 1) == 0)
      at[lane / 2] = v[0];
  }

  // The place of row `col` of the part among the parts' rows (times 1: of m and l,
  // times D: of its output), or -1.
  __device__ __forceinline__ int64_t place(const AtPart& a, int rows, int col) const {
    if (col >= rows) return -1;
    if (a.t0 != 0) {
      const int cta = static_cast<int>(blockIdx.x);
      return in_bounds(cta < p.n_ctas && col < p.slab_rows, p.batch.status) ? static_cast<int64_t>(cta) * p.slab_rows + col : -1;
    }
    const int tok = col / p.group;
    if (!in_bounds(a.first >= 0 && a.first + tok < p.batch.N, p.batch.status)) return -1;
    return p.place(a.line, static_cast<int64_t>(a.first + tok) * p.n_q_heads + a.head * p.group + (col - tok * p.group));
  }
  __device__ __forceinline__ void store_ml(const AtPart& a, int64_t at, int col, float m, float l) const {
    if (at < 0) return;
    (a.t0 == 0 ? p.part_ml : p.slab_ml)[at] = make_float2(m, l);
    if (a.t0 == 0) p.part_meta[at] = row_item(a, static_cast<int>(blockIdx.x), col);
  }

  // A part, C columns a thread.  Wide: the groups share each tile, group g has
  // columns g C .. g C + C - 1.  Otherwise they alternate tiles, each with all
  // columns, a reference, sums and an O of its own, joined at the end, so that
  // their chains of scores, weights and products overlap.  `base`: tiles before it.
  template <int C, bool kWide>
  __device__ __forceinline__ void part(const AtPart& a, uint32_t base) {
    constexpr float kTop = kQ8Top<T>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int kStep = kWide ? 1 : 2;
    constexpr int kChunk = C < 32 ? C : 32;  // columns read from TMEM at a time
    float* const neg_ref = sh.neg_ref[g];
    float* const c0s = cross(g, 0);
    float* const c1s = cross(g, 1);
    float* const c2s = cross(g, 2);
    float* const c3s = cross(g, 3);
    uint8_t* const pt = pbuf + g * (kQ8PBytes / 2) + key * 128;
    const uint32_t tm_o = tmem + 256 + 64 * g + lanes();
    const int col0 = kWide ? g * C : 0;
    const int mine = quad * 32 + lane;  // this thread's column in what is done once a column
    const int tiles = a.t1 - a.t0, rows = a.n0 * p.group;
    // entries below this one are seen by all rows
    const int open = a.line == 0 ? a.len : p.draft_mask != nullptr ? a.old : a.old + (a.first - a.seq_first) + 1;
    if (mine < C) neg_ref[mine] = sh.ref[g][mine] = kQ8Unset;
    if (mine == 0) {
      sh.far[g] = -INFINITY;
      sh.columns[g] = rows - col0;
    }
    uint64_t l2[C / 2];
#pragma unroll
    for (int c = 0; c < C / 2; ++c) l2[c] = 0;
    group_any(g, false);
    int unit = 0;  // log2 of the unit of O
    const float q_scale = p.scale_log2 * two_to(q_exp);
    const int i0 = kWide ? 0 : static_cast<int>((base & 1) ^ g);  // tile j is in S buffer j & 1
#pragma unroll 1
    for (int i = i0; i < tiles; i += kStep) {
      const uint32_t j = base + i;
      const uint32_t tm_s = tmem + 128 * (j & 1) + col0 + lanes();
      const int t = a.t0 + i;
      ok = wait(&sh.s_full[j & 1], (j >> 1) & 1) && ok;
      tc_fence_after();
      // this key's scale (its converter's write came before its product)
      // Neither 0 nor infinite: a hidden score (-infinity) times 0 or a score of 0 times
      // infinity would be NaN.  (What is raised to 2^-126 has scores below 2^-90.)
      const float scale = fminf(fmaxf(q_scale * two_to(sh.key_exp[j & 3][key >> 3]), kQ8LeastFactor), kQ8MostFactor);
      const uint64_t scale2 = f32x2(scale, scale);
      const bool ragged = open - t * kAtTile < kAtTile;
      uint64_t bits = ~0ull;
      if (ragged) bits = seen(a, t, col0, C);
      auto scores = [&](int c0, uint32_t (&s)[kChunk]) {
        tmem_load<kChunk>(tm_s + c0, s);
        if (ragged) {
          const uint32_t see = static_cast<uint32_t>(bits >> c0);
#pragma unroll
          for (int c = 0; c < kChunk; ++c) s[c] = see >> c & 1 ? s[c] : 0xff800000u;
        }
      };
      float e[C];  // weights
      bool waited = next == 0, wide = false;
      // Weights by the references as they are.  If one is too large (or the unit of
      // the values changed) the references are set anew, and once more.
#pragma unroll 1
      for (int turn = 0;; ++turn) {
        float over[2] = {sh.far[g], -INFINITY};
#pragma unroll
        for (int c0 = 0; c0 < C; c0 += kChunk) {
          uint32_t s[kChunk];
          scores(c0, s);
#pragma unroll
          for (int c = 0; c < kChunk; c += 4) {
            const ulonglong2 n = *reinterpret_cast<const ulonglong2*>(neg_ref + c0 + c);
            float x[4];
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), scale2, n.x), x[0], x[1]);
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), scale2, n.y), x[2], x[3]);
            over[0] = max3(over[0], x[0], x[1]);
            over[1] = max3(over[1], x[2], x[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) e[c0 + c + k] = ex2(x[k]);
          }
        }
        int now = unit;
        if (kBf16 && turn == 0) {  // the tile's values: their unit and type
          ok = wait(&sh.vc_full[j & 1], (j >> 1) & 1) && ok;
          now = sh.v_unit[j & 1];
          wide = sh.v_wide[j & 1] != 0;
          if (i == i0) unit = now;
        }
        if (!group_any(g, fmaxf(over[0], over[1]) > kQ8Most || now != unit || !ok)) break;
        if (turn > 1) break;  // (far, or scores that are not finite: the references are right after one turn)
        // (O may be multiplied: the last product into it is complete)
        if (ok && !waited) ok = products_done();
        waited = true;
        if (group_any(g, !ok)) {
          ok = false;
          return;
        }
        tc_fence_after();
#pragma unroll 1
        for (int c0 = 0; c0 < C; c0 += kChunk) {
          uint32_t s[kChunk];
          float top[kChunk];
          scores(c0, s);
#pragma unroll
          for (int c = 0; c < kChunk; ++c) top[c] = __uint_as_float(s[c]) * scale;
          reduce_columns<kChunk>(top, lane, [](float x, float y) { return fmaxf(x, y); });
          to_cross<kChunk>(c0, top);
        }
        group_any(g, false);
        if (mine < C) {
          const float m = fmaxf(max3(c0s[mine], c1s[mine], c2s[mine]), c3s[mine]);
          const float n = sh.ref[g][mine];
          const bool up = m + n > kQ8Most;
          c0s[mine] = up ? ex2(kTop - (m + n)) : 1.f;  // (0 at a row's first keys)
          if (up) neg_ref[mine] = sh.ref[g][mine] = kTop - m;
          if (mine < sh.columns[g] && m > -INFINITY && fabsf(m) >= Attend8Params::kFar) sh.far[g] = INFINITY;
        }
        group_any(g, false);
        if (sh.far[g] > 0.f) {
          far_scores(tm_s, C, scale, sh.ref[g]);
          if (mine < C) neg_ref[mine] = 0.f;
          turn = 1;
        }
        if (i > i0) {
#pragma unroll
          for (int c = 0; c < C / 2; ++c) {
            float x, y;
            f32x2_split(l2[c], x, y);
            l2[c] = f32x2(x * c0s[2 * c], y * c0s[2 * c + 1]);
          }
          if (D == 128 || quad < 2) {
            // (units may be 2^220 apart: two steps, each a normal number)
            const float units = two_to(max(unit - now, -126)), more = two_to(min(unit - now + 126, 0));
#pragma unroll 1
            for (int c = 0; c < C; c += 16) {
              uint32_t o[16];
              tmem_load<16>(tm_o + c, o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * c0s[c + x] * units * more);
              tmem_st16(tm_o + c, o);
            }
            tmem_st_wait();
          }
        }
        unit = now;
        group_any(g, false);  // the maxima's place may be written again
      }
      if (!waited) ok = products_done() && ok;
      // the sums keep the weights in 32 bits, P ([key][64 rows], 128-byte swizzle)
      // in 16 (half a step off at most)
#pragma unroll
      for (int c = 0; c < C / 2; ++c) l2[c] = add_f32x2(l2[c], f32x2(e[2 * c], e[2 * c + 1]));
      auto put = [&](auto type) {
        using W = decltype(type);
#pragma unroll
        for (int c = 0; c < C; c += 8)
          *reinterpret_cast<uint4*>(pt + ((c / 8 ^ (key & 7)) << 4)) =
              make_uint4(Pack16<W>::pack(e[c], e[c + 1]), Pack16<W>::pack(e[c + 2], e[c + 3]),
                         Pack16<W>::pack(e[c + 4], e[c + 5]), Pack16<W>::pack(e[c + 6], e[c + 7]));
      };
      if (kBf16 && wide)
        put(__nv_bfloat16());
      else
        put(__half());
      fence_async_shared();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[g]);
      next = j + 1;
    }

    // ---- the part's results ----
    if (next > 0) ok = products_done() && ok;
    if (group_any(g, !ok)) {
      ok = false;
      return;
    }
#pragma unroll
    for (int c0 = 0; c0 < C; c0 += kChunk) {
      float sum[kChunk];
#pragma unroll
      for (int c = 0; c < kChunk / 2; ++c) f32x2_split(l2[c0 / 2 + c], sum[2 * c], sum[2 * c + 1]);
      reduce_columns<kChunk>(sum, lane, [](float x, float y) { return x + y; });
      to_cross<kChunk>(c0, sum);
    }
    group_any(g, false);
    float l = 0.f;
    if (mine < C) l = (c0s[mine] + c1s[mine]) + (c2s[mine] + c3s[mine]);
    float* const out = (a.t0 == 0 ? p.part_o : p.slab_o) + quad * 32 + lane;
    const bool has_dims = D == 128 || quad < 2;
    int64_t* const places = reinterpret_cast<int64_t*>(c1s);  // of the columns that this group writes
    if (kWide) {
      group_any(g, false);  // all sums have been read
      if (mine < C) {
        places[mine] = place(a, rows, col0 + mine);
        store_ml(a, places[mine], col0 + mine, sh.ref[g][mine] == kQ8Unset ? -INFINITY : -sh.ref[g][mine], l);
      }
      group_any(g, false);
      tc_fence_after();
      if (has_dims) {
#pragma unroll 1
        for (int c = 0; c < C; c += 8) {
          uint32_t o[8];
          tmem_load<8>(tm_o + c, o);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (places[c + x] >= 0) out[places[c + x] * D] = __uint_as_float(o[x]) * two_to(unit);
        }
      }
      tc_fence_before();
      group_any(g, false);  // the places and the references may be written again
    } else {
      if (mine < C) c0s[mine] = l;
      if (mine == 0) sh.unit[g] = two_to(unit);
      // both groups' references, sums and products are there
      auto meet = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.meet[i]);
        return wait(&sh.meet[i], meets & 1);
      };
      ok = meet(0) && ok;
      if (group_any(g, !ok)) {
        ok = false;
        return;
      }
      tc_fence_after();
      // group g joins its half of the columns; a group without a tile has sums of 0
      constexpr int kHalf = C / 2;
      float* const factor = c3s;  // [2][kHalf]
      if (mine < kHalf) {
        const int c = g * kHalf + mine;
        const float n0 = sh.ref[0][c], n1 = sh.ref[1][c], m = fmaxf(-n0, -n1);
        const float f0 = n0 == kQ8Unset ? 0.f : ex2(-n0 - m), f1 = n1 == kQ8Unset ? 0.f : ex2(-n1 - m);
        // (a part of one tile has one O, in the group of its buffer: the other is not looked at)
        factor[mine] = tiles > 1 || (base & 1) == 0 ? f0 * sh.unit[0] : -1.f;
        factor[kHalf + mine] = tiles > 1 || (base & 1) != 0 ? f1 * sh.unit[1] : -1.f;
        places[mine] = place(a, rows, c);
        store_ml(a, places[mine], c, m == -kQ8Unset ? -INFINITY : m, cross(0, 0)[c] * f0 + cross(1, 0)[c] * f1);
      }
      group_any(g, false);
      if (has_dims) {
        const uint32_t from = tmem + 256 + lanes() + g * kHalf;
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 8) {
          uint32_t x0[8], x1[8];
          tmem_load<8>(from + c, x0);
          tmem_load<8>(from + 64 + c, x1);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            const float f0 = factor[c + x], f1 = factor[kHalf + c + x];
            float v = f0 < 0.f ? 0.f : __uint_as_float(x0[x]) * f0;
            if (f1 >= 0.f) v += __uint_as_float(x1[x]) * f1;
            if (places[c + x] >= 0) out[places[c + x] * D] = v;
          }
        }
      }
      tc_fence_before();
      ok = meet(1) && ok;  // the sums' places and the references may be written again
      ++meets;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.o_free);
  }
};

// columns of a part's products; above 64 the softmax groups share each tile
__device__ __forceinline__ int q8_columns(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

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
      mbar_init(&sh.vc_full[v], 4);
      mbar_init(&sh.s_full[v], 1);
      mbar_init(&sh.q_full[v], 1);
      mbar_init(&sh.q_empty[v], 1);
    }
    for (int i = 0; i < kQ8Queue; ++i) {
      mbar_init(&sh.part_full[i], 1);
      mbar_init(&sh.part_empty[i], 15);  // eight softmax warps, four converters, the issuer, the two loaders
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sh.p_full[g], 4);
      mbar_init(&sh.pv_done[g], 1);
      mbar_init(&sh.meet[g], 8);
      mbar_init(&sh.q_ready[g], 4);
    }
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
      a.fixed = fixed_weight<Attend8Params>(pl.tiles_alone * p.n_heads + own, p.n_ctas);
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
              a.t0 = tiles_before<Attend8Params>(lo, off, w, a.fixed, tiles);
              a.t1 = tiles_before<Attend8Params>(hi, off, w, a.fixed, tiles);
              off += item_weight<Attend8Params>(tiles, w, a.fixed);
              if (a.t0 >= a.t1) continue;
              // the part that the item's last tile begins in
              a.last = cta;
              if (a.t0 == 0 && a.t1 < tiles)
                a.last = static_cast<int>(((off - tile_weight<Attend8Params>(w) + 1) * p.n_ctas - 1) / total);
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
      uint32_t ph_p[2] = {0, 0};
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
        const int columns = q8_columns(__shfl_sync(0xffffffffu, sh.parts[q].n0, 0) * p.group);
        const bool wide = columns == 128;
        if (lane == 0) mbar_arrive(&sh.part_empty[q]);
        if (line < 0) break;
        if (!wait(kBf16 ? &sh.q_ready[n & 1] : &sh.q_full[n & 1], (n >> 1) & 1)) break;
        const uint32_t id_qk = idesc_f16_f32(kBf16 && __shfl_sync(0xffffffffu, static_cast<int>(sh.q_bf16[n & 1]), 0) != 0, false,
                                             kAtTile, columns);
        // A (the values) too has K over its rows
        const uint32_t id_pv = idesc_f16_f32(false, true, kAtTile, columns) | 1u << 15,
                       id_pv_bf16 = idesc_f16_f32(true, true, kAtTile, columns) | 1u << 15;
        // scores of the part's tile i
        auto qk = [&](int i) {
          const uint32_t j = base + i, b = j & 1;
          if (!wait(&sh.kc_full[b], (j >> 1) & 1)) return;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t bd = q_desc + (n & 1) * (kTileBytes >> 4);
#pragma unroll 1
            for (int k = 0; k < D / 16; ++k)
              tc_mma_ts(utm + 128 * b, utm + 384 + (D / 2) * b + 8 * k, bd + (k / 4) * (kHalfBytes >> 4) + (k % 4) * 2, id_qk, k > 0);
            tc_commit(&sh.s_full[b]);
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
          // the weights: of both groups, or of the one that has this tile
          if ((wide || b == 0) && !wait(&sh.p_full[0], ph_p[0]++ & 1)) break;
          if ((wide || b == 1) && !wait(&sh.p_full[1], ph_p[1]++ & 1)) break;
          tc_fence_after();
          const uint32_t id = kBf16 && __shfl_sync(0xffffffffu, static_cast<int>(sh.v_wide[b]), 0) != 0 ? id_pv_bf16 : id_pv;
          if (elect_one()) {
            const uint32_t g = wide ? 0 : b;
            const uint64_t ad = v_desc + b * (kTileBytes >> 4), bd = p_desc + g * (kQ8PBytes / 2 >> 4);
            const bool more = i >= (wide ? 1 : 2);
#pragma unroll 1
            for (int k = 0; k < kAtTile / 16; ++k)
              tc_mma(utm + 256 + 64 * g, ad + k * (2048 >> 4), bd + k * (2048 >> 4), id, more || k > 0);
            tc_commit(&sh.pv_done[b]);
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
      // The values' unit (bf16 caches): they are converted to fp16 as multiples of
      // 2^unit, exact for blocks whose exponents are within unit - 15 .. unit + 7.
      // It is the first tile's largest exponent and rises where one passes that range;
      // a tile with a block below it is converted to bf16 instead.  So are all tiles after
      // one of either kind: weights too small for fp16 may count there, since the ones that
      // the references were set at may stand before much smaller values.
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
        // (256: no scale, its keys are none)
        auto scale_of = [&](int i, int page) -> uint32_t {
          const uint32_t key = static_cast<uint32_t>(t0 + i) * kAtTile + my_key;
          return page < p.n_pages ? scales[p.c8.scale_at(page, static_cast<int>(key % page_size), head)] : 256;
        };
        int unit = 0;
        int low = -1000;  // tiles with a block below it have bf16 values (-1000: the unit is not set)
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
          const bool none = scale == 256 || lane >= 16;
          const int e = none ? 0 : stored_exponent<T>(scale);
          int wide = 0;
          if (kBf16 && values) {
            const int most = __reduce_max_sync(0xffffffffu, none ? -1000 : e), least = __reduce_min_sync(0xffffffffu, none ? 1000 : e);
            if (most > -1000 && (low == -1000 || most > unit + 7)) {
              low = low == -1000 ? most - 15 : 1000;
              unit = most;
            }
            wide = least < low;
            if (wide) low = 1000;
          }
          if (lane < 16) sh.scales[values][slot][lane] = static_cast<int8_t>(none && values ? unit : e);
          if (values && lane == 0) {
            sh.raw_unit[slot] = static_cast<int16_t>(unit);
            sh.raw_wide[slot] = static_cast<int8_t>(wide);
          }
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
    for (uint32_t n = 0;; ++n) {
      const int q = n % kQ8Queue;
      wait(&sh.part_full[q], (n / kQ8Queue) & 1);
      if (group_any(2, !ok)) break;
      const int line = sh.parts[q].line, t0 = sh.parts[q].t0, tiles = sh.parts[q].t1 - t0, len = sh.parts[q].len,
                rows = sh.parts[q].n0 * p.group, columns = q8_columns(rows);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.part_empty[q]);
      if (line < 0) break;
      bool k_bf16 = false;
      if (kBf16) {
        // The queries as fp16 times 2^unit: the largest gets 2^14 or more, and what has an
        // exponent up to 31 below its, 2^-17 or more, has bf16's 8 bits above fp16's last,
        // 2^-24.  With smaller ones (zeros are none), or any not finite, all stay bf16, and
        // so do the keys: either way the products are exact, whatever rows share the part.
        wait(&sh.q_full[n & 1], (n >> 1) & 1);
        uint8_t* const qt = qbuf + (n & 1) * kTileBytes;
        // of this thread's row, two values at a time: magnitudes with bit 15 set, the largest;
        // less 1 and signed, where zero is the largest, the smallest
        uint32_t top2 = 0, low2 = 0x7fff7fffu;
        if (ok && key < rows) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint4 w = *reinterpret_cast<const uint4*>(qt + (c / 8) * kHalfBytes + key * 128 + (((c % 8) ^ (key & 7)) << 4));
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t y = x[i] | 0x80008000u;
              top2 = __vmaxu2(top2, y);
              low2 = __vmins2(low2, y - 0x00010001u);
            }
          }
        }
        sh.row_ends[key] = __vmaxu2(top2 & 0x7fff7fffu, top2 >> 16 & 0x7fffu) & 0xffffu |
                           (__vmins2(low2, low2 >> 16 | low2 << 16) ^ 0x80008000u) << 16;
        if (group_any(2, !ok)) break;
        uint32_t most = 0, least = 0xffff;
#pragma unroll
        for (int r = 0; r < kAtTile; r += 32) {
          const uint32_t x = sh.row_ends[r + lane];
          most = max(most, x & 0xffffu);
          least = min(least, x >> 16);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        least = __reduce_min_sync(0xffffffffu, least);
        k_bf16 = most >= 0x7f80u || (least + 1 >> 7) + 31 < (most >> 7);
        const int e = most == 0 || k_bf16 ? 0 : max(static_cast<int>(most >> 7) - 127 - 14, -120);
        if (!k_bf16) {
          const float f = two_to(-e);
          for (int x = key; x < columns * 8 * kHalves; x += 128) {
            uint4* const at = reinterpret_cast<uint4*>(qt + (x / (columns * 8)) * kHalfBytes + (x % (columns * 8)) * 16);
            float v[8];
            unpack8<__nv_bfloat16>(*at, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= f;
            *at = pack8<__half>(v);
          }
        }
        if (key == 0) {
          sh.q_exp[n & 1] = static_cast<int16_t>(e);
          sh.q_bf16[n & 1] = k_bf16;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_ready[n & 1]);
      }
#pragma unroll 1
      for (int i = 0; i < tiles && ok; ++i) {
        const uint32_t j = base + i, b = j & 1, slot = j % kSlots, use = j / kSlots;
        // keys, to TMEM: the codes' values, their scales count in the scores
        if (!wait(&sh.raw_full[0][slot], use & 1)) break;
        if (j >= 2 && !wait(&sh.s_full[b], ((j >> 1) & 1) ^ 1)) break;
        tc_fence_after();
        {
          const uint8_t* const tile = ring + slot * kRawBytes;
          const uint32_t dst = tmem + lanes + 384 + (D / 2) * b;
          if ((lane & 7) == 0) sh.key_exp[j & 3][key >> 3] = sh.scales[0][slot][key >> 3];
          if (!kBf16 || !k_bf16) {
#pragma unroll 1
            for (int c = 0; c < D / 16; c += 4) {
              uint32_t d[32];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint4 w = codes(tile, c + x);
                codes_f16(w.x, d[8 * x], d[8 * x + 1]);
                codes_f16(w.y, d[8 * x + 2], d[8 * x + 3]);
                codes_f16(w.z, d[8 * x + 4], d[8 * x + 5]);
                codes_f16(w.w, d[8 * x + 6], d[8 * x + 7]);
              }
              tmem_st32(dst + 8 * c, d);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              const uint4 x = codes(tile, c);
              uint32_t d[8];
              codes_bf16(x.x, 0, d[0], d[1]);
              codes_bf16(x.y, 0, d[2], d[3]);
              codes_bf16(x.z, 0, d[4], d[5]);
              codes_bf16(x.w, 0, d[6], d[7]);
              tmem_st8(dst + 8 * c, d);
            }
          }
          tmem_st_wait();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.kc_full[b]);
          mbar_arrive(&sh.raw_empty[0][slot]);
        }
        // values, to a swizzled tile, as multiples of their unit; past the last entry
        // zeros (zero times what stands there must be zero)
        if (!wait(&sh.raw_full[1][slot], use & 1)) break;
        if (j >= 2 && !wait(&sh.pv_done[b], ((j >> 1) & 1) ^ 1)) break;
        {
          const uint8_t* const tile = ring + (kSlots + slot) * kRawBytes;
          const int e = sh.scales[1][slot][key >> 3] - sh.raw_unit[slot];
          const bool live = (t0 + i) * kAtTile + key < len, wide = sh.raw_wide[slot] != 0;
          uint8_t* const dst = vbuf + b * kTileBytes + key * 128;
          // 8 dims: one 16-byte vector
          auto put = [&](int at, const uint32_t* d) {
            *reinterpret_cast<uint4*>(dst + (at / 8) * kHalfBytes + (((at % 8) ^ (key & 7)) << 4)) = make_uint4(d[0], d[1], d[2], d[3]);
          };
          if (!kBf16 || !wide) {
            const __half2 h = __float2half2_rn(two_to(e));  // e: -15 .. 8
            const uint32_t scale = *reinterpret_cast<const uint32_t*>(&h);
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              const uint4 w = live ? codes(tile, c) : make_uint4(0, 0, 0, 0);
              uint32_t d[8];
              codes_f16(w.x, d[0], d[1]);
              codes_f16(w.y, d[2], d[3]);
              codes_f16(w.z, d[4], d[5]);
              codes_f16(w.w, d[6], d[7]);
#pragma unroll
              for (int x = 0; x < 8; ++x) d[x] = mul_f16x2(d[x], scale);
              put(2 * c, d);
              put(2 * c + 1, d + 4);
            }
          } else {
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              const uint4 x = live ? codes(tile, c) : make_uint4(0, 0, 0, 0);
              uint32_t d[8];
              codes_bf16(x.x, e, d[0], d[1]);
              codes_bf16(x.y, e, d[2], d[3]);
              codes_bf16(x.z, e, d[4], d[5]);
              codes_bf16(x.w, e, d[6], d[7]);
              put(2 * c, d);
              put(2 * c + 1, d + 4);
            }
          }
          if (key == 0) {
            sh.v_unit[b] = sh.raw_unit[slot];
            sh.v_wide[b] = sh.raw_wide[slot];
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
    Q8Softmax<T, D> sm = {p, sh, pbuf, tmem, warp >> 2, warp & 3, lane, (warp & 3) * 32 + lane, true, 0, 0, 0};
    uint32_t base = 0;
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
      const int q = n % kQ8Queue;
      sm.ok = sm.wait(&sh.part_full[q], (n / kQ8Queue) & 1) && sm.ok;
      if (group_any(sm.g, !sm.ok)) break;
      const AtPart a = sh.parts[q];
      if (a.line < 0) break;
      if (kBf16) {
        // (before the part's place is free: the queries of the part after the next
        // complete the next phase of this barrier)
        sm.ok = sm.wait(&sh.q_ready[n & 1], (n >> 1) & 1) && sm.ok;
        sm.q_exp = sh.q_exp[n & 1];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.part_empty[q]);
      const int columns = q8_columns(a.n0 * p.group);
      if (columns == 16)
        sm.template part<16, false>(a, base);
      else if (columns == 32)
        sm.template part<32, false>(a, base);
      else if (columns == 64)
        sm.template part<64, false>(a, base);
      else
        sm.template part<64, true>(a, base);
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
