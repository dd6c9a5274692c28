// attend.cuh — attention of the new positions over a shared prefix and their
// sequences' pages, on the tcgen05 tensor cores.
//
// Work.  The rows of one key head are its (position, query head) pairs.  Over
// the prefix the rows of the whole batch are one matrix, so the prefix's keys
// and values are read once per row block and not once per sequence; over the
// sequences' own pages the rows of one sequence are.  An item is a block of
// up to two row tiles (128 rows each: whole positions) against all tiles of
// 128 keys that its rows see.  The items' key tiles, weighted by what they
// cost, form one line, the prefix's items first, and CTA c takes its c-th equal
// part: lengths are read on the device, so nothing is planned on the host, and
// one sequence or one head fills the GPU as well as many.  CTAs bound by the
// tensor cores (prefix) and CTAs bound by HBM (own pages) run side by side.
//
// A part of an item leaves, per row, the unnormalised output, its reference
// exponent m and the sum l: O = sum_t 2^(s_t - m) v_t, l = sum_t 2^(s_t - m)
// with s in units of log2.  The part that holds an item's first tile writes to
// the row's own place, any other to its CTA's slab (it is the CTA's first
// part); attend_join_kernel adds a row's parts in a fixed order, so results do
// not depend on timing.
//
// One CTA per SM:
//   warps 0-3, 4-7  softmax groups 0 and 1, one thread a row.  With two row
//                   tiles group g has tile g and both read each key tile; with
//                   one, the groups share its rows and alternate key tiles
//                   (their halves are joined at the end of the part), so that
//                   exponentials of one overlap products of the other.
//   warp 8          the scheduler: finds the CTA's parts, queues them for the
//                   others and loads their queries (TMA).
//   warp 9          issues the products: S = Q K^T (both operands
//                   from shared memory) and O += P V (P from TMEM, where the
//                   softmax group wrote it over S; V's rows are K).
//   warps 10, 11    load key and value tiles into a ring (TMA, one box per run
//                   of a page and 64 dims).
// TMEM: S0 S1 (128 columns each) and O0 O1 (D columns each).
//
// The reference m of a row rises only when a tile's maximum passes the one it
// was set at by more than 2^8, and only then is O (in TMEM) multiplied; weights
// stay below 2^8, fp16's (which begin higher) below 2^15; l and O are exact with
// respect to any m.  A NaN score raises no maximum (m may
// stay -inf) but makes l and O NaN, and so does an infinite one (inf - inf):
// l, not m, tells a row that saw nothing, by l = 0.
//
// What bounds it.  Own pages: HBM (16 caches of up to 32,768 entries, 944 MB:
// 150 us, 6.3 TB/s, 0.93 of the measured copy bandwidth).  Prefix: the chain of
// a key tile, scores -> weights (some 1,700 clocks: 128 columns from TMEM, their
// maximum, 128 exponentials at 8 a clock per SM quarter, the stores) -> O and the
// next scores (1,024 clocks of products).  P takes the place of S, so a group's
// chain is serial; the two groups overlap and take 3,250 clocks a tile where
// the products alone take 2,048 (B = 128, prefix 32,768: 366 to 387 us on five
// boxes, 0.92 to 0.97 PFLOP/s of the pairs that exist).  A softmax thread holds
// 128 scores: 100 bytes a thread spill at D = 128, 52 at D = 64.  Tried and not kept: 64-key steps with two score
// buffers (scores of 64 keys cost 48 clocks an instruction against 64 for 128:
// 474 us then against 435), halves of a row in two threads (701), the first 64
// keys' weights announced early (no change), an issuer per group (432: products
// of both groups interleave and each group's finish later).
#pragma once

#include <type_traits>

#include "kvappend.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace specv {

constexpr int kAtTile = 128;        // rows of a row tile, keys of a key tile
constexpr int kAtThreads = 384;     // three warpgroups
// Registers: the launch gives 168 a thread (65,536 / 384, by 8); the softmax
// groups hold a row's 128 scores and take 216, the third warpgroup keeps 72:
// 216 + 216 + 72 = 3 x 168.
constexpr int kAtSoftmaxRegs = 216, kAtOtherRegs = 72;
constexpr int kAtRingBytes = 160 * 1024;
constexpr int kAtMaxCtas = 160;     // slabs in the workspace
constexpr int kAtQueue = 4;         // parts queued ahead
constexpr int kAtFixed = 15;        // weight of a part's fixed cost
constexpr float kAtRise = 8.f;      // log2 of how far a row's maximum may pass the one its reference was set at
// log2 of the weight that a maximum gets when the reference is set at it.  fp16
// weights reach 2^15 of the 65,504 that the type holds: below 2^-14 they lose
// bits, below 2^-25 all, so the higher they stand the longer the tail that counts
// (8,192 keys of 2^-25.5 of the largest weight each, values 2,048 times the
// largest's: 1.18 for 1.35 with 0 here).  bf16 has fp32's exponents.
template <typename T>
constexpr float kAtTop = std::is_same<T, __half>::value ? 7.f : 0.f;

struct AttendParams {
  CUtensorMap tmK, tmV;  // [page, head, slot, dim], boxes of 64 dims x box_rows slots
  CUtensorMap tmQ;       // [position, head, dim], boxes of 64 dims x group heads x tok_tile positions
  uint16_t* out;
  int64_t o_ps, o_hs;
  float* lse;
  PagedBatch batch;
  int n_pages, box_rows;
  const int32_t* prefix_table;
  int prefix_len;
  int slab_rows;     // rows of a block, at most
  const uint64_t* draft_mask;
  float scale_log2;  // scale * log2(e)
  int n_q_heads, n_heads, group;
  int tok_tile;      // positions of a row tile: 128 / group
  int n_ctas;
  int64_t* begin;    // [n_ctas + 1] where the CTAs' parts begin
  // rows' own places: [0] for the prefix, if there is one, then for their
  // sequences' pages
  int4* part_meta;   // [1 or 2][N * n_q_heads] RowItem of each row
  float* part_o;     // [1 or 2][N * n_q_heads][D]
  float2* part_ml;   // [1 or 2][N * n_q_heads]
  float* slab_o;     // [n_ctas][slab_rows][D]
  float2* slab_ml;   // [n_ctas][slab_rows]
  // the queries and the cache as they are, for rows that are summed again (last:
  // nothing else reads here)
  const uint16_t* q;
  int64_t q_ps, q_hs;
  PagedView cache;

  // a row's index in part_* (row: of [N * n_q_heads])
  __device__ __forceinline__ int64_t place(int line, int64_t row) const {
    return line == 1 && prefix_len > 0 ? static_cast<int64_t>(batch.N) * n_q_heads + row : row;
  }
};

// ---------------------------------------------------------------------------
// the line of work
// ---------------------------------------------------------------------------
__device__ __forceinline__ int new_positions(const PagedBatch& p) {
  return min(max(p.q_indptr[p.B], 0), p.N);
}

// Key tiles that row block rb of a sequence sees.
__device__ __forceinline__ int block_tiles(const AttendParams& p, const SeqSpan& s, int rb) {
  const int kv = static_cast<int>(s.kv);
  const int64_t last = p.draft_mask != nullptr
                           ? kv
                           : static_cast<int64_t>(kv) - s.n + min(static_cast<int64_t>(s.n), static_cast<int64_t>(rb + 1) * 2 * p.tok_tile);
  return last <= 0 ? 0 : static_cast<int>((last + kAtTile - 1) / kAtTile);
}

// Row tiles of a block.
__device__ __forceinline__ int block_rows(int positions, int tok_tile, int rb) {
  return positions - rb * 2 * tok_tile > tok_tile ? 2 : 1;
}

// Weights are in units of some 400 clocks: a key tile took 3,250 with two row
// tiles and 2,000 with one.  A part's queries, first scores and results took
// some 6,000: an item weighs that much more, all on its first tile, where the
// CTAs have several tiles each; where they have few the tiles alone are dealt
// out, which uses more CTAs (candidates_d64: 28 us against 31.5).
__device__ __forceinline__ int tile_weight(int row_tiles) { return row_tiles == 2 ? 8 : 5; }
__device__ __forceinline__ int fixed_weight(int64_t tiles_alone, int n_ctas) {
  return tiles_alone < 30LL * n_ctas ? 0 : kAtFixed;
}
__device__ __forceinline__ int64_t item_weight(int tiles, int row_tiles, int fixed) {
  return tiles == 0 ? 0 : static_cast<int64_t>(tiles) * tile_weight(row_tiles) + fixed;
}

// One key head's items of a sequence: the weight of their tiles alone, and how
// many there are.
struct SeqWeight {
  int64_t tiles_alone;
  int items;
  __device__ __forceinline__ int64_t per_head(int fixed) const { return tiles_alone + static_cast<int64_t>(items) * fixed; }
};
__device__ __forceinline__ SeqWeight seq_weight(const AttendParams& p, const SeqSpan& s) {
  SeqWeight w = {0, 0};
  for (int rb = 0; rb * 2 * p.tok_tile < s.n; ++rb) {
    const int tiles = block_tiles(p, s, rb);
    w.tiles_alone += static_cast<int64_t>(tiles) * tile_weight(block_rows(s.n, p.tok_tile, rb));
    w.items += tiles > 0;
  }
  return w;
}

// The rows of the blocks that see no key at all (fewer entries than new
// positions, which the status word reports): the join finds no parts there.
__device__ __noinline__ void no_tiles(const AttendParams& p, const SeqSpan& s) {
  for (int i = 0; i < s.n; ++i) {
    if (block_tiles(p, s, i / (2 * p.tok_tile)) > 0) continue;
    for (int h = 0; h < p.n_q_heads; ++h)
      if (in_bounds(s.first >= 0 && s.first + i < p.batch.N, p.batch.status))
        p.part_meta[p.place(1, static_cast<int64_t>(s.first + i) * p.n_q_heads + h)] = make_int4(-1, 0, 0, 0);
  }
}

// The prefix's items: the same for each head.
struct PrefixItems {
  int positions, blocks, tiles;
  int64_t tiles_alone;  // weight of one head's, without fixed cost
  __device__ __forceinline__ int64_t per_head(int fixed) const {
    return tiles == 0 ? 0 : tiles_alone + static_cast<int64_t>(blocks) * fixed;
  }
};
__device__ __forceinline__ PrefixItems prefix_items(const AttendParams& p) {
  PrefixItems L;
  L.positions = new_positions(p.batch);
  L.tiles = (p.prefix_len + kAtTile - 1) / kAtTile;
  L.blocks = (L.positions + 2 * p.tok_tile - 1) / (2 * p.tok_tile);
  L.tiles_alone = L.blocks == 0 ? 0
                                : static_cast<int64_t>(L.tiles) *
                                      ((L.blocks - 1) * tile_weight(2) +
                                       tile_weight(block_rows(L.positions, p.tok_tile, L.blocks - 1)));
  return L;
}

// Part c of n of the line of weight W begins at W * c / n; tiles belong to the
// part that their first unit of weight lies in.  (The 64-bit division takes
// some hundred clocks, before the first load of a CTA.)
__device__ __forceinline__ int64_t part_begin(int64_t W, int c, int n) {
  if (W < (1 << 24)) return static_cast<uint32_t>(W) * static_cast<uint32_t>(c) / static_cast<uint32_t>(n);  // n <= 160
  return W * c / n;
}
// Tile t of an item begins at its `off` (t = 0) or at off + fixed + t * weight:
// the tiles that begin before x.
__device__ __forceinline__ int tiles_before(int64_t x, int64_t off, int row_tiles, int fixed, int tiles) {
  if (x <= off || tiles == 0) return 0;
  const int64_t y = x - off - fixed;
  if (y <= 0) return 1;
  if (y >= static_cast<int64_t>(tiles) * 8) return tiles;
  const uint32_t z = static_cast<uint32_t>(y);
  const int t = static_cast<int>(row_tiles == 2 ? (z + 7) / 8 : (z + 4) / 5);
  return min(t, tiles);
}

// A part of an item, as the scheduler queues it.
struct AtPart {
  int64_t off;        // the item's place in the line
  int tiles, w;       // all its key tiles, its row tiles
  int fixed;          // the fixed cost that counts in the line
  int last;           // for the part with the first tile: the last part that holds any
  int line;           // 0 prefix, 1 own pages, -1 no more
  int head, first;    // key head, first position
  int n0, n1;         // positions of the two row tiles (n1 = 0: one tile)
  int t0, t1;         // key tiles
  int len, old;       // entries, entries older than the new positions
  int seq_first, seq_n;
  int seq;
};

// What the join needs of a row's item, written with the item's first tile:
// x: the parts that hold its first and last tile, and the row's place in their
// slabs (8 bits each), or -1: no tiles.  y: 4 * tiles, 2 where the fixed cost counts, row tiles - 1.
// z, w: the item's place in the line.
__device__ __forceinline__ int4 row_item(const AtPart& a, int part, int slab_row) {
  return make_int4(part | a.last << 8 | slab_row << 16, 4 * a.tiles + (a.fixed > 0 ? 2 : 0) + a.w - 1, static_cast<int>(a.off),
                   static_cast<int>(a.off >> 32));
}


__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// two fp32 operations at once
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// 32-byte global store (eight fp32; the address 32-byte aligned)
__device__ __forceinline__ void st_global_f8(float* q, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(q), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// ---------------------------------------------------------------------------
// kernel
// ---------------------------------------------------------------------------
// What follows the query tiles and the ring in shared memory.
template <int kSlots>
struct AtShared {
  uint64_t kv_full[kSlots], kv_empty[kSlots], part_full[kAtQueue], part_empty[kAtQueue];
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], meet[2], done;
  float2 xch[2][kAtTile];  // the groups' (m, l)
  AtPart parts[kAtQueue];
  uint32_t tmem;
};
template <int D>
constexpr int kAtSlots = kAtRingBytes / (kAtTile * D * 2);
static_assert(kAtSlots<128> >= 5 && kAtSlots<64> >= 5, "the loaders' waits count on it");
template <int D>
constexpr uint32_t at_smem_bytes() {
  return 2u * kAtTile * D * 2 + kAtRingBytes + sizeof(AtShared<kAtSlots<D>>);
}
static_assert(at_smem_bytes<128>() <= 227 * 1024, "one CTA's shared memory");

template <typename T, int D>
__global__ void __launch_bounds__(kAtThreads, 1) attend_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kHalves = D / 64;                       // 64-dim halves of a tile
  constexpr uint32_t kHalfBytes = kAtTile * 128;        // 16 KB
  constexpr uint32_t kTileBytes = kHalves * kHalfBytes;
  constexpr int kSlots = kAtSlots<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  // no static shared memory: the swizzled tiles begin at its (1024-byte aligned) start
  extern __shared__ __align__(1024) uint8_t at_smem[];
  uint8_t* const qbuf = at_smem;                   // [2] query tiles
  uint8_t* const ring = at_smem + 2 * kTileBytes;  // [kSlots] key and value tiles
  AtShared<kSlots>& sh = *reinterpret_cast<AtShared<kSlots>*>(ring + kAtRingBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const status = p.batch.status;
  const int cta = static_cast<int>(blockIdx.x);
  grid_dep_launch();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sh.kv_full[i], 1);
      mbar_init(&sh.kv_empty[i], 1);
    }
    for (int i = 0; i < kAtQueue; ++i) {
      mbar_init(&sh.part_full[i], 1);
      mbar_init(&sh.part_empty[i], 11);  // eight softmax warps, the issuer, the two loaders
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sh.q_full[g], 1);
      mbar_init(&sh.q_empty[g], 1);
      mbar_init(&sh.s_full[g], 1);
      mbar_init(&sh.p_full[g], 4);
      mbar_init(&sh.o_full[g], 1);
      mbar_init(&sh.meet[g], 8);
    }
    mbar_init(&sh.done, 1);
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  grid_dep_wait();
  auto tm_s = [&](int g) { return tmem + 128 * g; };
  auto tm_o = [&](int g) { return tmem + 256 + D * g; };
  if (warp >= 8) {
    regs_down<kAtOtherRegs>();
    if (warp == 8) {
      // ---------------- scheduler (the whole warp): parts, and their queries ----------------
      const PrefixItems pl = prefix_items(p);
      int queued = 0;
      uint32_t q_loads[2] = {0, 0};
      bool ok = true;
      // The queries of a part whose first positions are `first`: row tile g of
      // two, or (-1) none for a group without key tiles.
      auto load_queries = [&](int head, int first0, int first1) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int first = g == 0 ? first0 : first1;
          if (first < 0) continue;
          if (q_loads[g] > 0)
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&sh.q_empty[g], (q_loads[g] & 1) ^ 1, status, kWaitLimitCycles));
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[g], kHalves * 128u * p.group * p.tok_tile);
          __syncwarp();
          // (tiled copies stay inside their tensor by themselves: recorded only)
          in_bounds(first >= 0 && first < p.batch.N && (head + 1) * p.group <= p.n_q_heads, status);
          if (lane < kHalves)
            tma_load_3d(smem_u32(qbuf) + g * kTileBytes + lane * kHalfBytes, &p.tmQ, lane * 64, head * p.group, first,
                        &sh.q_full[g]);
          ++q_loads[g];
        }
      };
      // After the first part the queries come one part behind the queue: their
      // buffers come free late, and the key and value loads need not wait.
      int late_head = 0, late0 = -1, late1 = -1;
      // a free place of the queue
      auto queue_place = [&]() {
        const int q = queued % kAtQueue;
        if (queued >= kAtQueue)
          ok = ok && mbar_wait(&sh.part_empty[q], ((queued / kAtQueue) & 1) ^ 1, status, kWaitLimitCycles);
        ok = __all_sync(0xffffffffu, ok);
        ++queued;
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
      if (ok && lane == 0 && in_bounds(cta < p.n_ctas, status)) {
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
            for (int at = 0; at < s.n && ok; at += 2 * p.tok_tile) {
              const int rb = at / (2 * p.tok_tile);
              const int tiles = a.line == 0 ? pl.tiles : block_tiles(p, s, rb), w = block_rows(s.n, p.tok_tile, rb);
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
              a.n0 = min(p.tok_tile, s.n - at);
              a.n1 = min(p.tok_tile, s.n - at - a.n0);
              const int q = queue_place();
              if (!ok) break;
              if (lane == 0) {
                sh.parts[q] = a;
                mbar_arrive(&sh.part_full[q]);
              }
              const int first1 = a.n1 > 0 ? a.first + a.n0 : a.t1 - a.t0 > 1 ? a.first : -1;
              if (queued == 1) {
                load_queries(a.head, a.first, first1);
              } else {
                if (late0 >= 0) load_queries(late_head, late0, late1);
                late_head = a.head;
                late0 = a.first;
                late1 = first1;
              }
            }
          }
        }
      }
      if (ok && late0 >= 0) load_queries(late_head, late0, late1);
      if (ok) {
        const int q = queue_place();
        if (ok && lane == 0) {
          sh.parts[q].line = -1;
          mbar_arrive(&sh.part_full[q]);
        }
      }
#pragma unroll
      for (int g = 0; g < 2; ++g)  // the last copies land before the CTA exits
        if (q_loads[g] > 0) mbar_wait(&sh.q_full[g], (q_loads[g] & 1) ^ 1, status, kWaitLimitCycles);
    } else if (warp == 9) {
      // ---------------- issuer (the whole warp; one thread issues) ----------------
      constexpr uint32_t id_qk = idesc_f16_f32(kBf16, false, kAtTile, kAtTile);
      constexpr uint32_t id_pv = idesc_f16_f32(kBf16, true, kAtTile, D);
      const uint32_t utm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = smem_desc_k128(smem_u32(qbuf)), k_desc = smem_desc_k128(smem_u32(ring)),
                     v_desc = smem_desc_mn128(smem_u32(ring), kHalfBytes);
      uint32_t base = 0, waited = 0;  // tiles of the ring before this part, tiles known to have landed
      uint32_t ph_q[2] = {0, 0}, ph_p[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, status, kWaitLimitCycles));
        return ok;
      };
      auto landed = [&](uint32_t i) {
        for (; ok && waited <= i; ++waited) wait(&sh.kv_full[waited % kSlots], (waited / kSlots) & 1);
        return ok;
      };
      // group g's scores of ring tile i, in one thread; `free_tile`: the tile's
      // last reader, `free_q`: the queries' last use
      auto qk = [&](int g, uint32_t slot, bool free_tile, bool free_q) {
        const uint64_t ad = q_desc + g * (kTileBytes >> 4), bd = k_desc + slot * (kTileBytes >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t step = (k / 4) * (kHalfBytes >> 4) + (k % 4) * 2;
          tc_mma(utm + 128 * g, ad + step, bd + step, id_qk, k > 0);
        }
        tc_commit(&sh.s_full[g]);
        if (free_tile) tc_commit(&sh.kv_empty[slot]);
        if (free_q) tc_commit(&sh.q_empty[g]);
      };
      auto pv = [&](int g, uint32_t slot, bool first) {
        const uint64_t bd = v_desc + slot * (kTileBytes >> 4);
#pragma unroll
        for (int k = 0; k < kAtTile / 16; ++k)
          tc_mma_ts(utm + 256 + D * g, utm + 128 * g + 8 * k, bd + k * (2048 >> 4), id_pv, !first || k > 0);
      };
#pragma unroll 1
      for (int n = 0; ok; ++n) {
        const int q = n % kAtQueue;
        if (!wait(&sh.part_full[q], (n / kAtQueue) & 1)) break;
        const int line = __shfl_sync(0xffffffffu, sh.parts[q].line, 0);
        const int tiles = __shfl_sync(0xffffffffu, sh.parts[q].t1 - sh.parts[q].t0, 0);
        const bool two = __shfl_sync(0xffffffffu, sh.parts[q].n1, 0) > 0;
        if (lane == 0) mbar_arrive(&sh.part_empty[q]);
        if (line < 0) break;
        const int per = two ? tiles : (tiles + 1) / 2;  // key tiles of group 0
        auto tile_of = [&](int g, int j) { return two ? j : 2 * j + g; };
        auto k_at = [&](int t) { return base + (two ? 2 * t : (t == 0 ? 0 : 2 * t - 1)); };
        auto v_at = [&](int t) { return base + (two ? 2 * t + 1 : min(2 * t + 2, 2 * tiles - 1)); };
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (tile_of(g, 0) >= tiles || !ok) continue;
          const uint32_t i = k_at(tile_of(g, 0));
          if (!wait(&sh.q_full[g], ph_q[g]) || !landed(i)) continue;
          ph_q[g] ^= 1;
          tc_fence_after();
          if (elect_one()) qk(g, i % kSlots, !two || g == 1, tile_of(g, 1) >= tiles);
          __syncwarp();
        }
#pragma unroll 1
        for (int j = 0; j < per && ok; ++j) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int t = tile_of(g, j);
            if (t >= tiles || !ok) continue;
            // everything that can be waited for before the weights is, so that
            // both products follow them without a pause
            const int next = tile_of(g, j + 1);
            const bool more = next < tiles;
            const uint32_t vi = v_at(t), ki = more ? k_at(next) : vi;
            const uint32_t vslot = vi % kSlots, kslot = ki % kSlots;
            const bool free_q = tile_of(g, j + 2) >= tiles;
            if (!landed(vi) || !landed(ki) || !wait(&sh.p_full[g], ph_p[g])) continue;
            ph_p[g] ^= 1;
            tc_fence_after();
            if (elect_one()) {
              pv(g, vslot, j == 0);
              if (!two || g == 1) tc_commit(&sh.kv_empty[vslot]);
              if (more)
                qk(g, kslot, !two || g == 1, free_q);
              else
                tc_commit(&sh.o_full[g]);
            }
            __syncwarp();
          }
        }
        base += 2 * tiles;
      }
      // nothing is in flight when the TMEM is freed
      if (elect_one()) tc_commit(&sh.done);
      __syncwarp();
      mbar_wait(&sh.done, 0, status, kWaitLimitCycles);
    } else {
      // ---------------- key loads (warp 10) and value loads (warp 11) ----------------
      // One box a lane: a run of a page's slots, 64 dims.  (One warp for both
      // could not keep up with pages of 16: 3,300 clocks a key tile.)
      const bool values = warp == 11;
      const CUtensorMap* const map = values ? &p.tmV : &p.tmK;
      const int n_boxes = kAtTile / p.box_rows;
      const int my_box = lane % n_boxes, my_half = lane / n_boxes;
      const bool loads = my_half < kHalves;
      const uint32_t my_dst = smem_u32(ring) + my_half * kHalfBytes + my_box * p.box_rows * 128;
      const uint32_t page_size = p.batch.page_size;
      uint32_t base = 0, last = 0;  // tiles of the ring before this part; 1 + the last one this warp put in slot `lane`
      bool ok = true;
#pragma unroll 1
      for (int n = 0; ok; ++n) {
        const int q = n % kAtQueue;
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.part_full[q], (n / kAtQueue) & 1, status, kWaitLimitCycles));
        if (!ok) break;
        const int line = sh.parts[q].line, head = sh.parts[q].head, t0 = sh.parts[q].t0, tiles = sh.parts[q].t1 - t0,
                  len = sh.parts[q].len, seq = sh.parts[q].seq;
        const bool two = sh.parts[q].n1 > 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.part_empty[q]);
        if (line < 0) break;
        const int32_t* const table =
            line == 0 ? p.prefix_table : p.batch.block_table + static_cast<int64_t>(seq) * p.batch.table_width;
        // the page of this lane's box in the part's tile i, loaded three tiles
        // ahead; past the entries n_pages, where the copy fills zeros
        const uint32_t table_end = line == 0 ? (p.prefix_len - 1u) / page_size + 1 : p.batch.table_width;
        auto page_at = [&](int i) {
          const uint32_t key = static_cast<uint32_t>(t0 + i) * kAtTile + my_box * p.box_rows;
          return loads && i < tiles && key < static_cast<uint32_t>(len) &&
                         in_bounds(key / page_size < table_end && seq >= 0 && seq < p.batch.B, status)
                     ? table[key / page_size]
                     : p.n_pages;
        };
        int page0 = page_at(0), page1 = page_at(1), page2 = page_at(2);
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          // the order the products want the tiles in: with two row tiles
          // K V K V ...; with one the groups alternate and the next keys come
          // before these values: K0 K1 V0 K2 V1 ... V
          const uint32_t at = base + (values ? (two ? 2 * i + 1 : min(2 * i + 2, 2 * tiles - 1))
                                             : (two ? 2 * i : (i == 0 ? 0 : 2 * i - 1)));
          const uint32_t slot = at % kSlots, use = at / kSlots;
          int page = page0;
          page0 = page1;
          page1 = page2;
          page2 = page_at(i + 3);
          const uint32_t key = static_cast<uint32_t>(t0 + i) * kAtTile + my_box * p.box_rows;
          if (page < 0 || page >= p.n_pages) {
            if (loads && key < static_cast<uint32_t>(len)) atomicOr(status, kStatusBadCache);
            page = p.n_pages;
          }
          const int at_slot = static_cast<int>(key % page_size);
          // (A wait tells neighbouring phases apart: the slot's occupant before
          // the last one is free, since the tile that this warp loaded before,
          // at most three places back, came after a later one was.)
          if (use > 0)
            ok = __all_sync(0xffffffffu, mbar_wait(&sh.kv_empty[slot], (use & 1) ^ 1, status, kWaitLimitCycles));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[slot], kTileBytes);
          __syncwarp();
          in_bounds(slot < kSlots && at_slot + p.box_rows <= static_cast<int>(page_size) && head >= 0 && head < p.n_heads,
                    status);
          if (loads) tma_load_4d(my_dst + slot * kTileBytes, map, my_half * 64, at_slot, head, page, &sh.kv_full[slot]);
          if (lane == static_cast<int>(slot)) last = at + 1;
        }
        base += 2 * tiles;
      }
      // Copies land before the CTA exits: the issuer waits for every tile, unless
      // a wait ran out.  (Only then: a slot that the other loader has filled since
      // is past the phase waited for here.)
      if (!ok && lane < kSlots && last > 0)
        mbar_wait(&sh.kv_full[lane], ((last - 1) / kSlots) & 1, status, kWaitLimitCycles);
      __syncwarp();
    }
  } else {
    regs_up<kAtSoftmaxRegs>();
    // ---------------- softmax groups ----------------
    const int g = warp >> 2, quad = warp & 3, r = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int row_tok = r / p.group, row_head = r % p.group;
    uint32_t ph_s = 0, ph_o[2] = {0, 0}, ph_meet = 0, base = 0;
    bool ok = true;
    // all eight warps meet (a wait with a limit, unlike a barrier instruction)
    auto meet_all = [&](int i) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.meet[i]);
      return __all_sync(0xffffffffu, mbar_wait(&sh.meet[i], ph_meet, status, kWaitLimitCycles)) != 0;
    };
    auto products_done = [&](int o) {
      const bool got = __all_sync(0xffffffffu, mbar_wait(&sh.o_full[o], ph_o[o], status, kWaitLimitCycles));
      ph_o[o] ^= 1;
      return got;
    };
    for (int n = 0; ok; ++n) {
      const int qi = n % kAtQueue;
      ok = __all_sync(0xffffffffu, mbar_wait(&sh.part_full[qi], (n / kAtQueue) & 1, status, kWaitLimitCycles));
      if (!ok) break;
      const AtPart a = sh.parts[qi];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.part_empty[qi]);
      if (a.line < 0) break;
      const int tiles = a.t1 - a.t0;
      const bool two = a.n1 > 0;
      const int first = a.first + (two && g == 1 ? a.n0 : 0);
      const int rows = (two && g == 1 ? a.n1 : a.n0) * p.group;
      const int mine = two ? tiles : (tiles + 1 - g) / 2;
      const bool warp_live = quad * 32 < rows;
      const int tok = first + row_tok, gq = row_head;
      float m = -INFINITY, l = 0.f;

      // entries this row sees: all below `lim`, then the mask's bits from `lim` on
      int lim = a.len;
      uint64_t bits = 0;
      if (a.line == 1 && r < rows) {
        if (p.draft_mask == nullptr) {
          lim = a.old + (tok - a.seq_first) + 1;
        } else {
          lim = a.old;
          bits = in_bounds(tok >= 0 && tok < p.batch.N, status) ? p.draft_mask[tok] : 0;
          if (a.seq_n < 64) bits &= (1ull << a.seq_n) - 1;
        }
      }
      // Values past the last entry, in its page, may be anything: zero times that
      // must be zero.  The tile in question, and its rows live .. end - 1.
      const int live = a.len & (kAtTile - 1), end = (live + p.box_rows - 1) & -p.box_rows;  // box_rows: a power of two
      const int ragged = live < end ? a.len >> 7 : -1;
      for (int i = 0; i < mine && ok; ++i) {
        const int t = a.t0 + (two ? i : 2 * i + g);
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.s_full[g], ph_s, status, kWaitLimitCycles));
        if (!ok) break;
        ph_s ^= 1;
        tc_fence_after();
        if (warp_live) {
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_start(tm_s(g) + lanes + 32 * c, s[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32_wait(s[c]);
          const int left = lim - t * kAtTile;  // len + 127 is below 2^31
          if (__any_sync(0xffffffffu, left < kAtTile)) {
            const int below = left < -128 ? -128 : left;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int x = below - 32 * c;  // entries of this run below lim
              uint32_t see = x >= 32 ? 0xffffffffu : x <= 0 ? 0u : (1u << x) - 1;
              if (bits != 0) {
                if (x >= 0 && x < 32) see |= static_cast<uint32_t>(bits << x);
                if (x < 0 && x > -64) see |= static_cast<uint32_t>(bits >> -x);
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) s[c][j] = (see >> j) & 1 ? s[c][j] : 0xff800000u;  // -inf
            }
          }
          float tops[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tops[c] = max3(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]), __uint_as_float(s[c][2]));
#pragma unroll
            for (int j = 3; j < 31; j += 2) tops[c] = max3(tops[c], __uint_as_float(s[c][j]), __uint_as_float(s[c][j + 1]));
            tops[c] = fmaxf(tops[c], __uint_as_float(s[c][31]));
          }
          const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * p.scale_log2;
          const bool rise = top > m + (kAtTop<T> + kAtRise) || (m == -INFINITY && top > -INFINITY);
          if (__any_sync(0xffffffffu, rise)) {
            const float nm = rise ? top - kAtTop<T> : m;
            const float al = rise ? ex2(m - nm) : 1.f;  // 0 at a row's first keys
            l *= al;
            m = nm;
            if (i > 0) {  // the last product into O is complete: S came after it
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32_start(tm_o(g) + lanes + 32 * c, o);
                tmem_ld32_wait(o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * al);
                tmem_st32(tm_o(g) + lanes + 32 * c, o);
              }
            }
          }
          const float sub = m == -INFINITY ? 0.f : m;
          const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2), sub2 = f32x2(-sub, -sub);
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              // 16-bit weights for the product with V, half a step off at most;
              // the sum keeps them in 32 bits
              float e0, e1;
              f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[c][2 * j]), __uint_as_float(s[c][2 * j + 1])), scale2, sub2),
                          e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum[j % 4] = add_f32x2(sum[j % 4], f32x2(e0, e1));
              w[j] = Pack16<T>::pack(e0, e1);
            }
            tmem_st16(tm_s(g) + lanes + 16 * c, w);
          }
          float l0, l1;
          f32x2_split(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), l0, l1);
          l += l0 + l1;
          tmem_st_wait();
        }
        if (t == ragged) {
          const uint32_t at = base + (two ? 2 * (t - a.t0) + 1 : min(2 * (t - a.t0) + 2, 2 * tiles - 1));
          ok = __all_sync(0xffffffffu, mbar_wait(&sh.kv_full[at % kSlots], (at / kSlots) & 1, status, kWaitLimitCycles));
          if (!ok) break;
          uint8_t* v = ring + (at % kSlots) * kTileBytes;
          for (int x = r; x < (end - live) * 8 * kHalves; x += 128) {
            const int row = live + x / (8 * kHalves), c = x % (8 * kHalves);
            if (!in_bounds(row < kAtTile, status)) continue;
            *reinterpret_cast<uint4*>(v + (c / 8) * kHalfBytes + row * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[g]);
      }
      if (!ok) break;

      // ---- the part's results ----
      float* dst_o;
      float2* dst_ml;
      int4* dst_meta = nullptr;
      const int slab_row = (two && g == 1 ? a.n0 * p.group : 0) + r;  // < slab_rows where r < rows
      if (a.t0 == 0) {
        const int64_t row = p.place(a.line, static_cast<int64_t>(tok) * p.n_q_heads + a.head * p.group + gq);
        dst_o = p.part_o + row * D;
        dst_ml = p.part_ml + row;
        dst_meta = p.part_meta + row;
      } else {
        const int64_t row = static_cast<int64_t>(cta) * p.slab_rows + slab_row;
        dst_o = p.slab_o + row * D;
        dst_ml = p.slab_ml + row;
      }
      // With one row tile a group waits for both groups' products, with two for
      // its own: the other's phase is only counted.  (A wait there could come two
      // phases late and never end: group 0 needs nothing of group 1 for a next
      // part of one tile, and completes its phase again.)  A wait tells
      // neighbouring phases apart, and no phase before the one waited for is open:
      // products complete in the order in which one thread issued them, and
      // this group's of the last part or of this one came after them.
      ok = products_done(two ? g : 0);
      if (!two && tiles > 1) ok = products_done(1) && ok;
      if (!ok) break;
      tc_fence_after();
      float f0 = 1.f, f1 = 0.f;
      if (!two) {
        sh.xch[g][r] = make_float2(m, l);
        ok = meet_all(0);
        if (!ok) break;
        const float2 o = sh.xch[g ^ 1][r];
        const float mm = fmaxf(m, o.x);
        const float fm = m == -INFINITY ? 0.f : ex2(m - mm), fo = o.x == -INFINITY ? 0.f : ex2(o.x - mm);
        l = g == 0 ? l * fm + o.y * fo : o.y * fo + l * fm;
        m = mm;
        f0 = g == 0 ? fm : fo;
        f1 = g == 0 ? fo : fm;
      }
      if (warp_live) {
        const bool mine_to_write =
            r < rows && in_bounds(a.t0 == 0 ? tok >= 0 && tok < p.batch.N && a.head * p.group + gq < p.n_q_heads
                                            : cta < p.n_ctas && slab_row < p.slab_rows,
                                  status);
        if (two) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            float v[32];
            tmem_ld32(tm_o(g) + lanes + 32 * c, v);
            if (mine_to_write) {
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                st_global_f8(dst_o + 32 * c + j, v + j);
            }
          }
        } else {
          // group g joins its half of the columns
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const int col = g * (D / 2) + 32 * c;
            float v[32], x[32];
            tmem_ld32(tm_o(0) + lanes + col, v);
            if (tiles > 1) {
              tmem_ld32(tm_o(1) + lanes + col, x);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = v[j] * f0 + x[j] * f1;
            }
            if (mine_to_write) {
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                st_global_f8(dst_o + col + j, v + j);
            }
          }
        }
        if (mine_to_write && (two || g == 0)) {
          *dst_ml = make_float2(m, l);
          if (a.t0 == 0) *dst_meta = row_item(a, cta, slab_row);
        }
      }
      tc_fence_before();
      if (two) {
        ph_o[g ^ 1] ^= 1;
      } else {  // O and the exchanged values are free again once all have read them
        ok = meet_all(1);
        ph_meet ^= 1;
      }
      base += 2 * tiles;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// A row whose output is not finite although its sum of weights is: an entry that
// the row does not see may hold an infinity or a NaN, which the tensor cores take
// times a weight of 0, or the sum passed the largest fp32 before its division.
// The warp sums the row again, only over what it sees and with the weights
// divided first: scores with a key a lane, then the values with dims over the
// lanes.  The prefix's sum (m0, o0) stands where it is finite.  In a verify pass
// this keeps a bad draft out of the rows before it: some 0.5 us a key of the
// sequence (the verify batch with one bad draft behind 510 entries: 274 us for
// 46).  Kept short: with the keys' steps unrolled by eight the join's code cost every
// launch 1 us, called or not.
// ---------------------------------------------------------------------------
template <typename T, int D>
__device__ __noinline__ void sum_row_again(const AttendParams& p, int n, int hq, float m, float inv, float m0, float4 o0) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31, b = find_seq(p.batch, n, lane);
  if (b < 0) return;
  const SeqSpan s = seq_span(p.batch, b);
  const int kv = static_cast<int>(s.kv), first = s.first, count = s.n;
  const int64_t in_page = (hq / p.group) * p.cache.head_stride;
  const uint16_t* const q = p.q + n * p.q_ps + hq * p.q_hs;
  float sum[kPer] = {};
  // the prefix's sum stands if it is finite
  const bool stands = fabsf(o0.x) < INFINITY && fabsf(o0.y) < INFINITY && fabsf(o0.z) < INFINITY && fabsf(o0.w) < INFINITY;
  const int from = __all_sync(0xffffffffu, stands) ? 1 : 0;
  if (from == 1) {
    const float f = m0 == -INFINITY ? 0.f : ex2(m0 - m) * inv;
    sum[0] = o0.x * f;
    sum[1] = o0.y * f;
    sum[kPer - 2] = o0.z * f;
    sum[kPer - 1] = o0.w * f;
  }
#pragma unroll 1
  for (int line = from; line < 2; ++line) {
    // entries below `lim` are seen, then those of the mask's bits
    const int32_t* const table =
        line == 0 ? p.prefix_table : p.batch.block_table + static_cast<int64_t>(b) * p.batch.table_width;
    const int entries = line == 0 ? p.prefix_len : kv, old = entries - (line == 0 ? 0 : count);
    const bool masked = line == 1 && p.draft_mask != nullptr;
    const int lim = line == 0 || masked ? old : old + (n - first) + 1;
    const uint64_t bits = masked ? p.draft_mask[n] : 0;
#pragma unroll 1
    for (int t0 = 0; t0 < entries; t0 += 32) {
      const int t = t0 + lane, j = t - old;
      const bool seen = t < entries && (t < lim || (j >= 0 && j < 64 && (bits >> j & 1) != 0));
      const bool inside = in_bounds(line == 0 || t >= entries || t / p.batch.page_size < p.batch.table_width, p.batch.status);
      const int page = seen && inside ? table[t / p.batch.page_size] : -1;
      const bool valid = page >= 0 && page < p.n_pages;  // others' keys and values read as zero (and are reported)
      const int64_t at = valid ? page * p.cache.page_stride + (t % p.batch.page_size) * p.cache.slot_stride + in_page : 0;
      float dot = 0.f;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {  // four loads in flight
        uint4 k[4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (valid) k[i] = *reinterpret_cast<const uint4*>(p.cache.k + at + c + 8 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x[8], y[8];
          unpack8<T>(*reinterpret_cast<const uint4*>(q + c + 8 * i), x);
          unpack8<T>(k[i], y);
#pragma unroll
          for (int e = 0; e < 8; ++e) dot = fmaf(x[e], y[e], dot);
        }
      }
      const float w = ex2(fmaf(dot, p.scale_log2, -m)) * inv;
      const unsigned any = __ballot_sync(0xffffffffu, valid);
#pragma unroll 1
      for (int u = 0; u < 32; u += 4) {
        if ((any >> u & 15) == 0) continue;
        float wu[4];
        uint32_t v[4][kPer / 2] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool there = any >> (u + i) & 1;
          wu[i] = __shfl_sync(0xffffffffu, w, u + i);
          const uint16_t* from = p.cache.v + __shfl_sync(0xffffffffu, at, u + i) + lane * kPer;
          if (there) {
#pragma unroll
            for (int x = 0; x < kPer / 2; ++x) v[i][x] = reinterpret_cast<const uint32_t*>(from)[x];
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if ((any >> (u + i) & 1) == 0) continue;
#pragma unroll
          for (int x = 0; x < kPer / 2; ++x) {
            float v0, v1;
            Pack16<T>::unpack(v[i][x], v0, v1);
            sum[2 * x] = fmaf(wu[i], v0, sum[2 * x]);
            sum[2 * x + 1] = fmaf(wu[i], v1, sum[2 * x + 1]);
          }
        }
      }
    }
  }
  uint16_t* const dst = p.out + n * p.o_ps + hq * p.o_hs + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) = Pack16<T>::pack(sum[i], sum[i + 1]);
}

// ---------------------------------------------------------------------------
// join: one warp per row adds the row's parts.  Each item's first part says
// where the others are, so a row whose items were not split takes one round of
// loads.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kPer = D / 32;  // dims of a lane
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(p.batch.N) * p.n_q_heads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  grid_dep_launch();
  grid_dep_wait();
  if (row >= rows) return;
  const int n = static_cast<int>(row / p.n_q_heads), hq = static_cast<int>(row - static_cast<int64_t>(n) * p.n_q_heads);

  auto load = [&](const float* src, float (&x)[kPer]) {
    if (kPer == 4)
      *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(src);
    else
      *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(src);
  };
  float x[2][kPer];
  float2 ml[2];
  int4 item[2];
#pragma unroll
  for (int line = 0; line < 2; ++line) {
    item[line] = make_int4(-1, 0, 0, 0);
    if (line == 0 && p.prefix_len == 0) continue;
    const int64_t at = p.place(line, row);
    item[line] = p.part_meta[at];
    ml[line] = p.part_ml[at];
    load(p.part_o + at * D + lane * kPer, x[line]);
  }
  if (!in_batch(p.batch, n)) return;  // padding, or (reported) before the first sequence: nothing was left for it

  float o[kPer] = {}, m = -INFINITY, l = 0.f, m0 = -INFINITY, o0[kPer] = {};  // 0: of the prefix
  auto add = [&](const float2& a, const float (&v)[kPer]) {
    // Nothing seen: a.y is 0, its O is not looked at.  (A part whose every score
    // is NaN has a.x = -inf too, but a.y NaN, which reaches l and o.)
    if (a.y == 0.f) return;
    const float mm = fmaxf(m, a.x);
    const float fo = m == -INFINITY ? 0.f : ex2(m - mm), fx = ex2(a.x - mm);
    m = mm;
    l = l * fo + a.y * fx;
#pragma unroll
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * fo + v[i] * fx;
  };
#pragma unroll
  for (int line = 0; line < 2; ++line) {
    if (line == 1) {
      m0 = m;
#pragma unroll
      for (int i = 0; i < kPer; ++i) o0[i] = o[i];
    }
    if (item[line].x < 0) continue;
    add(ml[line], x[line]);
    const int first = item[line].x & 255, last = min(item[line].x >> 8 & 255, p.n_ctas - 1);
    const int slab_row = min(item[line].x >> 16 & 255, p.slab_rows - 1), tiles = item[line].y >> 2, w = 1 + (item[line].y & 1),
              fixed = item[line].y & 2 ? kAtFixed : 0;
    const int64_t off = static_cast<int64_t>(item[line].w) << 32 | static_cast<uint32_t>(item[line].z);
    const int64_t* const begin = p.begin;
    for (int c0 = first + 1; c0 <= last; c0 += 32) {
      // lane i: whether part c0 + i holds a tile's beginning
      const int c = c0 + lane;
      const bool has = c <= last && tiles_before(begin[c], off, w, fixed, tiles) <
                                        tiles_before(begin[c + 1], off, w, fixed, tiles);
      unsigned parts = __ballot_sync(0xffffffffu, has);
      while (parts != 0u) {
        // up to four parts' loads in flight, added in ascending order
        float v[4][kPer];
        float2 a[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a[k] = make_float2(-INFINITY, 0.f);
          if (parts == 0u) continue;
          const int part = c0 + __ffs(parts) - 1;
          parts &= parts - 1;
          if (!in_bounds(part < p.n_ctas && slab_row >= 0 && slab_row < p.slab_rows, p.batch.status)) continue;
          const int64_t at = static_cast<int64_t>(part) * p.slab_rows + slab_row;
          a[k] = p.slab_ml[at];
          load(p.slab_o + at * D + lane * kPer, v[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) add(a[k], v[k]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;  // l: 0 where nothing was seen, else at least 1, or NaN
  uint16_t* dst = p.out + n * p.o_ps + hq * p.o_hs + lane * kPer;
  if (kPer == 4)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(Pack16<T>::pack(o[0] * inv, o[1] * inv), Pack16<T>::pack(o[kPer - 2] * inv, o[kPer - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = Pack16<T>::pack(o[0] * inv, o[1] * inv);
  if (lane == 0 && p.lse != nullptr) p.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < kPer; ++i) finite = finite && fabsf(o[i]) < INFINITY;
  if (__any_sync(0xffffffffu, !finite) && l < INFINITY)  // l: as in all lanes
    sum_row_again<T, D>(p, n, hq, m, inv, m0, make_float4(o0[0], o0[1], o0[kPer - 2], o0[kPer - 1]));
}

}  // namespace specv
