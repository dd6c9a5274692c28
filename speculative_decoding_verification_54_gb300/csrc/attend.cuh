// attend.cuh — attention of the new positions over a shared prefix and their
// sequences' pages, on the tcgen05 tensor cores.
//
// Work.  The rows of one key head are its (position, query head) pairs.  Over
// the prefix the rows of the whole batch are one matrix, so the prefix's keys
// and values are read once per row block and not once per sequence; over the
// sequences' own pages the rows of one sequence are.  An item is a block of
// up to two row tiles (128 rows each: whole positions) against all tiles of
// 128 keys that its rows see.  The items' key tiles, weighted by their row
// tiles, form two lines, one over the prefix and one over the own pages, and
// CTA c takes the c-th equal part of each: lengths are read on the device, so
// nothing is planned on the host, and one sequence or one head fills the GPU
// as well as many.  Even CTAs begin with their prefix part (bound by the
// tensor cores), odd ones with their own-pages part (bound by HBM), so the two
// overlap.
//
// A part of an item leaves, per row, the unnormalised output, its reference
// exponent m and the sum l: O = sum_t 2^(s_t - m) v_t, l = sum_t 2^(s_t - m)
// with s in units of log2.  The part that holds an item's first tile writes to
// the row's own place, any other to its CTA's slab (it is the CTA's first in
// that line); attend_join_kernel adds a row's parts in a fixed order, so
// results do not depend on timing.
//
// One CTA per SM:
//   warps 0-3, 4-7  softmax groups 0 and 1, one thread a row.  With two row
//                   tiles group g has tile g and both read each key tile; with
//                   one, the groups share its rows and alternate key tiles
//                   (their halves are joined at the end of the part), so that
//                   exponentials of one overlap products of the other.
//   warp 8          the scheduler and producer: finds the CTA's parts, queues
//                   them for the others and loads key and value tiles (TMA,
//                   one box per run of a page and 64 dims) into a ring.
//   warp 9          issues the products: S = Q K^T (both operands
//                   from shared memory) and O += P V (P from TMEM, where the
//                   softmax group wrote it over S; V's rows are K).
//   warps 10, 11    only fill their warpgroup.
// TMEM: S0 S1 (128 columns each) and O0 O1 (D columns each).
//
// The reference m of a row rises only when a tile's maximum passes it by more
// than 2^8, and only then is O (in TMEM) multiplied; weights stay below 256, l
// and O are exact with respect to any m.
#pragma once

#include <type_traits>

#include "kvappend.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace specv {

constexpr int kAtTile = 128;        // rows of a row tile, keys of a key tile
constexpr int kAtStep = 64;         // keys of one step of a softmax group
constexpr int kAtThreads = 384;     // three warpgroups
// Registers: the launch gives 168 a thread (65,536 / 384, by 8); the softmax
// groups take 192, the third warpgroup keeps 120: 192 + 192 + 120 = 3 x 168.
constexpr int kAtSoftmaxRegs = 192, kAtOtherRegs = 120;
constexpr int kAtRingBytes = 160 * 1024;
constexpr int kAtMaxCtas = 160;     // slabs in the workspace
constexpr int kAtQueue = 4;         // parts queued ahead
constexpr float kAtRise = 8.f;      // log2 of the largest weight

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
  const uint64_t* draft_mask;
  float scale_log2;  // scale * log2(e)
  int n_q_heads, n_heads, group;
  int tok_tile;      // positions of a row tile: 128 / group
  int n_ctas;
  int64_t* off;      // [B + 1] where each sequence begins in the own-pages line
  int64_t* begin;    // [2][n_ctas + 1] where the parts begin in each line
  float* part_o;     // [2][N * n_q_heads][D]
  float2* part_ml;   // [2][N * n_q_heads]
  float* slab_o;     // [n_ctas][2][256][D]
  float2* slab_ml;   // [n_ctas][2][256]
};

// ---------------------------------------------------------------------------
// the two lines of work
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

// Row tiles of the block: its weight per key tile.
__device__ __forceinline__ int block_weight(int positions, int tok_tile, int rb) {
  return positions - rb * 2 * tok_tile > tok_tile ? 2 : 1;
}

// Weight of one key head's items of a sequence.
__device__ __forceinline__ int64_t seq_head_weight(const AttendParams& p, const SeqSpan& s) {
  int64_t w = 0;
  for (int rb = 0; rb * 2 * p.tok_tile < s.n; ++rb)
    w += static_cast<int64_t>(block_tiles(p, s, rb)) * block_weight(s.n, p.tok_tile, rb);
  return w;
}

struct PrefixLine {
  int positions, blocks, tiles;
  int64_t per_head, total;
};
__device__ __forceinline__ PrefixLine prefix_line(const AttendParams& p) {
  PrefixLine L;
  L.positions = new_positions(p.batch);
  L.tiles = (p.prefix_len + kAtTile - 1) / kAtTile;
  L.blocks = (L.positions + 2 * p.tok_tile - 1) / (2 * p.tok_tile);
  L.per_head = L.blocks > 0
                   ? static_cast<int64_t>(L.tiles) * (2 * (L.blocks - 1) + block_weight(L.positions, p.tok_tile, L.blocks - 1))
                   : 0;
  L.total = L.per_head * p.n_heads;
  return L;
}

// Part c of n of a line of weight W begins at W * c / n; tiles belong to the
// part that their first unit of weight lies in.
__device__ __forceinline__ int64_t part_begin(int64_t W, int c, int n) { return W * c / n; }
__device__ __forceinline__ int tiles_before(int64_t x, int64_t off, int w, int tiles) {
  if (x <= off) return 0;
  const int64_t t = w == 2 ? (x - off + 1) >> 1 : x - off;
  return t < tiles ? static_cast<int>(t) : tiles;
}

// A part of an item, as the scheduler queues it.
struct AtPart {
  int line;           // 0 prefix, 1 own pages, -1 no more
  int head, first;    // key head, first position
  int n0, n1;         // positions of the two row tiles (n1 = 0: one tile)
  int t0, t1;         // key tiles
  int len, old;       // entries, entries older than the new positions
  int seq_first, seq_n;
  int seq;
};

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
  uint64_t q_full[2], q_empty[2], s_full[4], p_full[4], o_done[4], meet[2], done;
  float2 xch[2][kAtTile];  // the groups' (m, l)
  AtPart parts[kAtQueue];
  int64_t warp_sum[kAtThreads / 32], total, off;
  int seq;
  uint32_t tmem;
};
template <int D>
constexpr int kAtSlots = kAtRingBytes / (kAtTile * D * 2);
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
      mbar_init(&sh.part_empty[i], 9);  // eight softmax warps and the issuer
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sh.q_full[g], 1);
      mbar_init(&sh.q_empty[g], 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sh.s_full[2 * g + b], 1);
        mbar_init(&sh.p_full[2 * g + b], 4);
        mbar_init(&sh.o_done[2 * g + b], 1);
      }
      mbar_init(&sh.meet[g], 8);
    }
    mbar_init(&sh.done, 1);
    fence_mbar_init();
    sh.seq = p.batch.B;
    sh.off = 0;
  }
  if (warp == 9) tmem_alloc(&sh.tmem, 512);
  grid_dep_wait();

  // ---- the own-pages line: its weight, and where this CTA's part begins ----
  const int own_cta = p.n_ctas - 1 - cta;  // mirrored, so that short lines meet on different CTAs
  int64_t first_weight = 0;
  {
    int64_t w = 0;
    for (int b = threadIdx.x; b < p.batch.B; b += kAtThreads) {
      const int64_t one = seq_head_weight(p, seq_span(p.batch, b)) * p.n_heads;
      if (b == static_cast<int>(threadIdx.x)) first_weight = one;
      w += one;
    }
    for (int x = 16; x; x >>= 1) w += __shfl_xor_sync(0xffffffffu, w, x);
    if (lane == 0) sh.warp_sum[warp] = w;
    __syncthreads();
    if (threadIdx.x == 0) {
      int64_t t = 0;
      for (int i = 0; i < kAtThreads / 32; ++i) t += sh.warp_sum[i];
      sh.total = t;
    }
    __syncthreads();
    const int64_t total = sh.total, lo = part_begin(total, own_cta, p.n_ctas);
    int64_t before = 0;  // weight of the chunks before this one
    for (int b0 = 0; b0 < p.batch.B; b0 += kAtThreads) {
      const int b = b0 + threadIdx.x;
      int64_t one = 0;
      if (b < p.batch.B) one = b0 == 0 ? first_weight : seq_head_weight(p, seq_span(p.batch, b)) * p.n_heads;
      int64_t inc = one;
      for (int x = 1; x < 32; x <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, x);
        if (lane >= x) inc += o;
      }
      if (lane == 31) sh.warp_sum[warp] = inc;
      __syncthreads();
      int64_t base = before;
      for (int i = 0; i < warp; ++i) base += sh.warp_sum[i];
      const int64_t off = base + inc - one;
      if (b < p.batch.B) {
        if (off <= lo && lo < off + one) {
          sh.seq = b;
          sh.off = off;
        }
        if (cta == 0) {
          p.off[b] = off;
          if (b == p.batch.B - 1) p.off[b + 1] = off + one;
        }
      }
      for (int i = 0; i < kAtThreads / 32; ++i) before += sh.warp_sum[i];
      __syncthreads();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  auto tm_s = [&](int g, uint32_t u) { return tmem + 128 * g + 64 * (u & 1); };
  auto tm_o = [&](int g) { return tmem + 256 + D * g; };
  if (warp >= 8) {
    regs_down<kAtOtherRegs>();
    if (warp == 8) {
      // ---------------- scheduler and producer (the whole warp) ----------------
      const PrefixLine pl = prefix_line(p);
      const int n_boxes = kAtTile / p.box_rows;
      const int my_box = lane % n_boxes, my_half = lane / n_boxes;
      const bool loads = my_half < kHalves;
      const uint32_t box_bytes = static_cast<uint32_t>(p.box_rows) * 128u;
      int slot = 0, queued = 0;
      uint32_t loaded = 0;  // tiles, for the ring's phases
      bool ok = true;

      // one tile (keys or values) of 128 entries from `key0` on, of which `len`
      // are live; boxes past them read as zero
      auto load_tile = [&](const CUtensorMap* map, int head, int page, int key0) {
        if (loaded >= kSlots) ok = ok && mbar_wait(&sh.kv_empty[slot], ((loaded / kSlots) & 1) ^ 1, status, kWaitLimitCycles);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect_tx(&sh.kv_full[slot], kTileBytes);
        __syncwarp();
        if (loads)
          tma_load_4d(smem_u32(ring) + slot * kTileBytes + my_half * kHalfBytes + my_box * box_bytes, map, my_half * 64,
                      static_cast<uint32_t>(key0 + my_box * p.box_rows) % static_cast<uint32_t>(p.batch.page_size), head, page, &sh.kv_full[slot]);
        ++loaded;
        if (++slot == kSlots) slot = 0;
      };
      // the queries of a part: row tile g of two, or the one tile for each group
      uint32_t q_loads[2] = {0, 0};
      auto load_queries = [&](const AtPart& a) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (q_loads[g] > 0) ok = ok && mbar_wait(&sh.q_empty[g], (q_loads[g] & 1) ^ 1, status, kWaitLimitCycles);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) return;
          if (lane == 0) mbar_arrive_expect_tx(&sh.q_full[g], kHalves * 128u * p.group * p.tok_tile);
          __syncwarp();
          if (lane < kHalves)
            tma_load_3d(smem_u32(qbuf) + g * kTileBytes + lane * kHalfBytes, &p.tmQ, lane * 64, a.head * p.group,
                        a.first + (a.n1 > 0 && g == 1 ? a.n0 : 0), &sh.q_full[g]);
          ++q_loads[g];
        }
      };
      auto page_of = [&](const AtPart& a, int t) {
        const uint32_t key = static_cast<uint32_t>(t) * kAtTile + my_box * p.box_rows;
        if (!loads || t >= a.t1 || key >= static_cast<uint32_t>(a.len)) return p.n_pages;  // the copy fills zeros
        const uint32_t i = key / static_cast<uint32_t>(p.batch.page_size);
        const int page = a.line == 0 ? p.prefix_table[i]
                                     : p.batch.block_table[static_cast<int64_t>(a.seq) * p.batch.table_width + i];
        if (page >= 0 && page < p.n_pages) return page;
        atomicOr(status, kStatusBadCache);
        return p.n_pages;
      };
      // a free place of the queue
      auto queue_place = [&]() {
        const int q = queued % kAtQueue;
        if (queued >= kAtQueue)
          ok = ok && mbar_wait(&sh.part_empty[q], ((queued / kAtQueue) & 1) ^ 1, status, kWaitLimitCycles);
        ok = __all_sync(0xffffffffu, ok);
        ++queued;
        return q;
      };
#pragma unroll 1
      for (int turn = 0; turn < 2 && ok; ++turn) {
        // the prefix's line is that of one sequence of all new positions
        AtPart a;
        a.line = (turn ^ cta) & 1;
        const int64_t total = a.line == 0 ? pl.total : sh.total;
        const int c = a.line == 0 ? cta : own_cta;
        const int64_t lo = part_begin(total, c, p.n_ctas), hi = part_begin(total, c + 1, p.n_ctas);
        if (lane == 0) {
          int64_t* const begin = p.begin + a.line * (p.n_ctas + 1);
          begin[c] = lo;
          if (c == p.n_ctas - 1) begin[c + 1] = hi;
        }
        int64_t off = a.line == 0 ? 0 : sh.off;
        a.seq = a.line == 0 ? 0 : sh.seq;
#pragma unroll 1
        for (; off < hi && lo < hi && ok; ++a.seq) {
          SeqSpan s = {0, pl.positions, 0};
          int64_t hw = pl.per_head;
          if (a.line == 1) {
            s = seq_span(p.batch, a.seq);
            hw = seq_head_weight(p, s);
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
              const int tiles = a.line == 0 ? pl.tiles : block_tiles(p, s, rb), w = block_weight(s.n, p.tok_tile, rb);
              a.t0 = tiles_before(lo, off, w, tiles);
              a.t1 = tiles_before(hi, off, w, tiles);
              off += static_cast<int64_t>(tiles) * w;
              if (a.t0 >= a.t1) continue;
              a.first = s.first + at;
              a.n0 = min(p.tok_tile, s.n - at);
              a.n1 = min(p.tok_tile, s.n - at - a.n0);
              const int q = queue_place();
              if (!ok) break;
              if (lane == 0) {
                sh.parts[q] = a;
                mbar_arrive(&sh.part_full[q]);
              }
              // The order the products want the tiles in (scores run two halves
              // of a tile ahead): with two row tiles K V K V ..., with one K0 K1
              // V0 K2 V1 ... V.
              const int lead = a.n1 > 0 ? 0 : 1;
              int page = page_of(a, a.t0), vpage = page;
#pragma unroll 1
              for (int kt = a.t0; kt < a.t1 + lead && ok; ++kt) {
                const int vt = kt - lead, next = page_of(a, kt + 1);
                if (kt < a.t1) load_tile(&p.tmK, a.head, page, kt * kAtTile);
                if (kt == a.t0 + lead && ok) load_queries(a);  // after the first keys: the buffers may still be in use
              if (vt >= a.t0 && ok) load_tile(&p.tmV, a.head, lead ? vpage : page, vt * kAtTile);
                vpage = page;
                page = next;
              }
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
#pragma unroll
      for (int g = 0; g < 2; ++g)
        if (q_loads[g] > 0) mbar_wait(&sh.q_full[g], (q_loads[g] & 1) ^ 1, status, kWaitLimitCycles);
      // the copies of the last tiles land before the CTA exits
#pragma unroll 1
      for (uint32_t i = loaded > kSlots ? loaded - kSlots : 0; i < loaded; ++i)
        mbar_wait(&sh.kv_full[i % kSlots], (i / kSlots) & 1, status, kWaitLimitCycles);
    } else if (warp == 9) {
      // ---------------- issuer (the whole warp; one thread issues) ----------------
      constexpr uint32_t id_qk = idesc_f16_f32(kBf16, false, kAtTile, kAtStep);
      constexpr uint32_t id_pv = idesc_f16_f32(kBf16, true, kAtTile, D);
      const uint32_t utm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t q_desc = smem_desc_k128(smem_u32(qbuf)), k_desc = smem_desc_k128(smem_u32(ring)),
                     v_desc = smem_desc_mn128(smem_u32(ring), kHalfBytes);
      uint32_t base = 0, waited = 0;  // tiles of the ring before this part, tiles known to have landed
      uint32_t u0 = 0, parts = 0;     // steps of a group before this part; parts so far
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, status, kWaitLimitCycles));
      };
      auto landed = [&](uint32_t i) {
        for (; ok && waited <= i; ++waited) wait(&sh.kv_full[waited % kSlots], (waited / kSlots) & 1);
        tc_fence_after();
      };
      // scores of group g's step u: the 64 keys from row `row` of ring tile i on;
      // `free_tile`: the tile's last reader, `free_q`: the queries' last use
      auto qk = [&](int g, uint32_t u, uint32_t i, int row, bool free_tile, bool free_q) {
        landed(i);
        if (!ok) return;
        const uint64_t ad = q_desc + g * (kTileBytes >> 4);
        const uint64_t bd = k_desc + (i % kSlots) * (kTileBytes >> 4) + row * (128 >> 4);
        const uint32_t d = utm + 128 * g + 64 * (u & 1);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t step = (k / 4) * (kHalfBytes >> 4) + (k % 4) * 2;
            tc_mma(d, ad + step, bd + step, id_qk, k > 0);
          }
          tc_commit(&sh.s_full[2 * g + (u & 1)]);
          if (free_tile) tc_commit(&sh.kv_empty[i % kSlots]);
          if (free_q) tc_commit(&sh.q_empty[g]);
        }
        __syncwarp();
      };
      auto pv = [&](int g, uint32_t u, uint32_t i, int row, bool first, bool free_tile) {
        landed(i);
        wait(&sh.p_full[2 * g + (u & 1)], (u >> 1) & 1);
        if (!ok) return;
        tc_fence_after();
        const uint64_t bd = v_desc + (i % kSlots) * (kTileBytes >> 4) + row * (128 >> 4);
        const uint32_t d = utm + 256 + D * g, w = utm + 128 * g + 64 * (u & 1);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kAtStep / 16; ++k) tc_mma_ts(d, w + 8 * k, bd + k * (2048 >> 4), id_pv, !first || k > 0);
          tc_commit(&sh.o_done[2 * g + (u & 1)]);
          if (free_tile) tc_commit(&sh.kv_empty[i % kSlots]);
        }
        __syncwarp();
      };
#pragma unroll 1
      for (; ok; ++parts) {
        const int q = parts % kAtQueue;
        wait(&sh.part_full[q], (parts / kAtQueue) & 1);
        if (!ok) break;
        const int line = __shfl_sync(0xffffffffu, sh.parts[q].line, 0);
        const int tiles = __shfl_sync(0xffffffffu, sh.parts[q].t1 - sh.parts[q].t0, 0);
        const bool two = __shfl_sync(0xffffffffu, sh.parts[q].n1, 0) > 0;
        if (lane == 0) mbar_arrive(&sh.part_empty[q]);
        if (line < 0) break;
        const int steps = two ? 2 * tiles : tiles;
        // both groups are through with a tile after group 1's (last) step on it
        auto scores = [&](int g, int j) {
          const int t = two ? j >> 1 : j;
          qk(g, u0 + j, base + (two ? 2 * t : (t == 0 ? 0 : 2 * t - 1)), (two ? j & 1 : g) * kAtStep,
             g == 1 && (!two || (j & 1)), j == steps - 1);
        };
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (j >= steps) continue;
            if (j == 0) wait(&sh.q_full[g], parts & 1);
            if (ok) scores(g, j);
          }
        }
#pragma unroll 1
        for (int j = 0; j < steps && ok; ++j) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int t = two ? j >> 1 : j;
            if (ok)
              pv(g, u0 + j, base + (two ? 2 * t + 1 : min(2 * t + 2, 2 * tiles - 1)), (two ? j & 1 : g) * kAtStep,
                 j == 0, g == 1 && (!two || (j & 1)));
            if (ok && j + 2 < steps) scores(g, j + 2);
          }
        }
        base += 2 * tiles;
        u0 += steps;
      }
      // nothing is in flight when the TMEM is freed
      if (elect_one()) tc_commit(&sh.done);
      __syncwarp();
      mbar_wait(&sh.done, 0, status, kWaitLimitCycles);
    }
  } else {
    regs_up<kAtSoftmaxRegs>();
    // ---------------- softmax groups ----------------
    const int g = warp >> 2, quad = warp & 3, r = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t u0 = 0, ph_meet = 0, base = 0;
    bool ok = true;
    // all eight warps meet (a wait with a limit, unlike a barrier instruction)
    auto meet_all = [&](int i) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.meet[i]);
      return __all_sync(0xffffffffu, mbar_wait(&sh.meet[i], ph_meet, status, kWaitLimitCycles)) != 0;
    };
    // Group o's product of step u (and all before it).  A wait tells
    // neighbouring phases apart only: u - 2, the phase before, is complete
    // wherever this is called, because the scores of u came after it.
    auto product_done = [&](int o, uint32_t u) {
      return __all_sync(0xffffffffu, mbar_wait(&sh.o_done[2 * o + (u & 1)], (u >> 1) & 1, status, kWaitLimitCycles)) != 0;
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
      const int steps = two ? 2 * tiles : tiles;
      const bool warp_live = quad * 32 < rows;
      const int tok = first + r / p.group, gq = r % p.group;
      float m = -INFINITY, l = 0.f;

      // entries this row sees: all below `lim`, then the mask's bits from `lim` on
      int lim = a.len;
      uint64_t bits = 0;
      if (a.line == 1 && r < rows) {
        if (p.draft_mask == nullptr) {
          lim = a.old + (tok - a.seq_first) + 1;
        } else {
          lim = a.old;
          bits = p.draft_mask[tok];
          if (a.seq_n < 64) bits &= (1ull << a.seq_n) - 1;
        }
      }
      for (int j = 0; j < steps && ok; ++j) {
        const uint32_t u = u0 + j;
        const int i = two ? j >> 1 : j, t = a.t0 + i, row0 = (two ? j & 1 : g) * kAtStep;
        ok = __all_sync(0xffffffffu, mbar_wait(&sh.s_full[2 * g + (u & 1)], (u >> 1) & 1, status, kWaitLimitCycles));
        if (!ok) break;
        tc_fence_after();
        // values past the last entry, in its page, may be anything: zero times
        // that must be zero
        const int live = static_cast<int>(min(static_cast<int64_t>(kAtTile), a.len - static_cast<int64_t>(t) * kAtTile));
        const int z0 = max(live, row0), z1 = min((live + p.box_rows - 1) / p.box_rows * p.box_rows, row0 + kAtStep);
        if (z0 < z1) {
          const uint32_t at = base + (two ? 2 * i + 1 : min(2 * i + 2, 2 * tiles - 1));
          ok = __all_sync(0xffffffffu, mbar_wait(&sh.kv_full[at % kSlots], (at / kSlots) & 1, status, kWaitLimitCycles));
          if (!ok) break;
          uint8_t* v = ring + (at % kSlots) * kTileBytes;
          for (int x = r; x < (z1 - z0) * 8 * kHalves; x += 128) {
            const int row = z0 + x / (8 * kHalves), c = x % (8 * kHalves);
            *reinterpret_cast<uint4*>(v + (c / 8) * kHalfBytes + row * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
        }
        auto weights_ready = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.p_full[2 * g + (u & 1)]);
        };
        if (!warp_live) {
          weights_ready();
          continue;
        }
        const uint32_t ts = tm_s(g, u) + lanes;
        uint32_t s[2][32];
        tmem_ld32_start(ts, s[0]);
        tmem_ld32_start(ts + 32, s[1]);
        tmem_ld32_wait(s[0]);
        tmem_ld32_wait(s[1]);
        const int64_t left = static_cast<int64_t>(lim) - static_cast<int64_t>(t) * kAtTile - row0;
        if (__any_sync(0xffffffffu, left < kAtStep)) {
          const int below = left < -64 ? -64 : left > 64 ? 64 : static_cast<int>(left);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int x = below - 32 * c;  // entries of this run below lim
            uint32_t see = x >= 32 ? 0xffffffffu : x <= 0 ? 0u : (1u << x) - 1;
            if (bits != 0) {
              if (x >= 0 && x < 32) see |= static_cast<uint32_t>(bits << x);
              if (x < 0 && x > -64) see |= static_cast<uint32_t>(bits >> -x);
            }
#pragma unroll
            for (int k = 0; k < 32; ++k) s[c][k] = (see >> k) & 1 ? s[c][k] : 0xff800000u;  // -inf
          }
        }
        // The weights against the reference m: 16-bit values for the product
        // with V, half a step off at most; their sum stays in 32 bits.
        const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2);
        auto weights = [&]() {
          const float sub = m == -INFINITY ? 0.f : -m;
          const uint64_t sub2 = f32x2(sub, sub);
          uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float e0, e1;
              f32x2_split(fma_f32x2(f32x2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), scale2, sub2),
                          e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              sum[k % 4] = add_f32x2(sum[k % 4], f32x2(e0, e1));
              w[k] = Pack16<T>::pack(e0, e1);
            }
            tmem_st16(ts + 16 * c, w);
          }
          float l0, l1;
          f32x2_split(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), l0, l1);
          return l0 + l1;
        };
        // They go ahead with the reference so far while the step's maximum is
        // found beside them, and are done again in the few steps where the
        // reference has to rise.
        float now = weights();
        float tops[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t* x = &s[c / 2][16 * (c % 2)];
          tops[c] = __uint_as_float(x[0]);
#pragma unroll
          for (int k = 1; k < 15; k += 2) tops[c] = max3(tops[c], __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
          tops[c] = fmaxf(tops[c], __uint_as_float(x[15]));
        }
        const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * p.scale_log2;
        const bool rise = top > m + kAtRise || (m == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, rise)) {
          const float nm = rise ? top : m;
          const float al = rise ? ex2(m - nm) : 1.f;  // 0 at a row's first keys
          l *= al;
          m = nm;
          if (j > 0) {
            ok = product_done(g, u - 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32_start(tm_o(g) + lanes + 32 * c, o);
              tmem_ld32_wait(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
              tmem_st32(tm_o(g) + lanes + 32 * c, o);
            }
          }
          now = weights();
        }
        l += now;
        tmem_st_wait();
        weights_ready();
      }
      if (!ok) break;

      // ---- the part's results ----
      float* dst_o;
      float2* dst_ml;
      if (a.t0 == 0) {
        const int64_t row = (static_cast<int64_t>(a.line) * p.batch.N + tok) * p.n_q_heads + a.head * p.group + gq;
        dst_o = p.part_o + row * D;
        dst_ml = p.part_ml + row;
      } else {
        const int64_t row = (static_cast<int64_t>(cta) * 2 + a.line) * 256 + (two ? g * 128 : 0) + r;
        dst_o = p.slab_o + row * D;
        dst_ml = p.slab_ml + row;
      }
      // the last products; with one row tile both groups'
      ok = product_done(g, u0 + steps - 1) && (two || product_done(g ^ 1, u0 + steps - 1));
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
        const bool mine_to_write = r < rows;
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
            tmem_ld32(tm_o(1) + lanes + col, x);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = v[j] * f0 + x[j] * f1;
            if (mine_to_write) {
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                st_global_f8(dst_o + col + j, v + j);
            }
          }
        }
        if (mine_to_write && (two || g == 0)) *dst_ml = make_float2(m, l);
      }
      tc_fence_before();
      if (!two) {  // O and the exchanged values are free again once all have read them
        ok = meet_all(1);
        ph_meet ^= 1;
      }
      u0 += steps;
      base += 2 * tiles;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// join: one warp per row adds its parts
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(256) attend_join_kernel(const __grid_constant__ AttendParams p) {
  constexpr int kPer = D / 32;  // dims of a lane
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int n = static_cast<int>(row / p.n_q_heads), hq = static_cast<int>(row % p.n_q_heads);
  grid_dep_launch();
  grid_dep_wait();
  if (n >= p.batch.N) return;
  const int b = find_seq(p.batch.q_indptr, p.batch.B, n, lane);
  if (b < 0) return;
  const SeqSpan s = seq_span(p.batch, b);
  if (n < s.first || n >= s.first + s.n) return;
  const int head = hq / p.group, gq = hq % p.group;

  float o[kPer] = {}, m = -INFINITY, l = 0.f;
  // adds the parts of one item: `tiles` tiles of weight w from `off` on; `pos`
  // is the row's position in the item's block
  auto add = [&](int line, int64_t off, int tiles, int w, int pos) {
    if (tiles == 0) return;
    const int tile_row = pos % p.tok_tile * p.group + gq + (w == 2 ? pos / p.tok_tile * 128 : 0);
    const int64_t* begin = p.begin + line * (p.n_ctas + 1);
    for (int c0 = 0; c0 < p.n_ctas; c0 += 32) {
      // lane i: whether part c0 + i holds tiles of the item, and the item's first
      const int c = c0 + lane;
      int t0 = 0, t1 = 0;
      if (c < p.n_ctas) {
        t0 = tiles_before(begin[c], off, w, tiles);
        t1 = tiles_before(begin[c + 1], off, w, tiles);
      }
      unsigned parts = __ballot_sync(0xffffffffu, t0 < t1);
      const unsigned firsts = __ballot_sync(0xffffffffu, t0 == 0);
      while (parts != 0u) {
        // up to four parts' loads in flight, added in ascending order
        float x[4][kPer];
        float2 ml[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          ml[k] = make_float2(-INFINITY, 0.f);
          if (parts == 0u) continue;
          const int i = __ffs(parts) - 1;
          parts &= parts - 1;
          const bool first = (firsts >> i) & 1;
          const int cta = line == 0 ? c0 + i : p.n_ctas - 1 - (c0 + i);
          const int64_t at = first ? (static_cast<int64_t>(line) * p.batch.N + n) * p.n_q_heads + hq
                                   : (static_cast<int64_t>(cta) * 2 + line) * 256 + tile_row;
          ml[k] = (first ? p.part_ml : p.slab_ml)[at];
          const float* src = (first ? p.part_o : p.slab_o) + at * D + lane * kPer;
          if (kPer == 4)
            *reinterpret_cast<float4*>(x[k]) = *reinterpret_cast<const float4*>(src);
          else
            *reinterpret_cast<float2*>(x[k]) = *reinterpret_cast<const float2*>(src);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (ml[k].x == -INFINITY) continue;  // nothing seen: its O is not looked at
          const float mm = fmaxf(m, ml[k].x);
          const float fo = m == -INFINITY ? 0.f : ex2(m - mm), fx = ex2(ml[k].x - mm);
          m = mm;
          l = l * fo + ml[k].y * fx;
#pragma unroll
          for (int i = 0; i < kPer; ++i) o[i] = o[i] * fo + x[k][i] * fx;
        }
      }
    }
  };
  if (p.prefix_len > 0) {
    const PrefixLine pl = prefix_line(p);
    const int rb = n / (2 * p.tok_tile);
    add(0, head * pl.per_head + rb * 2LL * pl.tiles, pl.tiles, block_weight(pl.positions, p.tok_tile, rb),
        n - rb * 2 * p.tok_tile);
  }
  const int64_t begin = p.off[b], weight = p.off[b + 1] - begin;
  if (weight > 0) {
    const int rb = (n - s.first) / (2 * p.tok_tile);
    int64_t off = begin + head * (weight / p.n_heads);
    for (int i = 0; i < rb; ++i)
      off += static_cast<int64_t>(block_tiles(p, s, i)) * block_weight(s.n, p.tok_tile, i);
    add(1, off, block_tiles(p, s, rb), block_weight(s.n, p.tok_tile, rb), n - s.first - rb * 2 * p.tok_tile);
  }

  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* dst = p.out + n * p.o_ps + hq * p.o_hs + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) = Pack16<T>::pack(o[i] * inv, o[i + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[static_cast<int64_t>(n) * p.n_q_heads + hq] = l > 0.f ? (m + log2f(l)) * 0.693147180559945f : -INFINITY;
}

}  // namespace specv
