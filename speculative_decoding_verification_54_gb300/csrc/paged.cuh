// paged.cuh — what the kernels of the paged key/value cache share: the cache's
// view, the sequence a new position belongs to, and its entries' lengths.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace specv {

struct PagedView {
  uint16_t* k;  // 16-bit elements of either type
  uint16_t* v;
  int64_t page_stride, slot_stride, head_stride;  // elements
  int64_t n_pages;
  int page_size, n_heads;
};

// The new positions and pages of a call's sequences (device arrays).
struct PagedBatch {
  const int32_t* q_indptr;     // [B + 1]
  const int32_t* block_table;  // [B, table_width]
  const int32_t* kv_len;       // [B]
  int B, N, table_width, page_size;
  int* status;
};

// entries of a sequence: key tiles past them still count in 32 bits
constexpr int64_t kMaxEntries = 0x7fffffff - 255;

// Sequence b's rows and lengths, with every value that the host cannot check
// clamped into its range (the status word records that).
struct SeqSpan {
  int first, n;  // rows first .. first + n - 1 of the new positions
  int64_t kv;    // entries of its own pages, the new ones among them
  int64_t shift; // new position n is entry n + shift, by the lengths as given: not clamped
};

__device__ __forceinline__ SeqSpan seq_span(const PagedBatch& p, int b) {
  SeqSpan s;
  const int a = p.q_indptr[b], e = p.q_indptr[b + 1], kv = p.kv_len[b];
  s.first = min(max(a, 0), p.N);
  s.n = min(max(e, s.first), p.N) - s.first;
  s.kv = min(static_cast<int64_t>(max(kv, 0)), static_cast<int64_t>(p.table_width) * p.page_size);
  s.kv = min(s.kv, kMaxEntries);
  s.shift = static_cast<int64_t>(kv) - e;
  if (s.first != a || s.first + s.n != e || s.kv != kv || s.kv < s.n || (b == 0 && a != 0))
    atomicOr(p.status, kStatusBadCache);
  return s;
}

// The rows that belong to a sequence: from the first one's to the last one's.
__device__ __forceinline__ bool in_batch(const PagedBatch& p, int n) {
  const int first = p.q_indptr[0], end = p.q_indptr[p.B];  // both loads at once
  return (n >= first) & (n < end);
}

// The sequence whose rows hold `n`, found by a whole warp in steps of 32 (two
// dependent loads up to 1,024 sequences); -1 where none does (padding).
__device__ __forceinline__ int find_seq(const PagedBatch& p, int n, int lane) {
  const int32_t* const q_indptr = p.q_indptr;
  int lo = 0, len = p.B;  // the last b of [lo, lo + len) with q_indptr[b] <= n
  if (!in_batch(p, n)) return -1;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lane * step;
    const unsigned below = __ballot_sync(0xffffffffu, at < len && q_indptr[lo + at] <= n);
    const int hop = (below == 0u ? 0 : 31 - __clz(below)) * step;
    lo += hop;
    len = min(step, len - hop);
  }
  return lo;
}

}  // namespace specv
