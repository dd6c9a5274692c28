// attend.cuh — attention of the new positions over a shared prefix and their
// sequences' pages.
#pragma once

#include <cfloat>

#include "kvappend.cuh"
#include "paged.cuh"

namespace specv {

struct AttendParams {
  const uint16_t* q;
  int64_t q_ps, q_hs;
  uint16_t* out;
  int64_t o_ps, o_hs;
  float* lse;
  PagedView cache;
  PagedBatch batch;
  const int32_t* prefix_table;
  int64_t prefix_len;
  const uint64_t* draft_mask;
  float scale;
  int n_q_heads, group, D;
};

// One warp per new position and query head; lane i scores key 32 k + i.
template <typename T, int D>
__global__ void __launch_bounds__(128) attend_simple_kernel(const __grid_constant__ AttendParams p) {
  __shared__ float s_q[4][D];
  __shared__ int64_t s_row[4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_launch();
  grid_dep_wait();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  const int n = static_cast<int>(item / p.n_q_heads), h = static_cast<int>(item % p.n_q_heads);
  if (n >= p.batch.N) return;
  const int b = find_seq(p.batch.q_indptr, p.batch.B, n, lane);
  if (b < 0) return;
  const SeqSpan sp = seq_span(p.batch, b);
  if (n < sp.first || n >= sp.first + sp.n) return;
  const int hk = h / p.group;
  for (int d = lane; d < D; d += 32) s_q[warp][d] = Pack16<T>::up(p.q[n * p.q_ps + h * p.q_hs + d]);
  __syncwarp();
  float o[D / 32] = {}, m = -INFINITY, l = 0.f;
  const int64_t old = sp.kv - sp.n;
  for (int phase = 0; phase < 2; ++phase) {
    const int64_t len = phase == 0 ? p.prefix_len : sp.kv;
    for (int64_t k0 = 0; k0 < len; k0 += 32) {
      const int64_t key = k0 + lane;
      int64_t row = -1;
      bool seen = false;
      if (key < len) {
        const int page = phase == 0 ? p.prefix_table[key / p.batch.page_size]
                                    : p.batch.block_table[static_cast<int64_t>(b) * p.batch.table_width +
                                                          key / p.batch.page_size];
        if (page >= 0 && page < p.cache.n_pages)
          row = page * p.cache.page_stride + (key % p.batch.page_size) * p.cache.slot_stride + hk * p.cache.head_stride;
        else
          atomicOr(p.batch.status, kStatusBadCache);
        const int64_t nw = key - old;
        seen = phase == 0 || nw < 0 ||
               (p.draft_mask != nullptr ? nw < 64 && ((p.draft_mask[n] >> nw) & 1) : nw <= n - sp.first);
      }
      float s = 0.f;
      if (row >= 0)
        for (int d = 0; d < D; ++d) s = fmaf(s_q[warp][d], Pack16<T>::up(p.cache.k[row + d]), s);
      s = seen ? s * p.scale : -INFINITY;
      float mt = s;
      for (int x = 16; x; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
      const float mn = fmaxf(m, mt);
      if (mn == -INFINITY) continue;
      const float al = ex2((m - mn) * kLog2e), w = ex2((s - mn) * kLog2e);
      m = mn;
      l *= al;
      for (int i = 0; i < D / 32; ++i) o[i] *= al;
      float lt = w;
      for (int x = 16; x; x >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, x);
      l += lt;
      s_row[warp][lane] = row;
      __syncwarp();
      for (int t = 0; t < 32; ++t) {
        const float wt = __shfl_sync(0xffffffffu, w, t);
        const int64_t rt = s_row[warp][t];
        if (rt < 0 || wt == 0.f) continue;
        for (int i = 0; i < D / 32; ++i) o[i] = fmaf(wt, Pack16<T>::up(p.cache.v[rt + i * 32 + lane]), o[i]);
      }
      __syncwarp();
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < D / 32; ++i)
    p.out[n * p.o_ps + h * p.o_hs + i * 32 + lane] =
        static_cast<uint16_t>(Pack16<T>::pack(o[i] * inv, 0.f) & 0xffffu);
  if (lane == 0 && p.lse != nullptr)
    p.lse[static_cast<int64_t>(n) * p.n_q_heads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace specv
