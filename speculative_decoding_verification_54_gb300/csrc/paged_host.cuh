// paged_host.cuh — what the host sides of the paged cache's calls share: sizes,
// the attention's workspace, the batch's view and the queries' tensor map.
#pragma once

#include "attend.cuh"
#include "host.cuh"
#include "paged.cuh"
#include "spec_verify.h"

namespace specv {

struct AttnLayout {
  size_t header, begin, part_meta, part_o, part_ml, slab_o, slab_ml, total;
  int slab_rows;
};

// The parts of the rows (one place per row for the prefix, if there is any,
// and one for its own pages) and of the CTAs (one slab each: the rows of a block,
// which are two row tiles or all there are).
inline AttnLayout attn_layout(int N, int n_q_heads, int D, bool prefix) {
  AttnLayout L;
  const int64_t places = static_cast<int64_t>(N) * n_q_heads;
  L.slab_rows = static_cast<int>(places < 2 * kAtTile ? places : 2 * kAtTile);
  const size_t rows = (prefix ? 2 : 1) * static_cast<size_t>(places), slab_rows = size_t(kAtMaxCtas) * L.slab_rows;
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, 256);
    return at;
  };
  L.header = take(sizeof(WsHeader));
  L.begin = take((size_t(kAtMaxCtas) + 1) * sizeof(int64_t));
  L.part_meta = take(rows * sizeof(int4));
  L.part_o = take(rows * D * sizeof(float));
  L.part_ml = take(rows * sizeof(float2));
  L.slab_o = take(slab_rows * D * sizeof(float));
  L.slab_ml = take(slab_rows * sizeof(float2));
  L.total = off;
  return L;
}

constexpr int kMaxRowsPerCall = 1 << 24;

inline int check_sizes(int B, int N, int n_q_heads, int D) {
  if (B < 1 || B > 65535 || N < 1 || N > kMaxRowsPerCall || n_q_heads < 1 || n_q_heads > 4096 || D < 8 || D > 512 ||
      (D % 8) != 0)
    return SPEC_ERR_INVALID_ARG;
  return SPEC_OK;
}

inline bool vec8(int64_t stride) { return (stride & 7) == 0; }

// What the calls check of the cache and the batch.
inline int check_common(const spec_kv_cache* c, int n_q_heads, int N, const int32_t* q_indptr, int B,
                        const int32_t* block_table, int table_width, const int32_t* kv_len) {
  if (c == nullptr || c->k_pages == nullptr || c->v_pages == nullptr || q_indptr == nullptr ||
      block_table == nullptr || kv_len == nullptr)
    return SPEC_ERR_INVALID_ARG;
  if (c->dtype != SPEC_BF16 && c->dtype != SPEC_F16) return SPEC_ERR_UNSUPPORTED;
  if (int e = check_sizes(B, N, n_q_heads, c->head_dim)) return e;
  if (c->n_heads < 1 || c->n_heads > n_q_heads || c->page_size < 1 || c->n_pages < 1 || c->n_pages > INT32_MAX ||
      table_width < 1)
    return SPEC_ERR_INVALID_ARG;
  if (c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !vec8(c->page_stride) || !vec8(c->slot_stride) ||
      !vec8(c->head_stride))
    return SPEC_ERR_ALIGNMENT;
  return SPEC_OK;
}

inline int check_workspace(const void* ws, size_t bytes, size_t needed) {
  return ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < needed ? SPEC_ERR_WORKSPACE : SPEC_OK;
}

inline PagedView view_of(const spec_kv_cache* c) {
  PagedView v;
  v.k = static_cast<uint16_t*>(c->k_pages);
  v.v = static_cast<uint16_t*>(c->v_pages);
  v.page_stride = c->page_stride;
  v.slot_stride = c->slot_stride;
  v.head_stride = c->head_stride;
  v.n_pages = c->n_pages;
  v.page_size = c->page_size;
  v.n_heads = c->n_heads;
  return v;
}

inline PagedBatch batch_of(int page_size, int N, const int32_t* q_indptr, int B, const int32_t* block_table,
                           int table_width, const int32_t* kv_len, void* ws) {
  PagedBatch b;
  b.q_indptr = q_indptr;
  b.block_table = block_table;
  b.kv_len = kv_len;
  b.B = B;
  b.N = N;
  b.table_width = table_width;
  b.page_size = page_size;
  b.status = reinterpret_cast<int*>(ws);
  return b;
}

// The queries [position, head, dim] in boxes of one row tile: 64 dims of
// `group` heads of `positions` positions; past the last position zeros.
inline bool encode_queries(CUtensorMap* m, const void* q, int dtype, int head_dim, int N, int n_q_heads,
                           int64_t pos_stride, int64_t head_stride, int group, int positions) {
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(n_q_heads),
                              static_cast<cuuint64_t>(N)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(n_q_heads == 1 ? head_dim : head_stride) * 2,
                                 static_cast<cuuint64_t>(N == 1 ? head_dim : pos_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(positions)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
             const_cast<void*>(q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The appends' checks of everything but the cache and the batch, and their
// parameters (p's cache and batch stand already).
inline int append_params(AppendParams& p, int D, const void* q, int64_t q_pos_stride, int64_t q_head_stride, const void* k,
                         int64_t k_pos_stride, int64_t k_head_stride, const void* v, int64_t v_pos_stride,
                         int64_t v_head_stride, int n_q_heads, const float* inv_freq, const int32_t* positions, int n_axes,
                         const int32_t* axis, int rot_dim, int interleaved, int64_t position_base, void* q_out) {
  if (rot_dim < 0 || rot_dim > D || (rot_dim & 1) != 0 || (rot_dim > 0 && inv_freq == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return SPEC_ERR_INVALID_ARG;
  // without positions there is one axis; with several, each frequency names its own
  if (n_axes < 1 || n_axes > 16 || (positions == nullptr && n_axes != 1) ||
      (n_axes > 1 && axis == nullptr && rot_dim > 0) || position_base < 0)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !vec8(q_pos_stride) ||
      !vec8(q_head_stride) || !vec8(k_pos_stride) || !vec8(k_head_stride) || !vec8(v_pos_stride) ||
      !vec8(v_head_stride))
    return SPEC_ERR_ALIGNMENT;
  // a head's second half is read after its first half may have been written
  if (q == q_out) return SPEC_ERR_INVALID_ARG;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_ps = q_pos_stride;
  p.q_hs = q_head_stride;
  p.k_ps = k_pos_stride;
  p.k_hs = k_head_stride;
  p.v_ps = v_pos_stride;
  p.v_hs = v_head_stride;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.axis = axis;
  p.position_base = position_base;
  p.n_axes = n_axes;
  p.n_q_heads = n_q_heads;
  p.D = D;
  p.half = rot_dim / 2;
  return SPEC_OK;
}

// Where the attention keeps what in its workspace.
inline void workspace_params(AttendParams& p, const AttnLayout& L, void* workspace) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.begin = reinterpret_cast<int64_t*>(ws + L.begin);
  p.part_meta = reinterpret_cast<int4*>(ws + L.part_meta);
  p.part_o = reinterpret_cast<float*>(ws + L.part_o);
  p.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
  p.slab_o = reinterpret_cast<float*>(ws + L.slab_o);
  p.slab_ml = reinterpret_cast<float2*>(ws + L.slab_ml);
  p.slab_rows = L.slab_rows;
}

}  // namespace specv
