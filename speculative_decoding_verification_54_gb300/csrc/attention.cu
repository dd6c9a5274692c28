// attention.cu — host side of the paged cache's calls: argument checks,
// workspace layout and launches behind spec_kv_append and
// spec_prefix_attention.
#include <cuda.h>
#include <cmath>
#include <mutex>

#include "attend.cuh"
#include "common.cuh"
#include "host.cuh"
#include "kvappend.cuh"
#include "paged_host.cuh"
#include "spec_verify.h"

using namespace specv;

namespace {

struct AttnDevice {
  int sms = 0;
  bool ready = false;
};

// SMs of the current device; the first call on a device raises the attention
// kernels' shared-memory limits.
int device_sms(int* sms) {
  constexpr int kMaxDevices = 64;
  static AttnDevice devices[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPEC_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  AttnDevice& d = devices[dev];
  if (!d.ready) {
    auto raise = [](auto kernel, uint32_t bytes) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) ==
             cudaSuccess;
    };
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        !raise(attend_kernel<__nv_bfloat16, 64>, at_smem_bytes<64>()) ||
        !raise(attend_kernel<__nv_bfloat16, 128>, at_smem_bytes<128>()) ||
        !raise(attend_kernel<__half, 64>, at_smem_bytes<64>()) ||
        !raise(attend_kernel<__half, 128>, at_smem_bytes<128>()))
      return SPEC_ERR_CUDA;
    d.ready = true;
  }
  *sms = d.sms;
  return SPEC_OK;
}

// The pool [page, head, slot, dim] in boxes of 64 dims x `rows` slots of one
// head and page (128-byte rows, swizzled); pages past the last read as zero.
bool encode_pool(CUtensorMap* m, const void* base, const spec_kv_cache* c, int rows) {
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->head_dim), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->n_heads), static_cast<cuuint64_t>(c->n_pages)};
  // a dimension of one entry may have any stride, zero too: it is not used
  auto bytes = [&](int64_t stride, int64_t n) {
    return static_cast<cuuint64_t>(n == 1 ? c->head_dim : stride) * 2;
  };
  const cuuint64_t strides[3] = {bytes(c->slot_stride, c->page_size), bytes(c->head_stride, c->n_heads),
                                 bytes(c->page_stride, c->n_pages)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, c->dtype == SPEC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
int launch_append(const AppendParams& p, int interleaved, cudaStream_t s) {
  const dim3 grid((p.batch.N + p.tile - 1) / p.tile);
  const size_t smem = static_cast<size_t>(p.tile) * p.half * sizeof(float2);
  const cudaError_t e = interleaved ? launch_pdl(kv_append_kernel<T, true>, grid, dim3(kAppendThreads), smem, s, p)
                                    : launch_pdl(kv_append_kernel<T, false>, grid, dim3(kAppendThreads), smem, s, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

template <typename T, int D>
int launch_attend(const AttendParams& p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.batch.N) * p.n_q_heads;
  if (launch_pdl(attend_kernel<T, D>, dim3(p.n_ctas), dim3(kAtThreads), at_smem_bytes<D>(), s, p) != cudaSuccess ||
      launch_pdl(attend_join_kernel<T, D, AttendParams>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, s, p) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // namespace

extern "C" {

int spec_prefix_attention_workspace_bytes(int B, int N, int n_q_heads, int head_dim, int64_t prefix_len,
                                          size_t* bytes) {
  if (bytes == nullptr || prefix_len < 0) return SPEC_ERR_INVALID_ARG;
  if (int e = check_sizes(B, N, n_q_heads, head_dim)) return e;
  *bytes = attn_layout(N, n_q_heads, head_dim, prefix_len > 0).total;
  return SPEC_OK;
}

int spec_attention_workspace_bytes(int B, int N, int n_q_heads, int head_dim, size_t* bytes) {
  return spec_prefix_attention_workspace_bytes(B, N, n_q_heads, head_dim, 1, bytes);
}

int spec_kv_append_workspace_bytes(size_t* bytes) {
  if (bytes == nullptr) return SPEC_ERR_INVALID_ARG;
  *bytes = sizeof(WsHeader);  // the status word's
  return SPEC_OK;
}

int spec_kv_append(const spec_kv_cache* cache, const void* q, int64_t q_pos_stride, int64_t q_head_stride,
                   const void* k, int64_t k_pos_stride, int64_t k_head_stride, const void* v, int64_t v_pos_stride,
                   int64_t v_head_stride, int n_q_heads, int N, const int32_t* q_indptr, int B,
                   const int32_t* block_table, int table_width, const int32_t* kv_len, const float* inv_freq,
                   const int32_t* positions, int n_axes, const int32_t* axis, int rot_dim, int interleaved,
                   int64_t position_base, void* q_out, void* workspace, size_t workspace_bytes, void* stream) {
  if (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr) return SPEC_ERR_INVALID_ARG;
  if (int e = check_common(cache, n_q_heads, N, q_indptr, B, block_table, table_width, kv_len)) return e;
  if (int e = check_workspace(workspace, workspace_bytes, sizeof(WsHeader))) return e;
  AppendParams p = {};
  p.cache = view_of(cache);
  p.batch = batch_of(cache->page_size, N, q_indptr, B, block_table, table_width, kv_len, workspace);
  if (int e = append_params(p, cache->head_dim, q, q_pos_stride, q_head_stride, k, k_pos_stride, k_head_stride, v,
                            v_pos_stride, v_head_stride, n_q_heads, inv_freq, positions, n_axes, axis, rot_dim,
                            interleaved, position_base, q_out))
    return e;
  // Positions a CTA takes: as few as fill the GPU once with three CTAs an SM,
  // at most 24 (32,768 positions of 256 dims: 24 a CTA 188 us, 8 186 us, 4 195
  // us, 2 232 us; 5,528 of 128, where 13 fill the GPU once: 13 20.0 us, 8 22.2
  // us, 4 26.5 us), and no more than 32 KB of cosines and sines.
  int sms = 0;
  if (int e = device_sms(&sms)) return e;
  p.tile = (N + 3 * sms - 1) / (3 * sms);
  const int most = p.half > 0 ? 32 * 1024 / (p.half * static_cast<int>(sizeof(float2))) : kAppendMaxTile;
  if (p.tile > most) p.tile = most;
  if (p.tile > kAppendMaxTile) p.tile = kAppendMaxTile;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cache->dtype == SPEC_BF16 ? launch_append<__nv_bfloat16>(p, interleaved, s)
                                   : launch_append<__half>(p, interleaved, s);
}

int spec_prefix_attention(const spec_kv_cache* cache, const void* q, int64_t q_pos_stride, int64_t q_head_stride,
                          int n_q_heads, int N, const int32_t* q_indptr, int B, const int32_t* prefix_table,
                          int64_t prefix_len, const int32_t* block_table, int table_width, const int32_t* kv_len,
                          const uint64_t* draft_mask, float scale, void* out, int64_t out_pos_stride,
                          int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (q == nullptr || out == nullptr) return SPEC_ERR_INVALID_ARG;
  if (int e = check_common(cache, n_q_heads, N, q_indptr, B, block_table, table_width, kv_len)) return e;
  const AttnLayout L = attn_layout(N, n_q_heads, cache->head_dim, prefix_len > 0);
  if (int e = check_workspace(workspace, workspace_bytes, L.total)) return e;
  if (prefix_len < 0 || prefix_len > INT32_MAX - kAtTile || (prefix_len > 0 && prefix_table == nullptr) || !(scale > 0.f) || !std::isfinite(scale))
    return SPEC_ERR_INVALID_ARG;
  if (n_q_heads % cache->n_heads != 0 || q_pos_stride < 0 || q_head_stride < 0) return SPEC_ERR_INVALID_ARG;
  if ((cache->head_dim != 64 && cache->head_dim != 128) || cache->page_size % 8 != 0 ||
      n_q_heads / cache->n_heads > 128)
    return SPEC_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out) || !vec8(q_pos_stride) || !vec8(q_head_stride) || !vec8(out_pos_stride) ||
      !vec8(out_head_stride))
    return SPEC_ERR_ALIGNMENT;
  int sms = 0;
  if (int e = device_sms(&sms)) return e;
  AttendParams p = {};
  // a box lies inside one page and one key tile
  p.box_rows = 8;
  while (p.box_rows < kAtTile && cache->page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
  p.group = n_q_heads / cache->n_heads;
  p.tok_tile = kAtTile / p.group;
  p.block = 2 * p.tok_tile;
  p.narrow = p.tok_tile;
  if (!encode_pool(&p.tmK, cache->k_pages, cache, p.box_rows) ||
      !encode_pool(&p.tmV, cache->v_pages, cache, p.box_rows) ||
      !encode_queries(&p.tmQ, q, cache->dtype, cache->head_dim, N, n_q_heads, q_pos_stride, q_head_stride, p.group, p.tok_tile))
    return SPEC_ERR_INVALID_ARG;  // strides beyond what a tensor map takes
  p.out = static_cast<uint16_t*>(out);
  p.o_ps = out_pos_stride;
  p.o_hs = out_head_stride;
  p.lse = lse;
  p.q = static_cast<const uint16_t*>(q);
  p.q_ps = q_pos_stride;
  p.q_hs = q_head_stride;
  p.cache = view_of(cache);
  p.batch = batch_of(cache->page_size, N, q_indptr, B, block_table, table_width, kv_len, workspace);
  p.n_pages = static_cast<int>(cache->n_pages);
  p.prefix_table = prefix_table;
  p.prefix_len = static_cast<int>(prefix_len);
  p.draft_mask = draft_mask;
  p.scale_log2 = scale * kLog2e;
  p.n_q_heads = n_q_heads;
  p.n_heads = cache->n_heads;
  p.n_ctas = sms < kAtMaxCtas ? sms : kAtMaxCtas;
  workspace_params(p, L, workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = cache->dtype == SPEC_BF16;
  if (cache->head_dim == 64)
    return bf16 ? launch_attend<__nv_bfloat16, 64>(p, s) : launch_attend<__half, 64>(p, s);
  return bf16 ? launch_attend<__nv_bfloat16, 128>(p, s) : launch_attend<__half, 128>(p, s);
}

}  // extern "C"
