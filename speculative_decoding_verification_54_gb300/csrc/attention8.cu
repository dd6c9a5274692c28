// attention8.cu — host side of the 8-bit paged cache's calls and of the append with
// norms: argument checks and launches behind spec_kv_append_norm, spec_kv_append8,
// spec_kv_read8 and spec_prefix_attention8.
#include <cuda.h>
#include <cmath>
#include <mutex>

#include "append8.cuh"
#include "attend8.cuh"
#include "common.cuh"
#include "host.cuh"
#include "paged_host.cuh"
#include "spec_verify.h"

using namespace specv;

namespace {

constexpr int kAppendSmem = 32 * 1024;
constexpr int kAppend8Smem = kA8MaxOwn * 128 * static_cast<int>(sizeof(float2));  // rotated pairs of up to 256 dims

struct Device8 {
  int sms = 0;
  bool ready = false;
};

// SMs of the current device; the first call on a device raises the kernels'
// shared-memory limits.
int device8_sms(int* sms) {
  constexpr int kMaxDevices = 64;
  static Device8 devices[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPEC_ERR_CUDA;
  std::lock_guard<std::mutex> lk(mu);
  Device8& d = devices[dev];
  if (!d.ready) {
    auto raise = [](auto kernel, uint32_t bytes) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) ==
             cudaSuccess;
    };
    // the attention's warpgroups share out the registers it is launched with
    auto regs_fit = [](auto kernel) {
      cudaFuncAttributes a;
      return cudaFuncGetAttributes(&a, kernel) == cudaSuccess && a.numRegs == kQ8LaunchRegs;
    };
    if (!regs_fit(attend8_kernel<__nv_bfloat16, 64>) || !regs_fit(attend8_kernel<__nv_bfloat16, 128>) ||
        !regs_fit(attend8_kernel<__half, 64>) || !regs_fit(attend8_kernel<__half, 128>))
      return SPEC_ERR_CUDA;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        !raise(attend8_kernel<__nv_bfloat16, 64>, q8_smem_bytes<64>()) ||
        !raise(attend8_kernel<__nv_bfloat16, 128>, q8_smem_bytes<128>()) ||
        !raise(attend8_kernel<__half, 64>, q8_smem_bytes<64>()) ||
        !raise(attend8_kernel<__half, 128>, q8_smem_bytes<128>()) ||
        !raise(append_norm_kernel<__nv_bfloat16, kApart8, true>, kAppend8Smem) ||
        !raise(append_norm_kernel<__nv_bfloat16, kNeighbours, true>, kAppend8Smem) ||
        !raise(append_norm_kernel<__nv_bfloat16, kAnywhere, true>, kAppend8Smem) ||
        !raise(append_norm_kernel<__half, kApart8, true>, kAppend8Smem) ||
        !raise(append_norm_kernel<__half, kNeighbours, true>, kAppend8Smem) ||
        !raise(append_norm_kernel<__half, kAnywhere, true>, kAppend8Smem))
      return SPEC_ERR_CUDA;
    d.ready = true;
  }
  *sms = d.sms;
  return SPEC_OK;
}

bool vec16(int64_t stride) { return (stride & 15) == 0; }

// What the calls on an 8-bit cache check of it and of the batch.
int check_common8(const spec_kv_cache8* c, int n_q_heads, int N, const int32_t* q_indptr, int B, const int32_t* block_table,
                  int table_width) {
  if (c == nullptr || c->k_pages == nullptr || c->v_pages == nullptr || c->k_scales == nullptr || c->v_scales == nullptr ||
      q_indptr == nullptr || block_table == nullptr)
    return SPEC_ERR_INVALID_ARG;
  if (c->dtype != SPEC_BF16 && c->dtype != SPEC_F16) return SPEC_ERR_UNSUPPORTED;
  if (int e = check_sizes(B, N, n_q_heads, c->head_dim)) return e;
  if (c->n_heads < 1 || c->n_heads > n_q_heads || c->page_size < 1 || c->n_pages < 1 || c->n_pages > INT32_MAX ||
      table_width < 1)
    return SPEC_ERR_INVALID_ARG;
  if (c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0 || c->scale_page_stride < 0 ||
      c->scale_block_stride < 0 || c->scale_head_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  if ((c->block != 8 && c->block != 16 && c->block != 32 && c->block != 64) || c->head_dim % 16 != 0 || c->head_dim > 256)
    return SPEC_ERR_UNSUPPORTED;
  if (c->page_size % c->block != 0) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !vec16(c->page_stride) || !vec16(c->slot_stride) ||
      !vec16(c->head_stride))
    return SPEC_ERR_ALIGNMENT;
  return SPEC_OK;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

Paged8View view8_of(const spec_kv_cache8* c) {
  Paged8View v;
  v.k = static_cast<uint8_t*>(c->k_pages);
  v.v = static_cast<uint8_t*>(c->v_pages);
  v.k_scales = static_cast<uint8_t*>(c->k_scales);
  v.v_scales = static_cast<uint8_t*>(c->v_scales);
  v.page_stride = c->page_stride;
  v.slot_stride = c->slot_stride;
  v.head_stride = c->head_stride;
  v.s_page = c->scale_page_stride;
  v.s_block = c->scale_block_stride;
  v.s_head = c->scale_head_stride;
  v.n_pages = c->n_pages;
  v.page_size = c->page_size;
  v.n_heads = c->n_heads;
  v.block_shift = log2_of(c->block);
  return v;
}

// The pool [page, head, slot, dim] of codes in boxes of all dims x `rows` slots of
// one head and page (swizzled rows); pages past the last read as zero.
bool encode_pool8(CUtensorMap* m, const void* base, const spec_kv_cache8* c, int rows) {
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->head_dim), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->n_heads), static_cast<cuuint64_t>(c->n_pages)};
  // a dimension of one entry may have any stride, zero too: it is not used
  auto bytes = [&](int64_t stride, int64_t n) { return static_cast<cuuint64_t>(n == 1 ? c->head_dim : stride); };
  const cuuint64_t strides[3] = {bytes(c->slot_stride, c->page_size), bytes(c->head_stride, c->n_heads),
                                 bytes(c->page_stride, c->n_pages)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(c->head_dim), static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, c->head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool k8>
int launch_norm(const Append8Params& p, int interleaved, size_t smem, cudaStream_t s) {
  const dim3 grid((p.a.batch.N + p.a.tile - 1) / p.a.tile);
  const cudaError_t e = interleaved ? launch_pdl(append_norm_kernel<T, kNeighbours, k8>, grid, dim3(kA8Threads), smem, s, p)
                        : p.a.half % 8 == 0 ? launch_pdl(append_norm_kernel<T, kApart8, k8>, grid, dim3(kA8Threads), smem, s, p)
                                            : launch_pdl(append_norm_kernel<T, kAnywhere, k8>, grid, dim3(kA8Threads), smem, s, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// The norms' arguments and the launch, for a cache of either kind (p's cache,
// batch and rotation stand).  `block`: entries of a scale's block, 1 with 16 bits.
template <bool k8>
int append_norm(Append8Params& p, int dtype, int block, const float* q_weight, const float* k_weight, float eps,
                int interleaved, void* stream) {
  if (!(eps >= 0.f) || !std::isfinite(eps)) return SPEC_ERR_INVALID_ARG;
  int sms = 0;
  if (int e = device8_sms(&sms)) return e;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  const int per_row = (p.a.D / 8 + 1) / 2;  // lanes that hold two vectors each
  p.lanes = 1;
  while (p.lanes < per_row) p.lanes *= 2;
  // a unit's rows in kA8Steps steps of 32 / lanes rows a warp
  p.unit_warps = k8 ? block * p.lanes / (32 * kA8Steps) : 1;
  if (p.unit_warps < 1) p.unit_warps = 1;
  p.a.tile = (p.a.batch.N + 3 * sms - 1) / (3 * sms);
  // the cosines and sines of a position: vectors of eight angles, but for pairs anywhere
  p.unit_floats = !interleaved && p.a.half % 8 != 0 ? 2 * p.a.half : 16 * ((p.a.half + 7) / 8);
  p.inv_dims = 1.f / static_cast<float>(p.a.D);
  const int bytes = p.unit_floats * static_cast<int>(sizeof(float)), rest = k8 ? block - 1 : 0;
  const int most = !k8 && p.a.half > 0 ? kAppendSmem / bytes : kAppendMaxTile;
  if (p.a.tile > most) p.a.tile = most;
  if (p.a.tile > kAppendMaxTile) p.a.tile = kAppendMaxTile;
  // whole blocks, so that the CTAs have equally many
  if (k8 && p.a.tile > block) p.a.tile -= p.a.tile % block;
  const size_t smem = static_cast<size_t>(p.a.tile + rest) * bytes;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == SPEC_BF16 ? launch_norm<__nv_bfloat16, k8>(p, interleaved, smem, s)
                            : launch_norm<__half, k8>(p, interleaved, smem, s);
}

template <typename T, int D>
int launch_attend8(const Attend8Params& p, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.batch.N) * p.n_q_heads;
  if (launch_pdl(attend8_kernel<T, D>, dim3(p.n_ctas), dim3(kQ8Threads), q8_smem_bytes<D>(), s, p) != cudaSuccess ||
      launch_pdl(attend_join_kernel<T, D, Attend8Params>, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, s,
                 p) != cudaSuccess)
    return SPEC_ERR_CUDA;
  return SPEC_OK;
}

}  // namespace

extern "C" {

int spec_kv_append_norm(const spec_kv_cache* cache, const void* q, int64_t q_pos_stride, int64_t q_head_stride,
                        const void* k, int64_t k_pos_stride, int64_t k_head_stride, const void* v, int64_t v_pos_stride,
                        int64_t v_head_stride, int n_q_heads, int N, const int32_t* q_indptr, int B,
                        const int32_t* block_table, int table_width, const int32_t* kv_len, const float* inv_freq,
                        const int32_t* positions, int n_axes, const int32_t* axis, int rot_dim, int interleaved,
                        int64_t position_base, const float* q_weight, const float* k_weight, float norm_eps, void* q_out,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr) return SPEC_ERR_INVALID_ARG;
  if (int e = check_common(cache, n_q_heads, N, q_indptr, B, block_table, table_width, kv_len)) return e;
  if (int e = check_workspace(workspace, workspace_bytes, sizeof(WsHeader))) return e;
  Append8Params p = {};
  p.a.cache = view_of(cache);
  p.a.batch = batch_of(cache->page_size, N, q_indptr, B, block_table, table_width, kv_len, workspace);
  if (int e = append_params(p.a, cache->head_dim, q, q_pos_stride, q_head_stride, k, k_pos_stride, k_head_stride, v,
                            v_pos_stride, v_head_stride, n_q_heads, inv_freq, positions, n_axes, axis, rot_dim,
                            interleaved, position_base, q_out))
    return e;
  return append_norm<false>(p, cache->dtype, 1, q_weight, k_weight, norm_eps, interleaved, stream);
}

int spec_kv_append8(const spec_kv_cache8* cache, const void* q, int64_t q_pos_stride, int64_t q_head_stride,
                    const void* k, int64_t k_pos_stride, int64_t k_head_stride, const void* v, int64_t v_pos_stride,
                    int64_t v_head_stride, int n_q_heads, int N, const int32_t* q_indptr, int B,
                    const int32_t* block_table, int table_width, const int32_t* kv_len, const float* inv_freq,
                    const int32_t* positions, int n_axes, const int32_t* axis, int rot_dim, int interleaved,
                    int64_t position_base, const float* q_weight, const float* k_weight, float norm_eps, void* q_out,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr || kv_len == nullptr) return SPEC_ERR_INVALID_ARG;
  if (int e = check_common8(cache, n_q_heads, N, q_indptr, B, block_table, table_width)) return e;
  if (int e = check_workspace(workspace, workspace_bytes, sizeof(WsHeader))) return e;
  Append8Params p = {};
  p.c8 = view8_of(cache);
  p.a.cache.n_heads = cache->n_heads;
  p.a.batch = batch_of(cache->page_size, N, q_indptr, B, block_table, table_width, kv_len, workspace);
  if (int e = append_params(p.a, cache->head_dim, q, q_pos_stride, q_head_stride, k, k_pos_stride, k_head_stride, v,
                            v_pos_stride, v_head_stride, n_q_heads, inv_freq, positions, n_axes, axis, rot_dim,
                            interleaved, position_base, q_out))
    return e;
  return append_norm<true>(p, cache->dtype, cache->block, q_weight, k_weight, norm_eps, interleaved, stream);
}

int spec_kv_read8(const spec_kv_cache8* cache, const int32_t* out_indptr, int R, int B, const int32_t* block_table,
                  int table_width, const int32_t* first, void* k_out, int64_t k_pos_stride, int64_t k_head_stride,
                  void* v_out, int64_t v_pos_stride, int64_t v_head_stride, void* workspace, size_t workspace_bytes,
                  void* stream) {
  if (cache == nullptr || (k_out == nullptr && v_out == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (int e = check_common8(cache, cache->n_heads, R, out_indptr, B, block_table, table_width)) return e;
  if (int e = check_workspace(workspace, workspace_bytes, sizeof(WsHeader))) return e;
  if (!aligned16(k_out) || !aligned16(v_out) || !vec8(k_pos_stride) || !vec8(k_head_stride) || !vec8(v_pos_stride) ||
      !vec8(v_head_stride))
    return SPEC_ERR_ALIGNMENT;
  int sms = 0;
  if (int e = device8_sms(&sms)) return e;
  Read8Params p = {};
  p.c8 = view8_of(cache);
  p.batch = batch_of(cache->page_size, R, out_indptr, B, block_table, table_width, nullptr, workspace);
  p.first = first;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.k_ps = k_pos_stride;
  p.k_hs = k_head_stride;
  p.v_ps = v_pos_stride;
  p.v_hs = v_head_stride;
  p.D = cache->head_dim;
  p.tile = (R + 4 * sms - 1) / (4 * sms);
  if (p.tile > kR8MaxTile) p.tile = kR8MaxTile;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((R + p.tile - 1) / p.tile);
  const cudaError_t e = cache->dtype == SPEC_BF16 ? launch_pdl(read8_kernel<__nv_bfloat16>, grid, dim3(kR8Threads), 0, s, p)
                                                  : launch_pdl(read8_kernel<__half>, grid, dim3(kR8Threads), 0, s, p);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

int spec_prefix_attention8(const spec_kv_cache8* cache, const void* q, int64_t q_pos_stride, int64_t q_head_stride,
                           int n_q_heads, int N, const int32_t* q_indptr, int B, const int32_t* prefix_table,
                           int64_t prefix_len, const int32_t* block_table, int table_width, const int32_t* kv_len,
                           const uint64_t* draft_mask, float scale, void* out, int64_t out_pos_stride,
                           int64_t out_head_stride, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (q == nullptr || out == nullptr || kv_len == nullptr) return SPEC_ERR_INVALID_ARG;
  if (int e = check_common8(cache, n_q_heads, N, q_indptr, B, block_table, table_width)) return e;
  const AttnLayout L = attn_layout(N, n_q_heads, cache->head_dim, prefix_len > 0);
  if (int e = check_workspace(workspace, workspace_bytes, L.total)) return e;
  if (prefix_len < 0 || prefix_len > INT32_MAX - kAtTile || (prefix_len > 0 && prefix_table == nullptr) || !(scale > 0.f) ||
      !std::isfinite(scale))
    return SPEC_ERR_INVALID_ARG;
  if (n_q_heads % cache->n_heads != 0 || q_pos_stride < 0 || q_head_stride < 0) return SPEC_ERR_INVALID_ARG;
  if ((cache->head_dim != 64 && cache->head_dim != 128) || n_q_heads / cache->n_heads > 128) return SPEC_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(out) || !vec8(q_pos_stride) || !vec8(q_head_stride) || !vec8(out_pos_stride) ||
      !vec8(out_head_stride))
    return SPEC_ERR_ALIGNMENT;
  int sms = 0;
  if (int e = device8_sms(&sms)) return e;
  Attend8Params p = {};
  // a box lies inside one page and one key tile
  p.box_rows = 8;
  while (p.box_rows < kAtTile && cache->page_size % (2 * p.box_rows) == 0) p.box_rows *= 2;
  p.group = n_q_heads / cache->n_heads;
  p.tok_tile = kAtTile / p.group;
  p.block = p.tok_tile;
  p.narrow = 64 / p.group;
  if (!encode_pool8(&p.tmK, cache->k_pages, cache, p.box_rows) || !encode_pool8(&p.tmV, cache->v_pages, cache, p.box_rows) ||
      !encode_queries(&p.tmQ, q, cache->dtype, cache->head_dim, N, n_q_heads, q_pos_stride, q_head_stride, p.group,
                      p.tok_tile))
    return SPEC_ERR_INVALID_ARG;  // strides beyond what a tensor map takes
  p.out = static_cast<uint16_t*>(out);
  p.o_ps = out_pos_stride;
  p.o_hs = out_head_stride;
  p.lse = lse;
  p.q = static_cast<const uint16_t*>(q);
  p.q_ps = q_pos_stride;
  p.q_hs = q_head_stride;
  p.c8 = view8_of(cache);
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
    return bf16 ? launch_attend8<__nv_bfloat16, 64>(p, s) : launch_attend8<__half, 64>(p, s);
  return bf16 ? launch_attend8<__nv_bfloat16, 128>(p, s) : launch_attend8<__half, 128>(p, s);
}

}  // extern "C"
