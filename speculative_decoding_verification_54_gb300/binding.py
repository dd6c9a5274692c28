"""Thin ctypes binding of libspecverify (spec_verify.h), same names as the C ABI.

Argument marshalling only: every step of the verify path runs in the CUDA
kernels of the shared library.  Tensors are torch CUDA tensors (PyTorch is
used for device memory and streams); raw integer device addresses are also
accepted where noted.  A missing or unloadable library raises immediately —
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

SPEC_F32, SPEC_BF16, SPEC_F16 = 0, 1, 2
SPEC_OK = 0
SPEC_ERR_INVALID_ARG = -1
SPEC_ERR_UNSUPPORTED = -2
SPEC_ERR_ALIGNMENT = -3
SPEC_ERR_WORKSPACE = -4
SPEC_ERR_CUDA = -5
SPEC_ERR_TIMEOUT = -6
SPEC_ERR_DEVICE_INPUT = -7
SPEC_ERR_STATE = -8
SPEC_ERR_DEVICE_BOUNDS = -9
MAX_GAMMA = 31

EXPORTED = (
    "spec_verify_workspace_bytes", "spec_verify_workspace_init", "spec_verify_greedy",
    "spec_verify_sample", "spec_verify_status", "spec_verify_error_string",
    "spec_verify_version", "spec_verify_selftest_timeout", "spec_verify_sample_reduce_only",
    "spec_verify_sample_noalloc", "spec_verify_lmhead_sample", "spec_verify_lmhead_gemm_only",
    "spec_verify_greedy_multi", "spec_round_update", "spec_verify_topkp_workspace_bytes",
    "spec_verify_sample_topkp", "spec_centroid_head_workspace_bytes", "spec_centroid_head",
    "spec_verify_sparse_workspace_bytes", "spec_verify_sample_sparse",
    "spec_attention_workspace_bytes", "spec_kv_append", "spec_prefix_attention",
    "spec_kv_append_workspace_bytes", "spec_prefix_attention_workspace_bytes",
    "spec_kv_append_norm", "spec_kv_append8", "spec_kv_read8", "spec_prefix_attention8",
)


class SpecVerifyError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        super().__init__(f"{what}: {error_string(code)} ({code})" if what else f"{error_string(code)} ({code})")


_lib = None
_vp, _sz, _i, _i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64


def lib_path() -> str:
    return _build.LIB


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the shared library (built by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libspecverify not built ({path} missing); run __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    lib.spec_verify_workspace_bytes.argtypes = [_i, _i, _i, _i, ctypes.POINTER(_sz)]
    lib.spec_verify_workspace_init.argtypes = [_vp, _sz, _vp]
    lib.spec_verify_greedy.argtypes = [_vp, _i, _vp, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]
    lib.spec_verify_greedy_multi.argtypes = [_vp, _i, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _sz, _vp]
    lib.spec_verify_sample.argtypes = [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i,
                                       _vp, _vp, _vp, _vp, _sz, _vp]
    lib.spec_verify_sample_reduce_only.argtypes = list(lib.spec_verify_sample.argtypes)
    lib.spec_verify_sample_noalloc.argtypes = [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i,
                                               _vp, _vp, _vp, _vp]
    lib.spec_verify_lmhead_sample.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i,
                                              _vp, _vp, _vp, _vp, _sz, _vp]
    lib.spec_verify_lmhead_gemm_only.argtypes = list(lib.spec_verify_lmhead_sample.argtypes)
    lib.spec_round_update.argtypes = [_vp, _vp, _i, _i, _i, _vp, _vp]
    lib.spec_verify_topkp_workspace_bytes.argtypes = [_i, _i, _i, ctypes.POINTER(_sz)]
    lib.spec_verify_sample_topkp.argtypes = [_vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, ctypes.c_float,
                                             _vp, _vp, _vp, _vp, _sz, _vp]
    lib.spec_centroid_head_workspace_bytes.argtypes = [_i, _i, _i, ctypes.POINTER(_sz)]
    lib.spec_centroid_head.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                                       _vp, _sz, _vp]
    lib.spec_verify_sparse_workspace_bytes.argtypes = [_i, _i, _i, ctypes.POINTER(_sz)]
    lib.spec_verify_sample_sparse.argtypes = [_vp, _i, _vp, _vp, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i,
                                              _vp, _vp, _vp, _vp, _sz, _vp]
    lib.spec_attention_workspace_bytes.argtypes = [_i, _i, _i, _i, ctypes.POINTER(_sz)]
    lib.spec_kv_append_workspace_bytes.argtypes = [ctypes.POINTER(_sz)]
    lib.spec_prefix_attention_workspace_bytes.argtypes = [_i, _i, _i, _i, _i64, ctypes.POINTER(_sz)]
    lib.spec_kv_append.argtypes = [_vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i, _i, _vp, _i, _vp, _i, _vp,
                                   _vp, _vp, _i, _vp, _i, _i, _i64, _vp, _vp, _sz, _vp]
    lib.spec_prefix_attention.argtypes = [_vp, _vp, _i64, _i64, _i, _i, _vp, _i, _vp, _i64, _vp, _i, _vp, _vp,
                                          ctypes.c_float, _vp, _i64, _i64, _vp, _vp, _sz, _vp]
    lib.spec_kv_append_norm.argtypes = lib.spec_kv_append.argtypes[:24] + [_vp, _vp, ctypes.c_float, _vp, _vp, _sz, _vp]
    lib.spec_kv_append8.argtypes = list(lib.spec_kv_append_norm.argtypes)
    lib.spec_kv_read8.argtypes = [_vp, _vp, _i, _i, _vp, _i, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _sz, _vp]
    lib.spec_prefix_attention8.argtypes = list(lib.spec_prefix_attention.argtypes)
    lib.spec_verify_status.argtypes = [_vp, _vp]
    lib.spec_verify_error_string.argtypes = [_i]
    lib.spec_verify_error_string.restype = ctypes.c_char_p
    lib.spec_verify_version.argtypes = []
    lib.spec_verify_selftest_timeout.argtypes = [_vp, _sz, _vp]
    for name in EXPORTED:
        if name not in ("spec_verify_error_string",):
            getattr(lib, name).restype = _i
    _lib = lib
    return lib


def error_string(code: int) -> str:
    return load().spec_verify_error_string(int(code)).decode()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _ptr(t):
    """Device address of a tensor (or an int address), None for None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.float32:
        return SPEC_F32
    if t.dtype == torch.bfloat16:
        return SPEC_BF16
    raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, f"logits dtype {t.dtype}")


def _check(code: int, what: str) -> int:
    if code != SPEC_OK:
        raise SpecVerifyError(code, what)
    return code


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


# ---------------------------------------------------------------------------
# the C ABI, one wrapper per entry point
# ---------------------------------------------------------------------------
def spec_verify_workspace_bytes(B: int, gamma: int, V: int, H: int = 0) -> int:
    out = _sz(0)
    _check(load().spec_verify_workspace_bytes(B, gamma, V, H, ctypes.byref(out)),
           "spec_verify_workspace_bytes")
    return out.value


def spec_verify_workspace_init(workspace, stream=None) -> None:
    _check(load().spec_verify_workspace_init(_ptr(workspace), _nbytes(workspace), _stream(stream)),
           "spec_verify_workspace_init")


def make_workspace(B: int, gamma: int, V: int, H: int = 0, device="cuda"):
    """Allocate (torch) and zero a workspace big enough for (B, gamma, V, H)."""
    import torch
    n = spec_verify_workspace_bytes(B, gamma, V, H)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def spec_verify_greedy(target_logits, draft_tokens, out_tokens, out_num_accepted, workspace,
                       stream=None) -> None:
    """target_logits [B, gamma+1, V] (fp32/bf16), draft_tokens [B, gamma] int32."""
    B, g1, V = target_logits.shape
    gamma = g1 - 1
    _check(load().spec_verify_greedy(_ptr(target_logits), _dtype_code(target_logits),
                                     _ptr(draft_tokens), B, gamma, V, _ptr(out_tokens),
                                     _ptr(out_num_accepted), _ptr(workspace), _nbytes(workspace),
                                     _stream(stream)), "spec_verify_greedy")


def spec_verify_greedy_multi(target_logits, draft_tokens, out_tokens, out_num_accepted, workspace,
                             out_choice=None, stream=None) -> None:
    """target_logits [B, n_cand, gamma+1, V] (fp32/bf16), draft_tokens
    [B, n_cand, gamma] int32; out_tokens [B, gamma+1], out_num_accepted [B],
    optional out_choice [B] int32.  Workspace: make_workspace(B * n_cand, gamma, V)."""
    B, n_cand, g1, V = target_logits.shape
    _check(load().spec_verify_greedy_multi(_ptr(target_logits), _dtype_code(target_logits),
                                           _ptr(draft_tokens), B, n_cand, g1 - 1, V, _ptr(out_tokens),
                                           _ptr(out_num_accepted), _ptr(out_choice), _ptr(workspace),
                                           _nbytes(workspace), _stream(stream)), "spec_verify_greedy_multi")


def spec_verify_sample(target_logits, draft_logits, draft_tokens, temperature, u_accept,
                       u_resample, out_tokens, out_num_accepted, workspace, out_debug=None,
                       stream=None) -> None:
    """target_logits [B, gamma+1, V], draft_logits [B, gamma, V] (same dtype),
    draft_tokens [B, gamma] int32, temperature [B], u_accept [B, gamma],
    u_resample [B] (float32); out_tokens [B, gamma+1], out_num_accepted [B]
    int32; optional out_debug [B, gamma+1, 4] float32."""
    B, g1, V = target_logits.shape
    gamma = g1 - 1
    if draft_logits.dtype != target_logits.dtype:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, "target and draft logits differ in dtype")
    _check(load().spec_verify_sample(_ptr(target_logits), _ptr(draft_logits),
                                     _dtype_code(target_logits), _ptr(draft_tokens),
                                     _ptr(temperature), _ptr(u_accept), _ptr(u_resample), B, gamma, V,
                                     _ptr(out_tokens), _ptr(out_num_accepted), _ptr(out_debug),
                                     _ptr(workspace), _nbytes(workspace), _stream(stream)),
           "spec_verify_sample")


def spec_verify_topkp_workspace_bytes(B: int, gamma: int, V: int) -> int:
    out = _sz(0)
    _check(load().spec_verify_topkp_workspace_bytes(B, gamma, V, ctypes.byref(out)),
           "spec_verify_topkp_workspace_bytes")
    return out.value


def make_topkp_workspace(B: int, gamma: int, V: int, device="cuda"):
    """Allocate (torch) and zero a workspace for spec_verify_sample_topkp."""
    import torch
    n = spec_verify_topkp_workspace_bytes(B, gamma, V)
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def spec_verify_sample_topkp(target_logits, draft_logits, draft_tokens, temperature, u_accept,
                             u_resample, top_k, top_p, out_tokens, out_num_accepted, workspace,
                             out_debug=None, stream=None) -> None:
    """spec_verify_sample with top-k / top-p truncation of p and q (same
    arguments plus top_k, top_p).  Workspace: make_topkp_workspace(B, gamma, V)."""
    B, g1, V = target_logits.shape
    if draft_logits.dtype != target_logits.dtype:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, "target and draft logits differ in dtype")
    _check(load().spec_verify_sample_topkp(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), _ptr(draft_tokens),
        _ptr(temperature), _ptr(u_accept), _ptr(u_resample), B, g1 - 1, V, int(top_k), float(top_p),
        _ptr(out_tokens), _ptr(out_num_accepted), _ptr(out_debug), _ptr(workspace), _nbytes(workspace),
        _stream(stream)), "spec_verify_sample_topkp")


def spec_verify_sample_reduce_only(target_logits, draft_logits, draft_tokens, temperature,
                                   u_accept, u_resample, out_tokens, out_num_accepted, workspace,
                                   out_debug=None, stream=None) -> None:
    """Enqueue only the row-reducer kernel of spec_verify_sample (timing aid)."""
    B, g1, V = target_logits.shape
    _check(load().spec_verify_sample_reduce_only(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), _ptr(draft_tokens),
        _ptr(temperature), _ptr(u_accept), _ptr(u_resample), B, g1 - 1, V, _ptr(out_tokens),
        _ptr(out_num_accepted), _ptr(out_debug), _ptr(workspace), _nbytes(workspace),
        _stream(stream)), "spec_verify_sample_reduce_only")


def spec_verify_sample_noalloc(target_logits, draft_logits, draft_tokens, temperature, u_accept,
                               u_resample, out_tokens, out_num_accepted, out_debug=None,
                               stream=None) -> None:
    """spec_verify_sample for callers that cannot allocate device memory: no
    workspace, the library's built-in 16 MiB scratch instead.  Calls must not
    overlap on the GPU (they share that scratch)."""
    B, g1, V = target_logits.shape
    if draft_logits.dtype != target_logits.dtype:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, "target and draft logits differ in dtype")
    _check(load().spec_verify_sample_noalloc(
        _ptr(target_logits), _ptr(draft_logits), _dtype_code(target_logits), _ptr(draft_tokens),
        _ptr(temperature), _ptr(u_accept), _ptr(u_resample), B, g1 - 1, V, _ptr(out_tokens),
        _ptr(out_num_accepted), _ptr(out_debug), _stream(stream)), "spec_verify_sample_noalloc")


def _lmhead_call(fn, name, hidden, W, draft_logits, draft_tokens, temperature, u_accept,
                 u_resample, out_tokens, out_num_accepted, workspace, out_debug, stream):
    import torch
    B, gamma, V = draft_logits.shape
    H = W.shape[1]
    for t, what in ((hidden, "hidden"), (W, "W"), (draft_logits, "draft_logits")):
        if t.dtype != torch.bfloat16:
            raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, f"{what} must be bfloat16, got {t.dtype}")
    if tuple(hidden.shape) != (B * (gamma + 1), H) or W.shape[0] != V:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: hidden {tuple(hidden.shape)}, "
                              f"W {tuple(W.shape)}, draft_logits {tuple(draft_logits.shape)}")
    _check(fn(_ptr(hidden), _ptr(W), _ptr(draft_logits), _ptr(draft_tokens), _ptr(temperature),
              _ptr(u_accept), _ptr(u_resample), B, gamma, V, H, _ptr(out_tokens),
              _ptr(out_num_accepted), _ptr(out_debug), _ptr(workspace), _nbytes(workspace),
              _stream(stream)), name)


def spec_verify_lmhead_sample(hidden, W, draft_logits, draft_tokens, temperature, u_accept,
                              u_resample, out_tokens, out_num_accepted, workspace, out_debug=None,
                              stream=None) -> None:
    """Sampling verification with the target logits computed in the call as
    hidden @ W^T: hidden [B*(gamma+1), H], W [V, H], draft_logits [B, gamma, V]
    (all bfloat16); the other arguments as spec_verify_sample.  The workspace
    comes from make_workspace(B, gamma, V, H)."""
    _lmhead_call(load().spec_verify_lmhead_sample, "spec_verify_lmhead_sample", hidden, W,
                 draft_logits, draft_tokens, temperature, u_accept, u_resample, out_tokens,
                 out_num_accepted, workspace, out_debug, stream)


def spec_verify_lmhead_gemm_only(hidden, W, draft_logits, draft_tokens, temperature, u_accept,
                                 u_resample, out_tokens, out_num_accepted, workspace,
                                 out_debug=None, stream=None) -> None:
    """Enqueue only the lm_head GEMM kernel of spec_verify_lmhead_sample (timing aid)."""
    _lmhead_call(load().spec_verify_lmhead_gemm_only, "spec_verify_lmhead_gemm_only", hidden, W,
                 draft_logits, draft_tokens, temperature, u_accept, u_resample, out_tokens,
                 out_num_accepted, workspace, out_debug, stream)


class SpecRoundState(ctypes.Structure):
    """spec_round_state: per-sequence host bookkeeping of the round driver."""
    _fields_ = [("gamma", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("seq_len", ctypes.c_int64), ("kv_len", ctypes.c_int64)]


def spec_round_update(states, num_accepted, gamma_min: int, gamma_max: int):
    """Host round bookkeeping.  ``states``: a ctypes array of SpecRoundState
    (updated in place); ``num_accepted``: host int sequence.  Returns the
    number of KV entries to keep per sequence.  Raises SpecVerifyError
    (SPEC_ERR_STATE, with the first inconsistent sequence) on bad bookkeeping."""
    B = len(states)
    n = (ctypes.c_int32 * B)(*[int(x) for x in num_accepted])
    keep = (ctypes.c_int64 * B)()
    bad = ctypes.c_int(-1)
    code = load().spec_round_update(ctypes.cast(states, _vp) if B else None, ctypes.cast(n, _vp),
                                    B, gamma_min, gamma_max, ctypes.cast(keep, _vp), ctypes.byref(bad))
    _check(code, f"spec_round_update (first bad sequence {bad.value})" if code == SPEC_ERR_STATE
           else "spec_round_update")
    return list(keep)


def spec_verify_status(workspace, stream=None) -> int:
    """Synchronise and return (and clear) the device-side status code."""
    return load().spec_verify_status(_ptr(workspace), _stream(stream))


def spec_verify_version() -> int:
    return load().spec_verify_version()


def spec_verify_selftest_timeout(workspace, stream=None) -> None:
    _check(load().spec_verify_selftest_timeout(_ptr(workspace), _nbytes(workspace), _stream(stream)),
           "spec_verify_selftest_timeout")


# ---------------------------------------------------------------------------
# centroid-masked sparse draft head and verification against its sparse rows
# ---------------------------------------------------------------------------
def _aligned_zeros(n: int, device):
    import torch
    ws = torch.zeros(n + 256, dtype=torch.uint8, device=device)
    off = (-ws.data_ptr()) % 256
    return ws[off:off + n]


def spec_centroid_head_workspace_bytes(R: int, n_clusters: int, top_k: int) -> int:
    out = _sz(0)
    _check(load().spec_centroid_head_workspace_bytes(R, n_clusters, top_k, ctypes.byref(out)),
           "spec_centroid_head_workspace_bytes")
    return out.value


def make_centroid_head_workspace(R: int, n_clusters: int, top_k: int, device="cuda"):
    """Allocate (torch) and zero a workspace for spec_centroid_head."""
    return _aligned_zeros(spec_centroid_head_workspace_bytes(R, n_clusters, top_k), device)


def spec_centroid_head(hidden, centroids, W_ord, cluster_off, ord2tok, top_k, out_tok, out_logit,
                       out_count, workspace, stream=None) -> None:
    """hidden [R, H], centroids [n_clusters, H], W_ord [V, H] (bf16); cluster_off
    int32 [n_clusters+1]; ord2tok int32 [V]; out_tok int32 / out_logit f32
    [R, max_cand]; out_count int32 [R]."""
    R, H = hidden.shape
    V = W_ord.shape[0]
    n_clusters = centroids.shape[0]
    max_cand = out_tok.shape[1]
    _check(load().spec_centroid_head(
        _ptr(hidden), _ptr(centroids), _ptr(W_ord), _ptr(cluster_off), _ptr(ord2tok), R, H, V, n_clusters,
        int(top_k), max_cand, _ptr(out_tok), _ptr(out_logit), _ptr(out_count), _ptr(workspace),
        _nbytes(workspace), _stream(stream)), "spec_centroid_head")


def spec_verify_sparse_workspace_bytes(B: int, gamma: int, V: int) -> int:
    out = _sz(0)
    _check(load().spec_verify_sparse_workspace_bytes(B, gamma, V, ctypes.byref(out)),
           "spec_verify_sparse_workspace_bytes")
    return out.value


def make_sparse_workspace(B: int, gamma: int, V: int, device="cuda"):
    """Allocate (torch) and zero a workspace for spec_verify_sample_sparse."""
    return _aligned_zeros(spec_verify_sparse_workspace_bytes(B, gamma, V), device)


def spec_verify_sample_sparse(target_logits, cand_tok, cand_logit, cand_count, draft_tokens, temperature,
                              u_accept, u_resample, out_tokens, out_num_accepted, workspace, out_debug=None,
                              stream=None) -> None:
    """target_logits [B, gamma+1, V] (fp32/bf16); cand_tok int32 / cand_logit
    f32 [B*gamma, stride] (tokens ascending per row); cand_count int32
    [B*gamma]; the rest as spec_verify_sample."""
    B, g1, V = target_logits.shape
    _check(load().spec_verify_sample_sparse(
        _ptr(target_logits), _dtype_code(target_logits), _ptr(cand_tok), _ptr(cand_logit), _ptr(cand_count),
        cand_tok.shape[1], _ptr(draft_tokens), _ptr(temperature), _ptr(u_accept), _ptr(u_resample), B, g1 - 1, V,
        _ptr(out_tokens), _ptr(out_num_accepted), _ptr(out_debug), _ptr(workspace), _nbytes(workspace),
        _stream(stream)), "spec_verify_sample_sparse")


# ---------------------------------------------------------------------------
# the paged key/value cache: append with rotary positions, shared-prefix attention
# ---------------------------------------------------------------------------
class SpecKvCache(ctypes.Structure):
    """spec_kv_cache: the pools of a paged cache (strides in elements)."""
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("page_stride", _i64), ("slot_stride", _i64),
                ("head_stride", _i64), ("n_pages", _i64), ("page_size", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


def make_kv_cache(k_pages, v_pages) -> SpecKvCache:
    """The cache over pools [n_pages, page_size, n_heads, head_dim] (bf16 or
    fp16, any strides but the last; both alike).  A pool stored
    [n_pages, n_heads, page_size, head_dim] is passed as its transpose(1, 2).
    The struct keeps the tensors alive."""
    import torch
    codes = {torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}
    if k_pages.dtype not in codes or v_pages.dtype != k_pages.dtype:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, f"cache dtypes {k_pages.dtype}, {v_pages.dtype}")
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride() \
            or k_pages.stride(3) != 1:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"cache pools {tuple(k_pages.shape)} with strides "
                              f"{k_pages.stride()}, {tuple(v_pages.shape)} with {v_pages.stride()}")
    if k_pages.device != v_pages.device:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"cache pools on {k_pages.device} and {v_pages.device}")
    n_pages, page_size, n_heads, head_dim = k_pages.shape
    page_stride, slot_stride, head_stride, _ = k_pages.stride()
    cache = SpecKvCache(k_pages.data_ptr(), v_pages.data_ptr(), page_stride, slot_stride, head_stride, n_pages,
                        page_size, n_heads, head_dim, codes[k_pages.dtype])
    cache.tensors = (k_pages, v_pages)
    cache.address = ctypes.addressof(cache)
    # what every call compares with, read once
    cache.expected = (k_pages.dtype, n_heads, head_dim, page_size, k_pages.device.index, torch.int32, torch.float32,
                      torch.int64)
    return cache


def spec_attention_workspace_bytes(B: int, N: int, n_q_heads: int, head_dim: int, prefix: bool = True) -> int:
    """Bytes for spec_prefix_attention (without a shared prefix: prefix=False,
    about half); they do for spec_kv_append too."""
    return spec_prefix_attention_workspace_bytes(B, N, n_q_heads, head_dim, 1 if prefix else 0)


def spec_prefix_attention_workspace_bytes(B: int, N: int, n_q_heads: int, head_dim: int, prefix_len: int) -> int:
    out = _sz(0)
    _check(load().spec_prefix_attention_workspace_bytes(B, N, n_q_heads, head_dim, prefix_len, ctypes.byref(out)),
           "spec_prefix_attention_workspace_bytes")
    return out.value


def spec_kv_append_workspace_bytes() -> int:
    out = _sz(0)
    _check(load().spec_kv_append_workspace_bytes(ctypes.byref(out)), "spec_kv_append_workspace_bytes")
    return out.value


def make_attention_workspace(B: int, N: int, n_q_heads: int, head_dim: int, device="cuda", prefix: bool = True):
    """Allocate (torch) and zero a workspace for spec_prefix_attention (and spec_kv_append)."""
    return _aligned_zeros(spec_attention_workspace_bytes(B, N, n_q_heads, head_dim, prefix), device)


def make_append_workspace(device="cuda"):
    """Allocate (torch) and zero a workspace for spec_kv_append alone."""
    return _aligned_zeros(spec_kv_append_workspace_bytes(), device)


# PyTorch's raw getters, looked up once (every call asks both)
_raw_stream = _raw_device = None


def _call_stream(stream, device_index):
    """The caller's stream, or PyTorch's current one (its raw handle: building
    the Stream object costs as much as the launch)."""
    global _raw_stream
    if stream is not None:
        return _stream(stream)
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw_stream(device_index)


def _current_device() -> int:
    global _raw_device
    if _raw_device is None:
        import torch
        _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _raw_device()


def _cache_of(name, cache, kind, maker):
    """A cache of the other kind is another struct: never handed on."""
    if not isinstance(cache, kind):
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: a cache of {maker} is wanted, not {type(cache).__name__}")


def _positions_first(name, cache, *tensors):
    """Shared checks of [N, heads, head_dim] tensors: the cache's dtype and
    head_dim, one N, adjacent dims."""
    dtype, D = cache.expected[0], cache.expected[2]
    N = tensors[0].shape[0]
    for t in tensors:
        if t.dtype != dtype:
            raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, f"{name}: dtype {t.dtype}, cache {dtype}")
        if t.dim() != 3 or t.shape[0] != N or t.shape[2] != D or t.stride(2) != 1:
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: shape {tuple(t.shape)} strides {t.stride()}, "
                                  f"expected [{N}, heads, {D}] with adjacent dims")


def _batch_checks(name, q_indptr, block_table, kv_len):
    import torch
    B = kv_len.numel()
    for t, shape in ((q_indptr, (B + 1,)), (kv_len, (B,)), (block_table, (B, block_table.shape[-1]))):
        if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: {t.dtype} {tuple(t.shape)}, expected contiguous "
                                  f"int32 {shape}")
    return B


def _refuse_place(name, cache, **tensors):
    """Which tensor is not on the cache's GPU, or that GPU is not the current one."""
    device = cache.expected[4]
    if device is None:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: the cache is not on the GPU")
    for key, t in tensors.items():
        if t is not None and t.get_device() != device:
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: {key} is on {t.device}, the cache on cuda:{device}")
    raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: the cache is on cuda:{device}, which is not the current device")


def spec_kv_append(cache, q, k, v, q_out, q_indptr, block_table, kv_len, workspace, inv_freq=None, positions=None,
                   axis=None, interleaved=False, position_base=0, stream=None) -> None:
    """Rotate the new queries and keys and append keys and values to the cache.

    cache from make_kv_cache; q [N, n_q_heads, D], k and v [N, n_heads, D]
    (views of one projection's output are fine); q_out [N, n_q_heads, D]
    contiguous; q_indptr int32 [B+1], block_table int32 [B, width], kv_len
    int32 [B] (the new positions counted); inv_freq float32 [rot_dim / 2] (None:
    no rotation); positions int32 [n_axes, N] and axis int32 [rot_dim / 2], or
    None for position_base + the entry's index."""
    if not isinstance(cache, SpecKvCache):
        _cache_of("spec_kv_append", cache, SpecKvCache, "make_kv_cache")
    dt, n_heads, D, _, device, i32, f32, _ = cache.expected
    q_shape, k_shape, table_shape, B = q.shape, k.shape, block_table.shape, kv_len.numel()
    # one pass over what has to hold; which one does not is found out after
    if not (q.dtype is dt and k.dtype is dt and v.dtype is dt and q_out.dtype is dt
            and len(q_shape) == 3 and q_shape[2] == D and k_shape == (q_shape[0], n_heads, D) and v.shape == k_shape
            and q_out.shape == q_shape and q_out.is_contiguous()
            and q_indptr.dtype is i32 and kv_len.dtype is i32 and block_table.dtype is i32
            and kv_len.dim() == 1 and q_indptr.dim() == 1 and q_indptr.numel() == B + 1
            and len(table_shape) == 2 and table_shape[0] == B
            and q_indptr.is_contiguous() and kv_len.is_contiguous() and block_table.is_contiguous()):
        _refuse_append(cache, q, k, v, q_out, q_indptr, block_table, kv_len)
    q_stride, k_stride, v_stride = q.stride(), k.stride(), v.stride()
    if q_stride[2] != 1 or k_stride[2] != 1 or v_stride[2] != 1:
        _refuse_append(cache, q, k, v, q_out, q_indptr, block_table, kv_len)
    n_axes, rot, freq, pos, ax = 1, 0, None, None, None
    if inv_freq is not None:
        rot = 2 * inv_freq.shape[0]
        if inv_freq.dtype is not f32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, "spec_kv_append: inv_freq must be contiguous float32")
        freq = inv_freq.data_ptr()
    if positions is not None:
        n_axes = positions.shape[0]
        if positions.dtype is not i32 or tuple(positions.shape) != (n_axes, q_shape[0]) \
                or not positions.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"spec_kv_append: positions {positions.dtype} "
                                  f"{tuple(positions.shape)}, expected contiguous int32 [n_axes, {q_shape[0]}]")
        pos = positions.data_ptr()
    if axis is not None:
        if axis.dtype is not i32 or 2 * axis.numel() != rot or not axis.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"spec_kv_append: axis {axis.dtype} {tuple(axis.shape)}, "
                                  f"expected contiguous int32 [{rot // 2}]")
        ax = axis.data_ptr()
    # last, so that every other refusal can be had without a GPU
    if not (q.get_device() == k.get_device() == v.get_device() == q_out.get_device() == q_indptr.get_device()
            == kv_len.get_device() == block_table.get_device() == workspace.get_device() == device == _current_device()
            and (freq is None or inv_freq.get_device() == device) and (pos is None or positions.get_device() == device)
            and (ax is None or axis.get_device() == device)):
        _refuse_place("spec_kv_append", cache, q=q, k=k, v=v, q_out=q_out, q_indptr=q_indptr, block_table=block_table,
                      kv_len=kv_len, workspace=workspace, inv_freq=inv_freq, positions=positions, axis=axis)
    lib = _lib or load()
    code = lib.spec_kv_append(
        cache.address, q.data_ptr(), q_stride[0], q_stride[1], k.data_ptr(), k_stride[0], k_stride[1], v.data_ptr(),
        v_stride[0], v_stride[1], q_shape[1], q_shape[0], q_indptr.data_ptr(), B, block_table.data_ptr(),
        table_shape[1], kv_len.data_ptr(), freq, pos, n_axes, ax, rot, 1 if interleaved else 0, position_base,
        q_out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _call_stream(stream, device))
    if code != SPEC_OK:
        _check(code, "spec_kv_append")


def _refuse_append(cache, q, k, v, q_out, q_indptr, block_table, kv_len, name="spec_kv_append"):
    n_heads = cache.n_heads
    _positions_first(name, cache, q, k, v, q_out)
    _batch_checks(name, q_indptr, block_table, kv_len)
    if k.shape[1] != n_heads or v.shape[1] != n_heads or q_out.shape != q.shape or not q_out.is_contiguous():
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: q {tuple(q.shape)}, k {tuple(k.shape)}, "
                              f"v {tuple(v.shape)}, q_out {tuple(q_out.shape)}, {n_heads} cache heads")
    raise SpecVerifyError(SPEC_ERR_INVALID_ARG, name)


def spec_prefix_attention(cache, q, out, q_indptr, block_table, kv_len, workspace, prefix_table=None, prefix_len=0,
                          draft_mask=None, scale=None, lse=None, stream=None) -> None:
    """Attention of the new positions over the shared prefix and their
    sequences' pages.

    cache from make_kv_cache; q, out [N, n_q_heads, D] in the cache's dtype; prefix_table int32
    [>= ceil(prefix_len / page_size)]; draft_mask int64 [N] (64 bits, bit j: the
    position sees new entry j) or None for a chain; scale defaults to
    D ** -0.5; lse float32 [N, n_q_heads] or None.  The rest as spec_kv_append."""
    _cache_of("spec_prefix_attention", cache, SpecKvCache, "make_kv_cache")
    _attention((_lib or load()).spec_prefix_attention, "spec_prefix_attention", cache, q, out, q_indptr, block_table, kv_len,
               workspace, prefix_table, prefix_len, draft_mask, scale, lse, stream)


def _attention(call, name, cache, q, out, q_indptr, block_table, kv_len, workspace, prefix_table, prefix_len, draft_mask,
               scale, lse, stream):
    dt, n_heads, D, page_size, device, i32, f32, i64 = cache.expected
    q_shape, table_shape, B = q.shape, block_table.shape, kv_len.numel()
    if not (q.dtype is dt and out.dtype is dt and len(q_shape) == 3 and q_shape[2] == D and out.shape == q_shape
            and q_indptr.dtype is i32 and kv_len.dtype is i32 and block_table.dtype is i32
            and kv_len.dim() == 1 and q_indptr.dim() == 1 and q_indptr.numel() == B + 1
            and len(table_shape) == 2 and table_shape[0] == B
            and q_indptr.is_contiguous() and kv_len.is_contiguous() and block_table.is_contiguous()):
        _refuse_attention(cache, q, out, q_indptr, block_table, kv_len, name)
    q_stride, out_stride = q.stride(), out.stride()
    if q_stride[2] != 1 or out_stride[2] != 1:
        _refuse_attention(cache, q, out, q_indptr, block_table, kv_len, name)
    N, n_q_heads = q_shape[0], q_shape[1]
    shared = mask = stats = None
    if prefix_len > 0:
        if prefix_table is None or prefix_table.dtype is not i32 or prefix_table.dim() != 1 \
                or not prefix_table.is_contiguous() or prefix_table.shape[0] * page_size < prefix_len:
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: prefix_table does not hold the pages "
                                  f"of {prefix_len} entries")
        shared = prefix_table.data_ptr()
    if draft_mask is not None:
        if draft_mask.dtype is not i64 or draft_mask.shape != (N,) or not draft_mask.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: draft_mask {draft_mask.dtype} "
                                  f"{tuple(draft_mask.shape)}, expected contiguous int64 [{N}]")
        mask = draft_mask.data_ptr()
    if lse is not None:
        if lse.dtype is not f32 or lse.shape != (N, n_q_heads) or not lse.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: lse {lse.dtype} {tuple(lse.shape)}, "
                                  f"expected contiguous float32 [{N}, {n_q_heads}]")
        stats = lse.data_ptr()
    if not (q.get_device() == out.get_device() == q_indptr.get_device() == kv_len.get_device()
            == block_table.get_device() == workspace.get_device() == device == _current_device()
            and (shared is None or prefix_table.get_device() == device)
            and (mask is None or draft_mask.get_device() == device) and (stats is None or lse.get_device() == device)):
        _refuse_place(name, cache, q=q, out=out, q_indptr=q_indptr, block_table=block_table,
                      kv_len=kv_len, workspace=workspace, prefix_table=prefix_table if prefix_len > 0 else None,
                      draft_mask=draft_mask, lse=lse)
    code = call(
        cache.address, q.data_ptr(), q_stride[0], q_stride[1], n_q_heads, N, q_indptr.data_ptr(), B,
        shared, prefix_len, block_table.data_ptr(), table_shape[1], kv_len.data_ptr(), mask,
        D ** -0.5 if scale is None else scale, out.data_ptr(), out_stride[0], out_stride[1], stats,
        workspace.data_ptr(), workspace.nbytes, _call_stream(stream, device))
    if code != SPEC_OK:
        _check(code, name)


def _refuse_attention(cache, q, out, q_indptr, block_table, kv_len, name):
    _positions_first(name, cache, q, out)
    _batch_checks(name, q_indptr, block_table, kv_len)
    if out.shape != q.shape:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: q {tuple(q.shape)}, out {tuple(out.shape)}: shapes differ")
    raise SpecVerifyError(SPEC_ERR_INVALID_ARG, name)


# ---------------------------------------------------------------------------
# norms in the append, and the cache in 8 bits
# ---------------------------------------------------------------------------
class SpecKvCache8(ctypes.Structure):
    """spec_kv_cache8: the pools of codes and of scales (strides in bytes)."""
    _fields_ = [("k_pages", _vp), ("v_pages", _vp), ("k_scales", _vp), ("v_scales", _vp), ("page_stride", _i64),
                ("slot_stride", _i64), ("head_stride", _i64), ("scale_page_stride", _i64), ("scale_block_stride", _i64),
                ("scale_head_stride", _i64), ("n_pages", _i64), ("page_size", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("block", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


def make_kv_cache8(k_pages, v_pages, k_scales, v_scales, dtype=None) -> SpecKvCache8:
    """The 8-bit cache over pools [n_pages, page_size, n_heads, head_dim] of
    float8_e4m3fn codes (or uint8, the same bytes; any strides but the last, both
    alike) and scales [n_pages, page_size / block, n_heads] of float8_e8m0fnu (or
    uint8; any strides, both alike), for queries, keys, values and outputs of
    `dtype` (bfloat16, the default, or float16).  The block is what the shapes
    say: 8, 16, 32 or 64 entries.  The struct keeps the tensors alive."""
    import torch
    dtype = torch.bfloat16 if dtype is None else dtype
    codes = {torch.bfloat16: SPEC_BF16, torch.float16: SPEC_F16}
    if dtype not in codes:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, f"cache of {dtype}")
    if k_pages.dtype not in (torch.float8_e4m3fn, torch.uint8) or v_pages.dtype != k_pages.dtype:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, f"cache dtypes {k_pages.dtype}, {v_pages.dtype}: float8_e4m3fn codes")
    if k_scales.dtype not in (torch.float8_e8m0fnu, torch.uint8) or v_scales.dtype != k_scales.dtype:
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, f"scale dtypes {k_scales.dtype}, {v_scales.dtype}: float8_e8m0fnu")
    if k_pages.dim() != 4 or k_pages.shape != v_pages.shape or k_pages.stride() != v_pages.stride() \
            or k_pages.stride(3) != 1:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"cache pools {tuple(k_pages.shape)} with strides "
                              f"{k_pages.stride()}, {tuple(v_pages.shape)} with {v_pages.stride()}")
    n_pages, page_size, n_heads, head_dim = k_pages.shape
    if k_scales.dim() != 3 or k_scales.shape != v_scales.shape or k_scales.stride() != v_scales.stride() \
            or k_scales.shape[0] != n_pages or k_scales.shape[2] != n_heads or k_scales.shape[1] < 1 \
            or page_size % k_scales.shape[1]:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"scales {tuple(k_scales.shape)} with strides {k_scales.stride()}, "
                              f"{tuple(v_scales.shape)} with {v_scales.stride()}: expected [{n_pages}, {page_size} / "
                              f"block, {n_heads}]")
    if not k_pages.device == v_pages.device == k_scales.device == v_scales.device:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"cache pools on {k_pages.device}, {v_pages.device}, scales on "
                              f"{k_scales.device}, {v_scales.device}")
    block = page_size // k_scales.shape[1]
    if block not in (8, 16, 32, 64):
        raise SpecVerifyError(SPEC_ERR_UNSUPPORTED, f"blocks of {block} entries: 8, 16, 32 or 64")
    page_stride, slot_stride, head_stride, _ = k_pages.stride()
    cache = SpecKvCache8(k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), page_stride,
                         slot_stride, head_stride, *k_scales.stride(), n_pages, page_size, n_heads, head_dim, block,
                         codes[dtype])
    cache.tensors = (k_pages, v_pages, k_scales, v_scales)
    cache.address = ctypes.addressof(cache)
    cache.expected = (dtype, n_heads, head_dim, page_size, k_pages.device.index, torch.int32, torch.float32, torch.int64)
    return cache


def spec_kv_append_norm(cache, q, k, v, q_out, q_indptr, block_table, kv_len, workspace, inv_freq=None, positions=None,
                        axis=None, interleaved=False, position_base=0, q_weight=None, k_weight=None, norm_eps=1e-6,
                        stream=None) -> None:
    """spec_kv_append with root-mean-square norms of each query and key head
    before the rotation: q_weight, k_weight float32 [D], None for no norm of that
    side.  The rest as spec_kv_append."""
    _cache_of("spec_kv_append_norm", cache, SpecKvCache, "make_kv_cache")
    _append_norm((_lib or load()).spec_kv_append_norm, "spec_kv_append_norm", cache, q, k, v, q_out, q_indptr, block_table,
                 kv_len, workspace, inv_freq, positions, axis, interleaved, position_base, q_weight, k_weight, norm_eps,
                 stream)


def spec_kv_append8(cache, q, k, v, q_out, q_indptr, block_table, kv_len, workspace, inv_freq=None, positions=None,
                    axis=None, interleaved=False, position_base=0, q_weight=None, k_weight=None, norm_eps=1e-6,
                    stream=None) -> None:
    """spec_kv_append_norm to an 8-bit cache (from make_kv_cache8): keys and values
    are quantised as they are written, with a scale for each block of entries."""
    _cache_of("spec_kv_append8", cache, SpecKvCache8, "make_kv_cache8")
    _append_norm((_lib or load()).spec_kv_append8, "spec_kv_append8", cache, q, k, v, q_out, q_indptr, block_table, kv_len,
                 workspace, inv_freq, positions, axis, interleaved, position_base, q_weight, k_weight, norm_eps, stream)


def _append_norm(call, name, cache, q, k, v, q_out, q_indptr, block_table, kv_len, workspace, inv_freq, positions, axis,
                 interleaved, position_base, q_weight, k_weight, norm_eps, stream):
    dt, n_heads, D, _, device, i32, f32, _ = cache.expected
    q_shape, k_shape, table_shape, B = q.shape, k.shape, block_table.shape, kv_len.numel()
    if not (q.dtype is dt and k.dtype is dt and v.dtype is dt and q_out.dtype is dt
            and len(q_shape) == 3 and q_shape[2] == D and k_shape == (q_shape[0], n_heads, D) and v.shape == k_shape
            and q_out.shape == q_shape and q_out.is_contiguous()
            and q_indptr.dtype is i32 and kv_len.dtype is i32 and block_table.dtype is i32
            and kv_len.dim() == 1 and q_indptr.dim() == 1 and q_indptr.numel() == B + 1
            and len(table_shape) == 2 and table_shape[0] == B
            and q_indptr.is_contiguous() and kv_len.is_contiguous() and block_table.is_contiguous()):
        _refuse_append(cache, q, k, v, q_out, q_indptr, block_table, kv_len, name)
    q_stride, k_stride, v_stride = q.stride(), k.stride(), v.stride()
    if q_stride[2] != 1 or k_stride[2] != 1 or v_stride[2] != 1:
        _refuse_append(cache, q, k, v, q_out, q_indptr, block_table, kv_len, name)
    n_axes, rot, freq, pos, ax, qw, kw = 1, 0, None, None, None, None, None
    if inv_freq is not None:
        rot = 2 * inv_freq.shape[0]
        if inv_freq.dtype is not f32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: inv_freq must be contiguous float32")
        freq = inv_freq.data_ptr()
    if positions is not None:
        n_axes = positions.shape[0]
        if positions.dtype is not i32 or positions.shape != (n_axes, q_shape[0]) or not positions.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: positions {positions.dtype} "
                                  f"{tuple(positions.shape)}, expected contiguous int32 [n_axes, {q_shape[0]}]")
        pos = positions.data_ptr()
    if axis is not None:
        if axis.dtype is not i32 or 2 * axis.numel() != rot or not axis.is_contiguous():
            raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: axis {axis.dtype} {tuple(axis.shape)}, "
                                  f"expected contiguous int32 [{rot // 2}]")
        ax = axis.data_ptr()
    if q_weight is not None:
        qw = _norm_weight(name, "q_weight", q_weight, D, f32)
    if k_weight is not None:
        kw = _norm_weight(name, "k_weight", k_weight, D, f32)
    if not (q.get_device() == k.get_device() == v.get_device() == q_out.get_device() == q_indptr.get_device()
            == kv_len.get_device() == block_table.get_device() == workspace.get_device() == device == _current_device()
            and (freq is None or inv_freq.get_device() == device) and (pos is None or positions.get_device() == device)
            and (ax is None or axis.get_device() == device) and (qw is None or q_weight.get_device() == device)
            and (kw is None or k_weight.get_device() == device)):
        _refuse_place(name, cache, q=q, k=k, v=v, q_out=q_out, q_indptr=q_indptr, block_table=block_table, kv_len=kv_len,
                      workspace=workspace, inv_freq=inv_freq, positions=positions, axis=axis, q_weight=q_weight,
                      k_weight=k_weight)
    code = call(
        cache.address, q.data_ptr(), q_stride[0], q_stride[1], k.data_ptr(), k_stride[0], k_stride[1], v.data_ptr(),
        v_stride[0], v_stride[1], q_shape[1], q_shape[0], q_indptr.data_ptr(), B, block_table.data_ptr(),
        table_shape[1], kv_len.data_ptr(), freq, pos, n_axes, ax, rot, 1 if interleaved else 0, position_base, qw, kw,
        norm_eps, q_out.data_ptr(), workspace.data_ptr(), workspace.nbytes, _call_stream(stream, device))
    if code != SPEC_OK:
        _check(code, name)


def _norm_weight(name, key, w, D, f32):
    if w.dtype is not f32 or w.shape != (D,) or not w.is_contiguous():
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: {key} {w.dtype} {tuple(w.shape)}, expected contiguous "
                              f"float32 [{D}]")
    return w.data_ptr()


def spec_kv_read8(cache, k_out, v_out, out_indptr, block_table, workspace, first=None, stream=None) -> None:
    """Entries of an 8-bit cache back in 16 bits: rows out_indptr[b] ..
    out_indptr[b+1]-1 of k_out and v_out [R, n_heads, D] (the cache's dtype; either
    may be None) become the entries of sequence b from first[b] (int32 [B], None: 0)
    on.  out_indptr int32 [B+1], block_table int32 [B, width]; a workspace of
    make_append_workspace."""
    name = "spec_kv_read8"
    _cache_of(name, cache, SpecKvCache8, "make_kv_cache8")
    dt, n_heads, D, _, device, i32, _, _ = cache.expected
    outs = [t for t in (k_out, v_out) if t is not None]
    if not outs:
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: no output")
    _positions_first(name, cache, *outs)
    if any(t.shape[1] != n_heads for t in outs):
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: outputs {[tuple(t.shape) for t in outs]}, {n_heads} cache heads")
    B = out_indptr.numel() - 1
    if out_indptr.dtype is not i32 or out_indptr.dim() != 1 or B < 1 or not out_indptr.is_contiguous() \
            or block_table.dtype is not i32 or block_table.dim() != 2 or block_table.shape[0] != B \
            or not block_table.is_contiguous():
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: out_indptr {out_indptr.dtype} {tuple(out_indptr.shape)}, "
                              f"block_table {block_table.dtype} {tuple(block_table.shape)}, expected contiguous int32 "
                              f"[B + 1] and [B, width]")
    if first is not None and (first.dtype is not i32 or first.shape != (B,) or not first.is_contiguous()):
        raise SpecVerifyError(SPEC_ERR_INVALID_ARG, f"{name}: first {first.dtype} {tuple(first.shape)}, expected "
                              f"contiguous int32 [{B}]")
    if not (all(t.get_device() == device for t in outs) and out_indptr.get_device() == block_table.get_device()
            == workspace.get_device() == device == _current_device() and (first is None or first.get_device() == device)):
        _refuse_place(name, cache, k_out=k_out, v_out=v_out, out_indptr=out_indptr, block_table=block_table,
                      workspace=workspace, first=first)
    strides = [(None, 0, 0) if t is None else (t.data_ptr(), t.stride(0), t.stride(1)) for t in (k_out, v_out)]
    _check((_lib or load()).spec_kv_read8(
        cache.address, out_indptr.data_ptr(), outs[0].shape[0], B, block_table.data_ptr(), block_table.shape[1],
        None if first is None else first.data_ptr(), *strides[0], *strides[1], workspace.data_ptr(), workspace.nbytes,
        _call_stream(stream, device)), name)


def spec_prefix_attention8(cache, q, out, q_indptr, block_table, kv_len, workspace, prefix_table=None, prefix_len=0,
                           draft_mask=None, scale=None, lse=None, stream=None) -> None:
    """spec_prefix_attention over an 8-bit cache (from make_kv_cache8); q and out
    in the cache's 16-bit dtype, the rest alike."""
    _cache_of("spec_prefix_attention8", cache, SpecKvCache8, "make_kv_cache8")
    _attention((_lib or load()).spec_prefix_attention8, "spec_prefix_attention8", cache, q, out, q_indptr, block_table,
               kv_len, workspace, prefix_table, prefix_len, draft_mask, scale, lse, stream)
