"""The 8-bit cache in other layouts: scales and codes in one allocation, scales head by
head, offsets past 32 bits; a first call inside a graph's capture."""
import os
import subprocess
import sys

import numpy as np
import pytest

from oracle import paged8
from tests import test_gpu_paged as t16
from tests.paged8_util import Problem8
from tests.test_gpu_paged import _f64, sv  # noqa: F401
from tests.test_gpu_paged8 import Rotation, _append8, _attend8, _check_append8, _weights

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _all_three(sv, pr, norm=True):  # noqa: F811
    """Append, attend, read back, each against the oracle."""
    import torch
    ro, w = Rotation(pr, pr.D, 1, 1), _weights(pr.D, 2)
    before = [(c.clone(), s.clone()) for c, s in zip(pr.codes, pr.scales)]
    _, ws = _append8(sv, pr, ro, False, 3, w[0], w[1])
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_append8(pr, before, ro, False, 3, w[1])
    pr.refresh()
    out, lse, ws = _attend8(sv, pr)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    t16._check_attend(pr, out, lse)
    rows = np.concatenate([[0], np.cumsum(pr.kv_lens)]).astype(np.int32)
    back = [torch.empty((int(rows[-1]), pr.Hk, pr.D), dtype=pr.q.dtype, device="cuda") for _ in "kv"]
    sv.spec_kv_read8(pr.cache(sv), *back, torch.from_numpy(rows).cuda(), pr.table, ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    for x, c, s in zip(back, pr.codes, pr.scales):
        assert np.array_equal(_f64(x), paged8.read8(c.cpu().numpy(), s.cpu().numpy(), rows, pr.table_np, [0] * len(pr.kv_lens)))


@pytest.mark.parametrize("dtype,D,page,block", [("bf16", 128, 16, 8), ("fp16", 64, 64, 32)])
def test_one_allocation_and_scales_head_by_head(sv, dtype, D, page, block):  # noqa: F811
    """A page's record holds its key codes, value codes and both scales; the scales head
    by head."""
    import torch
    pr = Problem8(301, dtype, D, 3, 6, page, block, [5, 20, 1], [70, 33, 1], prefix=50, pad_rows=1)
    n, Hk, blocks = pr.codes[0].shape[0], 3, page // block
    code, scale = page * Hk * D, blocks * Hk
    record = 2 * code + -(-2 * scale // 16) * 16 + 32
    memory = torch.full((n, record), 0x7F, dtype=torch.uint8, device="cuda")
    for i in range(2):
        c = memory[:, i * code:(i + 1) * code].unflatten(1, (page, Hk, D))
        s = memory[:, 2 * code + i * scale:2 * code + (i + 1) * scale].unflatten(1, (Hk, blocks)).transpose(1, 2)
        c.copy_(pr.codes[i])
        s.copy_(pr.scales[i])
        pr.codes[i], pr.scales[i] = c, s
    tail = memory[:, 2 * code + 2 * scale:].clone()
    _all_three(sv, pr)
    assert torch.equal(memory[:, 2 * code + 2 * scale:], tail)


def test_offsets_past_32_bits(sv):  # noqa: F811
    """The problem's pages spread over pools of 6 GB each."""
    import torch
    pr = Problem8(311, "bf16", 128, 8, 16, 64, 64, [4, 70], [300, 130], prefix=100)
    n = pr.codes[0].shape[0]
    total = 96 * 1024
    spread = np.linspace(0, total - 1, n).astype(np.int64)
    for i in range(2):
        big = torch.empty((total, 64, 8, 128), dtype=torch.uint8, device="cuda")
        scales = torch.empty((total, 1, 8), dtype=torch.uint8, device="cuda")
        at = torch.from_numpy(spread).cuda()
        big[at] = pr.codes[i]
        scales[at] = pr.scales[i]
        pr.codes[i], pr.scales[i] = big, scales
    assert pr.codes[0].numel() > 2 ** 32
    move = lambda t: torch.from_numpy(np.where(t < n, spread[np.minimum(t, n - 1)], t).astype(np.int32)).cuda()  # noqa: E731
    table, ptable = pr.table.clone(), pr.ptable.clone()
    pr.table, pr.ptable = move(pr.table_np), move(pr.ptable_np)
    ro, w = Rotation(pr, 128, 1, 1), _weights(128, 2)
    _, ws = _append8(sv, pr, ro, False, 3, w[0], w[1])
    out, lse, aws = _attend8(sv, pr)
    rows = torch.tensor([0, 300, 430], dtype=torch.int32, device="cuda")
    back = torch.empty((430, 8, 128), dtype=torch.bfloat16, device="cuda")
    sv.spec_kv_read8(pr.cache(sv), back, None, rows, pr.table, ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK and sv.spec_verify_status(aws) == sv.SPEC_OK
    # the same on the small pools gives the same bits
    small = Problem8(311, "bf16", 128, 8, 16, 64, 64, [4, 70], [300, 130], prefix=100)
    _append8(sv, small, ro, False, 3, w[0], w[1])
    want, want_lse, _ = _attend8(sv, small)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    at = torch.from_numpy(spread).cuda()
    for i in range(2):
        assert torch.equal(pr.codes[i][at], small.codes[i]) and torch.equal(pr.scales[i][at], small.scales[i])
    small_back = torch.empty_like(back)
    sv.spec_kv_read8(small.cache(sv), small_back, None, rows, table, ws)
    assert torch.equal(back, small_back) and ptable.shape == pr.ptable.shape


_CHILD = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
import speculative_decoding_verification_54_gb300 as sv
from speculative_decoding_verification_54_gb300 import _build
_build.build()
sv.load()
torch.cuda.set_device(0)
codes = [torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device="cuda") for _ in "kv"]
scales = [torch.full((4, 1, 2), 127, dtype=torch.uint8, device="cuda") for _ in "kv"]
cache = sv.make_kv_cache8(*codes, *scales)
q = torch.ones(3, 4, 64, dtype=torch.bfloat16, device="cuda")
k, v = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda"), 3 * torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
q_out, out = torch.empty_like(q), torch.empty_like(q)
i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
indptr, table, lens, ws = i32(0, 3), i32(2, 1)[None], i32(20), sv.make_attention_workspace(1, 3, 4, 64)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    sv.spec_kv_append8(cache, q, k, v, q_out, indptr, table, lens, ws)
    sv.spec_prefix_attention8(cache, q_out, out, indptr, table, lens, ws)
graph.replay()
torch.cuda.synchronize()
assert sv.spec_verify_status(ws) == sv.SPEC_OK
assert torch.isfinite(out).all() and out.max() > 0.2, out
print("ok")
"""


def test_first_calls_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", _CHILD, ROOT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), (r.stdout[-500:], r.stderr[-2000:])
