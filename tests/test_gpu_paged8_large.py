"""spec_prefix_attention8 with many tiles and parts on every CTA, so that rings, queues
and buffers go round: against float64 on the GPU, and against itself; and the 8-bit
calls' small cases in the bounds-checked build."""
import os
import re
import subprocess
import sys

import numpy as np
import pytest

from oracle import paged
from tests import test_gpu_paged as t16
from tests.paged8_util import Problem8
from tests.test_gpu_paged import sv  # noqa: F401
from tests.test_gpu_paged8 import _attend8

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_54_gb300", "csrc")

LARGE = [
    # dtype, D, Hk, Hq, page, block, B, q_len, prefix, most own entries, mask
    ("bf16", 128, 8, 32, 64, 32, 24, 8, 8192, 700, False),
    ("bf16", 128, 4, 8, 16, 16, 64, 5, 1500, 2500, False),
    ("fp16", 64, 16, 16, 32, 8, 64, 1, 4000, 300, False),
    ("fp16", 64, 4, 28, 24, 8, 40, 12, 3001, 900, True),
    ("bf16", 128, 8, 16, 16, 16, 3, 700, 2050, 1400, False),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,Hk,Hq,page,block,B,q_len,prefix,most,mask", LARGE)
def test_attention8_large(sv, dtype, D, Hk, Hq, page, block, B, q_len, prefix, most, mask):  # noqa: F811
    """The tolerance is _check_attend's with the row's largest sums in place of each row's own."""
    import torch
    rng = np.random.default_rng(71)
    q_lens = rng.integers(1, q_len + 1, B).tolist()
    kv_lens = [int(rng.integers(n, most + 1)) for n in q_lens]
    pr = Problem8(72, dtype, D, Hk, Hq, page, block, q_lens, kv_lens, prefix=prefix)
    words = t16._random_mask(rng, q_lens, pr.N) if mask else None
    ws = sv.make_attention_workspace(B, pr.N, Hq, D)
    for _ in range(3):
        out, lse, _ = _attend8(sv, pr, words, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    u = torch.finfo(pr.q.dtype).eps / 2
    flat = [p.reshape(-1, Hk, D) for p in pr.pools]
    shared = [int(pr.ptable_np[t // page]) * page + t % page for t in range(prefix)]
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        rows = torch.tensor(shared + [int(pr.table_np[b, t // page]) * page + t % page for t in range(kv)], device="cuda")
        K, V = (x[rows].permute(1, 0, 2) for x in flat)
        a = int(pr.indptr_np[b])
        q = pr.q[a:a + n].double().reshape(n, Hk, Hq // Hk, D).permute(1, 2, 0, 3)
        new = torch.tensor([[paged.sees(i, j, None if words is None else words[a + i]) for j in range(n)] for i in range(n)],
                           device="cuda")
        s = torch.einsum("hgnd,hkd->hgnk", q, K) * D ** -0.5
        s[..., prefix + kv - n:] = s[..., prefix + kv - n:].masked_fill(~new, -float("inf"))
        want_lse = torch.logsumexp(s, dim=-1)
        w = torch.exp(s - want_lse[..., None])
        want, absv = torch.einsum("hgnk,hkd->hgnd", w, V), torch.einsum("hgnk,hkd->hgnd", w, V.abs())
        es = D * 2.0 ** -23 * float((torch.einsum("hgnd,hkd->hgnk", q.abs(), K.abs()) * D ** -0.5).max())
        keys = prefix + kv
        tol = (u + 2 * es + 2.0 ** -20 + keys * 2.0 ** -23) * absv + u * want.abs() \
            + keys * 2.0 ** -25 * float(V.abs().max()) + 2.0 ** -25
        got = out[a:a + n].double().reshape(n, Hk, Hq // Hk, D).permute(1, 2, 0, 3)
        assert bool(((got - want).abs() <= tol).all()), (b, float(((got - want).abs() - tol).max()))
        got_lse = lse[a:a + n].double().reshape(n, Hk, Hq // Hk).permute(1, 2, 0)
        ltol = es + keys * 2.0 ** -23 + 2.0 ** -20 + want_lse.abs() * 2.0 ** -22
        assert bool(((got_lse - want_lse).abs() <= ltol).all()), b


# dtype, D, Hk, Hq, page, block, q_len, kv_len, prefix: parts of one tile or two, wide and narrow, one after the other
SHORT_PARTS = [
    ("bf16", 128, 8, 16, 16, 16, 64, 128, 0),
    ("bf16", 128, 8, 16, 16, 16, 9, 100, 0),
    ("fp16", 64, 8, 16, 32, 32, 70, 130, 0),
    ("bf16", 128, 4, 8, 64, 64, 100, 250, 300),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,D,Hk,Hq,page,block,q_len,kv_len,prefix", SHORT_PARTS)
def test_short_parts_in_a_row(sv, dtype, D, Hk, Hq, page, block, q_len, kv_len, prefix):  # noqa: F811
    """Many passes without a pause: no wait of the kernel may run out, and every pass
    gives the same bits."""
    import torch
    B = 64
    pr = Problem8(81, dtype, D, Hk, Hq, page, block, [q_len] * B, [kv_len] * B, prefix=prefix)
    ws = sv.make_attention_workspace(B, pr.N, Hq, D)
    out, lse, _ = _attend8(sv, pr, ws=ws)
    first, first_lse = out.clone(), lse.clone()
    other = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        _attend8(sv, pr, ws=ws, out=out, lse=lse)
        other += (out != first).sum() + (lse != first_lse).sum()
    torch.cuda.synchronize()
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert int(other) == 0


_CHILD = r"""
import sys
sys.path.insert(0, sys.argv[1])
import speculative_decoding_verification_54_gb300 as sv, torch
from speculative_decoding_verification_54_gb300 import _build
sv.load(_build.build(checked=True))
torch.cuda.set_device(0)
from tests import test_gpu_paged8 as t, test_gpu_paged8_edges as e, test_gpu_paged8_large as l
n = 0
for c in t.APPEND:
    t.test_append_norm(sv, *c)
    t.test_append8(sv, *c)
    n += 1
t.test_append8_many_sequences(sv)
for c in t.ATTEND:
    t.test_attention8(sv, *c)
    n += 1
for c in t.READ:
    t.test_read8(sv, *c)
    n += 1
for c in (l.LARGE[1], l.LARGE[3], l.LARGE[4]):
    l.test_attention8_large(sv, *c)
    n += 1
e.test_pages_and_lengths_out_of_range_are_reported(sv)
for c in e.SHAPES[2:4]:
    e.test_nan_values_that_a_mask_hides(sv, c, "last")
print("ok", n)
"""


@pytest.mark.gpu
def test_checked_build_of_the_8_bit_calls():
    r = subprocess.run([sys.executable, "-c", _CHILD, ROOT], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    assert r.stdout.startswith("ok"), r.stdout[-2000:]


@pytest.mark.parametrize("name,least", [("attend8.cuh", 6), ("append8.cuh", 6)])
def test_the_kernels_check_their_computed_indices(name, least):
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    assert len(re.findall(r"\bin_bounds\(", re.sub(r"//.*", "", text))) >= least
