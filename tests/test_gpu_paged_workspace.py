"""The paged calls stay inside a workspace of exactly the size that they ask
for, between guards."""
import numpy as np
import pytest

from tests.test_gpu_paged import Problem, _attend, _check_attend, sv  # noqa: F401

pytestmark = pytest.mark.gpu

GUARD = 4096


def _guarded(n):
    import torch
    buf = torch.full((n + 2 * GUARD + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    off = GUARD + (-(buf.data_ptr() + GUARD)) % 256
    ws = buf[off:off + n]
    ws.zero_()

    def untouched():
        return bool((buf[:off] == 0xA5).all()) and bool((buf[off + n:] == 0xA5).all())
    return ws, untouched


@pytest.mark.parametrize("dtype,D,Hk,Hq,page,q_lens,kv_lens,prefix", [
    ("bf16", 128, 8, 32, 16, [1], [9000], 0),                  # rows in many parts, 32 rows a slab
    ("bf16", 128, 8, 32, 16, [1], [300], 9000),
    ("fp16", 64, 1, 100, 16, [2], [5000], 7000),               # two row tiles of 100 rows
    ("bf16", 64, 2, 2, 16, [100, 60], [4000, 60], 0),          # 256-row blocks and single tiles
    ("bf16", 128, 2, 6, 32, [50, 3], [900, 2000], 3000),
])
def test_attention(sv, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix):  # noqa: F811
    pr = Problem(121, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix)
    ws, untouched = _guarded(sv.spec_attention_workspace_bytes(len(q_lens), pr.N, Hq, D, prefix=prefix > 0))
    out, lse, _ = _attend(sv, pr, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_attend(pr, out, lse)
    assert untouched()


def test_append(sv):  # noqa: F811
    import torch
    pr = Problem(122, "bf16", 128, 2, 6, 16, [500, 1], [600, 33])
    ws, untouched = _guarded(sv.spec_kv_append_workspace_bytes())
    q_out = torch.empty((pr.N, pr.Hq, pr.D), dtype=torch.bfloat16, device="cuda")
    sv.spec_kv_append(sv.make_kv_cache(*pr.pools), pr.q, pr.k, pr.v, q_out, pr.indptr, pr.table, pr.kv_len, ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert torch.equal(q_out, pr.q)
    for b, (n, kv) in enumerate(zip(pr.q_lens, pr.kv_lens)):
        at = np.arange(kv - n, kv)
        page, slot = pr.table_np[b][at // 16], at % 16
        a = int(pr.indptr_np[b])
        assert torch.equal(pr.pools[1][page, slot], pr.v[a:a + n]) and torch.equal(pr.pools[0][page, slot], pr.k[a:a + n])
    assert untouched()
