"""Lengths outside their ranges in spec_kv_append: reported, and no entry that
the cache held is lost."""
import numpy as np
import pytest

from oracle import paged
from tests.test_gpu_paged import Problem, _attend, _f64, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def _append(sv, pr, ws, base=0):
    import torch
    q_out = torch.full((pr.N, pr.Hq, pr.D), -7.0, dtype=pr.q.dtype, device="cuda")
    freq = torch.from_numpy((10000.0 ** (-np.arange(pr.D // 2) / (pr.D // 2))).astype(np.float32)).cuda()
    sv.spec_kv_append(sv.make_kv_cache(*pr.pools), pr.q, pr.k, pr.v, q_out, pr.indptr, pr.table, pr.kv_len, ws,
                      inv_freq=freq, position_base=base)
    return q_out, freq


@pytest.mark.parametrize("past", [1, 3, 4, 100, 2 ** 31 - 1])
def test_append_past_the_table_keeps_what_the_cache_holds(sv, past):  # noqa: F811
    """Sequence 1's length runs past its row of the table by `past` entries: what
    still has a place is written there, the rest nowhere."""
    import torch
    page, n = 16, 4
    pr = Problem(101, "bf16", 64, 2, 4, page, [2, n, 3], [40, 48, 30])
    capacity = 3 * page
    kv = min(capacity + past, 2 ** 31 - 1)
    pr.kv_len[1] = kv
    before = [p.clone() for p in pr.pools]
    ws = sv.make_attention_workspace(3, pr.N, pr.Hq, pr.D)
    q_out, freq = _append(sv, pr, ws, base=7)
    assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
    # the oracle's append, entry by entry, of what has a place
    new = np.zeros_like(pr.live)
    u, f = 2.0 ** -8, freq.double().cpu().numpy()
    k, q = _f64(pr.k), _f64(pr.q)
    # an angle is off by at most 5e-7, each product and sum by 2^-24, of |x| + |y| <= 2 max
    slack = 2 * max(np.abs(k).max(), np.abs(q).max()) * (5e-7 + 3 * 2.0 ** -24)
    for b, (ql, kl) in enumerate(zip(pr.q_lens, [40, kv, 30])):
        for i in range(ql):
            t, row = kl - ql + i, int(pr.indptr_np[b]) + i
            want_q = paged.rotate(q[row], [7 + t], f)
            assert (np.abs(_f64(q_out)[row] - want_q) <= u * (np.abs(want_q) + slack) + slack).all()
            if t >= capacity:
                continue
            where = int(pr.table_np[b, t // page]), t % page
            new[where] = True
            want = paged.rotate(k[row], [7 + t], f)
            assert (np.abs(_f64(pr.pools[0][where]) - want) <= u * (np.abs(want) + slack) + slack).all()
            assert torch.equal(pr.pools[1][where], pr.v[row])
    assert new.sum() == 2 + 3 + max(0, n - past)
    old = torch.from_numpy(~new).cuda()
    for p, was in zip(pr.pools, before):
        assert torch.equal(p[old].view(torch.int16), was[old].view(torch.int16))


def test_append_of_more_positions_than_entries_writes_what_has_a_place(sv):  # noqa: F811
    import torch
    pr = Problem(102, "fp16", 64, 1, 2, 8, [6, 2], [6, 10])
    pr.kv_len[0] = 4  # positions 0 and 1 would be entries -2 and -1
    before = [p.clone() for p in pr.pools]
    ws = sv.make_attention_workspace(2, pr.N, pr.Hq, pr.D)
    _append(sv, pr, ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
    new = np.zeros_like(pr.live)
    for row, (b, t) in {2: (0, 0), 3: (0, 1), 4: (0, 2), 5: (0, 3), 6: (1, 8), 7: (1, 9)}.items():
        where = int(pr.table_np[b, t // 8]), t % 8
        new[where] = True
        assert torch.equal(pr.pools[1][where], pr.v[row])
    old = torch.from_numpy(~new).cuda()
    for p, was in zip(pr.pools, before):
        assert torch.equal(p[old].view(torch.int16), was[old].view(torch.int16))
