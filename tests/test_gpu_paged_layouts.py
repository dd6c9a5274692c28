"""Layouts of the paged calls that a caller may come with: head-major queries and
outputs, both pools in one allocation, a pool of one page, bad pages in the
prefix's table."""
import numpy as np
import pytest

from tests.test_gpu_paged import Problem, _append_and_check, _attend, _check_attend, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def _head_major(t):
    """The same values, heads further apart than positions."""
    return t.transpose(0, 1).contiguous().transpose(0, 1)


def _interleave(pools):
    """Both pools in one allocation, a page's values behind its keys."""
    import torch
    both = torch.stack(pools, dim=1)  # [pages, 2, slots, heads, dim]
    return [both[:, 0], both[:, 1]]


@pytest.mark.parametrize("dtype,D,Hk,Hq,q_lens,kv_lens,prefix", [
    ("bf16", 128, 2, 8, [5, 3, 7], [100, 3, 333], 700),
    ("fp16", 64, 4, 4, [90, 1], [150, 1], 0),
])
def test_head_major_queries_and_outputs(sv, dtype, D, Hk, Hq, q_lens, kv_lens, prefix):  # noqa: F811
    import torch
    pr = Problem(131, dtype, D, Hk, Hq, 16, q_lens, kv_lens, prefix, pad_rows=2)
    pr.q = _head_major(pr.q)
    assert pr.q.stride(1) > pr.q.stride(0)
    out = _head_major(torch.full((pr.N, Hq, D), -7.0, dtype=pr.q.dtype, device="cuda"))
    out, lse, ws = _attend(sv, pr, out=out)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_attend(pr, out, lse)


def test_append_from_head_major_projections(sv):  # noqa: F811
    pr = Problem(132, "bf16", 128, 2, 6, 16, [9, 4], [20, 4], pad_rows=1)
    pr.q, pr.k, pr.v = _head_major(pr.q), _head_major(pr.k), _head_major(pr.v)
    _append_and_check(sv, pr, 128, False, 1, 5, 133)


@pytest.mark.parametrize("heads_first", [False, True])
def test_pools_in_one_allocation(sv, heads_first):  # noqa: F811
    pr = Problem(134, "bf16", 64, 2, 8, 24, [5, 3, 7], [100, 3, 333], 250, heads_first=heads_first)
    if heads_first:
        pr.pools = [p.transpose(1, 2) for p in _interleave([p.transpose(1, 2) for p in pr.pools])]
    else:
        pr.pools = _interleave(pr.pools)
    assert pr.pools[0].stride(0) == 2 * 24 * 2 * 64
    _append_and_check(sv, pr, 32, True, 1, 0, 135)
    out, lse, ws = _attend(sv, pr)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_attend(pr, out, lse)


@pytest.mark.parametrize("q_len,kv_len", [(1, 1), (3, 41), (64, 64)])
def test_a_pool_of_one_page(sv, q_len, kv_len):  # noqa: F811
    import torch
    pr = Problem(136, "fp16", 64, 1, 2, 64, [q_len], [kv_len])
    page = int(pr.table_np[0, 0])
    pr.pools = [p[page:page + 1].clone() for p in pr.pools]
    pr.live, pr.table_np = pr.live[page:page + 1], np.zeros((1, 1), dtype=np.int32)
    pr.table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    _append_and_check(sv, pr, 64, False, 1, 0, 137)
    out, lse, ws = _attend(sv, pr)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_attend(pr, out, lse)


def test_bad_pages_of_the_prefix_are_reported_and_read_as_zero(sv):  # noqa: F811
    import torch
    pr = Problem(138, "bf16", 128, 2, 4, 16, [4, 3], [50, 20], 300)
    for bad in (-1, 2 ** 30, pr.pools[0].shape[0]):
        pr.ptable = torch.from_numpy(pr.ptable_np.copy()).cuda()
        pr.ptable[7] = bad
        out, lse, ws = _attend(sv, pr)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        # keys and values of that page are zeros
        page = int(pr.ptable_np[7])
        kept = [p[page].clone() for p in pr.pools]
        for p in pr.pools:
            p[page] = 0
        _check_attend(pr, out, lse)
        for p, was in zip(pr.pools, kept):
            p[page] = was


def test_pools_whose_offsets_pass_32_bits(sv):  # noqa: F811
    """Pages 2^29 elements apart: element offsets to beyond 2^32, byte offsets to 2^33."""
    import torch
    pr = Problem(139, "bf16", 64, 2, 4, 16, [5, 2], [60, 33], 20)
    small = pr.pools
    pages = small[0].shape[0]
    assert pages > 8
    pr.pools = []
    for p in small:
        buf = torch.empty(((pages - 1) << 29) + p[0].numel(), dtype=p.dtype, device="cuda")
        wide = buf.as_strided(p.shape, (1 << 29, *p.stride()[1:]))
        wide.copy_(p)
        pr.pools.append(wide)
    _append_and_check(sv, pr, 64, False, 1, pr.prefix, 140)
    out, lse, ws = _attend(sv, pr)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_attend(pr, out, lse)
