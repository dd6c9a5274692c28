"""Values that are not finite, in entries that a mask hides from some rows: those
rows' outputs are as if the entry were not there; rows that see it get what the
sum gives.  And values near the type's largest, whose sums must not overflow."""
import numpy as np
import pytest

from oracle import paged
from tests.test_gpu_paged import Problem, _attend, _check_attend, _random_mask, sv  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [
    # dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, mask
    ("bf16", 128, 2, 8, 16, [5, 3, 7], [100, 63, 333], 0, False),     # one row tile
    ("fp16", 64, 2, 4, 16, [90, 4], [150, 70], 300, False),           # two row tiles
    ("bf16", 64, 1, 4, 32, [6, 5], [6000, 4000], 2000, False),        # rows of many parts
    ("fp16", 128, 2, 6, 24, [9, 12], [60, 150], 131, True),
    ("bf16", 128, 1, 2, 16, [300, 2], [400, 10], 40, False),          # several row blocks
    ("bf16", 64, 2, 2, 8, [70, 3], [70, 3], 5, True),                 # entries past the 64th, seen by none
]


def _bits(t):
    import torch
    return t.view(torch.int16)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_new_entries(sv, shape, place):  # noqa: F811
    """A NaN in one dim and an infinity in another of one new entry's values."""
    dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, mask = shape
    pr = Problem(151, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, pad_rows=2)
    words = _random_mask(np.random.default_rng(152), q_lens, pr.N) if mask else None
    first, n = 0, q_lens[0]
    j = {"first": 0, "middle": n // 2, "last": n - 1}[place]
    t = kv_lens[0] - n + j
    where = int(pr.table_np[0, t // page]), t % page
    pr.pools[1][where][0, 5] = 0.0
    pr.pools[1][where][Hk - 1, D - 2] = 0.0
    clean, clean_lse, ws = _attend(sv, pr, words)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    pr.pools[1][where][0, 5] = float("nan")
    pr.pools[1][where][Hk - 1, D - 2] = float("inf")
    out, lse, ws = _attend(sv, pr, words, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    import torch
    assert torch.equal(lse, clean_lse)
    group = Hq // Hk
    got = out.clone()
    for i in range(n):
        if not paged.sees(i, j, None if words is None else words[first + i]):
            continue
        nan, inf = got[first + i, :group, 5], got[first + i, Hq - group:, D - 2]
        # (a weight that vanished makes the infinity a NaN)
        assert torch.isnan(nan).all() and not torch.isfinite(inf).any()
        nan.copy_(clean[first + i, :group, 5])
        inf.copy_(clean[first + i, Hq - group:, D - 2])
    pr.pools[1][where][0, 5] = 0.0
    pr.pools[1][where][Hk - 1, D - 2] = 0.0
    _check_attend(pr, got, lse, words)
    # the other sequences keep their bits
    assert torch.equal(_bits(out[n:]), _bits(clean[n:]))


def test_values_near_the_largest(sv):  # noqa: F811
    """bf16 values of up to 2^126, all positive: weighted they are finite, the sum
    before its division by the weights' is not."""
    import torch
    pr = Problem(153, "bf16", 64, 2, 4, 16, [4, 1], [60, 300], 700)
    pr.pools[1].abs_()
    plain, plain_lse, ws = _attend(sv, pr)
    big = 2.0 ** 126 / 8
    pr.pools[1].mul_(big)  # powers of two: the exact sums scale by it
    out, lse, ws = _attend(sv, pr, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert torch.equal(lse, plain_lse) and torch.isfinite(out).all()
    pr.pools[1].div_(big)
    _check_attend(pr, (out.double() / big).to(torch.bfloat16), lse)


def test_old_entries_and_the_prefix_reach_all_that_see_them(sv):  # noqa: F811
    import torch
    pr = Problem(154, "fp16", 64, 2, 4, 16, [5, 3], [100, 60], 50)
    clean, clean_lse, ws = _attend(sv, pr)
    pr.pools[1][int(pr.table_np[0, 1]), 3, 0, 9] = float("-inf")
    pr.pools[1][int(pr.ptable_np[2]), 7, 1, 11] = float("nan")
    out, lse, ws = _attend(sv, pr, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert torch.equal(lse, clean_lse)
    assert (out[:5, :2, 9] == float("-inf")).all() and torch.isnan(out[:, 2:, 11]).all()
    fine = torch.ones_like(out, dtype=torch.bool)
    fine[:5, :2, 9] = False
    fine[:, 2:, 11] = False
    got = torch.where(fine, out, clean)
    pr.pools[1][int(pr.table_np[0, 1]), 3, 0, 9] = 0.0
    pr.pools[1][int(pr.ptable_np[2]), 7, 1, 11] = 0.0
    u = 2.0 ** -11
    # another order of the sums: two roundings apart
    assert torch.allclose(got.double(), clean.double(), rtol=4 * u, atol=4 * u)
