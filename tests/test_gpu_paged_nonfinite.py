"""Non-finite queries and keys in spec_prefix_attention: a row that sees a NaN
score, or an infinite one, gives NaN in both outputs as the formula does, and
every other row keeps its bits."""
import numpy as np
import pytest

from tests.test_gpu_paged import Problem, _attend, _random_mask, sv  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [
    # dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, mask
    ("bf16", 128, 2, 8, 16, [5, 3, 7], [100, 63, 333], 0, False),       # one row tile
    ("fp16", 64, 2, 4, 16, [90, 4], [150, 70], 300, False),             # two row tiles
    ("bf16", 64, 1, 4, 32, [6, 5], [6000, 4000], 9000, False),          # rows of many parts
    ("fp16", 128, 2, 6, 24, [9, 12], [60, 150], 131, True),
]


def _problem(shape):
    dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, mask = shape
    pr = Problem(91, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, pad_rows=2)
    words = _random_mask(np.random.default_rng(92), q_lens, pr.N) if mask else None
    return pr, words


def _check(sv, pr, words, touched):
    """`touched` [rows, Hq]: which outputs have to be NaN; the others keep the
    bits of the call before `change`."""
    import torch
    out, lse, ws = _attend(sv, pr, words)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    t = torch.from_numpy(touched).cuda()
    assert torch.isnan(lse[t]).all() and torch.isnan(out[t]).all()
    rest = ~t
    assert torch.equal(lse[rest], pr.base_lse[rest])
    assert torch.equal(out[rest].view(torch.int16), pr.base_out[rest].view(torch.int16))


def _with_base(sv, shape):
    pr, words = _problem(shape)
    pr.base_out, pr.base_lse, ws = _attend(sv, pr, words)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    return pr, words, np.zeros((pr.N, pr.Hq), dtype=bool)


@pytest.mark.parametrize("shape", SHAPES)
def test_queries(sv, shape):  # noqa: F811
    """A NaN in one dim, a whole row of infinities, one infinite dim."""
    pr, words, touched = _with_base(sv, shape)
    last = pr.rows() - 1
    pr.q[1, 0, 7] = float("nan")
    pr.q[last, pr.Hq - 1] = float("inf")
    pr.q[last, 0, 3] = float("-inf")
    touched[1, 0] = touched[last, pr.Hq - 1] = touched[last, 0] = True
    _check(sv, pr, words, touched)


@pytest.mark.parametrize("shape", SHAPES)
def test_one_old_key(sv, shape):  # noqa: F811
    """The second sequence's first entry, in the last key head."""
    pr, words, touched = _with_base(sv, shape)
    pr.pools[0][int(pr.table_np[1, 0]), 0, pr.Hk - 1, 5] = float("nan")
    group = pr.Hq // pr.Hk
    touched[pr.indptr_np[1]:pr.indptr_np[2], (pr.Hk - 1) * group:] = True
    _check(sv, pr, words, touched)


@pytest.mark.parametrize("shape", SHAPES)
def test_a_new_key_reaches_the_rows_that_see_it(sv, shape):  # noqa: F811
    from oracle import paged
    pr, words, touched = _with_base(sv, shape)
    first, n = int(pr.indptr_np[0]), pr.q_lens[0]
    j = n // 2
    t = pr.kv_lens[0] - n + j
    pr.pools[0][int(pr.table_np[0, t // pr.page]), t % pr.page, 0] = float("nan")
    for i in range(n):
        if paged.sees(i, j, None if words is None else words[first + i]):
            touched[first + i, :pr.Hq // pr.Hk] = True
    assert touched.any()
    _check(sv, pr, words, touched)


@pytest.mark.parametrize("shape", SHAPES[1:])
def test_a_prefix_without_one_finite_key(sv, shape):  # noqa: F811
    """Parts in which a row's every score is NaN."""
    import torch
    pr, words, touched = _with_base(sv, shape)
    for t in range(pr.prefix):
        pr.pools[0][int(pr.ptable_np[t // pr.page]), t % pr.page, 0, 0] = float("nan")
    torch.cuda.synchronize()
    touched[:pr.rows(), :pr.Hq // pr.Hk] = True
    _check(sv, pr, words, touched)
