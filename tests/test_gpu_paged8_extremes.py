"""Attention over the 8-bit cache at the ends of its ranges, with bounds that see every
row: factors of scores, scales of values and weights far apart, queries of many sizes,
scores past what fp32 resolves.

Each problem is one sequence, handed in many times over (`COPIES`), so that the CTAs' parts
hold several key tiles and are cut at different ones; every copy is held to the bound.

The bound of an output, per row (u = eps / 2 of the type, half a step; weights w of which the
largest is 1, l their sum): weights rounded to the type or fp16, u sum w|v| / l; fp16 weights
that are small, at most 2^-29 (bf16 caches, 2^-32 fp16 ones) and no more than the weight
itself, sum min(w, 2^-29) |v| / l over the keys named by `small`; the result rounded, u |ref|;
fp32 scores of D exact products, es = D 2^-23 sum|q k| scale, twice; n keys summed in fp32
and the exponential, n 2^-23 + 2^-20; fp16 results below 2^-14, 2^-25.
"""
import numpy as np
import pytest

from oracle import paged, paged8
from tests.paged8_util import Problem8
from tests.test_gpu_paged import _f64, sv  # noqa: F401

pytestmark = pytest.mark.gpu

COPIES = 160
SMALL = {"bf16": 2.0 ** -29, "fp16": 2.0 ** -32}

# key heads, query heads, new positions: parts of 20 rows, and of 96 (where the softmax groups share tiles)
FORM = pytest.mark.parametrize("form", [(2, 8, 5), (1, 32, 3)], ids=["narrow", "wide"])


def _make(seed, dtype, D, form, kv, prefix=0, block=16):
    Hk, Hq, n = form
    return Problem8(seed, dtype, D, Hk, Hq, 16, block, [n], [kv], prefix=prefix, spread=0)


def _where(pr, t):
    return int(pr.table_np[0, t // pr.page]), t % pr.page


def _edit(pr, side, codes=None, exponent=None):
    """Codes and block exponents of one side by entry: codes(t, old [Hk, D]) and
    exponent(t, old) of the block that begins at entry t; None keeps the old."""
    import torch
    c, s = pr.codes[side].cpu().numpy(), pr.scales[side].cpu().numpy()
    for t in range(pr.kv_lens[0]):
        page, slot = _where(pr, t)
        if codes is not None:
            new = codes(t, c[page, slot])
            c[page, slot] = c[page, slot] if new is None else new
        if exponent is not None and t % pr.block == 0:
            new = exponent(t, s[page, slot // pr.block].astype(int) - 127)
            s[page, slot // pr.block] = s[page, slot // pr.block] if new is None else np.asarray(new) + 127
    pr.codes[side].copy_(torch.from_numpy(c))
    pr.scales[side].copy_(torch.from_numpy(s))
    pr.refresh()


def _exact(pr, words=None, scale=None, small=None, exact_scores=False):
    """out, lse and their bounds [n, Hq, ...] of the one sequence in float64; small(t): keys
    (numbered with the prefix first) whose weights may be off where they are small;
    exact_scores: equal scores are equal in fp32, and no others count."""
    n, D, group = pr.q_lens[0], pr.D, pr.Hq // pr.Hk
    kv, P = pr.kv_lens[0], pr.prefix
    scale = D ** -0.5 if scale is None else scale
    at = [(int(pr.ptable_np[t // pr.page]), t % pr.page) for t in range(P)] + [_where(pr, t) for t in range(kv)]
    pages, slots = np.array(at).T
    K, V, q = (_f64(x) for x in (pr.pools[0], pr.pools[1], pr.q))
    K, V = K[pages, slots], V[pages, slots]
    import torch
    u = torch.finfo(pr.q.dtype).eps / 2
    may = np.array([small is None or small(t) for t in range(P + kv)])
    out, lse = np.zeros((n, pr.Hq, D)), np.full((n, pr.Hq), -np.inf)
    tol, ltol = np.zeros_like(out), np.zeros_like(lse)
    for i in range(n):
        old = P + kv - n
        seen = np.array([t < old or paged.sees(i, t - old, None if words is None else words[i]) for t in range(P + kv)])
        if not seen.any():
            continue
        for h in range(pr.Hq):
            k, v = K[seen, h // group], V[seen, h // group]
            s = scale * (k @ q[i, h])
            w = np.exp(s - s.max())
            l = w.sum()
            out[i, h], lse[i, h] = w @ v / l, s.max() + np.log(l)
            es = 0.0 if exact_scores else D * 2.0 ** -23 * scale * (np.abs(k) @ np.abs(q[i, h]))[w > 2.0 ** -60].max()
            rel = u + 2 * es + 2.0 ** -20 + len(s) * 2.0 ** -23
            lost = np.minimum(w, SMALL[pr.dtype]) * may[seen]
            tol[i, h] = rel * (w @ np.abs(v)) / l + u * np.abs(out[i, h]) + lost @ np.abs(v) / l \
                + (2.0 ** -25 if pr.dtype == "fp16" else 0.0)
            ltol[i, h] = es + len(s) * 2.0 ** -23 + 2.0 ** -20 + abs(lse[i, h]) * 2.0 ** -21
    return out, lse, tol, ltol


def _run(sv, pr, words=None, scale=None, copies=COPIES):  # noqa: F811
    """The sequence `copies` times over in one call."""
    import torch
    n = pr.q_lens[0]
    i32 = dict(dtype=torch.int32, device="cuda")
    q = pr.q[:n].repeat(copies, 1, 1)
    out, lse = torch.full_like(q, -7.0), torch.full((n * copies, pr.Hq), -7.0, device="cuda")
    ws = sv.make_attention_workspace(copies, n * copies, pr.Hq, pr.D)
    mask = None if words is None else torch.from_numpy(np.tile(words[:n], copies).view(np.int64)).cuda()
    sv.spec_prefix_attention8(pr.cache(sv), q, out, torch.arange(copies + 1, **i32) * n, pr.table.repeat(copies, 1),
                              pr.kv_len.repeat(copies), ws, prefix_table=pr.ptable if pr.prefix else None,
                              prefix_len=pr.prefix, draft_mask=mask, scale=scale, lse=lse)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    return _f64(out).reshape(copies, n, pr.Hq, pr.D), _f64(lse).reshape(copies, n, pr.Hq)


def _check(sv, pr, words=None, scale=None, small=None, exact_scores=False):  # noqa: F811
    want, wl, tol, ltol = _exact(pr, words, scale, small, exact_scores)
    empty = np.isneginf(wl)
    # the bound can tell: an answer of zeros does not pass it
    assert (np.abs(want) > 2 * tol)[~empty].mean() > 0.75
    for copies in (COPIES, 1):
        got, gl = _run(sv, pr, words, scale, copies)
        assert (np.isneginf(gl) == empty).all() and (got[:, empty] == 0).all()
        gl, flat = np.where(empty, 0, gl), np.where(empty, 0, wl)
        bad = ~(np.abs(gl - flat) <= ltol)
        assert not bad.any(), (np.argwhere(bad)[:4], gl[bad][:4], np.broadcast_to(flat, gl.shape)[bad][:4])
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], np.broadcast_to(want, got.shape)[bad][:4],
                               np.broadcast_to(tol, got.shape)[bad][:4])


# ---------------------------------------------------------------------------
# the factor of a score: scale * log2(e) * the queries' unit * the key's scale
# ---------------------------------------------------------------------------
@FORM
@pytest.mark.parametrize("factor,scale", [(-40, None), (-60, None), (-110, None), (0, 1e-12), (-40, 1e-30)])
@pytest.mark.parametrize("prefix,masked", [(0, False), (130, False), (0, True), (130, True)])
def test_factors_of_scores_near_zero(sv, form, factor, scale, prefix, masked):  # noqa: F811
    """Queries so small (or such a scale) that a block of zero keys, whose exponent is -100, has
    a factor below fp32: its hidden and missing entries do not count, the others as 0."""
    pr = _make(11, "bf16", 128, form, 693, prefix)
    pr.q = pr.q * 2.0 ** factor
    new = 693 - form[2]
    zero = lambda t: t // 16 in (0, 20, new // 16, 692 // 16)  # noqa: E731  the last blocks: new entries, and past the end
    _edit(pr, 0, lambda t, c: np.where(zero(t), 0, c), lambda t, e: np.where(zero(t), -100, e))
    words = np.array([0, 1, 0b110, 0b1000, 0b11111][:form[2]], dtype=np.uint64) if masked else None
    _check(sv, pr, words, scale)


def test_a_row_that_sees_nothing_beside_zero_keys(sv):  # noqa: F811
    pr = _make(12, "bf16", 64, (2, 8, 3), 3)
    pr.q = pr.q * 2.0 ** -60
    _edit(pr, 0, lambda t, c: 0 * c, lambda t, e: -100)
    _check(sv, pr, np.array([0, 0b1, 0], dtype=np.uint64))


@FORM
def test_factors_of_scores_past_the_largest(sv, form):  # noqa: F811
    """Queries of 2^40 along a dim in which keys of the largest exponent are zero, and a row
    of zeros beside them: every score is 0."""
    pr = _make(13, "bf16", 128, form, 437, 130)
    pr.q = pr.q * 0
    pr.q[::2, :, 0] = 2.0 ** 40
    zero = lambda c: np.where(np.arange(128) == 0, 0, c)  # noqa: E731
    _edit(pr, 0, lambda t, c: zero(c), lambda t, e: 120)
    for page in pr.ptable_np:
        pr.codes[0][int(page), :, :, 0] = 0
    pr.scales[0][pr.ptable.long()] = 120 + 127
    pr.refresh()
    _check(sv, pr)


# ---------------------------------------------------------------------------
# values of blocks that are far apart
# ---------------------------------------------------------------------------
@FORM
@pytest.mark.parametrize("dtype,low,high", [("bf16", -30, 30), ("bf16", -6, 6), ("fp16", -6, 6)])
def test_value_scales_far_apart_row_by_row(sv, form, dtype, low, high):  # noqa: F811
    rng = np.random.default_rng(5)
    for how in range(4):
        pr = _make(21 + how, dtype, 64, form, 700)
        far = [lambda t: low + (high - low) * t // 700, lambda t: high - (high - low) * t // 700,
               lambda t: int(rng.integers(low, high + 1)), lambda t: high if 300 <= t < 316 else low][how]
        _edit(pr, 1, None, lambda t, e: np.clip(e + far(t), paged8.LOW[dtype], paged8.HIGH[dtype]))
        _check(sv, pr)


def _weightless(pr, first, count):
    """Keys first .. first + count - 1 whose weights are nothing: -128 in every dim, before
    queries of ones (whose other scores are small)."""
    pr.q = pr.q * 0 + 1.0
    inside = lambda t: first <= t < first + count  # noqa: E731
    _edit(pr, 0, lambda t, c: np.full_like(c, 0xF0) if inside(t) else None, lambda t, e: 0 if inside(t) else None)


@FORM
@pytest.mark.parametrize("at", [0, 128, 320, 688])
def test_rows_of_small_values_beside_weightless_large_ones(sv, form, at):  # noqa: F811
    """A block of values 2^40 times the others', at which every row's weight is nothing."""
    pr = _make(31, "bf16", 64, form, 704)
    _weightless(pr, at, 16)
    _edit(pr, 1, None, lambda t, e: e + 40 if t == at else None)
    _check(sv, pr)


@FORM
@pytest.mark.parametrize("apart", [100, 120, 131, 150, 200])
def test_a_hidden_block_of_much_larger_values(sv, form, apart):  # noqa: F811
    """The last block's values are 2^apart times the others' and have no weight: what the tiles
    before it gave stands (where fp32 can hold it beside them), or is lost; it is not enlarged.
    In the last tile small values may be lost from 2^110 on."""
    pr = _make(41, "bf16", 64, form, 704)
    _weightless(pr, 688, 16)
    _edit(pr, 1, lambda t, c: c & 0x7F, lambda t, e: e - 80 if t < 688 else e - 80 + apart)  # (values of one sign)
    want, wl, tol, ltol = _exact(pr)
    got, gl = _run(sv, pr)
    assert (np.abs(gl - wl) <= ltol).all()
    # at most the last tile's values
    V, K, q = (_f64(x) for x in (pr.pools[1], pr.pools[0], pr.q))
    group, lost = pr.Hq // pr.Hk, np.zeros_like(want)
    for h in range(pr.Hq):
        for t in range(640, 688):
            page, slot = _where(pr, t)
            w = np.exp(pr.D ** -0.5 * (K[page, slot, h // group] @ q[0, h]) - wl[:, h])
            lost[:, h] += w[:, None] * np.abs(V[page, slot, h // group])
    if apart <= 110:
        lost *= 0
    assert (np.abs(want) > 4 * (tol + lost)).all()
    if apart <= 131:  # (sums in units of 2^(apart - 87) are not below 2^-126)
        assert (np.abs(got - want) <= tol + lost).all()
    else:
        assert (np.abs(got) <= np.abs(want) + tol + lost).all()


@FORM
@pytest.mark.parametrize("log2", [6, 20, 28, 30, 31, 34, 40])
@pytest.mark.parametrize("first,count", [(16, 16), (128, 128), (256, 128), (304, 16), (384, 256), (512, 192)])
def test_small_weights_of_large_values(sv, form, log2, first, count):  # noqa: F811
    """One key of the first tile has the weight 1, all others 2^-log2, and some have values of
    2^log2 (a block, whole tiles): they count as much as the one."""
    pr = _make(51, "bf16", 64, form, 704)
    one, large = 7, lambda t: first <= t < first + count  # noqa: E731
    # scores: q_0 k_0, keys of 0 but the one's 4
    keys = lambda t, c: np.broadcast_to(np.where((np.arange(64) == 0) & (t == one), 0x48, 0), c.shape)  # noqa: E731
    _edit(pr, 0, keys, lambda t, e: 0)
    _edit(pr, 1, None, lambda t, e: -7 + (log2 if large(t) else 0))
    pr.q = pr.q * 0
    pr.q[..., 0] = log2 * np.log(2.0) * 8 / 4
    _check(sv, pr, small=lambda t: not large(t))


@FORM
@pytest.mark.parametrize("log2", [20, 28, 30, 31, 34, 40])
def test_small_weights_of_large_values_on_both_sides(sv, form, log2):  # noqa: F811
    """The same with large values first: two tiles of them, two of small ones that have the keys
    of weight 1, two of large ones again."""
    pr = _make(52, "bf16", 64, form, 704)
    large = lambda t: t < 256 or t >= 512  # noqa: E731
    keys = lambda t, c: np.broadcast_to(np.where((np.arange(64) == 0) & (t in (260, 390)), 0x48, 0), c.shape)  # noqa: E731
    _edit(pr, 0, keys, lambda t, e: 0)
    _edit(pr, 1, None, lambda t, e: -7 + (log2 if large(t) else 0))
    pr.q = pr.q * 0
    pr.q[..., 0] = log2 * np.log(2.0) * 8 / 4
    _check(sv, pr, small=lambda t: not large(t))


# ---------------------------------------------------------------------------
# queries whose dims are far apart
# ---------------------------------------------------------------------------
@FORM
@pytest.mark.parametrize("apart", [20, 28, 31, 32, 33, 35, 37, 45])
@pytest.mark.parametrize("rows", ["each", "beside"])
def test_small_dims_of_queries_against_large_keys(sv, form, apart, rows):  # noqa: F811
    """Dims 2^apart below the largest one of their row (or of another row), which decide the
    scores: keys are 2^apart times larger there, and 0 where the largest is."""
    import torch
    pr = _make(61, "bf16", 64, form, 460)
    rng = np.random.default_rng(apart)
    small = rng.uniform(1, 2, pr.q.shape) * rng.choice([-1.0, 1.0], pr.q.shape) * 2.0 ** -apart
    small[..., 0] = 1.0 if rows == "each" else 2.0 ** -20
    small[..., 1] = 0.0
    if rows == "beside":
        small[0] = 0.0
        small[0, :, 1] = 1.0  # the first position's rows: the largest dim alone, hidden by keys of 0
    pr.q = torch.from_numpy(small).to(torch.bfloat16).cuda()
    _edit(pr, 0, lambda t, c: np.where(np.arange(64) < 2, 0, c), lambda t, e: e + apart)
    _check(sv, pr)


# ---------------------------------------------------------------------------
# scores larger than fp32 resolves
# ---------------------------------------------------------------------------
@FORM
@pytest.mark.parametrize("dtype,log2", [("bf16", x) for x in (20, 25, 27, 29, 31, 33, 36, 40, 60, 100)] +
                         [("fp16", x) for x in (20, 23, 26)])
@pytest.mark.parametrize("how", ["equal", "negative", "two", "rising"])
def test_large_scores(sv, form, dtype, log2, how):  # noqa: F811
    """Scores of some 2^log2 in one dim, exact as products: keys of the largest score share the
    weight, the others have none."""
    import torch
    pr = _make(71, dtype, 64, form, 700)
    rng = np.random.default_rng(log2)
    a = log2 // 2 if dtype == "bf16" else 14
    b = log2 - a  # the keys' part
    tiles = 6

    def keys(t, c):
        code = {"equal": 0x73, "negative": 0xF3, "two": 0x73 if t % 3 else 0x6B, "rising": 0x73}[how]
        return np.broadcast_to(np.where(np.arange(64) == 0, code, 0), c.shape)

    # 1.375 2^(b + 3), or half of that; rising: by a power of two a tile
    _edit(pr, 0, keys, lambda t, e: b - 4 - (0 if how != "rising" else tiles - 1 - t // 128))
    # every row a mantissa of its own
    pr.q = pr.q * 0
    m = torch.from_numpy(rng.integers(128, 256, pr.q.shape[:2]) / 128.0).cuda()
    pr.q[..., 0] = (m * 2.0 ** a).to(pr.q.dtype)
    _check(sv, pr, exact_scores=True)


@FORM
@pytest.mark.parametrize("log2", [25, 31, 40, 60])
def test_large_scores_beside_a_hidden_nan(sv, form, log2):  # noqa: F811
    """The same, summed again key by key, for a value that is not finite and that only the last
    row sees."""
    pr = _make(72, "bf16", 64, form, 700)
    _edit(pr, 0, lambda t, c: np.broadcast_to(np.where(np.arange(64) == 0, 0x73, 0), c.shape), lambda t, e: log2 // 2 - 4)
    pr.q = pr.q * 0
    pr.q[..., 0] = 1.59375 * 2.0 ** (log2 - log2 // 2)
    want, wl, tol, ltol = _exact(pr, exact_scores=True)
    page, slot = _where(pr, 699)
    pr.codes[1][page, slot, 0, 5] = 0x7F
    for copies in (COPIES, 1):
        got, gl = _run(sv, pr, copies=copies)
        assert (np.abs(gl - wl) <= ltol).all()
        assert (np.abs(got - want)[:, :-1] <= tol[:-1]).all()
        first = pr.Hq // pr.Hk  # the heads that read key head 0
        assert np.isnan(got[:, -1, :first, 5]).all()
        got[:, -1, :first, 5] = want[-1, :first, 5]
        assert (np.abs(got - want) <= tol).all()
