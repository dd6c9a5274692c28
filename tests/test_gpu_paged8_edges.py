"""The 8-bit cache's calls where they can go wrong: scales and queries that are far
apart, values that are not finite, references that rise, streams, graphs, row offsets,
pages and lengths out of range, many parts."""
import numpy as np
import pytest

from oracle import paged, paged8
from tests import test_gpu_paged as t16
from tests.paged8_util import Problem8
from tests.test_gpu_paged import _f64, sv  # noqa: F401
from tests.test_gpu_paged8 import EPS, Rotation, _append8, _attend8, _check_append8, _weights

pytestmark = pytest.mark.gpu


def _checked(sv, pr, words=None, ws=None):  # noqa: F811
    out, lse, ws = _attend8(sv, pr, words, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    t16._check_attend(pr, out, lse, words)
    return out, lse, ws


def _set_scales(pr, side, change):
    """change(scales) on one side's scale bytes of live blocks."""
    s = pr.scales[side].cpu().numpy().astype(int)
    live = s < 255
    s = np.where(live, change(s), 255)
    pr.scales[side].copy_(__import__("torch").from_numpy(s.astype(np.uint8)))
    pr.refresh()


SHAPES = [
    # dtype, D, Hk, Hq, page, block, q_lens, kv_lens, prefix, mask
    ("bf16", 128, 2, 8, 16, 16, [5, 3, 7], [100, 63, 333], 0, False),
    ("fp16", 64, 2, 4, 16, 8, [90, 4], [150, 70], 300, False),
    ("bf16", 64, 1, 4, 32, 8, [6, 5], [6000, 4000], 2000, False),           # rows of many parts
    ("fp16", 128, 2, 6, 24, 8, [9, 12], [60, 150], 131, True),
    ("bf16", 128, 1, 2, 16, 16, [300, 2], [400, 10], 40, False),            # several row blocks
]


def _problem(shape, seed, **kw):
    dtype, D, Hk, Hq, page, block, q_lens, kv_lens, prefix, mask = shape
    pr = Problem8(seed, dtype, D, Hk, Hq, page, block, q_lens, kv_lens, prefix=prefix, pad_rows=2, **kw)
    return pr, t16._random_mask(np.random.default_rng(seed + 1), q_lens, pr.N) if mask else None


@pytest.mark.parametrize("shape", SHAPES)
def test_value_scales_far_apart(sv, shape):  # noqa: F811
    """Blocks whose values differ by up to 2^60 (bf16), the largest first, last or
    anywhere: a row's output is right against its own weights' values."""
    for how in (0, 1, 2):
        pr, words = _problem(shape, 101 + how)
        rng = np.random.default_rng(how)
        low, high = (-30, 30) if pr.dtype == "bf16" else (-6, 6)
        shape_ = pr.scales[1].shape
        far = np.broadcast_to(np.linspace(low, high, shape_[0]).astype(int)[:, None, None], shape_)
        far = (far, -far, rng.integers(low, high + 1, shape_))[how]
        _set_scales(pr, 1, lambda s: np.clip(s + far, 127 + paged8.LOW[pr.dtype], 127 + paged8.HIGH[pr.dtype]))
        _checked(sv, pr, words)


def test_a_row_that_sees_only_small_values(sv):  # noqa: F811
    """One block of values 2^40 times the others', where every row's weight is nothing,
    before, among and behind them: the rows' outputs are of the small ones."""
    import torch
    for at in (0, 20, 39):
        pr = Problem8(111, "bf16", 64, 1, 4, 16, 16, [3], [700])
        s = pr.scales[1].cpu().numpy()
        s[pr.table_np[0, at]] += 40
        pr.scales[1].copy_(torch.from_numpy(s))
        # their keys against every query: scores far below the others'
        q = torch.ones_like(pr.q)
        pr.q = q
        codes = pr.codes[0].cpu().numpy()
        codes[pr.table_np[0, at]] = 0xF0   # -128 in every dim
        pr.codes[0].copy_(torch.from_numpy(codes))
        ks = pr.scales[0].cpu().numpy()
        ks[pr.table_np[0, at]] = 127
        pr.scales[0].copy_(torch.from_numpy(ks))
        pr.refresh()
        _checked(sv, pr)


@pytest.mark.parametrize("shape", SHAPES)
def test_key_scales_far_apart(sv, shape):  # noqa: F811
    """Keys of blocks that differ by 2^12 in length: scores from nearly 0 to hundreds,
    references that rise at any tile."""
    pr, words = _problem(shape, 121)
    rng = np.random.default_rng(5)
    _set_scales(pr, 0, lambda s: np.clip(s + rng.integers(-8, 5, s.shape), 127 - 15, 127 + 8))
    _checked(sv, pr, words)


def test_queries_far_apart(sv):  # noqa: F811
    """Rows 2^-40 and 2^30 times the others', a row of zeros, rows of one large dim:
    the scores of every row are its own.  (Keys scaled down so that they stay scores.)"""
    import torch
    for dtype, factors in (("bf16", [1.0, 2.0 ** -40, 0.0, 2.0 ** 30, 2.0 ** -100, 1.0]), ("bf16", [1.0, 2.0 ** -18, 3.0, 0.0, 1.0, 2.0]),
                           ("fp16", [1.0, 2.0 ** -12, 0.0, 2.0 ** 6, 1.0, 1.0])):
        pr = Problem8(131, dtype, 128, 2, 8, 16, 16, [6], [300], prefix=130)
        pr.q = (pr.q.double() * torch.tensor(factors, device="cuda", dtype=torch.float64)[:, None, None]).to(pr.q.dtype)
        pr.q[4, :, 5] = 2.0
        down = 30 if max(factors) > 2 ** 20 else 0
        _set_scales(pr, 0, lambda s: np.maximum(s - down, 127 + paged8.LOW[dtype]))
        _checked(sv, pr)


@pytest.mark.parametrize("dtype,move", [("bf16", 115), ("bf16", -80), ("fp16", 6)])
def test_values_near_the_ends_of_the_type(sv, dtype, move):  # noqa: F811
    """All values times 2^move, which scales the exact sums by as much; at 2^115 the sums
    before their division pass the largest fp32."""
    import torch
    pr = Problem8(141, dtype, 64, 2, 4, 16, 8, [4, 1], [60, 300], prefix=700)
    _, plain_lse, ws = _attend8(sv, pr)
    _set_scales(pr, 1, lambda s: s + move)
    out, lse, _ = _attend8(sv, pr, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert torch.equal(lse, plain_lse) and torch.isfinite(out).all()
    pr.pools[1] = pr.pools[1] * 2.0 ** -move
    rows = pr.rows()
    scaled = out.double()
    scaled[:rows] *= 2.0 ** -move
    t16._check_attend(pr, scaled.to(pr.q.dtype), lse)


@pytest.mark.parametrize("shape", SHAPES)
def test_nan_keys_reach_the_rows_that_see_them(sv, shape):  # noqa: F811
    import torch
    pr, words = _problem(shape, 151)
    base, base_lse, ws = _attend8(sv, pr, words)
    n, group = pr.q_lens[0], pr.Hq // pr.Hk
    touched = np.zeros((pr.N, pr.Hq), dtype=bool)
    j = n // 2
    t = pr.kv_lens[0] - n + j
    pr.codes[0][int(pr.table_np[0, t // pr.page]), t % pr.page, 0, 3] = 0xFF
    for i in range(n):
        if paged.sees(i, j, None if words is None else words[i]):
            touched[i, :group] = True
    # the second sequence's first entry, the last head: every row of it sees that
    pr.codes[0][int(pr.table_np[1, 0]), 0, pr.Hk - 1, pr.D - 1] = 0x7F
    if pr.kv_lens[1] > pr.q_lens[1]:
        touched[pr.indptr_np[1]:pr.indptr_np[2], (pr.Hk - 1) * group:] = True
    # and a query that is not finite
    last = pr.rows() - 1
    pr.q[last, 0, 7] = float("nan")
    touched[last, 0] = True
    out, lse, _ = _attend8(sv, pr, words, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    m = torch.from_numpy(touched).cuda()
    assert torch.isnan(lse[m]).all() and torch.isnan(out[m]).all()
    # the others' queries may have been taken in the other type: the same to rounding
    rest = ~m[:pr.rows()]
    u = torch.finfo(pr.q.dtype).eps / 2
    assert torch.allclose(lse[:pr.rows()][rest], base_lse[:pr.rows()][rest], rtol=2.0 ** -20, atol=2.0 ** -14)
    # weights rounded to 2^-9 (bf16) or 2^-12 each way, the result as well
    assert torch.allclose(out[:pr.rows()][rest].double(), base[:pr.rows()][rest].double(), rtol=4 * u, atol=16 * u * 8)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("place", ["first", "middle", "last"])
def test_nan_values_that_a_mask_hides(sv, shape, place):  # noqa: F811
    """A NaN among one new entry's values: rows that see it get NaN in that dim, the
    others what they get without it."""
    import torch
    pr, words = _problem(shape, 161)
    n, D = pr.q_lens[0], pr.D
    j = {"first": 0, "middle": n // 2, "last": n - 1}[place]
    t = pr.kv_lens[0] - n + j
    where = int(pr.table_np[0, t // pr.page]), t % pr.page
    pr.codes[1][where][0, 5] = 0
    pr.codes[1][where][pr.Hk - 1, D - 2] = 0
    pr.refresh()
    clean, clean_lse, ws = _checked(sv, pr, words)
    pr.codes[1][where][0, 5] = 0x7F
    pr.codes[1][where][pr.Hk - 1, D - 2] = 0xFF
    out, lse, _ = _attend8(sv, pr, words, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert torch.equal(lse, clean_lse)
    group, got = pr.Hq // pr.Hk, out.clone()
    for i in range(n):
        if not paged.sees(i, j, None if words is None else words[i]):
            continue
        for heads, dim in ((slice(0, group), 5), (slice(pr.Hq - group, pr.Hq), D - 2)):
            assert torch.isnan(got[i, heads, dim]).all()
            got[i, heads, dim] = clean[i, heads, dim]
    t16._check_attend(pr, got, lse, words)
    assert torch.equal(out[n:], clean[n:])


def test_peaked_scores(sv):  # noqa: F811
    """Queries along single keys: references that rise by hundreds, early, late and at a
    tile's border, in one group's tiles and in the other's."""
    import torch
    for Hq in (4, 40):  # one narrow part, and a wide one
        pr = Problem8(171, "bf16", 128, 1, Hq, 16, 16, [4], [520], prefix=400)
        for i, (table, t) in enumerate(((pr.ptable_np, 3), (pr.ptable_np, 399), (pr.table_np[0], 128), (pr.table_np[0], 510))):
            pr.q[i] = (20 * pr.pools[0][int(table[t // 16]), t % 16, 0]).to(torch.bfloat16)[None].expand(Hq, -1)
        _checked(sv, pr)


def test_small_weights_count(sv):  # noqa: F811
    """Thousands of keys whose weights are 2^-20 (bf16) or 2^-24 (fp16) of one key's and
    whose values are large: they do not vanish."""
    import torch
    for dtype, far in (("bf16", 20.0), ("fp16", 24.0)):
        pr = Problem8(181, dtype, 64, 1, 4, 64, 64, [1], [8192])
        for side in (0, 1):
            pr.codes[side].fill_(0x38)  # ones
            pr.scales[side].fill_(127)
        t = 77
        page, slot = int(pr.table_np[0, t // 64]), t % 64
        pr.codes[0][page, slot, 0, 0] = 0x48  # 4: its score is 3 q_0 scale above the others'
        pr.codes[1][:] = 0x48                 # values of 4, its own of 2^-5
        pr.codes[1][page, slot] = 0x10
        pr.refresh()
        pr.q.zero_()
        pr.q[..., 0] = far * 0.6931471805599453 * 8 / 3
        _checked(sv, pr)


def test_strided_rows_other_stream_and_repeats(sv):  # noqa: F811
    import torch
    pr = Problem8(191, "bf16", 64, 2, 8, 16, 8, [5, 3, 7], [100, 3, 333], prefix=700)
    wide = torch.full((pr.N, pr.Hq + 2, 2 * pr.D), -7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = wide[:, 1:-1, :pr.D], torch.empty((pr.N, pr.Hq), device="cuda")
    ws = sv.make_attention_workspace(3, pr.N, pr.Hq, pr.D)
    torch.cuda.synchronize()
    s, first = torch.cuda.Stream(), None
    for _ in range(4):
        out.fill_(0)
        torch.cuda.synchronize()
        _attend8(sv, pr, ws=ws, out=out, lse=lse, stream=s)
        assert sv.spec_verify_status(ws, s) == sv.SPEC_OK
        now = (out.clone(), lse.clone())
        first = first or now
        assert torch.equal(now[0], first[0]) and torch.equal(now[1], first[1])
    t16._check_attend(pr, out, lse)
    assert (wide[:, 0] == -7.0).all() and (wide[:, -1] == -7.0).all() and (wide[..., pr.D:] == -7.0).all()


def test_two_streams_at_once(sv):  # noqa: F811
    """Two calls with workspaces of their own on one cache, side by side."""
    import torch
    a = Problem8(201, "bf16", 128, 2, 8, 16, 16, [5, 3], [900, 1300], prefix=600)
    want, want_lse, ws = _attend8(sv, a)
    wss = [ws, sv.make_attention_workspace(2, a.N, a.Hq, a.D)]
    outs = [[torch.empty_like(want), torch.empty_like(want_lse)] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, (out, lse) in zip(streams, wss, outs):
            _attend8(sv, a, ws=w, out=out, lse=lse, stream=s)
    torch.cuda.synchronize()
    for s, w, (out, lse) in zip(streams, wss, outs):
        assert sv.spec_verify_status(w, s) == sv.SPEC_OK
        assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_append_attend_and_read_in_a_graph(sv):  # noqa: F811
    """The three calls captured once and replayed for rounds whose lengths differ."""
    import torch
    pr = Problem8(211, "bf16", 128, 2, 8, 16, 16, [4, 4, 4], [60, 60, 60], prefix=40)
    q_out = torch.empty((pr.N, pr.Hq, pr.D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q_out), torch.empty((pr.N, pr.Hq), device="cuda")
    back = [torch.empty((12, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    ws, cache = sv.make_attention_workspace(3, pr.N, pr.Hq, pr.D), pr.cache(sv)
    first = torch.zeros(3, dtype=torch.int32, device="cuda")
    ro, w = Rotation(pr, 128, 1, 1), torch.from_numpy(_weights(128, 2)).cuda()
    args = ro.args()

    def all_three():
        sv.spec_kv_append8(cache, pr.q, pr.k, pr.v, q_out, pr.indptr, pr.table, pr.kv_len, ws, q_weight=w[0], k_weight=w[1],
                           norm_eps=EPS, position_base=pr.prefix, **args)
        sv.spec_prefix_attention8(cache, q_out, out, pr.indptr, pr.table, pr.kv_len, ws, prefix_table=pr.ptable,
                                  prefix_len=pr.prefix, lse=lse)
        sv.spec_kv_read8(cache, *back, pr.indptr, pr.table, ws, first=first)

    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        all_three()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            all_three()
    torch.cuda.synchronize()
    projected = pr.q
    for kv in ([4, 20, 60], [8, 33, 59]):
        pr.kv_lens = kv
        pr.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        first.copy_(torch.tensor([n - 4 for n in kv], dtype=torch.int32))
        before = [(c.clone(), x.clone()) for c, x in zip(pr.codes, pr.scales)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert sv.spec_verify_status(ws) == sv.SPEC_OK
        _check_append8(pr, before, ro, False, pr.prefix, w[1].cpu().numpy())
        pr.refresh()
        pr.q = q_out
        t16._check_attend(pr, out, lse)
        pr.q = projected
        for side in (0, 1):
            want = paged8.read8(pr.codes[side].cpu().numpy(), pr.scales[side].cpu().numpy(), pr.indptr_np, pr.table_np, [n - 4 for n in kv])
            assert np.array_equal(_f64(back[side]), want)


def test_a_larger_draft_and_its_rejection(sv):  # noqa: F811
    """A block's scale rises with a large new entry and stays when the entry is dropped;
    older entries keep what half a step of the new scale leaves."""
    import torch
    pr = Problem8(221, "bf16", 64, 2, 2, 16, 16, [1], [6])
    ro, older = Rotation(pr, 0, 1, 1), pr.pools[0][int(pr.table_np[0, 0]), :5].clone()
    pr.k *= 1000.0
    _, ws = _append8(sv, pr, ro, False, 0, None, None)
    scale = pr.scales[0][int(pr.table_np[0, 0]), 0].clone()
    pr.k /= 1000.0
    _append8(sv, pr, ro, False, 0, None, None, ws=ws)  # the same entry again
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert torch.equal(pr.scales[0][int(pr.table_np[0, 0]), 0], scale)
    pr.refresh()
    now = pr.pools[0][int(pr.table_np[0, 0]), :5]
    step = 2.0 ** (scale.double() - 127 - 10)[None, :, None]
    assert ((now - older).abs() <= older.abs() * 2.0 ** -4 + step).all()


def test_pages_and_lengths_out_of_range_are_reported(sv):  # noqa: F811
    """A page that is none and lengths past the table: reported, skipped, and the other
    sequence's results stand; codes and scales of other pages keep their bits."""
    import torch
    pr = Problem8(231, "bf16", 64, 1, 4, 16, 8, [2, 2], [40, 33])
    good, _, ws = _attend8(sv, pr)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    keep, ro = pr.table.clone(), Rotation(pr, 64, 1, 1)
    rows = torch.tensor([0, 40, 73], dtype=torch.int32, device="cuda")
    back = [torch.full((73, 1, 64), -7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for bad in (-1, 2 ** 30, pr.codes[0].shape[0]):
        pr.table.copy_(keep)
        pr.table[1, 1] = bad
        out, _, _ = _attend8(sv, pr, ws=ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        assert torch.equal(out[:2], good[:2])
        sv.spec_kv_read8(pr.cache(sv), *back, rows, pr.table, ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        assert (back[0][40 + 16:40 + 32] == 0).all() and torch.equal(back[1][:40].double(), pr.pools[1][pr.table[0].long()].flatten(0, 1)[:40])
        pr.table[1, 2] = bad  # the page that the append would write to
        before = [(c.clone(), s.clone()) for c, s in zip(pr.codes, pr.scales)]
        _append8(sv, pr, ro, False, 0, None, None, ws=ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        touched = [int(pr.table_np[0, 2]), int(pr.table_np[1, 1])]  # entries 38, 39; entry 31 may go where it was
        rest = torch.ones(pr.codes[0].shape[0], dtype=torch.bool, device="cuda")
        rest[touched] = False
        for (c, s), (wc, wsc) in zip(zip(pr.codes, pr.scales), before):
            assert torch.equal(c[rest], wc[rest]) and torch.equal(s[rest], wsc[rest])
            c.copy_(wc)
            s.copy_(wsc)
    pr.table.copy_(keep)
    for bad_len in (1, -5, 10 ** 6):  # fewer than the new positions, negative, past the table
        pr.kv_len[1] = bad_len
        pr.table[1, 2:] = pr.table[1, 1]
        out, _, _ = _attend8(sv, pr, ws=ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        assert torch.equal(out[:2], good[:2])
        before = [(c.clone(), s.clone()) for c, s in zip(pr.codes, pr.scales)]
        _append8(sv, pr, ro, False, 0, None, None, ws=ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        own = [int(pr.table_np[0, 2]), int(pr.table_np[1, 0])]  # sequence 1's first entry may be new (length 1)
        rest = torch.ones(pr.codes[0].shape[0], dtype=torch.bool, device="cuda")
        rest[own] = False
        for (c, s), (wc, wsc) in zip(zip(pr.codes, pr.scales), before):
            assert torch.equal(c[rest], wc[rest]) and torch.equal(s[rest], wsc[rest])
            c.copy_(wc)
            s.copy_(wsc)


def test_row_offsets_that_do_not_ascend(sv):  # noqa: F811
    """Reported; nothing is written outside the tables' pages."""
    import torch
    pr = Problem8(241, "bf16", 64, 1, 2, 8, 8, [3, 3, 3], [8, 8, 8])
    ro, keep = Rotation(pr, 64, 1, 1), pr.indptr.clone()
    pages = torch.zeros(pr.codes[0].shape[0], dtype=torch.bool, device="cuda")
    pages[pr.table[:, 0].long()] = True
    before = [(c.clone(), s.clone()) for c, s in zip(pr.codes, pr.scales)]
    for bad in ([1, 3, 6, 9], [0, 6, 3, 9], [0, 9, 9, 3], [0, 3, 6, 100], [-5, 3, 6, 9]):
        pr.indptr.copy_(torch.tensor(bad, dtype=torch.int32))
        _, ws = _append8(sv, pr, ro, False, 0, None, None)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT, bad
        back = torch.full((pr.N, 1, 64), -7.0, dtype=torch.bfloat16, device="cuda")
        sv.spec_kv_read8(pr.cache(sv), back, None, pr.indptr, pr.table, ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT, bad
        for (c, s), (wc, wsc) in zip(zip(pr.codes, pr.scales), before):
            assert torch.equal(c[~pages], wc[~pages]) and torch.equal(s[~pages], wsc[~pages])
            c.copy_(wc)
            s.copy_(wsc)
    pr.indptr.copy_(keep)
