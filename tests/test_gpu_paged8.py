"""GPU (C ABI) vs the float64 oracle for the append with norms and the 8-bit paged
cache: spec_kv_append_norm, spec_kv_append8, spec_kv_read8, spec_prefix_attention8.

Tolerances (u = eps / 2 of the type, half a step):
* norm and rotation: the sum of squares of D fp32 values (D 2^-24 of it, half of
  that in its root), the reciprocal root (2^-23), two products: a value x is off
  by |x| (D / 2 + 5) 2^-24 =: n; then the rotation's (|x| + |y|) (5e-7 + 3 * 2^-24)
  as in test_gpu_paged.py, of the normalised pair; n of both dims passes through
  it.  The sum of both is d.
* 16-bit outputs: one rounding more, u (|ref| + d) (+ 2^-25 where fp16 is subnormal).
* codes: a value within d of the exact one, rounded to e4m3 of its block's scale:
  half a step is 2^-4 |x| or, below 2^-6, 2^-10 of the scale.  The scale is the one of a
  largest value within d of the exact one.
* values are not computed with, so their codes and scales are equal.
* attention: the tolerances of test_gpu_paged.py over the values that the codes stand for.
"""
import numpy as np
import pytest

from oracle import paged, paged8
from tests import test_gpu_paged as t16
from tests.paged8_util import Problem8
from tests.test_gpu_paged import Problem, _dt, _f64, sv  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = 1e-5

# dtype, D, Hk, Hq, page, block, rot, interleaved, axes, q_lens, kv_lens, heads_first, base, norm
APPEND = [
    ("bf16", 128, 8, 32, 16, 16, 128, False, 1, [1], [1], False, 0, True),
    ("bf16", 128, 8, 32, 16, 8, 128, False, 1, [5, 5, 5], [5, 16, 33], False, 1000000, True),
    ("fp16", 64, 4, 28, 24, 8, 32, True, 1, [3, 0, 7, 1], [30, 0, 7, 49], True, 77, True),
    ("fp16", 64, 1, 1, 8, 8, 64, False, 1, [2, 1], [3, 1], False, 0, False),
    ("bf16", 128, 2, 6, 32, 32, 102, False, 3, [9, 4], [20, 4], False, 0, True),
    ("bf16", 80, 3, 9, 40, 8, 20, True, 2, [1, 6], [41, 80], True, 0, True),
    ("fp16", 256, 2, 4, 64, 64, 256, False, 1, [130], [200], False, 2 ** 31 - 500, True),
    ("bf16", 16, 1, 3, 16, 16, 16, True, 1, [4], [12], False, 0, True),
    ("bf16", 96, 3, 6, 64, 32, 96, False, 1, [40, 3], [45, 80], False, 5, False),
    ("bf16", 64, 2, 4, 16, 16, 0, False, 1, [6], [40], False, 0, True),
    ("fp16", 128, 4, 8, 16, 16, 128, False, 1, [600, 1, 700], [650, 1, 701], False, 9, True),
    ("bf16", 64, 3, 3, 128, 64, 64, False, 1, [200, 63, 1], [263, 63, 64], True, 0, True),
]


class Rotation:
    def __init__(self, pr, rot, axes, seed):
        rng = np.random.default_rng(seed)
        self.half, self.axes = rot // 2, axes
        self.freq = (10000.0 ** (-np.arange(self.half) / max(self.half, 1))).astype(np.float32)
        self.positions = self.axis = None
        if axes > 1:
            self.positions = rng.integers(0, 2 ** 20, (axes, pr.N)).astype(np.int32)
            self.axis = (np.arange(self.half) % axes).astype(np.int32)

    def args(self):
        import torch
        dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
        return dict(inv_freq=dev(self.freq) if self.half else None, positions=dev(self.positions), axis=dev(self.axis))


def _weights(D, seed):
    return np.random.default_rng(seed).uniform(0.25, 1.5, (2, D)).astype(np.float32)


def _turned(pr, ro, x, weight, interleaved, base):
    """x [N, heads, D] normalised and rotated, and how far fp32 may be from it."""
    y = paged8.norm(x, None if weight is None else weight.astype(np.float64), EPS)
    near = np.abs(y) * ((pr.D / 2 + 5) * 2.0 ** -24 if weight is not None else 0.0)
    out, off = y.copy(), near.copy()
    for b, (ql, kl) in enumerate(zip(pr.q_lens, pr.kv_lens)):
        for i in range(ql):
            n = pr.indptr_np[b] + i
            pos = [base + kl - ql + i] if ro.positions is None else ro.positions[:, n]
            out[n] = paged.rotate(y[n], pos, ro.freq, ro.axis, interleaved)
    for f in range(ro.half):
        a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + ro.half)
        off[..., a] = off[..., b] = (np.abs(y[..., a]) + np.abs(y[..., b])) * (5e-7 + 3 * 2.0 ** -24) + near[..., a] + near[..., b]
    return out, off


def _new_entries(pr):
    """(row, sequence, entry) of every new position."""
    for b, (ql, kl) in enumerate(zip(pr.q_lens, pr.kv_lens)):
        for i in range(ql):
            yield pr.indptr_np[b] + i, b, kl - ql + i


@pytest.mark.parametrize("dtype,D,Hk,Hq,page,block,rot,interleaved,axes,q_lens,kv_lens,heads_first,base,norm", APPEND + [
    ("bf16", 72, 2, 4, 5, 0, 36, False, 1, [7], [9], False, 0, True),      # the last lane holds one vector
    ("fp16", 512, 1, 3, 7, 0, 512, False, 1, [5], [5], False, 3, True),
])
def test_append_norm(sv, dtype, D, Hk, Hq, page, block, rot, interleaved, axes, q_lens, kv_lens, heads_first, base, norm):  # noqa: F811
    import torch
    pr = Problem(21, dtype, D, Hk, Hq, page, q_lens, kv_lens, heads_first=heads_first, pad_rows=2)
    ro, w = Rotation(pr, rot, axes, 22), _weights(D, 23)
    qw, kw = (w[0], w[1]) if norm else (w[0], None)  # without: one side only
    before = [p.clone() for p in pr.pools]
    q_out = torch.full((pr.N, Hq, D), -7.0, dtype=pr.q.dtype, device="cuda")
    ws = sv.make_append_workspace()
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    sv.spec_kv_append_norm(sv.make_kv_cache(*pr.pools), pr.q, pr.k, pr.v, q_out, pr.indptr, pr.table, pr.kv_len, ws,
                           interleaved=interleaved, position_base=base, q_weight=dev(qw), k_weight=dev(kw), norm_eps=EPS,
                           **ro.args())
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    u, rows = torch.finfo(pr.q.dtype).eps / 2, pr.rows()
    want, off = _turned(pr, ro, _f64(pr.q), qw, interleaved, base)
    assert (np.abs(_f64(q_out) - want)[:rows] <= (u * (np.abs(want) + off) + off + 2.0 ** -25)[:rows]).all()
    assert (q_out[rows:] == -7.0).all()
    want, off = _turned(pr, ro, _f64(pr.k), kw, interleaved, base)
    got, new = _f64(pr.pools[0]), np.zeros_like(pr.live)
    for n, b, t in _new_entries(pr):
        at = pr.table_np[b, t // page], t % page
        new[at] = True
        assert (np.abs(got[at] - want[n]) <= u * (np.abs(want[n]) + off[n]) + off[n] + 2.0 ** -25).all()
        assert torch.equal(pr.pools[1][at], pr.v[n])
    old = torch.from_numpy(~new).cuda()
    for p, was in zip(pr.pools, before):
        assert torch.equal(p[old].view(torch.int16), was[old].view(torch.int16))


def _append8(sv, pr, ro, interleaved, base, qw, kw, ws=None, q_out=None):  # noqa: F811
    import torch
    if q_out is None:
        q_out = torch.full((pr.N, pr.Hq, pr.D), -7.0, dtype=pr.q.dtype, device="cuda")
    ws = sv.make_append_workspace() if ws is None else ws
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    sv.spec_kv_append8(pr.cache(sv), pr.q, pr.k, pr.v, q_out, pr.indptr, pr.table, pr.kv_len, ws, interleaved=interleaved,
                       position_base=base, q_weight=dev(qw), k_weight=dev(kw), norm_eps=EPS, **ro.args())
    return q_out, ws


def _check_append8(pr, before, ro, interleaved, base, kw):
    """Keys within their tolerance, values bit by bit, everything else as it was."""
    was = [[t.cpu().numpy() for t in side] for side in before]
    v_codes, v_scales = paged8.append8(was[1][0], was[1][1], _f64(pr.v), pr.indptr_np, pr.table_np, pr.kv_lens, pr.dtype)
    assert np.array_equal(pr.codes[1].cpu().numpy(), v_codes) and np.array_equal(pr.scales[1].cpu().numpy(), v_scales)
    want, off = _turned(pr, ro, _f64(pr.k), kw, interleaved, base)
    codes, scales = pr.codes[0].cpu().numpy(), pr.scales[0].cpu().numpy()
    new = np.zeros_like(pr.live)
    blocks = {}
    for n, b, t in _new_entries(pr):
        page, slot = pr.table_np[b, t // pr.page], t % pr.page
        new[page, slot] = True
        blocks.setdefault((page, slot // pr.block), []).append((n, slot))
    touched = np.zeros(scales.shape[:2], dtype=bool)
    for (page, k), rows in blocks.items():
        touched[page, k] = True
        behind = rows[0][1] % pr.block
        for h in range(pr.Hk):
            x, d = want[[n for n, _ in rows], h], off[[n for n, _ in rows], h]
            low, high = (paged8.exponent((np.abs(x) + s * d).clip(0), pr.dtype) for s in (-1, 1))
            old_e = -1000
            if behind:
                old_e = int(np.clip(int(was[0][1][page, k, h]) - 127, paged8.LOW[pr.dtype], paged8.HIGH[pr.dtype]))
            e = int(scales[page, k, h]) - 127
            assert max(low, old_e) <= e <= max(high, old_e)
            got = paged8.VALUES[codes[page, [s for _, s in rows], h]] * 2.0 ** e
            bound = (np.abs(x) + d) * 2.0 ** -4 + 2.0 ** (e - 10) + d
            assert (np.abs(got - x) <= bound).all()
            if behind:
                older = slice(k * pr.block, k * pr.block + behind)
                kept = was[0][0][page, older, h]
                assert np.array_equal(codes[page, older, h],
                                      paged8.encode(paged8.VALUES[kept] * 2.0 ** (old_e - e)) if e > old_e else kept)
    # older entries of the touched blocks were looked at
    free = ~new
    for page, k in np.argwhere(touched):
        free[page, k * pr.block:(k + 1) * pr.block] = False
    assert np.array_equal(codes[free], was[0][0][free]) and np.array_equal(scales[~touched], was[0][1][~touched])


@pytest.mark.parametrize("dtype,D,Hk,Hq,page,block,rot,interleaved,axes,q_lens,kv_lens,heads_first,base,norm", APPEND)
def test_append8(sv, dtype, D, Hk, Hq, page, block, rot, interleaved, axes, q_lens, kv_lens, heads_first, base, norm):  # noqa: F811
    import torch
    pr = Problem8(31, dtype, D, Hk, Hq, page, block, q_lens, kv_lens, heads_first=heads_first, pad_rows=2)
    ro, w = Rotation(pr, rot, axes, 32), _weights(D, 33)
    qw, kw = (w[0], w[1]) if norm else (None, None)
    before = [(c.clone(), s.clone()) for c, s in zip(pr.codes, pr.scales)]
    q_out, ws = _append8(sv, pr, ro, interleaved, base, qw, kw)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    u, rows = torch.finfo(pr.q.dtype).eps / 2, pr.rows()
    want, off = _turned(pr, ro, _f64(pr.q), qw, interleaved, base)
    assert (np.abs(_f64(q_out) - want)[:rows] <= (u * (np.abs(want) + off) + off + 2.0 ** -25)[:rows]).all()
    assert (q_out[rows:] == -7.0).all()
    _check_append8(pr, before, ro, interleaved, base, kw)


def test_append8_many_sequences(sv):  # noqa: F811
    rng = np.random.default_rng(5)
    q_lens = rng.integers(0, 3, 1500).tolist()
    kv_lens = [n + int(rng.integers(0, 20)) for n in q_lens]
    pr = Problem8(3, "bf16", 64, 1, 2, 8, 8, q_lens, kv_lens)
    ro, w = Rotation(pr, 64, 1, 4), _weights(64, 6)
    before = [(c.clone(), s.clone()) for c, s in zip(pr.codes, pr.scales)]
    _, ws = _append8(sv, pr, ro, False, 0, w[0], w[1])
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_append8(pr, before, ro, False, 0, w[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append8_values_at_the_ends_of_the_range(sv, dtype):  # noqa: F811
    """Zeros, the smallest and largest numbers of the type, NaN and infinities, each
    in blocks with ordinary neighbours and behind older entries."""
    import torch
    pr = Problem8(41, dtype, 64, 2, 2, 32, 8, [30, 9], [33, 12], spread=8)
    info, g = torch.finfo(_dt(dtype)), torch.Generator(device="cuda").manual_seed(1)
    kinds = [0.0, -0.0, info.tiny, info.smallest_normal * 8, -info.tiny * info.eps, info.max, -info.max, info.max / 2, float("inf"),
             float("-inf"), float("nan"), 1.0, 2.0 ** -8, 255.9, 256.0]
    for x in (pr.k, pr.v):
        pick = torch.randint(0, len(kinds), x.shape, generator=g, device="cuda")
        wild = torch.tensor(kinds, device="cuda", dtype=torch.float64).to(x.dtype)[pick]
        some = torch.rand(x.shape, generator=g, device="cuda") < 0.1
        some &= (torch.arange(x.shape[0], device="cuda") % 3 > 0)[:, None, None]
        x.copy_(torch.where(some, wild, x))
    pr.k[8:16] = 0.0  # a block of nothing
    pr.v[8:16] = float("nan")
    before = [(c.clone(), s.clone()) for c, s in zip(pr.codes, pr.scales)]
    ro = Rotation(pr, 0, 1, 2)
    _, ws = _append8(sv, pr, ro, False, 0, None, None)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    for i, x in enumerate((pr.k, pr.v)):  # nothing is computed with either
        codes, scales = paged8.append8(*(t.cpu().numpy() for t in before[i]), _f64(x), pr.indptr_np, pr.table_np, pr.kv_lens, dtype)
        got = pr.codes[i].cpu().numpy()
        assert np.array_equal(pr.scales[i].cpu().numpy(), scales)
        nan = codes & 0x7F == 0x7F  # either sign
        assert np.array_equal(got[~nan], codes[~nan]) and (got[nan] & 0x7F == 0x7F).all()


# dtype, D, Hk, Hq, page, block, q_lens, kv_lens, prefix, mask, heads_first
ATTEND = [
    ("bf16", 128, 1, 1, 16, 16, [1], [1], 0, False, False),
    ("bf16", 128, 8, 32, 16, 16, [1], [37], 512, False, False),
    ("bf16", 64, 2, 2, 8, 8, [1, 1, 1], [1, 127, 128], 0, False, True),
    ("fp16", 64, 2, 8, 24, 8, [5, 1, 3], [129, 300, 3], 1, False, False),
    ("fp16", 128, 4, 28, 40, 8, [5, 0, 5], [5, 0, 261], 127, False, True),
    ("bf16", 128, 2, 8, 64, 32, [5] * 7, [5, 64, 65, 200, 128, 256, 257], 129, False, False),
    ("bf16", 64, 1, 71, 16, 16, [1, 2, 3], [9, 40, 200], 300, False, False),     # one key head, 71 query heads
    ("fp16", 64, 1, 128, 16, 8, [3], [20], 40, False, False),
    ("bf16", 128, 2, 2, 128, 64, [300], [300], 0, False, False),                 # several row blocks, causal
    ("bf16", 128, 1, 3, 256, 64, [200, 90], [700, 90], 260, False, True),
    ("fp16", 64, 2, 10, 136, 8, [64, 1], [100, 400], 1000, False, False),
    ("bf16", 128, 2, 4, 16, 16, [12, 9, 6], [12, 50, 133], 0, True, False),      # rows that see nothing
    ("fp16", 64, 4, 28, 24, 8, [12] * 5, [12, 13, 140, 24, 129], 131, True, True),
    ("bf16", 64, 1, 4, 8, 8, [64], [64], 0, True, False),
    ("bf16", 64, 1, 2, 8, 8, [70, 65], [200, 65], 3, True, False),               # new entries past the 64th
    ("bf16", 128, 1, 1, 16, 16, [1] * 40, [130] * 40, 2000, False, False),
    ("bf16", 128, 2, 10, 32, 32, [6, 7, 12, 13, 25], [900, 70, 12, 500, 333], 0, False, False),  # 30 to 125 rows an item
]


def _attend8(sv, pr, words=None, ws=None, out=None, lse=None, stream=None):  # noqa: F811
    import torch
    if ws is None:
        ws = sv.make_attention_workspace(len(pr.q_lens), pr.N, pr.Hq, pr.D)
    if out is None:
        out = torch.full((pr.N, pr.Hq, pr.D), -7.0, dtype=pr.q.dtype, device="cuda")
    if lse is None:
        lse = torch.full((pr.N, pr.Hq), -7.0, device="cuda")
    mask = None if words is None else torch.from_numpy(words.view(np.int64)).cuda()
    sv.spec_prefix_attention8(pr.cache(sv), pr.q, out, pr.indptr, pr.table, pr.kv_len, ws,
                              prefix_table=pr.ptable if pr.prefix else None, prefix_len=pr.prefix, draft_mask=mask,
                              lse=lse, stream=stream)
    return out, lse, ws


@pytest.mark.parametrize("dtype,D,Hk,Hq,page,block,q_lens,kv_lens,prefix,mask,heads_first", ATTEND)
def test_attention8(sv, dtype, D, Hk, Hq, page, block, q_lens, kv_lens, prefix, mask, heads_first):  # noqa: F811
    pr = Problem8(7, dtype, D, Hk, Hq, page, block, q_lens, kv_lens, prefix=prefix, heads_first=heads_first, pad_rows=3)
    words = t16._random_mask(np.random.default_rng(8), q_lens, pr.N) if mask else None
    out, lse, ws = _attend8(sv, pr, words)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    t16._check_attend(pr, out, lse, words)
    rows = pr.rows()
    assert (out[rows:] == -7.0).all()


# dtype, D, Hk, page, block, kv_lens, firsts, counts, heads_first
READ = [
    ("bf16", 128, 8, 16, 16, [37], [0], [37], False),
    ("fp16", 64, 3, 24, 8, [100, 3, 50], [7, 0, 49], [93, 0, 1], True),
    ("bf16", 256, 2, 64, 64, [300, 64], [1, 63], [299, 1], False),
    ("fp16", 16, 1, 8, 8, [9], [0], [9], False),
    ("bf16", 80, 5, 40, 8, [500] * 9, [0] * 9, [500] * 9, True),
]


@pytest.mark.parametrize("dtype,D,Hk,page,block,kv_lens,firsts,counts,heads_first", READ)
def test_read8(sv, dtype, D, Hk, page, block, kv_lens, firsts, counts, heads_first):  # noqa: F811
    import torch
    pr = Problem8(9, dtype, D, Hk, Hk, page, block, [0] * len(kv_lens), kv_lens, heads_first=heads_first, pad_rows=1)
    indptr = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    rows = int(indptr[-1])
    wide = torch.full((2, rows + 2, Hk + 1, D + 8), -7.0, dtype=_dt(dtype), device="cuda")
    k, v = (w[:, :Hk, :D] for w in wide)  # strides of their own, two rows of padding
    ws = sv.make_append_workspace()
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    first = None if not any(firsts) else dev(firsts)
    sv.spec_kv_read8(pr.cache(sv), k, v, dev(indptr.tolist()), pr.table, ws, first=first)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    for out, side in ((k, 0), (v, 1)):
        want = paged8.read8(pr.codes[side].cpu().numpy(), pr.scales[side].cpu().numpy(), indptr, pr.table_np, firsts)
        assert np.array_equal(_f64(out)[:rows], want)
    assert (wide[:, rows:] == -7.0).all() and (wide[:, :, Hk:] == -7.0).all() and (wide[..., D:] == -7.0).all()
    only = torch.full_like(k, -7.0)
    sv.spec_kv_read8(pr.cache(sv), None, only, dev(indptr.tolist()), pr.table, ws, first=first)
    assert torch.equal(only[:rows], v[:rows])


def test_a_pass_through_the_cache(sv):  # noqa: F811
    """Rounds of append and attention on one cache, as a verify loop runs them: the
    attention sees what the appends left, the read-back gives the same."""
    import torch
    rounds, B, Hk, Hq, D, page, block = 5, 3, 2, 8, 64, 24, 8
    q_lens, kept = [6, 1, 4], [0, 0, 0]
    width, dt = 4, torch.bfloat16
    pool = lambda d: torch.full((B * width, page, Hk, D), d, dtype=torch.uint8, device="cuda")  # noqa: E731
    codes, scales = [pool(0x7F), pool(0x7F)], [torch.full((B * width, page // block, Hk), 255, dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache = sv.make_kv_cache8(*codes, *scales, dt)
    order = np.random.default_rng(0).permutation(B * width).reshape(B, width).astype(np.int32)
    table = torch.from_numpy(order).cuda()
    g = torch.Generator(device="cuda").manual_seed(3)
    freq = torch.tensor([1.0, 0.1] * 16, device="cuda")
    w = torch.rand(2, D, generator=g, device="cuda") + 0.5
    ws = sv.make_attention_workspace(B, sum(q_lens), Hq, D)
    for r in range(rounds):
        kv = [k + n for k, n in zip(kept, q_lens)]
        n = sum(q_lens)
        qkv = torch.randn(n, (Hq + 2 * Hk) * D, generator=g, device="cuda").to(dt) * (r + 1)
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hk * D, Hk * D], 1))
        indptr = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32, device="cuda")
        lens = torch.tensor(kv, dtype=torch.int32, device="cuda")
        q_out, out = torch.empty(n, Hq, D, dtype=dt, device="cuda"), torch.empty(n, Hq, D, dtype=dt, device="cuda")
        lse = torch.empty(n, Hq, device="cuda")
        sv.spec_kv_append8(cache, q, k, v, q_out, indptr, table, lens, ws, inv_freq=freq, q_weight=w[0], k_weight=w[1])
        sv.spec_prefix_attention8(cache, q_out, out, indptr, table, lens, ws, lse=lse)
        rows = torch.tensor(np.concatenate([[0], np.cumsum(kv)]), dtype=torch.int32, device="cuda")
        back = [torch.empty(sum(kv), Hk, D, dtype=dt, device="cuda") for _ in "kv"]
        sv.spec_kv_read8(cache, *back, rows, table, ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_OK

        class View:
            pass
        pr = View()
        pr.D, pr.q, pr.kv_lens, pr.prefix, pr.ptable_np, pr.table_np = D, q_out, kv, 0, None, order
        pr.indptr_np, pr.rows = indptr.cpu().numpy(), lambda: n
        pr.pools = [torch.from_numpy(paged8.values(c.cpu().numpy(), s.cpu().numpy())).cuda() for c, s in zip(codes, scales)]
        t16._check_attend(pr, out, lse)
        at = 0
        for b in range(B):
            for t in range(kv[b]):
                for x, side in zip(back, (0, 1)):
                    assert np.array_equal(_f64(x[at]), _f64(pr.pools[side][order[b, t // page], t % page]))
                at += 1
        kept = [k + min(n, r % 3 + 1) for k, n in zip(kept, q_lens)]  # some drafts are dropped
