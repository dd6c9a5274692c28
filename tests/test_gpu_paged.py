"""GPU (C ABI) vs the float64 oracle for the paged cache: spec_kv_append and
spec_prefix_attention, at the sizes, masks and layouts where they can go wrong.

Tolerances (u = eps / 2 of the type, half a step):
* append: the result is rounded once (u |ref|, 2^-25 absolute where fp16 goes
  subnormal); the angle is off by at most 5e-7 (fraction of a turn to 2^-53
  relative times a position below 2^31, its fp32 rounding, sincospi), each fp32
  product and sum by 2^-24: (|x| + |y|) (5e-7 + 3 * 2^-24).
* attention: weights rounded to the type (u sum w|v|; fp16 weights below 2^-14
  of the largest: 2^-25 absolute each), the result rounded (u |ref|); scores
  are fp32 sums of D exact products (D 2^-23 sum|q k| scale =: es, and the
  exponential 2^-21 relative), n keys summed in fp32 (n 2^-23).
"""
import numpy as np
import pytest

from oracle import paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_54_gb300 import _build
    _build.build()
    import speculative_decoding_verification_54_gb300 as m
    m.load()
    torch.cuda.set_device(0)
    return m


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _f64(t):
    return t.detach().double().cpu().numpy()


class Problem:
    """Pools with NaN wherever no live entry is, shuffled pages, table entries
    past the lengths pointing nowhere."""

    def __init__(self, seed, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix=0, heads_first=False, pad_rows=0):
        import torch
        self.dtype, self.D, self.Hk, self.Hq, self.page, self.prefix = dtype, D, Hk, Hq, page, prefix
        dt, rng = _dt(dtype), np.random.default_rng(seed)
        self.q_lens, self.kv_lens = q_lens, kv_lens
        self.N = sum(q_lens) + pad_rows
        B = len(q_lens)
        width = max(1, max(-(-n // page) for n in kv_lens))
        shared = -(-prefix // page)
        need = sum(-(-n // page) for n in kv_lens) + shared
        total = need + 2
        order = rng.permutation(total)
        table = np.full((B, width), 2 ** 30, dtype=np.int32)
        at = 0
        live = np.zeros((total, page), dtype=bool)
        for b, n in enumerate(kv_lens):
            c = -(-n // page)
            table[b, :c] = order[at:at + c]
            for t in range(n):
                live[table[b, t // page], t % page] = True
            at += c
        ptable = order[at:at + shared].astype(np.int32)
        for t in range(prefix):
            live[ptable[t // page], t % page] = True
        self.live = live
        g = torch.Generator().manual_seed(seed)
        shape = (total, Hk, page, D) if heads_first else (total, page, Hk, D)
        self.pools = []
        for _ in range(2):
            x = torch.randn(shape, generator=g).to(dt).cuda()
            x = x.transpose(1, 2) if heads_first else x
            x[torch.from_numpy(~live).cuda()] = float("nan")
            self.pools.append(x)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.indptr_np = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.table_np, self.ptable_np = table, ptable
        self.indptr, self.table, self.ptable, self.kv_len = i32(self.indptr_np), i32(table), i32(ptable), i32(kv_lens)
        # q, k and v of one projection's output
        qkv = torch.randn((self.N, (Hq + 2 * Hk) * D), generator=g).to(dt).cuda()
        q, k, v = qkv.split([Hq * D, Hk * D, Hk * D], dim=1)
        self.q, self.k, self.v = q.unflatten(1, (Hq, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (Hk, D))

    def rows(self):
        return int(self.indptr_np[-1])


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
APPEND = [
    # dtype, D, Hk, Hq, page, rot, interleaved, axes, q_lens, kv_lens, heads_first, base
    ("bf16", 128, 8, 32, 16, 128, False, 1, [1], [1], False, 0),
    ("bf16", 128, 8, 32, 16, 128, False, 1, [5, 5, 5], [5, 16, 33], False, 1000000),
    ("fp16", 64, 4, 28, 24, 32, True, 1, [3, 0, 7, 1], [30, 0, 7, 49], True, 77),
    ("fp16", 64, 1, 1, 1, 64, False, 1, [2, 1], [3, 1], False, 0),
    ("bf16", 128, 2, 6, 7, 102, False, 3, [9, 4], [20, 4], False, 0),
    ("bf16", 80, 3, 9, 40, 20, True, 2, [1, 6], [41, 80], True, 0),
    ("fp16", 256, 2, 4, 64, 256, False, 1, [130], [200], False, 2 ** 31 - 500),
    ("bf16", 8, 1, 3, 5, 8, True, 1, [4], [12], False, 0),
    ("bf16", 512, 1, 2, 8, 512, False, 4, [3], [3], False, 0),
    ("bf16", 64, 2, 4, 16, 0, False, 1, [6], [40], False, 0),
    ("fp16", 128, 4, 8, 16, 128, False, 1, [600, 1, 700], [650, 1, 701], False, 9),
]


def _append_and_check(sv, pr, rot, interleaved, axes, base, seed):
    import torch
    rng = np.random.default_rng(seed)
    half = rot // 2
    freq = (10000.0 ** (-np.arange(half) / max(half, 1))).astype(np.float32)
    positions = axis = None
    if axes > 1:
        positions = rng.integers(0, 2 ** 20, (axes, pr.N)).astype(np.int32)
        axis = (np.arange(half) % axes).astype(np.int32)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    before = [p.clone() for p in pr.pools]
    q_out = torch.full((pr.N, pr.Hq, pr.D), -7.0, dtype=pr.q.dtype, device="cuda")
    ws = sv.make_attention_workspace(len(pr.q_lens), pr.N, pr.Hq, pr.D)
    sv.spec_kv_append(sv.make_kv_cache(*pr.pools), pr.q, pr.k, pr.v, q_out, pr.indptr, pr.table, pr.kv_len, ws,
                      inv_freq=dev(freq) if rot else None, positions=dev(positions), axis=dev(axis),
                      interleaved=interleaved, position_base=base)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    q, k, v = _f64(pr.q), _f64(pr.k), _f64(pr.v)
    want = paged.kv_append(_f64(before[0]), _f64(before[1]), q, k, v, pr.indptr_np, pr.table_np, pr.kv_lens, freq,
                           positions, axis, interleaved, base)
    u = torch.finfo(pr.q.dtype).eps / 2
    # |x| + |y| of each rotated pair
    def other(x):
        y = np.zeros_like(x)
        for f in range(half):
            a, b = (2 * f, 2 * f + 1) if interleaved else (f, f + half)
            y[..., a] = y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
        return y
    rows = pr.rows()
    delta = other(q) * (5e-7 + 3 * 2.0 ** -24)
    tol = u * (np.abs(want[0]) + delta) + delta + 2.0 ** -25
    assert (np.abs(_f64(q_out) - want[0])[:rows] <= tol[:rows]).all()
    assert (q_out[rows:] == -7.0).all()
    if rot < pr.D:
        assert torch.equal(q_out[:rows, :, rot:], pr.q[:rows, :, rot:])
    got_k = _f64(pr.pools[0])
    new = np.zeros_like(pr.live)
    for b, (ql, kl) in enumerate(zip(pr.q_lens, pr.kv_lens)):
        for i in range(ql):
            t = kl - ql + i
            page, slot = pr.table_np[b, t // pr.page], t % pr.page
            new[page, slot] = True
            n = pr.indptr_np[b] + i
            d = other(k[n]) * (5e-7 + 3 * 2.0 ** -24)
            ref = want[1][page, slot]
            assert (np.abs(got_k[page, slot] - ref) <= u * (np.abs(ref) + d) + d + 2.0 ** -25).all()
            assert torch.equal(pr.pools[1][page, slot], pr.v[n])
    old = torch.from_numpy(~new).cuda()  # everything else keeps its bits, NaN too
    for p, was in zip(pr.pools, before):
        assert torch.equal(p[old].view(torch.int16), was[old].view(torch.int16))


@pytest.mark.parametrize("dtype,D,Hk,Hq,page,rot,interleaved,axes,q_lens,kv_lens,heads_first,base", APPEND)
def test_append(sv, dtype, D, Hk, Hq, page, rot, interleaved, axes, q_lens, kv_lens, heads_first, base):
    pr = Problem(11, dtype, D, Hk, Hq, page, q_lens, kv_lens, heads_first=heads_first, pad_rows=2)
    _append_and_check(sv, pr, rot, interleaved, axes, base, 12)


def test_append_many_sequences(sv):
    """More sequences than one step of the search for a position's sequence
    covers, some of them empty."""
    rng = np.random.default_rng(5)
    q_lens = rng.integers(0, 3, 1500).tolist()
    kv_lens = [n + int(rng.integers(0, 20)) for n in q_lens]
    pr = Problem(3, "bf16", 64, 1, 2, 8, q_lens, kv_lens)
    _append_and_check(sv, pr, 64, False, 1, 0, 4)


def test_append_keeps_infinite_dims_that_are_not_rotated(sv):
    import torch
    pr = Problem(4, "bf16", 64, 1, 2, 16, [2], [2])
    pr.q[..., 40:] = float("inf")
    _append_inf = torch.empty((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    ws = sv.make_attention_workspace(1, 2, 2, 64)
    freq = torch.ones(18, device="cuda")  # 36 of 64 dims: the border is inside a vector
    sv.spec_kv_append(sv.make_kv_cache(*pr.pools), pr.q, pr.k, pr.v, _append_inf, pr.indptr, pr.table, pr.kv_len, ws,
                      inv_freq=freq)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert torch.isfinite(_append_inf[..., :40]).all() and torch.isinf(_append_inf[..., 40:]).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
ATTEND = [
    # dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, mask, heads_first
    ("bf16", 128, 1, 1, 16, [1], [1], 0, False, False),
    ("bf16", 128, 8, 32, 16, [1], [37], 512, False, False),
    ("bf16", 64, 2, 2, 8, [1, 1, 1], [1, 127, 128], 0, False, True),
    ("fp16", 64, 2, 8, 24, [5, 1, 3], [129, 300, 3], 1, False, False),
    ("fp16", 128, 4, 28, 40, [5, 0, 5], [5, 0, 261], 127, False, True),
    ("bf16", 128, 2, 8, 64, [5] * 7, [5, 64, 65, 200, 128, 256, 257], 129, False, False),
    ("bf16", 64, 1, 71, 16, [1, 2, 3], [9, 40, 200], 300, False, False),      # one key head, 71 query heads
    ("fp16", 64, 1, 128, 16, [3], [20], 40, False, False),
    ("bf16", 128, 2, 2, 128, [300], [300], 0, False, False),                  # several row blocks, causal
    ("bf16", 128, 1, 3, 256, [200, 90], [700, 90], 260, False, True),
    ("fp16", 64, 2, 10, 136, [64, 1], [100, 400], 1000, False, False),
    ("bf16", 128, 2, 4, 16, [12, 9, 6], [12, 50, 133], 0, True, False),       # rows that see nothing
    ("fp16", 64, 4, 28, 24, [12] * 5, [12, 13, 140, 24, 129], 131, True, True),
    ("bf16", 64, 1, 4, 8, [64], [64], 0, True, False),
    ("bf16", 64, 1, 2, 8, [70, 65], [200, 65], 3, True, False),               # new entries past the 64th
    ("bf16", 128, 1, 1, 16, [1] * 40, [130] * 40, 2000, False, False),
]


def _random_mask(rng, q_lens, N):
    words = np.zeros(N, dtype=np.uint64)
    n = 0
    for ql in q_lens:
        for i in range(ql):
            if rng.random() > 0.2:  # the others see nothing new
                words[n] = rng.integers(0, 2 ** 63, dtype=np.uint64) | (np.uint64(1) << np.uint64(min(i, 63)))
            n += 1
    return words


def _attend(sv, pr, words=None, ws=None, out=None, lse=None, stream=None):
    import torch
    if ws is None:
        ws = sv.make_attention_workspace(len(pr.q_lens), pr.N, pr.Hq, pr.D)
    if out is None:
        out = torch.full((pr.N, pr.Hq, pr.D), -7.0, dtype=pr.q.dtype, device="cuda")
    if lse is None:
        lse = torch.full((pr.N, pr.Hq), -7.0, device="cuda")
    mask = None if words is None else torch.from_numpy(words.view(np.int64)).cuda()
    sv.spec_prefix_attention(sv.make_kv_cache(*pr.pools), pr.q, out, pr.indptr, pr.table, pr.kv_len, ws,
                             prefix_table=pr.ptable if pr.prefix else None, prefix_len=pr.prefix, draft_mask=mask,
                             lse=lse, stream=stream)
    return out, lse, ws


def _check_attend(pr, out, lse, words=None):
    import torch
    want, wl, absv, absqk, keys = paged.prefix_attention(
        np.nan_to_num(_f64(pr.pools[0])), np.nan_to_num(_f64(pr.pools[1])), _f64(pr.q), pr.indptr_np, pr.table_np,
        pr.kv_lens, pr.ptable_np, pr.prefix, words)
    u = torch.finfo(pr.q.dtype).eps / 2
    rows = pr.rows()
    got, gl = _f64(out), _f64(lse)
    n = keys[:, None]
    es = pr.D * 2.0 ** -23 * absqk
    vmax = max(1.0, float(np.nan_to_num(_f64(pr.pools[1])).__abs__().max()))
    rel = 2 * es + 2.0 ** -20 + n * 2.0 ** -23
    tol = (u + rel[..., None]) * absv + u * np.abs(want) + n[..., None] * 2.0 ** -25 * vmax + 2.0 ** -25
    bad = ~(np.abs(got - want)[:rows] <= tol[:rows])
    assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - want)[:rows][bad][:5], tol[:rows][bad][:5])
    empty = np.isneginf(wl[:rows])
    assert (np.isneginf(gl[:rows]) == empty).all() and (got[:rows][empty] == 0).all()
    ltol = (es + n * 2.0 ** -23 + 2.0 ** -20 + np.abs(np.where(np.isneginf(wl), 0, wl)) * 2.0 ** -22)[:rows]
    diff = np.abs(np.where(empty, 0, gl[:rows]) - np.where(empty, 0, wl[:rows]))
    assert (diff <= ltol).all(), (diff - ltol).max()
    assert (out[rows:] == -7.0).all() and (lse[rows:] == -7.0).all()


@pytest.mark.parametrize("dtype,D,Hk,Hq,page,q_lens,kv_lens,prefix,mask,heads_first", ATTEND)
def test_attention(sv, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, mask, heads_first):
    pr = Problem(21, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, heads_first, pad_rows=3)
    words = _random_mask(np.random.default_rng(22), q_lens, pr.N) if mask else None
    out, lse, ws = _attend(sv, pr, words)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_attend(pr, out, lse, words)


def test_attention_peaked_scores(sv):
    """Queries along single keys: the running maximum rises by hundreds within
    a row, early, late and at a tile's border."""
    pr = Problem(31, "bf16", 128, 1, 4, 16, [4], [520], 400)
    import torch
    for i, (pool_table, t) in enumerate(((pr.ptable_np, 3), (pr.ptable_np, 399), (pr.table_np[0], 128),
                                         (pr.table_np[0], 510))):
        pr.q[i] = 20 * pr.pools[0][int(pool_table[t // 16]), t % 16, 0][None].expand(4, -1)
    pr.q = pr.q.to(torch.bfloat16)
    out, lse, ws = _attend(sv, pr)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    _check_attend(pr, out, lse)


def test_attention_strided_rows_other_stream_and_repeats(sv):
    """Output rows inside a wider tensor, a stream of the caller's own, the same
    bits on every repeat with one workspace."""
    import torch
    pr = Problem(41, "bf16", 64, 2, 8, 16, [5, 3, 7], [100, 3, 333], 700)
    wide = torch.full((pr.N, pr.Hq + 2, 2 * pr.D), -7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 1:-1, :pr.D]
    lse = torch.empty((pr.N, pr.Hq), device="cuda")
    ws = sv.make_attention_workspace(3, pr.N, pr.Hq, pr.D)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    first = None
    for _ in range(4):
        out.fill_(0)
        torch.cuda.synchronize()
        _attend(sv, pr, ws=ws, out=out, lse=lse, stream=s)
        assert sv.spec_verify_status(ws, s) == sv.SPEC_OK
        now = (out.clone(), lse.clone())
        first = first or now
        assert torch.equal(now[0], first[0]) and torch.equal(now[1], first[1])
    _check_attend(pr, out, lse)
    assert (wide[:, 0] == -7.0).all() and (wide[:, -1] == -7.0).all() and (wide[..., pr.D:] == -7.0).all()


def test_append_then_attend_in_a_graph(sv):
    """Both calls captured once and replayed for rounds whose lengths differ."""
    import torch
    pr = Problem(51, "bf16", 128, 2, 8, 16, [4, 4, 4], [60, 60, 60], 40)
    q_out = torch.empty((pr.N, pr.Hq, pr.D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty_like(q_out), torch.empty((pr.N, pr.Hq), device="cuda")
    ws = sv.make_attention_workspace(3, pr.N, pr.Hq, pr.D)
    cache = sv.make_kv_cache(*pr.pools)
    freq = torch.from_numpy((10000.0 ** (-np.arange(64) / 64)).astype(np.float32)).cuda()

    def both():
        sv.spec_kv_append(cache, pr.q, pr.k, pr.v, q_out, pr.indptr, pr.table, pr.kv_len, ws, inv_freq=freq,
                          position_base=pr.prefix)
        sv.spec_prefix_attention(cache, q_out, out, pr.indptr, pr.table, pr.kv_len, ws, prefix_table=pr.ptable,
                                 prefix_len=pr.prefix, lse=lse)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        both()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            both()
    torch.cuda.synchronize()
    projected = pr.q
    for kv in ([4, 20, 60], [8, 33, 59]):
        pr.kv_lens = kv
        pr.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert sv.spec_verify_status(ws) == sv.SPEC_OK
        pr.q = q_out
        _check_attend(pr, out, lse)
        pr.q = projected


def test_pages_and_lengths_out_of_range_are_reported(sv):
    """A page that is none and a length past the table: reported, skipped, and
    the other sequences' results stand."""
    import torch
    pr = Problem(61, "bf16", 64, 1, 4, 16, [2, 2], [40, 33], 0)
    good, lse, ws = _attend(sv, pr)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    keep = pr.table.clone()
    for bad in (-1, 2 ** 30, pr.pools[0].shape[0]):
        pr.table.copy_(keep)
        pr.table[1, 1] = bad
        out, _, _ = _attend(sv, pr, ws=ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        assert torch.equal(out[:2], good[:2])
        pr.table[1, 2] = bad  # the page that the append would write to
        before = [p.clone() for p in pr.pools]
        q_out = torch.empty((4, 4, 64), dtype=torch.bfloat16, device="cuda")
        sv.spec_kv_append(sv.make_kv_cache(*pr.pools), pr.q, pr.k, pr.v, q_out, pr.indptr, pr.table, pr.kv_len, ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        touched = int(pr.table_np[0, 2])
        others = torch.arange(pr.pools[0].shape[0], device="cuda") != touched
        for p, was in zip(pr.pools, before):
            rest = others.clone()
            rest[int(pr.table_np[1, 1])] = False  # entry 31 of sequence 1 may go to the page that was there
            assert torch.equal(p[rest].view(torch.int16), was[rest].view(torch.int16))
            p.copy_(was)
    pr.table.copy_(keep)
    for bad_len in (1, -5, 10 ** 6):  # fewer than the new positions, negative, past the table
        pr.kv_len[1] = bad_len
        pr.table[1, 2:] = pr.table[1, 1]  # so that a clamped length reads pages that are there
        out, _, _ = _attend(sv, pr, ws=ws)
        assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
        assert torch.equal(out[:2], good[:2])


LARGE = [
    # dtype, D, Hk, Hq, page, B, q_len, prefix, most own entries, mask: many tiles
    # and parts on every CTA, so that rings, queues and slots go round
    ("bf16", 128, 8, 32, 64, 24, 8, 8192, 700, False),
    ("bf16", 128, 4, 8, 16, 96, 5, 1500, 2500, False),
    ("fp16", 64, 16, 16, 32, 64, 1, 4000, 300, False),
    ("fp16", 64, 4, 28, 24, 40, 12, 3001, 900, True),
    ("bf16", 128, 8, 16, 16, 3, 700, 2050, 1400, False),
]


@pytest.mark.parametrize("dtype,D,Hk,Hq,page,B,q_len,prefix,most,mask", LARGE)
def test_attention_large(sv, dtype, D, Hk, Hq, page, B, q_len, prefix, most, mask):
    """Against float64 on the GPU, head by head; the tolerance is
    _check_attend's with the row's largest sums in place of each row's own."""
    import torch
    rng = np.random.default_rng(71)
    q_lens = rng.integers(1, q_len + 1, B).tolist()
    kv_lens = [int(rng.integers(n, most + 1)) for n in q_lens]
    pr = Problem(72, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix)
    words = _random_mask(rng, q_lens, pr.N) if mask else None
    ws = sv.make_attention_workspace(B, pr.N, Hq, D)
    for _ in range(3):
        out, lse, _ = _attend(sv, pr, words, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    u = torch.finfo(pr.q.dtype).eps / 2
    flat = [p.reshape(-1, Hk, D) if p.is_contiguous() else p.contiguous().reshape(-1, Hk, D) for p in pr.pools]
    shared = [int(pr.ptable_np[t // page]) * page + t % page for t in range(prefix)]
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        rows = torch.tensor(shared + [int(pr.table_np[b, t // page]) * page + t % page for t in range(kv)], device="cuda")
        K, V = (x[rows].double().permute(1, 0, 2) for x in flat)                      # [Hk, keys, D]
        a = int(pr.indptr_np[b])
        q = pr.q[a:a + n].double().reshape(n, Hk, Hq // Hk, D).permute(1, 2, 0, 3)     # [Hk, group, n, D]
        new = torch.tensor([[paged.sees(i, j, None if words is None else words[a + i]) for j in range(n)]
                            for i in range(n)], device="cuda")
        s = torch.einsum("hgnd,hkd->hgnk", q, K) * D ** -0.5
        s[..., prefix + kv - n:] = s[..., prefix + kv - n:].masked_fill(~new, -float("inf"))
        want_lse = torch.logsumexp(s, dim=-1)
        w = torch.exp(s - want_lse[..., None])
        want = torch.einsum("hgnk,hkd->hgnd", w, V)
        absv = torch.einsum("hgnk,hkd->hgnd", w, V.abs())
        es = D * 2.0 ** -23 * float((torch.einsum("hgnd,hkd->hgnk", q.abs(), K.abs()) * D ** -0.5).max())
        keys = prefix + kv
        tol = (u + 2 * es + 2.0 ** -20 + keys * 2.0 ** -23) * absv + u * want.abs() \
            + keys * 2.0 ** -25 * float(V.abs().max()) + 2.0 ** -25
        got = out[a:a + n].double().reshape(n, Hk, Hq // Hk, D).permute(1, 2, 0, 3)
        assert bool(((got - want).abs() <= tol).all()), (b, float(((got - want).abs() - tol).max()))
        got_lse = lse[a:a + n].double().reshape(n, Hk, Hq // Hk).permute(1, 2, 0)
        ltol = es + keys * 2.0 ** -23 + 2.0 ** -20 + want_lse.abs() * 2.0 ** -22
        assert bool(((got_lse - want_lse).abs() <= ltol).all()), b


# dtype, D, Hk, Hq, page, q_len, kv_len, prefix: parts of one key tile, with one row tile or two, one after the other
SHORT_PARTS = [
    ("bf16", 128, 8, 16, 16, 128, 128, 0),
    ("bf16", 128, 8, 16, 16, 100, 128, 0),
    ("fp16", 64, 8, 16, 32, 128, 128, 0),
    ("bf16", 128, 4, 8, 64, 200, 250, 300),
]


@pytest.mark.parametrize("dtype,D,Hk,Hq,page,q_len,kv_len,prefix", SHORT_PARTS)
def test_attention_parts_of_one_tile_in_a_row(sv, dtype, D, Hk, Hq, page, q_len, kv_len, prefix):
    """Many passes without a pause: no wait of the kernel may run out, and every
    pass gives the same bits."""
    import torch
    B = 64
    pr = Problem(81, dtype, D, Hk, Hq, page, [q_len] * B, [kv_len] * B, prefix)
    ws = sv.make_attention_workspace(B, pr.N, Hq, D)
    out, lse, _ = _attend(sv, pr, ws=ws)
    first, first_lse = out.clone(), lse.clone()
    other = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        _attend(sv, pr, ws=ws, out=out, lse=lse)
        other += (out != first).sum() + (lse != first_lse).sum()
    torch.cuda.synchronize()
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    assert int(other) == 0
