"""The paged cache on the CPU: the float64 oracle's pins, planted mistakes that
they must catch, and the calls' refusals (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

import speculative_decoding_verification_54_gb300 as sv
from oracle import paged
from speculative_decoding_verification_54_gb300 import _build

torch = pytest.importorskip("torch")


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------
def _check_rotation():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 12))
    freq = np.array([1.0, 0.25, 0.03, 0.001])
    for inter in (False, True):
        y = paged.rotate(x, [17, 5], freq, axis=[0, 1, 0, 1], interleaved=inter)
        assert np.allclose(y[:, 8:], x[:, 8:])  # dims past rot_dim stay
        assert np.allclose((y ** 2).sum(1), (x ** 2).sum(1))
        a = [0, 2, 4, 6] if inter else [0, 1, 2, 3]
        b = [1, 3, 5, 7] if inter else [4, 5, 6, 7]
        z = (x[:, a] + 1j * x[:, b]) * np.exp(1j * np.array([17, 5, 17, 5]) * freq)
        assert np.allclose(y[:, a], z.real) and np.allclose(y[:, b], z.imag)
    # a product of two rotated heads depends on the distance alone
    q, k = rng.standard_normal((1, 8)), rng.standard_normal((1, 8))
    dots = [(paged.rotate(q, [p + 3], freq) * paged.rotate(k, [p], freq)).sum() for p in (0, 11, 4000)]
    assert np.allclose(dots, dots[0])


def _small(rng, mask):
    k_pages, v_pages = rng.standard_normal((2, 9, 4, 2, 8))
    q = rng.standard_normal((5, 4, 8))
    words = np.array([0b1, 0b101, 0, 0b11, 0b110], dtype=np.uint64) if mask else None
    return k_pages, v_pages, q, np.array([0, 3, 5]), np.array([[3, 1, 7], [0, 8, 2]]), np.array([9, 2]), words


def _check_attention():
    rng = np.random.default_rng(1)
    for mask in (False, True):
        for prefix in (0, 6):
            kp, vp, q, indptr, table, kv, words = _small(rng, mask)
            out, lse, *_ = paged.prefix_attention(kp, vp, q, indptr, table, kv, np.array([5, 6]), prefix, words)
            flat = lambda pool, pages, n: pool[pages].reshape(-1, 2, 8)[:n]  # noqa: E731
            for n in range(5):
                b = 0 if n < 3 else 1
                i, ql = n - indptr[b], indptr[b + 1] - indptr[b]
                K = np.concatenate([flat(kp, [5, 6], prefix), flat(kp, table[b], kv[b])])
                V = np.concatenate([flat(vp, [5, 6], prefix), flat(vp, table[b], kv[b])])
                vis = np.ones(len(K), dtype=bool)
                new = [bool((int(words[n]) >> j) & 1) if mask else j <= i for j in range(ql)]
                vis[len(K) - ql:] = new
                for h in range(4):
                    if not vis.any():
                        assert (out[n, h] == 0).all() and lse[n, h] == -math.inf
                        continue
                    e = np.where(vis, np.exp(K[:, h // 2] @ q[n, h] / math.sqrt(8)), 0.0)
                    assert np.allclose(out[n, h], e @ V[:, h // 2] / e.sum())
                    assert np.isclose(lse[n, h], math.log(e.sum()))


def _check_append():
    rng = np.random.default_rng(2)
    kp, vp, q, indptr, table, kv, _ = _small(rng, False)
    k, v = rng.standard_normal((2, 5, 2, 8))
    freq = np.array([1.0, 0.1])
    qo, ko, vo = paged.kv_append(kp, vp, q, k, v, indptr, table, kv, freq, position_base=100)
    # sequence 0: entries 6, 7, 8 (pages 1, 1, 7); sequence 1: entries 0, 1 (page 0)
    where = [(1, 2, 106), (1, 3, 107), (7, 0, 108), (0, 0, 100), (0, 1, 101)]
    untouched = np.ones(kp.shape[:2], dtype=bool)
    for n, (page, slot, pos) in enumerate(where):
        assert np.allclose(ko[page, slot], paged.rotate(k[n], [pos], freq))
        assert np.allclose(vo[page, slot], v[n])
        assert np.allclose(qo[n], paged.rotate(q[n], [pos], freq))
        untouched[page, slot] = False
    assert (ko[untouched] == kp[untouched]).all() and (vo[untouched] == vp[untouched]).all()


@pytest.mark.parametrize("check", [_check_rotation, _check_attention, _check_append])
def test_oracle_pins(check):
    check()


@pytest.mark.parametrize("name,wrong,check", [
    ("rotate", lambda x, p, f, axis=None, interleaved=False:
        _ROTATE(x, [-a for a in p], f, axis, interleaved), _check_rotation),           # turned the other way
    ("rotate", lambda x, p, f, axis=None, interleaved=False:
        _ROTATE(x, p, f, None, interleaved), _check_rotation),                         # one axis for all
    ("sees", lambda i, j, w=None: j < i if w is None else _SEES(i, j, w), _check_attention),   # not itself
    ("sees", lambda i, j, w=None: _SEES(i, j, None), _check_attention),                # the mask ignored
    ("entry_of", lambda q_len, kv_len, i: kv_len + i, _check_append),                  # kv_len without the new ones
])
def test_planted_mistakes_fail_a_pin(monkeypatch, name, wrong, check):
    monkeypatch.setattr(paged, name, wrong)
    with pytest.raises((AssertionError, IndexError)):
        check()


_ROTATE, _SEES = paged.rotate, paged.sees


# ---------------------------------------------------------------------------
# refusals: fake device addresses, rejected on the host before any CUDA call
# ---------------------------------------------------------------------------
A16, A8, WS = 0x10000, 0x10008, 0x20000


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sv.load()


def _cache(**kw):
    args = dict(k_pages=A16, v_pages=A16, page_stride=16 * 8 * 128, slot_stride=8 * 128, head_stride=128, n_pages=64,
                page_size=16, n_heads=8, head_dim=128, dtype=sv.SPEC_BF16)
    args.update({k: v for k, v in kw.items() if k in args})
    return sv.SpecKvCache(*[args[f] for f, _ in sv.SpecKvCache._fields_])


COMMON = [
    (dict(cache=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(k_pages=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(v_pages=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(q=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(out=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(ip=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(bt=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(kl=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(B=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(B=65536), sv.SPEC_ERR_INVALID_ARG),
    (dict(N=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(N=(1 << 24) + 1), sv.SPEC_ERR_INVALID_ARG),
    (dict(Hq=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_heads=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_heads=33), sv.SPEC_ERR_INVALID_ARG),
    (dict(tw=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(page_size=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_pages=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_pages=1 << 31), sv.SPEC_ERR_INVALID_ARG),
    (dict(head_dim=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(head_dim=100), sv.SPEC_ERR_INVALID_ARG),
    (dict(page_stride=-8), sv.SPEC_ERR_INVALID_ARG),
    (dict(dtype=sv.SPEC_F32), sv.SPEC_ERR_UNSUPPORTED),
    (dict(dtype=7), sv.SPEC_ERR_UNSUPPORTED),
    (dict(q=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(out=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(k_pages=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(qs=4100), sv.SPEC_ERR_ALIGNMENT),
    (dict(qh=132), sv.SPEC_ERR_ALIGNMENT),
    (dict(slot_stride=1028), sv.SPEC_ERR_ALIGNMENT),
    (dict(ws=None), sv.SPEC_ERR_WORKSPACE),
    (dict(ws=WS + 16), sv.SPEC_ERR_WORKSPACE),
    (dict(wsb=128), sv.SPEC_ERR_WORKSPACE),
]


def _append(lib, **kw):
    a = dict(cache=_cache(**kw), q=A16, qs=4096, qh=128, k=A16, ks=1024, kh=128, v=A16, vs=1024, vh=128, Hq=32, N=20,
             ip=A16, B=4, bt=A16, tw=8, kl=A16, freq=A16, pos=None, axes=1, axis=None, rot=128, inter=0, base=0,
             out=0x30000, ws=WS, wsb=1 << 32)
    a.update(kw)
    return lib.spec_kv_append(None if a["cache"] is None else ctypes.addressof(a["cache"]), a["q"], a["qs"], a["qh"],
                              a["k"], a["ks"], a["kh"], a["v"], a["vs"], a["vh"], a["Hq"], a["N"], a["ip"], a["B"],
                              a["bt"], a["tw"], a["kl"], a["freq"], a["pos"], a["axes"], a["axis"], a["rot"],
                              a["inter"], a["base"], a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(k=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(v=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(out=A16), sv.SPEC_ERR_INVALID_ARG),            # in place
    (dict(rot=127), sv.SPEC_ERR_INVALID_ARG),
    (dict(rot=130), sv.SPEC_ERR_INVALID_ARG),
    (dict(rot=-2), sv.SPEC_ERR_INVALID_ARG),
    (dict(freq=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(inter=2), sv.SPEC_ERR_INVALID_ARG),
    (dict(axes=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(axes=17, pos=A16, axis=A16), sv.SPEC_ERR_INVALID_ARG),
    (dict(axes=3), sv.SPEC_ERR_INVALID_ARG),             # several axes, no positions
    (dict(axes=3, pos=A16), sv.SPEC_ERR_INVALID_ARG),    # several axes, none dealt out
    (dict(base=-1), sv.SPEC_ERR_INVALID_ARG),
    (dict(head_dim=520), sv.SPEC_ERR_INVALID_ARG),
    (dict(k=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(vs=1026), sv.SPEC_ERR_ALIGNMENT),
])
def test_append_rejects_bad_arguments_on_host(lib, kw, code):
    assert _append(lib, **kw) == code


def _attend(lib, **kw):
    a = dict(cache=_cache(**kw), q=A16, qs=4096, qh=128, Hq=32, N=20, ip=A16, B=4, pt=A16, pl=100, bt=A16, tw=8, kl=A16,
             mask=None, scale=0.1, out=A16, os=4096, oh=128, lse=None, ws=WS, wsb=1 << 32)
    a.update(kw)
    return lib.spec_prefix_attention(None if a["cache"] is None else ctypes.addressof(a["cache"]), a["q"], a["qs"],
                                     a["qh"], a["Hq"], a["N"], a["ip"], a["B"], a["pt"], a["pl"], a["bt"], a["tw"],
                                     a["kl"], a["mask"], a["scale"], a["out"], a["os"], a["oh"], a["lse"], a["ws"],
                                     a["wsb"], None)


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(pl=-1), sv.SPEC_ERR_INVALID_ARG),
    (dict(pt=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(scale=0.0), sv.SPEC_ERR_INVALID_ARG),
    (dict(scale=-1.0), sv.SPEC_ERR_INVALID_ARG),
    (dict(scale=math.nan), sv.SPEC_ERR_INVALID_ARG),
    (dict(scale=math.inf), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_heads=5), sv.SPEC_ERR_INVALID_ARG),          # 32 heads over 5
    (dict(head_dim=96), sv.SPEC_ERR_UNSUPPORTED),
    (dict(page_size=12), sv.SPEC_ERR_UNSUPPORTED),
    (dict(Hq=129, n_heads=1), sv.SPEC_ERR_UNSUPPORTED),
    (dict(os=4100), sv.SPEC_ERR_ALIGNMENT),
    (dict(oh=4), sv.SPEC_ERR_ALIGNMENT),
])
def test_attention_rejects_bad_arguments_on_host(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_attention_workspace_bytes(lib):
    small = sv.spec_attention_workspace_bytes(1, 1, 8, 64)
    assert small >= 256 and small % 256 == 0
    assert sv.spec_attention_workspace_bytes(64, 320, 32, 128) >= small
    for bad in ((0, 1, 8, 64), (1, 0, 8, 64), (1, 1, 0, 64), (1, 1, 8, 60), (1, 1, 8, 520)):
        with pytest.raises(sv.SpecVerifyError) as e:
            sv.spec_attention_workspace_bytes(*bad)
        assert e.value.code == sv.SPEC_ERR_INVALID_ARG


def test_binding_refuses_wrong_shapes_and_types(lib):
    pool = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    for k, v, code in ((pool.float(), pool.float(), sv.SPEC_ERR_UNSUPPORTED), (pool, pool.half(), sv.SPEC_ERR_UNSUPPORTED),
                       (pool, pool[:4], sv.SPEC_ERR_INVALID_ARG), (pool[0], pool[0], sv.SPEC_ERR_INVALID_ARG),
                       (pool[..., ::2], pool[..., ::2], sv.SPEC_ERR_INVALID_ARG)):
        with pytest.raises(sv.SpecVerifyError) as e:
            sv.make_kv_cache(k, v)
        assert e.value.code == code
    cache = sv.make_kv_cache(pool, pool.clone())
    assert (cache.page_size, cache.n_heads, cache.head_dim, cache.slot_stride) == (16, 2, 64, 128)
    i32 = dict(dtype=torch.int32)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    good = dict(q=q, k=kv, v=kv, q_out=q.clone(), q_indptr=torch.zeros(2, **i32), block_table=torch.zeros(1, 4, **i32),
                kv_len=torch.zeros(1, **i32), workspace=torch.zeros(256, dtype=torch.uint8),
                inv_freq=torch.zeros(32), positions=torch.zeros(1, 3, **i32))
    for change, code in ((dict(q=q.float()), sv.SPEC_ERR_UNSUPPORTED), (dict(k=kv[:2]), sv.SPEC_ERR_INVALID_ARG),
                         (dict(k=q), sv.SPEC_ERR_INVALID_ARG), (dict(q_out=q[:, :2]), sv.SPEC_ERR_INVALID_ARG),
                         (dict(q_indptr=torch.zeros(1, **i32)), sv.SPEC_ERR_INVALID_ARG),
                         (dict(kv_len=torch.zeros(1, dtype=torch.int64)), sv.SPEC_ERR_INVALID_ARG),
                         (dict(inv_freq=torch.zeros(32, dtype=torch.float64)), sv.SPEC_ERR_INVALID_ARG),
                         (dict(positions=torch.zeros(3, **i32)), sv.SPEC_ERR_INVALID_ARG),
                         (dict(axis=torch.zeros(31, **i32)), sv.SPEC_ERR_INVALID_ARG),
                         ({}, sv.SPEC_ERR_INVALID_ARG)):  # everything fits, but it is not on the GPU
        with pytest.raises(sv.SpecVerifyError) as e:
            sv.spec_kv_append(cache, **{**good, **change})
        assert e.value.code == code
    good = dict(q=q, out=q.clone(), q_indptr=torch.zeros(2, **i32), block_table=torch.zeros(1, 4, **i32),
                kv_len=torch.zeros(1, **i32), workspace=torch.zeros(256, dtype=torch.uint8))
    for change in (dict(out=q[:2]), dict(prefix_len=17, prefix_table=torch.zeros(1, **i32)), dict(prefix_len=3),
                   dict(draft_mask=torch.zeros(3, **i32)), dict(lse=torch.zeros(3, 4, dtype=torch.float64)),
                   dict(lse=torch.zeros(3, 2)), {}):
        with pytest.raises(sv.SpecVerifyError) as e:
            sv.spec_prefix_attention(cache, **{**good, **change})
        assert e.value.code == sv.SPEC_ERR_INVALID_ARG
