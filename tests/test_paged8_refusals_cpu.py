"""Refusals of the append with norms and of the 8-bit cache's calls, on the host: by the
C ABI for fake device addresses, and by the binding for tensors that do not fit (no
GPU needed)."""
import ctypes
import math

import pytest

import speculative_decoding_verification_54_gb300 as sv
from speculative_decoding_verification_54_gb300 import _build
from tests import test_paged_cpu as t16
from tests.test_paged_devices_cpu import library, on  # noqa: F401

torch = pytest.importorskip("torch")

A16, A8, WS = t16.A16, t16.A8, t16.WS
I32, BF16, U8 = torch.int32, torch.bfloat16, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return sv.load()


# ---------------------------------------------------------------------------
# C ABI
# ---------------------------------------------------------------------------
def _cache8(**kw):
    args = dict(k_pages=A16, v_pages=A16, k_scales=A8, v_scales=A8, page_stride=16 * 8 * 128, slot_stride=8 * 128,
                head_stride=128, scale_page_stride=8, scale_block_stride=8, scale_head_stride=1, n_pages=64, page_size=16,
                n_heads=8, head_dim=128, block=16, dtype=sv.SPEC_BF16)
    args.update({k: v for k, v in kw.items() if k in args})
    return sv.SpecKvCache8(*[args[f] for f, _ in sv.SpecKvCache8._fields_])


def _address(cache):
    return None if cache is None else ctypes.addressof(cache)


def _append(call, made, **kw):
    a = dict(cache=made, q=A16, qs=4096, qh=128, k=A16, ks=1024, kh=128, v=A16, vs=1024, vh=128, Hq=32, N=20, ip=A16, B=4,
             bt=A16, tw=8, kl=A16, freq=A16, pos=None, axes=1, axis=None, rot=128, inter=0, base=0, qw=A16, kw=A16, eps=1e-6,
             out=0x30000, ws=WS, wsb=1 << 32)
    a.update(kw)
    return call(_address(a["cache"]), a["q"], a["qs"], a["qh"], a["k"], a["ks"], a["kh"], a["v"], a["vs"], a["vh"], a["Hq"],
                a["N"], a["ip"], a["B"], a["bt"], a["tw"], a["kl"], a["freq"], a["pos"], a["axes"], a["axis"], a["rot"],
                a["inter"], a["base"], a["qw"], a["kw"], a["eps"], a["out"], a["ws"], a["wsb"], None)


APPEND = [
    (dict(k=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(v=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(out=A16), sv.SPEC_ERR_INVALID_ARG),
    (dict(rot=127), sv.SPEC_ERR_INVALID_ARG),
    (dict(rot=130), sv.SPEC_ERR_INVALID_ARG),
    (dict(freq=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(inter=2), sv.SPEC_ERR_INVALID_ARG),
    (dict(axes=3), sv.SPEC_ERR_INVALID_ARG),
    (dict(axes=3, pos=A16), sv.SPEC_ERR_INVALID_ARG),
    (dict(base=-1), sv.SPEC_ERR_INVALID_ARG),
    (dict(eps=-1e-6), sv.SPEC_ERR_INVALID_ARG),
    (dict(eps=math.nan), sv.SPEC_ERR_INVALID_ARG),
    (dict(eps=math.inf), sv.SPEC_ERR_INVALID_ARG),
    (dict(k=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(vs=1026), sv.SPEC_ERR_ALIGNMENT),
    (dict(wsb=255), sv.SPEC_ERR_WORKSPACE),
]

# what the 8-bit cache's calls refuse of it and of the batch
CACHE8 = [
    (dict(cache=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(k_pages=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(v_pages=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(k_scales=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(v_scales=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(ip=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(bt=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(B=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(N=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(N=(1 << 24) + 1), sv.SPEC_ERR_INVALID_ARG),
    (dict(tw=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_heads=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_pages=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_pages=1 << 31), sv.SPEC_ERR_INVALID_ARG),
    (dict(page_size=24), sv.SPEC_ERR_INVALID_ARG),            # no whole blocks
    (dict(page_stride=-16), sv.SPEC_ERR_INVALID_ARG),
    (dict(scale_block_stride=-1), sv.SPEC_ERR_INVALID_ARG),
    (dict(block=4, page_size=16), sv.SPEC_ERR_UNSUPPORTED),
    (dict(block=128, page_size=128), sv.SPEC_ERR_UNSUPPORTED),
    (dict(head_dim=136), sv.SPEC_ERR_UNSUPPORTED),
    (dict(head_dim=512), sv.SPEC_ERR_UNSUPPORTED),
    (dict(dtype=sv.SPEC_F32), sv.SPEC_ERR_UNSUPPORTED),
    (dict(k_pages=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(slot_stride=1032), sv.SPEC_ERR_ALIGNMENT),          # 8 bytes are enough for 16 bits, not here
    (dict(head_stride=136), sv.SPEC_ERR_ALIGNMENT),
    (dict(ws=None), sv.SPEC_ERR_WORKSPACE),
    (dict(ws=WS + 16), sv.SPEC_ERR_WORKSPACE),
]


@pytest.mark.parametrize("kw,code", APPEND)
def test_append_norm(lib, kw, code):
    assert _append(lib.spec_kv_append_norm, t16._cache(), **kw) == code


def test_append_norm_refuses_what_the_append_does(lib):
    for kw, code in t16.COMMON:
        assert _append(lib.spec_kv_append_norm, t16._cache(**kw), **kw) == code, kw


@pytest.mark.parametrize("kw,code", APPEND + CACHE8 + [(dict(kl=None), sv.SPEC_ERR_INVALID_ARG), (dict(q=None), sv.SPEC_ERR_INVALID_ARG)])
def test_append8(lib, kw, code):
    assert _append(lib.spec_kv_append8, _cache8(**kw), **kw) == code


@pytest.mark.parametrize("kw,code", CACHE8 + [
    (dict(ko=None, vo=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(ko=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(vo=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(ks=1028), sv.SPEC_ERR_ALIGNMENT),
    (dict(vh=4), sv.SPEC_ERR_ALIGNMENT),
    (dict(wsb=255), sv.SPEC_ERR_WORKSPACE),
])
def test_read8(lib, kw, code):
    a = dict(cache=_cache8(**kw), ip=A16, N=20, B=4, bt=A16, tw=8, first=None, ko=A16, ks=1024, kh=128, vo=A16, vs=1024, vh=128,
             ws=WS, wsb=1 << 32)
    a.update(kw)
    got = lib.spec_kv_read8(_address(a["cache"]), a["ip"], a["N"], a["B"], a["bt"], a["tw"], a["first"], a["ko"], a["ks"],
                            a["kh"], a["vo"], a["vs"], a["vh"], a["ws"], a["wsb"], None)
    assert got == code


@pytest.mark.parametrize("kw,code", CACHE8 + [
    (dict(kl=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(q=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(out=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(pl=-1), sv.SPEC_ERR_INVALID_ARG),
    (dict(pt=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(scale=0.0), sv.SPEC_ERR_INVALID_ARG),
    (dict(scale=math.nan), sv.SPEC_ERR_INVALID_ARG),
    (dict(scale=math.inf), sv.SPEC_ERR_INVALID_ARG),
    (dict(n_heads=5), sv.SPEC_ERR_INVALID_ARG),
    (dict(head_dim=96), sv.SPEC_ERR_UNSUPPORTED),
    (dict(head_dim=256), sv.SPEC_ERR_UNSUPPORTED),
    (dict(Hq=129, n_heads=1), sv.SPEC_ERR_UNSUPPORTED),
    (dict(q=A8), sv.SPEC_ERR_ALIGNMENT),
    (dict(os=4100), sv.SPEC_ERR_ALIGNMENT),
    (dict(wsb=4096), sv.SPEC_ERR_WORKSPACE),
])
def test_attention8(lib, kw, code):
    a = dict(cache=_cache8(**kw), q=A16, qs=4096, qh=128, Hq=32, N=20, ip=A16, B=4, pt=A16, pl=100, bt=A16, tw=8, kl=A16,
             mask=None, scale=0.1, out=A16, os=4096, oh=128, lse=None, ws=WS, wsb=1 << 32)
    a.update(kw)
    got = lib.spec_prefix_attention8(_address(a["cache"]), a["q"], a["qs"], a["qh"], a["Hq"], a["N"], a["ip"], a["B"], a["pt"],
                                     a["pl"], a["bt"], a["tw"], a["kl"], a["mask"], a["scale"], a["out"], a["os"], a["oh"],
                                     a["lse"], a["ws"], a["wsb"], None)
    assert got == code


# ---------------------------------------------------------------------------
# binding
# ---------------------------------------------------------------------------
def _pools(block=8, page=16, dims=64):
    codes, scales = torch.zeros(8, page, 2, dims, dtype=U8), torch.zeros(8, page // block, 2, dtype=U8)
    return [codes, codes.clone(), scales, scales.clone()]


def test_the_cache_says_its_block():
    cache = sv.make_kv_cache8(*_pools())
    assert (cache.block, cache.page_size, cache.dtype) == (8, 16, sv.SPEC_BF16)
    k, v, ks, vs = _pools()
    typed = sv.make_kv_cache8(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks.view(torch.float8_e8m0fnu),
                              vs.view(torch.float8_e8m0fnu), torch.float16)
    assert typed.dtype == sv.SPEC_F16 and typed.k_pages == k.data_ptr() and typed.scale_block_stride == 2


@pytest.mark.parametrize("change,message", [
    (lambda p: p.__setitem__(0, p[0].to(torch.int8)), "dtypes"),
    (lambda p: p.__setitem__(1, p[1].view(torch.float8_e4m3fn)), "dtypes"),
    (lambda p: p.__setitem__(2, p[2].float()), "scale dtypes"),
    (lambda p: p.__setitem__(1, p[1][:, :8]), "cache pools"),
    (lambda p: p.__setitem__(1, p[1].transpose(1, 2).contiguous().transpose(1, 2)), "cache pools"),
    (lambda p: (p.__setitem__(0, p[0][..., ::2]), p.__setitem__(1, p[1][..., ::2])), "cache pools"),
    (lambda p: p.__setitem__(3, p[3][:4]), "scales"),
    (lambda p: (p.__setitem__(2, p[2][:4]), p.__setitem__(3, p[3][:4])), "scales"),
    (lambda p: (p.__setitem__(2, p[2][..., :1]), p.__setitem__(3, p[3][..., :1])), "scales"),
    (lambda p: [p.__setitem__(i, torch.zeros(8, 3, 2, dtype=U8)) for i in (2, 3)], "scales"),
    (lambda p: [p.__setitem__(i, torch.zeros(8, 0, 2, dtype=U8)) for i in (2, 3)], "scales"),
    (lambda p: [p.__setitem__(i, torch.zeros(8, 4, 2, dtype=U8)) for i in (2, 3)], "blocks of 4"),
])
def test_pools_that_do_not_fit_are_refused(change, message):
    pools = _pools()
    change(pools)
    with pytest.raises(sv.SpecVerifyError, match=message):
        sv.make_kv_cache8(*pools)
    with pytest.raises(sv.SpecVerifyError, match="cache of"):
        sv.make_kv_cache8(*_pools(), torch.float32)


def _tensors(place=None):
    q, kv = torch.zeros(3, 4, 64, dtype=BF16), torch.zeros(3, 2, 64, dtype=BF16)
    append = dict(q=q, k=kv, v=kv.clone(), q_out=q.clone(), q_indptr=torch.zeros(2, dtype=I32),
                  block_table=torch.zeros(1, 4, dtype=I32), kv_len=torch.zeros(1, dtype=I32),
                  workspace=torch.zeros(256, dtype=U8), inv_freq=torch.zeros(32), positions=torch.zeros(2, 3, dtype=I32),
                  axis=torch.zeros(32, dtype=I32), q_weight=torch.zeros(64), k_weight=torch.zeros(64))
    read = dict(k_out=kv.clone(), v_out=kv.clone(), out_indptr=torch.zeros(2, dtype=I32),
                block_table=torch.zeros(1, 4, dtype=I32), workspace=torch.zeros(256, dtype=U8), first=torch.zeros(1, dtype=I32))
    attend = dict(q=q.clone(), out=q.clone(), q_indptr=torch.zeros(2, dtype=I32), block_table=torch.zeros(1, 4, dtype=I32),
                  kv_len=torch.zeros(1, dtype=I32), workspace=torch.zeros(256, dtype=U8), prefix_table=torch.zeros(2, dtype=I32),
                  draft_mask=torch.zeros(3, dtype=torch.int64), lse=torch.zeros(3, 4))
    all_ = dict(append=append, read=read, attend=attend)
    if place is not None:
        all_ = {k: {n: on(place, t) for n, t in a.items()} for k, a in all_.items()}
    all_["attend"]["prefix_len"] = 32
    return all_


def _caches(place=None):
    pools = _pools()
    pool16 = [torch.zeros(8, 16, 2, 64, dtype=BF16) for _ in "kv"]
    if place is not None:
        pools, pool16 = [on(place, t) for t in pools], [on(place, t) for t in pool16]
    return sv.make_kv_cache8(*pools), sv.make_kv_cache(*pool16)


CALLS = [("spec_kv_append_norm", "append", 1), ("spec_kv_append8", "append", 0), ("spec_kv_read8", "read", 0),
         ("spec_prefix_attention8", "attend", 0)]


@pytest.mark.parametrize("name,kind,which", CALLS)
def test_a_cache_of_the_other_kind_is_refused(name, kind, which):
    with pytest.raises(sv.SpecVerifyError, match="make_kv_cache"):
        getattr(sv, name)(_caches()[1 - which], **_tensors()[kind])
    for old, args in ((sv.spec_kv_append, "append"), (sv.spec_prefix_attention, "attend")):
        kw = {k: v for k, v in _tensors()[args].items() if "weight" not in k}
        with pytest.raises(sv.SpecVerifyError, match="make_kv_cache"):
            old(_caches()[0], **kw)


@pytest.mark.parametrize("name,which", [("spec_kv_append_norm", 1), ("spec_kv_append8", 0)])
@pytest.mark.parametrize("change,message", [
    (dict(q_weight=torch.zeros(64, dtype=BF16)), "q_weight"),
    (dict(q_weight=torch.zeros(4, 64)), "q_weight"),
    (dict(k_weight=torch.zeros(32)), "k_weight"),
    (dict(k_weight=torch.zeros(128)[::2]), "k_weight"),
    (dict(inv_freq=torch.zeros(2, 16)), "inv_freq"),
    (dict(positions=torch.zeros(2, 2, dtype=I32)), "positions"),
    (dict(axis=torch.zeros(31, dtype=I32)), "axis"),
    (dict(q=torch.zeros(3, 4, 64)), "dtype"),
    (dict(k=torch.zeros(2, 2, 64, dtype=BF16)), "shape"),
    (dict(v=torch.zeros(3, 4, 64, dtype=BF16)), "cache heads"),
    (dict(q_out=torch.zeros(3, 4, 128, dtype=BF16)[..., :64]), "q_out"),
    (dict(q=torch.zeros(3, 4, 128, dtype=BF16)[..., ::2]), "adjacent"),
    (dict(kv_len=torch.zeros(1, dtype=torch.int64)), "int32"),
    (dict(block_table=torch.zeros(1, 8, dtype=I32)[:, ::2]), "contiguous"),
    (dict(), "GPU"),
])
def test_append_tensors(name, which, change, message):
    with pytest.raises(sv.SpecVerifyError, match=message):
        getattr(sv, name)(_caches()[which], **{**_tensors()["append"], **change})


@pytest.mark.parametrize("change,message", [
    (dict(k_out=None, v_out=None), "no output"),
    (dict(k_out=torch.zeros(3, 2, 64)), "dtype"),
    (dict(v_out=torch.zeros(4, 2, 64, dtype=BF16)), "shape"),
    (dict(k_out=torch.zeros(3, 3, 64, dtype=BF16)), "cache heads"),
    (dict(out_indptr=torch.zeros(3, dtype=I32)), "out_indptr"),
    (dict(out_indptr=torch.zeros(2, dtype=torch.int64)), "out_indptr"),
    (dict(out_indptr=torch.zeros(1, dtype=I32)), "out_indptr"),
    (dict(block_table=torch.zeros(4, dtype=I32)), "block_table"),
    (dict(first=torch.zeros(2, dtype=I32)), "first"),
    (dict(first=torch.zeros(1)), "first"),
    (dict(), "GPU"),
])
def test_read_tensors(change, message):
    with pytest.raises(sv.SpecVerifyError, match=message):
        sv.spec_kv_read8(_caches()[0], **{**_tensors()["read"], **change})


@pytest.mark.parametrize("change,message", [
    (dict(prefix_table=None), "prefix_table"),
    (dict(prefix_len=33), "prefix_table"),
    (dict(draft_mask=torch.zeros(2, dtype=torch.int64)), "draft_mask"),
    (dict(lse=torch.zeros(3, 2)), "lse"),
    (dict(out=torch.zeros(3, 2, 64, dtype=BF16)), "out"),
    (dict(q=torch.zeros(3, 4, 64, dtype=torch.float16)), "dtype"),
    (dict(), "GPU"),
])
def test_attention_tensors(change, message):
    with pytest.raises(sv.SpecVerifyError, match=message):
        sv.spec_prefix_attention8(_caches()[0], **{**_tensors()["attend"], **change})


@pytest.mark.parametrize("name,kind,which", CALLS)
def test_tensors_on_another_device_are_refused(library, name, kind, which):  # noqa: F811
    call = getattr(sv, name)
    call(_caches(1)[which], **_tensors(1)[kind], stream=5)
    assert library.calls == [name]
    for key, t in _tensors(1)[kind].items():
        if not isinstance(t, torch.Tensor):
            continue
        with pytest.raises(sv.SpecVerifyError, match=key):
            call(_caches(1)[which], **{**_tensors(1)[kind], key: on(0, t)}, stream=5)
    with pytest.raises(sv.SpecVerifyError, match="current device"):
        call(_caches(0)[which], **_tensors(0)[kind], stream=5)
    assert library.calls == [name]
