"""Tensors of several GPUs in the paged calls: refused on the host.  The tensors
only claim a device and the library is a stand-in that counts its calls, so
nothing is launched (no GPU needed)."""
import pytest

import speculative_decoding_verification_54_gb300 as sv
from speculative_decoding_verification_54_gb300 import binding

torch = pytest.importorskip("torch")

I32, BF16 = torch.int32, torch.bfloat16


class Claims(torch.Tensor):
    """A host tensor that says it is on cuda:`place`."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    place = 0

    def get_device(self):
        return self.place

    @property
    def device(self):
        return torch.device("cuda", self.place)

    @property
    def is_cuda(self):
        return True


def on(place, t):
    t = t.as_subclass(Claims)
    t.place = place
    return t


class Library:
    def __init__(self):
        self.calls = []

    def spec_verify_error_string(self, code):
        return b"code"

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(binding, "_lib", lib)
    monkeypatch.setattr(binding, "_current_device", lambda: 1, raising=False)
    return lib


def _append_args(place):
    q, kv = torch.zeros(3, 4, 64, dtype=BF16), torch.zeros(3, 2, 64, dtype=BF16)
    args = dict(q=q, k=kv, v=kv.clone(), q_out=q.clone(), q_indptr=torch.zeros(2, dtype=I32),
                block_table=torch.zeros(1, 4, dtype=I32), kv_len=torch.zeros(1, dtype=I32),
                workspace=torch.zeros(256, dtype=torch.uint8), inv_freq=torch.zeros(32),
                positions=torch.zeros(2, 3, dtype=I32), axis=torch.zeros(32, dtype=I32))
    return {k: on(place, t) for k, t in args.items()}


def _attend_args(place):
    q = torch.zeros(3, 4, 64, dtype=BF16)
    args = dict(q=q, out=q.clone(), q_indptr=torch.zeros(2, dtype=I32), block_table=torch.zeros(1, 4, dtype=I32),
                kv_len=torch.zeros(1, dtype=I32), workspace=torch.zeros(256, dtype=torch.uint8),
                prefix_table=torch.zeros(2, dtype=I32), draft_mask=torch.zeros(3, dtype=torch.int64),
                lse=torch.zeros(3, 4))
    return {**{k: on(place, t) for k, t in args.items()}, "prefix_len": 32}


def _cache(place, other=None):
    pool = torch.zeros(8, 16, 2, 64, dtype=BF16)
    return sv.make_kv_cache(on(place, pool), on(place if other is None else other, pool.clone()))


CALLS = [(sv.spec_kv_append, _append_args), (sv.spec_prefix_attention, _attend_args)]


@pytest.mark.parametrize("call,args", CALLS)
def test_one_device_is_called(library, call, args):
    call(_cache(1), **args(1), stream=5)
    assert library.calls == [call.__name__]


@pytest.mark.parametrize("call,name", [(c, k) for c, a in CALLS for k, t in a(0).items() if isinstance(t, torch.Tensor)])
def test_a_tensor_on_another_device_is_refused(library, call, name):
    args = dict(CALLS)[call]
    for place in (0, -1):
        bad = args(1)
        bad[name] = on(place, bad[name]) if place >= 0 else bad[name].as_subclass(torch.Tensor)
        with pytest.raises(sv.SpecVerifyError, match=name) as e:
            call(_cache(1), **bad, stream=5)
        assert e.value.code == sv.SPEC_ERR_INVALID_ARG
    assert library.calls == []


@pytest.mark.parametrize("call,args", CALLS)
def test_a_cache_that_is_not_on_the_current_device_is_refused(library, call, args):
    with pytest.raises(sv.SpecVerifyError, match="current device") as e:
        call(_cache(0), **args(0), stream=5)
    assert e.value.code == sv.SPEC_ERR_INVALID_ARG and library.calls == []


def test_pools_on_two_devices_are_refused():
    with pytest.raises(sv.SpecVerifyError, match="pools") as e:
        _cache(0, 1)
    assert e.value.code == sv.SPEC_ERR_INVALID_ARG
