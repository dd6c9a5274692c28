"""Caches of the right kind are taken by the paged calls, a program's own subclasses among
them (host only: the library is a stand-in that counts its calls)."""
import ctypes

import pytest

import speculative_decoding_verification_54_gb300 as sv
from tests.test_paged8_refusals_cpu import _caches, _tensors
from tests.test_paged_devices_cpu import library  # noqa: F401

torch = pytest.importorskip("torch")


class Layer16(sv.SpecKvCache):
    pass


class Layer8(sv.SpecKvCache8):
    pass


def _own(cache, kind):
    mine = kind(*(getattr(cache, f) for f, _ in cache._fields_))
    mine.tensors, mine.expected, mine.address = cache.tensors, cache.expected, ctypes.addressof(mine)
    return mine


CALLS = [("spec_kv_append", "append", 16), ("spec_kv_append_norm", "append", 16), ("spec_prefix_attention", "attend", 16),
         ("spec_kv_append8", "append", 8), ("spec_kv_read8", "read", 8), ("spec_prefix_attention8", "attend", 8)]


@pytest.mark.parametrize("name,kind,bits", CALLS)
def test_a_subclass_of_the_cache_is_taken(library, name, kind, bits):  # noqa: F811
    codes, halves = _caches(1)
    tensors = {k: t for k, t in _tensors(1)[kind].items() if name != "spec_kv_append" or "weight" not in k}
    getattr(sv, name)(_own(halves, Layer16) if bits == 16 else _own(codes, Layer8), **tensors, stream=5)
    assert library.calls == [name]
    with pytest.raises(sv.SpecVerifyError, match="make_kv_cache"):
        getattr(sv, name)(_own(codes, Layer8) if bits == 16 else _own(halves, Layer16), **tensors, stream=5)
    assert library.calls == [name]
