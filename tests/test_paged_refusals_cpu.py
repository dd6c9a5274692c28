"""Refusals of the paged calls' binding, each by its own message: the checks that
keep the kernels inside prefix_table, positions, axis, draft_mask and lse (no
GPU needed)."""
import pytest

import speculative_decoding_verification_54_gb300 as sv
from speculative_decoding_verification_54_gb300 import _build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    sv.load()


I32, BF16 = torch.int32, torch.bfloat16


def _cache():
    pool = torch.zeros(8, 16, 2, 64, dtype=BF16)
    return sv.make_kv_cache(pool, pool.clone())


def _append_args():
    q = torch.zeros(3, 4, 64, dtype=BF16)
    kv = torch.zeros(3, 2, 64, dtype=BF16)
    return dict(q=q, k=kv, v=kv.clone(), q_out=q.clone(), q_indptr=torch.zeros(2, dtype=I32),
                block_table=torch.zeros(1, 4, dtype=I32), kv_len=torch.zeros(1, dtype=I32),
                workspace=torch.zeros(256, dtype=torch.uint8), inv_freq=torch.zeros(32),
                positions=torch.zeros(2, 3, dtype=I32), axis=torch.zeros(32, dtype=I32))


def _attend_args():
    q = torch.zeros(3, 4, 64, dtype=BF16)
    return dict(q=q, out=q.clone(), q_indptr=torch.zeros(2, dtype=I32), block_table=torch.zeros(1, 4, dtype=I32),
                kv_len=torch.zeros(1, dtype=I32), workspace=torch.zeros(256, dtype=torch.uint8),
                prefix_table=torch.zeros(2, dtype=I32), prefix_len=32, draft_mask=torch.zeros(3, dtype=torch.int64),
                lse=torch.zeros(3, 4))


def _refused(call, args, change, message):
    with pytest.raises(sv.SpecVerifyError, match=message):
        call(_cache(), **{**args, **change})


@pytest.mark.parametrize("change,message", [
    (dict(inv_freq=torch.zeros(32, dtype=torch.float64)), "inv_freq"),
    (dict(inv_freq=torch.zeros(2, 16)), "inv_freq"),
    (dict(inv_freq=torch.zeros(64)[::2]), "inv_freq"),
    (dict(positions=torch.zeros(3, dtype=I32)), "positions"),
    (dict(positions=torch.zeros(2, 2, dtype=I32)), "positions"),
    (dict(positions=torch.zeros(2, 3, dtype=torch.int64)), "positions"),
    (dict(positions=torch.zeros(3, 2, dtype=I32).T), "positions"),
    (dict(axis=torch.zeros(31, dtype=I32)), "axis"),
    (dict(axis=torch.zeros(32, dtype=torch.int64)), "axis"),
    (dict(axis=torch.zeros(64, dtype=I32)[::2]), "axis"),
    (dict(inv_freq=None), "axis"),                       # an axis for frequencies that are not there
    (dict(q=torch.zeros(3, 4, 64)), "dtype"),
    (dict(q=torch.zeros(3, 4, 128, dtype=BF16)[..., ::2]), "adjacent"),
    (dict(q=torch.zeros(12, 64, dtype=BF16)), "shape"),
    (dict(k=torch.zeros(2, 2, 64, dtype=BF16)), "shape"),
    (dict(v=torch.zeros(3, 4, 64, dtype=BF16)), "cache heads"),
    (dict(q_out=torch.zeros(3, 4, 128, dtype=BF16)[..., :64]), "q_out"),
    (dict(q_indptr=torch.zeros(1, dtype=I32)), "int32"),
    (dict(kv_len=torch.zeros(1, dtype=torch.int64)), "int32"),
    (dict(block_table=torch.zeros(2, 4, dtype=I32)), "int32"),
    (dict(block_table=torch.zeros(1, 8, dtype=I32)[:, ::2]), "contiguous"),
    (dict(), "GPU"),                                     # everything fits, but it is not on the GPU
])
def test_append(change, message):
    _refused(sv.spec_kv_append, _append_args(), change, message)


@pytest.mark.parametrize("change,message", [
    (dict(prefix_table=None), "prefix_table"),
    (dict(prefix_table=torch.zeros(2, dtype=torch.int64)), "prefix_table"),
    (dict(prefix_table=torch.zeros(1, 2, dtype=I32)), "prefix_table"),
    (dict(prefix_table=torch.zeros(4, dtype=I32)[::2]), "prefix_table"),
    (dict(prefix_len=33), "prefix_table"),
    (dict(draft_mask=torch.zeros(3, dtype=I32)), "draft_mask"),
    (dict(draft_mask=torch.zeros(2, dtype=torch.int64)), "draft_mask"),
    (dict(draft_mask=torch.zeros(6, dtype=torch.int64)[::2]), "draft_mask"),
    (dict(lse=torch.zeros(3, 4, dtype=torch.float64)), "lse"),
    (dict(lse=torch.zeros(3, 2)), "lse"),
    (dict(lse=torch.zeros(3, 8)[:, ::2]), "lse"),
    (dict(out=torch.zeros(2, 4, 64, dtype=BF16)), "shape"),
    (dict(out=torch.zeros(3, 2, 64, dtype=BF16)), "out"),
    (dict(out=torch.zeros(3, 4, 64)), "dtype"),
    (dict(q_indptr=torch.zeros(3, dtype=I32)), "int32"),
    (dict(), "GPU"),
])
def test_attention(change, message):
    _refused(sv.spec_prefix_attention, _attend_args(), change, message)
