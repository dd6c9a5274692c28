"""Workspaces of the paged calls are in proportion to what each call keeps there
(no GPU needed: every call here is refused for another reason)."""
import pytest

import speculative_decoding_verification_54_gb300 as sv
from tests.test_paged_cpu import _append, _attend, lib  # noqa: F401

torch = pytest.importorskip("torch")


def test_append_needs_its_status_word_alone(lib):  # noqa: F811
    assert sv.spec_kv_append_workspace_bytes() == 256
    for N in (1, 32768):
        # rot_dim is refused after the workspace has been looked at
        assert _append(lib, N=N, wsb=256, rot=127) == sv.SPEC_ERR_INVALID_ARG
        assert _append(lib, N=N, wsb=255, rot=127) == sv.SPEC_ERR_WORKSPACE
    assert sv.make_append_workspace("cpu").nbytes == 256


@pytest.mark.parametrize("N", [1, 20, 5000])
def test_attention_without_a_prefix_needs_one_place_a_row(lib, N):  # noqa: F811
    both = sv.spec_attention_workspace_bytes(4, N, 32, 128)
    own = sv.spec_attention_workspace_bytes(4, N, 32, 128, prefix=False)
    rows = N * 32
    assert both - own == -(-rows * 16 // 256) * 256 + -(-rows * 8 // 256) * 256 + rows * 128 * 4
    for size, kw in ((both, dict()), (own, dict(pl=0, pt=None))):
        # scale is refused after the workspace has been looked at
        assert _attend(lib, N=N, wsb=size, scale=0.0, **kw) == sv.SPEC_ERR_INVALID_ARG
        assert _attend(lib, N=N, wsb=size - 1, scale=0.0, **kw) == sv.SPEC_ERR_WORKSPACE
    assert sv.make_attention_workspace(4, N, 32, 128, "cpu", prefix=False).nbytes == own
    assert sv.make_attention_workspace(4, N, 32, 128, "cpu").nbytes == both


def test_few_rows_need_small_slabs(lib):  # noqa: F811
    """A CTA's slab holds the rows of one block at most: 32 of them for one token."""
    assert sv.spec_attention_workspace_bytes(1, 1, 32, 128) < 3 << 20
    assert sv.spec_attention_workspace_bytes(1, 1, 32, 128) > 160 * 32 * 128 * 4
