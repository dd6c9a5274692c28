"""Row offsets (q_indptr) that leave rows without a sequence or do not ascend,
in the paged cache's calls: reported, and such rows are left alone."""
import pytest

from tests.test_gpu_paged import Problem, _attend, sv  # noqa: F401
from tests.test_gpu_paged_ranges import _append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefix", [0, 40])
def test_rows_before_the_first_sequence_are_reported_and_left_alone(sv, prefix):  # noqa: F811
    import torch
    pr = Problem(103, "bf16", 64, 2, 8, 16, [3, 2, 4], [50, 2, 140], prefix)
    ws = sv.make_attention_workspace(3, pr.N, pr.Hq, pr.D)
    good, good_lse, _ = _attend(sv, pr, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    # the first sequence loses its rows: they belong to none
    pr.indptr = torch.tensor([3, 5, 9], dtype=torch.int32, device="cuda")
    pr.table, pr.kv_len, pr.q_lens = pr.table[1:].contiguous(), pr.kv_len[1:].contiguous(), [2, 4]
    out, lse, _ = _attend(sv, pr, ws=ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
    assert (out[:3] == -7.0).all() and (lse[:3] == -7.0).all()
    # parts begin elsewhere: 32-bit sums in another order, then one rounding to 8 bits
    assert torch.allclose(out[3:].float(), good[3:].float(), rtol=2.0 ** -7, atol=2.0 ** -7)
    assert torch.allclose(lse[3:], good_lse[3:], rtol=1e-5, atol=1e-5)
    q_out, _ = _append(sv, pr, ws)
    assert sv.spec_verify_status(ws) == sv.SPEC_ERR_DEVICE_INPUT
    assert (q_out[:3] == -7.0).all() and (q_out[3:] != -7.0).any()


def test_append_reports_row_offsets_that_do_not_ascend(sv):  # noqa: F811
    import torch
    pr = Problem(104, "bf16", 64, 1, 2, 8, [3, 2, 4], [20, 20, 20])
    ws = sv.make_attention_workspace(3, pr.N, pr.Hq, pr.D)
    for offsets, code in (([0, 3, 5, 9], sv.SPEC_OK), ([0, 5, 3, 9], sv.SPEC_ERR_DEVICE_INPUT),
                          ([0, 3, 5, 10], sv.SPEC_ERR_DEVICE_INPUT), ([-1, 3, 5, 9], sv.SPEC_ERR_DEVICE_INPUT),
                          ([0, 9, 4, 4], sv.SPEC_ERR_DEVICE_INPUT)):
        pr.indptr = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        _append(sv, pr, ws)
        assert sv.spec_verify_status(ws) == code, offsets
