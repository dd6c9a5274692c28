"""Many small weights behind one large: a long tail that together counts must
not vanish from the output of spec_prefix_attention."""
import numpy as np
import pytest

from tests.test_gpu_paged import Problem, _attend, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("peak", [0, 5000, 8191])
def test_tail_of_small_weights(sv, dtype, peak):  # noqa: F811
    """8,192 keys of one score, 2^-25.5 of the peak's weight each, with values
    2,048 times the peak's.

    Tolerance, of the values' scale 2,048: weights rounded to the type (u, all
    the same way where they are equal) and, in fp16, off by 2^-32 of the largest
    each where subnormal; the result rounded (u); 32-bit sums of n weights
    (n 2^-23 of the sum); the exponentials 2^-20 relative."""
    import torch
    D, n, B, heads = 64, 8192, 64, 8  # items enough that a CTA takes many tiles of one
    pr = Problem(111, dtype, D, heads, heads, 16, [1], [n])
    pr.q_lens, pr.kv_lens, pr.N = [1] * B, [n] * B, B
    pr.table = pr.table.expand(B, -1).contiguous()  # the sequences share their pages
    pr.kv_len = pr.kv_len.expand(B).contiguous()
    pr.indptr = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    K, V = pr.pools
    K.zero_()
    V.fill_(2048.0)
    where = int(pr.table_np[0, peak // 16]), peak % 16
    # the score of the peak, times log2(e): 25.5, in values that 16 bits hold
    pr.q = torch.zeros((B, heads, D), dtype=K.dtype, device="cuda")
    pr.q[:, :, 0] = 8.0
    gap = float(torch.tensor(25.5 / 1.4426950408889634).to(K.dtype))
    K[where][:, 0] = gap
    V[where] = 1.0
    out, lse, ws = _attend(sv, pr)
    assert sv.spec_verify_status(ws) == sv.SPEC_OK
    w = np.exp(-gap)
    total = 1.0 + (n - 1) * w
    want = (1.0 + (n - 1) * w * 2048.0) / total
    assert 1.3 < want
    u = torch.finfo(K.dtype).eps / 2
    tail = (n - 1) * w * 2048.0 / total
    tol = tail * (u + 2.0 ** -20) + (n * 2.0 ** -32 * 2048.0 if dtype == "fp16" else 0.0) \
        + want * (u + n * 2.0 ** -23) + u
    diff = np.abs(out.double().cpu().numpy() - want)
    assert (diff <= tol).all(), (diff.max(), want, tol)
    assert ((lse.double().cpu() - (gap + np.log(total))).abs() <= 1e-5 * gap).all()
