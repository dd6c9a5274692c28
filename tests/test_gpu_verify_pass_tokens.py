"""The example's tokens on the GPU against the model's rule and against a dense
float64 pass: both depend on the attention over prefix and pages, the rotation
and the causal mask."""
import pytest

from tests.verify_pass_util import by_rule, dense_logits, example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gamma", [0, 1, 4])
def test_tokens_are_those_of_the_rule_and_of_a_dense_pass(gamma):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_54_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    ex = example()
    model = ex.Target()
    prefix, prompts = ex.inputs(model)
    tokens, passes = ex.generate(model, prefix, prompts, 48, gamma)
    assert tokens == by_rule(ex, model, prefix, prompts, 48)
    assert passes == 47 if gamma == 0 else passes < 47
    for p, new in zip(prompts, tokens):
        text = prefix.tolist() + p.tolist() + new
        logits = dense_logits(model, text)[len(text) - len(new) - 1:-1]
        top = logits.topk(2, dim=1)
        assert top.indices[:, 0].tolist() == new
        assert (top.values[:, 0] - top.values[:, 1] > 0.2 * top.values[:, 0]).all()
