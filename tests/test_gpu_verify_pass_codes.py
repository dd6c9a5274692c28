"""The example over a cache in 8 bits: its tokens are those of the rule, and the
drafts save as many passes as over 16 bits."""
import pytest

from tests.verify_pass_util import by_rule, example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gamma", [0, 4])
def test_tokens_are_those_of_the_rule(gamma):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_54_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    ex = example()
    model = ex.Target()
    prefix, prompts = ex.inputs(model)
    tokens, passes = ex.generate(model, prefix, prompts, 48, gamma, codes=True)
    assert tokens == by_rule(ex, model, prefix, prompts, 48)
    assert passes == 47 if gamma == 0 else passes < 47
