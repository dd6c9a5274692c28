"""The example's verify loop on the GPU: speculative greedy decoding through the
paged cache gives the tokens of plain decoding, in fewer passes."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_speculative_decoding_gives_the_plain_tokens():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_54_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("verify_pass", os.path.join(ROOT, "examples", "verify_pass.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    plain, fast, plain_passes, fast_passes = example.main()
    assert all(len(t) == 48 for t in plain + fast)
    # the passes' shapes differ, so their bf16 roundings do: a token may differ
    # only from the first near tie on, and the model's logits leave none here
    assert fast == plain
    assert fast_passes < plain_passes
