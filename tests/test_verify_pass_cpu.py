"""The example's verify loop on the CPU, its library calls replaced by stand-ins
in PyTorch and Python (no GPU needed)."""
import importlib.util
import os
import random

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("verify_pass", os.path.join(ROOT, "examples", "verify_pass.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


class StandIns:
    """The calls that generate() makes.  `accept` says how many of its drafts a
    sequence keeps in a round; appends are checked against the table."""

    def __init__(self, monkeypatch, example, accept=None):
        self.accept, self.longest, self.page = accept, 0, example.PAGE
        for name in ("spec_kv_append", "spec_prefix_attention", "spec_verify_greedy", "spec_verify_status",
                     "make_attention_workspace", "make_workspace"):
            monkeypatch.setattr(example.sv, name, getattr(self, name))

    def make_attention_workspace(self, *a, **k):
        return None

    make_workspace = make_attention_workspace

    def spec_verify_status(self, ws):
        return 0

    def spec_kv_append(self, cache, q, k, v, q_out, q_indptr, block_table, kv_len, ws, **kw):
        longest = int(kv_len.max())
        self.longest = max(self.longest, longest)
        assert longest <= block_table.shape[1] * self.page, f"{longest} entries in {block_table.shape[1]} pages"
        q_out.copy_(q)

    def spec_prefix_attention(self, cache, q, out, *a, **kw):
        out.zero_()

    def spec_verify_greedy(self, logits, drafts, out, n, ws):
        gamma = drafts.shape[1]
        best = logits.argmax(dim=2).to(torch.int32)
        for b in range(drafts.shape[0]):
            kept = min(self.accept(b), gamma)
            out[b] = best[b]
            out[b, :kept] = drafts[b, :kept]
            n[b] = kept


@pytest.mark.parametrize("longest", [40, 41, 42, 43])  # 43: the pages end with the last entry
@pytest.mark.parametrize("seed", range(6))
def test_sequences_that_finish_early_stay_in_their_pages(monkeypatch, longest, seed):
    example = _example()
    rng = random.Random(seed)
    StandIns(monkeypatch, example, accept=lambda b: rng.randint(0, 1) if b == 0 else rng.randint(0, 4))
    model = example.Target(vocab=64, hidden=32, n_q_heads=2, n_heads=1, head_dim=16, layers=1, device="cpu")
    prompts = [torch.randint(0, 64, (n,), dtype=torch.int32) for n in (5, longest, 17, longest - 1)]
    prefix = torch.randint(0, 64, (20,), dtype=torch.int32)
    tokens, passes = example.generate(model, prefix, prompts, 48, 4)
    assert all(len(t) == 48 for t in tokens) and passes > 10
