"""The example's verify loop on the CPU, its library calls replaced by stand-ins
in PyTorch and Python (no GPU needed)."""
import random

import pytest

torch = pytest.importorskip("torch")

from tests.verify_pass_util import by_rule, dense_logits  # noqa: E402
from tests.verify_pass_util import example as _example  # noqa: E402


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


# ---------------------------------------------------------------------------
# the tokens: with the right attention those of the model's rule, with a wrong
# one others
# ---------------------------------------------------------------------------
class Attention(StandIns):
    """Both paged calls in PyTorch; `wrong` names a mistake."""

    def __init__(self, monkeypatch, example, wrong=None):
        self.wrong = wrong
        super().__init__(monkeypatch, example)

    def spec_verify_greedy(self, logits, drafts, out, n, ws):
        best = logits.argmax(dim=2).to(torch.int32)
        n.copy_((best[:, :-1] == drafts).int().cumprod(dim=1).sum(dim=1))
        out.copy_(best)

    def _spans(self, q_indptr, kv_len):
        ends = q_indptr.tolist()
        return [(b, a, e, n) for b, (a, e, n) in enumerate(zip(ends, ends[1:], kv_len.tolist()))]

    def _rotated(self, x, positions, inv_freq):
        if self.wrong == "no rotation":
            return x
        angle = positions.double()[:, None] * inv_freq.double()
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = x.double().chunk(2, dim=-1)
        return torch.cat([a * c - b * s, a * s + b * c], dim=-1).to(x.dtype)

    def spec_kv_append(self, cache, q, k, v, q_out, q_indptr, block_table, kv_len, ws, inv_freq=None, position_base=0):
        for b, a, e, n in self._spans(q_indptr, kv_len):
            at = torch.arange(n - (e - a), n)
            base = 0 if self.wrong == "positions without the prefix" else position_base
            page, slot = block_table[b].long()[at // self.page], at % self.page
            q_out[a:e] = self._rotated(q[a:e], at + base, inv_freq)
            cache.tensors[0][page, slot] = self._rotated(k[a:e], at + base, inv_freq)
            cache.tensors[1][page, slot] = v[a:e]

    def spec_prefix_attention(self, cache, q, out, q_indptr, block_table, kv_len, ws, prefix_table=None, prefix_len=0):
        if self.wrong == "zeros":
            out.zero_()
            return
        if self.wrong == "noise":
            out.normal_()
            return
        group = q.shape[1] // cache.n_heads
        for b, a, e, n in self._spans(q_indptr, kv_len):
            at, shared = torch.arange(n), torch.arange(0 if self.wrong == "no prefix" else prefix_len)
            own = block_table[0 if self.wrong == "another sequence's pages" else b].long()
            page = torch.cat([prefix_table.long()[shared // self.page], own[at // self.page]])
            slot = torch.cat([shared, at]) % self.page
            K, V = (t[page, slot].float().repeat_interleave(group, dim=1) for t in cache.tensors)
            s = torch.einsum("ihd,jhd->hij", q[a:e].float(), K) * q.shape[2] ** -0.5
            last = len(shared) + n - (e - a) + torch.arange(e - a)
            seen = torch.arange(len(page)) <= last[:, None]
            if self.wrong == "no causal mask":
                seen[:] = True
            if self.wrong == "not itself":
                seen = torch.arange(len(page)) < last[:, None]
            p = torch.softmax(s.masked_fill(~seen, -1e30), dim=-1)
            out[a:e] = torch.einsum("hij,jhd->ihd", p, V).to(out.dtype)


def _run(monkeypatch, wrong, gamma, new_tokens=30):
    example = _example()
    Attention(monkeypatch, example, wrong)
    model = example.Target(device="cpu")
    prefix, prompts = example.inputs(model, device="cpu")
    tokens, passes = example.generate(model, prefix, prompts, new_tokens, gamma)
    return example, model, prefix, prompts, tokens, passes


def test_the_right_attention_gives_the_tokens_of_the_rule(monkeypatch):
    example, model, prefix, prompts, plain, plain_passes = _run(monkeypatch, None, 0)
    assert plain == by_rule(example, model, prefix, prompts, 30)
    *_, fast, fast_passes = _run(monkeypatch, None, 4)
    assert fast == plain and fast_passes < plain_passes == 29
    # the layers matter: without them every sequence would count on
    counting = [[(p.tolist()[-1] + 1 + i) % model.vocab for i in range(30)] for p in prompts]
    assert all(sum(a == b for a, b in zip(x, y)) < 3 for x, y in zip(plain, counting))


def test_the_model_leaves_no_near_ties(monkeypatch):
    """In float64 without a cache every token leads by a fifth of its logit: far
    more than roundings to 8 bits can move it."""
    example, model, prefix, prompts, plain, _ = _run(monkeypatch, None, 0)
    for p, new in zip(prompts, plain):
        text = prefix.tolist() + p.tolist() + new
        logits = dense_logits(model, text)[len(text) - len(new) - 1:-1]
        top = logits.topk(2, dim=1)
        assert top.indices[:, 0].tolist() == new
        assert (top.values[:, 0] - top.values[:, 1] > 0.2 * top.values[:, 0]).all()


@pytest.mark.parametrize("gamma", [0, 4])
@pytest.mark.parametrize("wrong", ["zeros", "noise", "no rotation", "positions without the prefix", "no causal mask",
                                   "not itself", "no prefix", "another sequence's pages"])
def test_a_wrong_attention_gives_other_tokens(monkeypatch, wrong, gamma):
    torch.manual_seed(0)
    example, model, prefix, prompts, tokens, _ = _run(monkeypatch, wrong, gamma)
    assert tokens != by_rule(example, model, prefix, prompts, 30)
