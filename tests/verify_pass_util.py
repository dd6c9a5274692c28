"""What the example's model says, computed apart from the library: by its rule,
and densely in float64."""
import importlib.util
import os

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("verify_pass", os.path.join(ROOT, "examples", "verify_pass.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def by_rule(ex, model, prefix, prompts, new_tokens):
    """Each token is the one HOP positions before its predecessor, plus one."""
    out = []
    for p in prompts:
        text = prefix.tolist() + p.tolist()
        first = len(text)
        for _ in range(new_tokens):
            text.append((text[len(text) - 1 - ex.HOP] + 1) % model.vocab)
        out.append(text[first:])
    return out


def dense_logits(model, tokens):
    """float64 [T, vocab]: the whole text in one pass, no cache, no pages."""
    import torch
    D, Hq, Hk, T = model.D, model.n_q_heads, model.n_heads, len(tokens)
    device = model.embed.device
    at = torch.tensor(tokens, device=device)
    h = model.embed[at].double()
    angle = torch.arange(T, device=device).double()[:, None] * model.inv_freq.double()
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]
    causal = torch.ones(T, T, dtype=torch.bool, device=device).tril()

    def turned(x):
        a, b = x.chunk(2, dim=-1)
        z = torch.complex(a, b) * unit
        return torch.cat([z.real, z.imag], dim=-1)

    for w_qkv, w_out in model.layers:
        x = h / (h ** 2).mean(dim=1, keepdim=True).sqrt()
        q, k, v = (x @ w_qkv.double().T).split([Hq * D, Hk * D, Hk * D], dim=1)
        q, k, v = turned(q.unflatten(1, (Hq, D))), turned(k.unflatten(1, (Hk, D))), v.unflatten(1, (Hk, D))
        k, v = (t.repeat_interleave(Hq // Hk, dim=1) for t in (k, v))
        s = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
        w = torch.softmax(s.masked_fill(~causal, -float("inf")), dim=-1)
        h = h + torch.einsum("hij,jhd->ihd", w, v).flatten(1) @ w_out.double().T
    h = h / (h ** 2).mean(dim=1, keepdim=True).sqrt()
    return model.logits(h.to(model.embed.dtype)).double()
