"""Speculative greedy decoding with a small target model: the paged cache, the
shared-prefix attention and the verify step run together.

Every sequence of a batch continues the same system prompt with a prompt of its
own.  Each round drafts gamma tokens by looking them up in the sequence's own
text, verifies them in one pass of the target (per layer: projections,
spec_kv_append, spec_prefix_attention), accepts with spec_verify_greedy, and
keeps the accepted cache entries by spec_round_update: the next append overwrites
the rest.

The model's weights are set by hand so that what it says can be known without
it: the token after position t is the one HOP positions before, plus one.  Its
first layer looks for the position after its own, and so finds itself as long as
no later one is visible; its last layer looks HOP positions back and copies what
the first one left there.  Without its layers it would count on from the newest
token.

    python examples/verify_pass.py            # needs the GPU and the built library
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_54_gb300 as sv  # noqa: E402

PAGE = 16
HOP = 20


class Target:
    """A decoder of `layers` layers over tied embeddings, bf16.

    Dim 0 of every embedding is ALWAYS, from which queries and keys are made, so
    that their products depend on positions alone: with keys (a, 0) and queries
    a (cos(-df), sin(-df)) in the pair of frequency f, two positions at distance x
    score a^2 sum_f cos((x - d) f), which is largest at x = d.  Values are the next
    n_heads * head_dim dims, which the output projection puts back in their place."""

    ALWAYS, SHARPNESS, COPY = 4.0, 8.0, (4.0, 3.0)  # COPY: the first layers' gain, the last one's

    def __init__(self, vocab=512, hidden=256, n_q_heads=8, n_heads=2, head_dim=64, layers=2, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.n_q_heads, self.n_heads, self.D, self.hidden, self.vocab = n_q_heads, n_heads, head_dim, hidden, vocab
        half, group, copied = head_dim // 2, n_q_heads // n_heads, n_heads * head_dim
        assert copied < hidden
        embed = torch.randn(vocab, hidden, generator=g, device=device)
        embed[:, 0] = self.ALWAYS
        # of one length for all tokens, or a key's length would count with its position
        for part in (embed[:, 1:1 + copied], embed[:, 1 + copied:]):
            part *= part.shape[1] ** 0.5 / part.norm(dim=1, keepdim=True)
        self.embed = embed.to(torch.bfloat16)
        self.inv_freq = (10000.0 ** (-torch.arange(half, device=device) / half)).float()
        mean_square = torch.ones(hidden)  # of the layer's input, dim by dim
        mean_square[0] = self.ALWAYS ** 2
        self.layers = []
        for i in range(layers):
            distance = HOP if i == layers - 1 else -1
            gain = self.COPY[1] if i == layers - 1 else self.COPY[0]
            rms = float(mean_square.mean().sqrt())
            a = (self.SHARPNESS * head_dim ** 0.5) ** 0.5 * rms / self.ALWAYS
            w_qkv = torch.zeros((n_q_heads + 2 * n_heads) * head_dim, hidden, device=device)
            q, k, v = w_qkv.split([n_q_heads * head_dim, copied, copied])
            angle = -distance * self.inv_freq
            q[:, 0] = a * torch.cat([angle.cos(), angle.sin()]).repeat(n_q_heads)
            k[:, 0] = a * torch.cat([torch.ones(half), torch.zeros(half)]).to(device).repeat(n_heads)
            v[:, 1:1 + copied] = torch.eye(copied, device=device)
            # the heads that share a key head see the same: each brings its part
            w_out = torch.zeros(hidden, n_q_heads * head_dim, device=device)
            back = torch.eye(copied, device=device).unflatten(1, (n_heads, 1, head_dim)).expand(-1, -1, group, -1)
            w_out[1:1 + copied] = gain * rms / group * back.flatten(1)
            mean_square[1:1 + copied] *= (1 + gain) ** 2
            self.layers.append((w_qkv.to(torch.bfloat16), w_out.to(torch.bfloat16)))

    def logits(self, h):
        # of a token's own embedding this makes the next token the likeliest
        return h @ torch.roll(self.embed, 1, dims=0).T


class Cache:
    """Pages of every layer, the prefix's and the sequences' tables."""

    def __init__(self, model, B, prefix_len, max_len, device="cuda"):
        shared, width = -(-prefix_len // PAGE), -(-max_len // PAGE)
        total = shared + B * width
        shape = (total, PAGE, model.n_heads, model.D)
        self.layers = [sv.make_kv_cache(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in "kv"))
                       for _ in model.layers]
        order = torch.randperm(total, device=device, dtype=torch.int32)
        self.prefix_table, self.prefix_len = order[:shared].contiguous(), prefix_len
        self.table = order[shared:].reshape(B, width).contiguous()


def forward(model, cache, tokens, q_len, kv_len, table, prefix_len, ws):
    """One pass over new tokens [N] (q_len of each sequence, kv_len entries of
    its own with them); returns hidden states [N, hidden]."""
    device = tokens.device
    N = tokens.shape[0]
    h = model.embed[tokens.long()]
    indptr = torch.tensor([0] + list(q_len), dtype=torch.int32).cumsum(0).to(torch.int32).to(device)
    lens = torch.tensor(list(kv_len), dtype=torch.int32, device=device)
    Hq, Hk, D = model.n_q_heads, model.n_heads, model.D
    q_turned = torch.empty(N, Hq, D, dtype=torch.bfloat16, device=device)
    out = torch.empty_like(q_turned)
    for (w_qkv, w_out), layer in zip(model.layers, cache.layers):
        x = torch.nn.functional.rms_norm(h, (model.hidden,))
        q, k, v = (x @ w_qkv.T).split([Hq * D, Hk * D, Hk * D], dim=1)
        sv.spec_kv_append(layer, q.unflatten(1, (Hq, D)), k.unflatten(1, (Hk, D)), v.unflatten(1, (Hk, D)), q_turned,
                          indptr, table, lens, ws, inv_freq=model.inv_freq, position_base=prefix_len)
        sv.spec_prefix_attention(layer, q_turned, out, indptr, table, lens, ws, prefix_table=cache.prefix_table,
                                 prefix_len=prefix_len)
        h = h + out.flatten(1) @ w_out.T
    return torch.nn.functional.rms_norm(h, (model.hidden,))


def draft(text, gamma, vocab):
    """The drafter knows a sequence's own text, not the prefix, and not every
    token: it looks up what stood HOP positions before, or counts on."""
    text, first = list(text), len(text)
    for i in range(first, first + gamma):
        seen = text[i - 1 - HOP] if i - 1 - HOP >= 0 else None
        text.append(((text[-1] if seen is None or seen % 8 == 0 else seen) + 1) % vocab)
    return text[first:]


def generate(model, prefix, prompts, new_tokens, gamma):
    """Greedy continuations of `prompts` behind the shared `prefix`, `gamma`
    drafts a round (0: plain decoding).  Returns the tokens and the number of
    passes of the target."""
    device = prefix.device
    B = len(prompts)
    max_len = max(p.shape[0] for p in prompts) + new_tokens + gamma + 1
    cache = Cache(model, B, prefix.shape[0], max_len, device)
    most = max(prefix.shape[0], sum(p.shape[0] for p in prompts), B * (gamma + 1))
    ws = sv.make_attention_workspace(B, most, model.n_q_heads, model.D, device)
    # the prefix once, as a sequence that lives in the shared pages
    forward(model, cache, prefix, [prefix.shape[0]], [prefix.shape[0]], cache.prefix_table[None], 0, ws)
    # the prompts
    q_len = [p.shape[0] for p in prompts]
    h = forward(model, cache, torch.cat(prompts), q_len, q_len, cache.table, cache.prefix_len, ws)
    last = torch.tensor(q_len).cumsum(0) - 1
    texts = [p.tolist() for p in prompts]
    done = [[int(t)] for t in model.logits(h[last.to(device)]).argmax(dim=1).cpu()]
    verify_ws = sv.make_workspace(B, max(gamma, 1), model.vocab, device=device)
    states = (sv.SpecRoundState * B)()
    for s, n in zip(states, q_len):
        s.gamma, s.seq_len, s.kv_len = max(gamma, 1), n + 1, n
    passes = 0
    while min(len(d) for d in done) < new_tokens:
        drafts = [draft(t + d, gamma, model.vocab) for t, d in zip(texts, done)]
        tokens = torch.tensor([[d[-1]] + x for d, x in zip(done, drafts)], dtype=torch.int32, device=device).flatten()
        # sequences that are finished go on until the others are
        h = forward(model, cache, tokens, [gamma + 1] * B, [s.kv_len + gamma + 1 for s in states], cache.table,
                    cache.prefix_len, ws)
        passes += 1
        logits = model.logits(h).unflatten(0, (B, gamma + 1)).contiguous()
        if gamma == 0:
            out, accepted = logits[:, 0].argmax(dim=1).to(torch.int32)[:, None].cpu(), [0] * B
            for s in states:
                s.seq_len += 1
                s.kv_len += 1
        else:
            out = torch.empty(B, gamma + 1, dtype=torch.int32, device=device)
            n = torch.empty(B, dtype=torch.int32, device=device)
            sv.spec_verify_greedy(logits, torch.tensor(drafts, dtype=torch.int32, device=device), out, n, verify_ws)
            if sv.spec_verify_status(verify_ws) != sv.SPEC_OK:
                raise RuntimeError("verification failed")
            out, accepted = out.cpu(), n.cpu().tolist()
            sv.spec_round_update(states, accepted, gamma, gamma)
        for b in range(B):
            done[b] += out[b, :accepted[b] + 1].tolist()
        # a pass appends up to entry prompt + len(done) + gamma, and the pages hold
        # max_len: a finished sequence drops what it has beyond new_tokens + 1
        for b, s in enumerate(states):
            extra = len(done[b]) - (new_tokens + 1)
            if extra > 0:
                del done[b][new_tokens + 1:]
                s.seq_len -= extra
                s.kv_len -= extra
    if sv.spec_verify_status(ws) != sv.SPEC_OK:
        raise RuntimeError("attention reported an error")
    return [d[:new_tokens] for d in done], passes


def inputs(model, device="cuda"):
    """A shared prefix and prompts, some shorter than HOP: their first tokens come
    from the prefix."""
    g = torch.Generator(device=device).manual_seed(1)
    prefix = torch.randint(0, model.vocab, (300,), generator=g, device=device, dtype=torch.int32)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g, device=device, dtype=torch.int32) for n in (5, 40, 17, 33)]
    return prefix, prompts


def main():
    torch.cuda.set_device(0)
    model = Target()
    prefix, prompts = inputs(model)
    plain, plain_passes = generate(model, prefix, prompts, 48, 0)
    spec, spec_passes = generate(model, prefix, prompts, 48, 4)
    same = sum(a == b for x, y in zip(plain, spec) for a, b in zip(x, y))
    print(f"plain: {plain_passes} passes, speculative: {spec_passes} passes, "
          f"{same} of {sum(map(len, plain))} tokens the same")
    return plain, spec, plain_passes, spec_passes


if __name__ == "__main__":
    main()
