"""Cases of the paged-cache operators of the verify pass, their plain forms, and their calls.

A target model verifies gamma + 1 drafted positions of every sequence in one
forward pass.  In each layer that pass rotates the new queries and keys to
their positions, writes keys and values into the sequence's pages
(spec_kv_append), and lets every new query attend to the prefix that the whole
batch shares, to its own sequence's pages, and to the new positions that the
draft mask shows it (spec_prefix_attention).

``own`` selects between the plain form (elementary torch operations in 32
bits, angles in 64) and the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _append(name, **kw):
    case = dict(name=name, op="append", dtype="bf16", B=1, q=1, ragged=False, Hq=32, Hk=8, D=128, rot=128, axes=1,
                interleaved=False, page=16, heads_first=False, suffix=64, prefix=0)
    case.update(kw)
    return case


def _attend(name, **kw):
    case = dict(name=name, op="attend", dtype="bf16", B=1, q=1, ragged=False, Hq=32, Hk=8, D=128, page=16,
                heads_first=False, suffix=64, prefix=0, mask=False)
    case.update(kw)
    return case


def listed():
    return [
        # one user's plain decode step: one token, a launch's latency
        _append("append_one", suffix=1000, prefix=512),
        # the verify pass of a served batch: 32 sequences x (gamma = 4) + 1
        _append("append_verify_b32", B=32, q=5, page=64, suffix=1024, prefix=8192),
        # drafts of different lengths, seven query heads a key head, a part of
        # each head rotated in neighbouring pairs, pages of no power of two
        _append("append_ragged_d64", dtype="fp16", B=48, q=9, ragged=True, Hq=28, Hk=4, D=64, rot=32, interleaved=True,
                page=24, suffix=777),
        # prompts with images: time, height and width positions
        _append("append_image_prompts", B=3, q=4097, ragged=True, Hq=28, Hk=4, axes=3, page=16, suffix=5000),
        # prompts entering the cache: bandwidth
        _append("append_prompts", B=8, q=4096, Hq=16, Hk=8, D=256, rot=256, page=64, heads_first=True, suffix=4096),
        # one user's plain decode step behind a system prompt: latency
        _attend("attend_one", prefix=512, suffix=37),
        # the verify pass of a served batch behind a shared system prompt
        _attend("attend_verify_b32", B=32, q=5, ragged=True, prefix=8192, suffix=1024),
        # long drafts and a long shared document: matrix products bound it
        _attend("attend_longdraft_b128", B=128, q=9, ragged=True, page=64, prefix=32768, suffix=2048),
        # long conversations with nothing shared: the cache's bytes bound it
        _attend("attend_long_caches", B=16, q=5, ragged=True, page=64, heads_first=True, suffix=32768),
        # several draft candidates a sequence in one pass, told apart by the mask
        _attend("attend_candidates_d64", dtype="fp16", B=24, q=12, Hq=28, Hk=4, D=64, page=24, prefix=2051, suffix=611,
                ragged=True, mask=True),
        # prompts entering behind the shared prefix: causal tiles
        _attend("attend_prompt_chunks", B=4, q=1024, ragged=True, Hq=16, Hk=8, page=16, prefix=4099, suffix=1500),
        # plain decoding of a wide batch, one query head a key head
        _attend("attend_decode_b64", B=64, q=1, ragged=True, Hq=16, Hk=16, D=64, page=32, prefix=16384, suffix=513),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    largest = {op: [max(_cost(c)[k] for c in listed() if c["op"] == op) for k in range(3)] for op in ("append", "attend")}
    while True:
        op = rng.choice(["append", "attend"])
        hk = rng.choice([1, 2, 3, 4, 5, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), B=_log_int(rng, 1, 128), Hk=hk, Hq=hk * group,
                    ragged=rng.random() < 0.75, heads_first=rng.random() < 0.4,
                    page=rng.choice([8, 16, 24, 32, 40, 64, 128, 256]))
        if op == "append":
            case.update(D=rng.choice([64, 128, 256]), axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4,
                        q=_log_int(rng, 1, 4096), prefix=rng.choice([0, 0, _log_int(rng, 1, 100000)]))
            case["rot"] = rng.choice([case["D"], case["D"] // 2, 2 * rng.randint(1, case["D"] // 2)])
            case["suffix"] = case["q"] + _log_int(rng, 1, 4096) - 1
        else:
            case.update(D=rng.choice([64, 128]), mask=rng.random() < 0.3)
            case["q"] = _log_int(rng, 1, 32) if case["mask"] or rng.random() < 0.7 else _log_int(rng, 1, 1024)
            case["prefix"] = 0 if rng.random() < 0.25 else _log_int(rng, 1, 32768)
            case["suffix"] = case["q"] + _log_int(rng, 1, 32768) - 1
        if all(x <= y for x, y in zip(_cost(case), largest[op])):
            return case


def _lengths(case):
    """New positions and cached positions (the new ones among them) of every sequence: sizes, so the case alone sets them."""
    rng = random.Random(",".join("%s=%s" % (k, case[k]) for k in ("op", "B", "q", "suffix", "ragged")))
    if not case["ragged"]:
        return [case["q"]] * case["B"], [case["suffix"]] * case["B"]
    q = [rng.randint(1, case["q"]) for _ in range(case["B"])]
    return q, [rng.randint(n, case["suffix"]) for n in q]


def work(case):
    size = 2  # both types
    q, kv = _lengths(case)
    n, Hq, Hk, D = sum(q), case["Hq"], case["Hk"], case["D"]
    if case["op"] == "append":
        moved = 2 * n * (Hq + 2 * Hk) * D * size + n * 4 * case["axes"]
        return {"bytes": moved, "flops": 6 * n * (Hq + Hk) * (case["rot"] // 2)}
    # new positions see every older one; among themselves the causal half, or
    # under a mask at most that
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, kv)) + n * case["prefix"]
    cached = (case["prefix"] + sum(kv)) * Hk * D * 2 * size
    return {"bytes": cached + 2 * n * Hq * D * size + 4 * n * Hq, "flops": 4 * pairs * Hq * D}


def _cost(case):
    """What bounds a drawn case: bytes, operations, and the plain form's largest table of scores (padded to the longest sequence)."""
    w = work(case)
    q, kv = _lengths(case)
    table = case["B"] * max(q) * case["Hq"] * (case["prefix"] + max(kv)) if case["op"] == "attend" else sum(q)
    return w["bytes"], w["flops"], table


def _pages(case, gen):
    """Pages dealt in random order: the pools (k, v), the sequences' table and the prefix's."""
    _, kv = _lengths(case)
    page, Hk, D = case["page"], case["Hk"], case["D"]
    width = max(-(-n // page) for n in kv)
    shared = -(-case["prefix"] // page) if case["op"] == "attend" else 0
    total = case["B"] * width + shared + 3
    order = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int32)
    shape = (total, Hk, page, D) if case["heads_first"] else (total, page, Hk, D)
    pools = [torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(_DTYPES[case["dtype"]]) for _ in "kv"]
    if case["heads_first"]:
        pools = [p.transpose(1, 2) for p in pools]  # seen as [pages, slots, heads, D] either way
    return pools, order[: case["B"] * width].reshape(case["B"], width).contiguous(), order[total - shared :].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q_len, kv_len = _lengths(case)
    n, Hq, Hk, D, dt = sum(q_len), case["Hq"], case["Hk"], case["D"], _DTYPES[case["dtype"]]
    (k_pages, v_pages), table, prefix_table = _pages(case, gen)
    indptr = torch.tensor([0] + q_len, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    lens = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    state = dict(case=case, k_pages=k_pages, v_pages=v_pages, table=table, prefix_table=prefix_table, indptr=indptr,
                 kv_len=lens, q_max=max(q_len), kept={})
    if case["op"] == "append":
        # q, k and v lie side by side in the output of one projection
        qkv = torch.randn((n, (Hq + 2 * Hk) * D), generator=gen, device="cuda").to(dt)
        q, k, v = qkv.split([Hq * D, Hk * D, Hk * D], dim=1)
        state.update(q=q.unflatten(1, (Hq, D)), k=k.unflatten(1, (Hk, D)), v=v.unflatten(1, (Hk, D)),
                     q_out=torch.empty((n, Hq, D), dtype=dt, device="cuda"))
        half = case["rot"] // 2
        state["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
        # text: one position a token, counted on from the prefix; images: a
        # position on each axis, frequencies dealt to the axes in turn
        state["axis"] = (torch.arange(half, device="cuda") % case["axes"]).to(torch.int32) if case["axes"] > 1 else None
        state["positions"] = None
        if case["axes"] > 1:
            state["positions"] = torch.randint(0, 40000, (case["axes"], n), generator=gen, device="cuda", dtype=torch.int32)
        return state
    # scores of a spread that softmax turns into peaks
    state["q"] = (2 * torch.randn((n, Hq, D), generator=gen, device="cuda")).to(dt)
    state["out"] = torch.empty((n, Hq, D), dtype=dt, device="cuda")
    state["lse"] = torch.empty((n, Hq), dtype=torch.float32, device="cuda")
    state["mask"] = None
    if case["mask"]:
        # three candidates a sequence: token i sees the tokens before it of its
        # own candidate, and itself; a few see nothing new at all
        local = torch.cat([torch.arange(x) for x in q_len])
        third = torch.repeat_interleave(torch.tensor([-(-x // 3) for x in q_len]), torch.tensor(q_len))
        bits = ((1 << (local + 1)) - 1) & ~((1 << (local // third * third)) - 1)
        hidden = torch.rand(n, generator=gen, device="cuda").cpu() < 0.02
        state["mask"] = torch.where(hidden, 0, bits).to(torch.int64).cuda()
    return state


def run(state):
    if own:
        return _call(state)
    return _plain_append(state) if state["case"]["op"] == "append" else _plain_attend(state)


def _call(s):
    import speculative_decoding_verification_54_gb300 as sv

    case, kept = s["case"], s["kept"]
    if not kept:  # what a program makes once for its cache
        kept["cache"] = sv.make_kv_cache(s["k_pages"], s["v_pages"])
        kept["ws"] = sv.make_attention_workspace(case["B"], s["q"].shape[0], case["Hq"], case["D"])
    if case["op"] == "append":
        sv.spec_kv_append(kept["cache"], s["q"], s["k"], s["v"], s["q_out"], s["indptr"], s["table"], s["kv_len"],
                          kept["ws"], inv_freq=s["inv_freq"], positions=s["positions"], axis=s["axis"],
                          interleaved=case["interleaved"], position_base=case["prefix"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    sv.spec_prefix_attention(kept["cache"], s["q"], s["out"], s["indptr"], s["table"], s["kv_len"], kept["ws"],
                             prefix_table=s["prefix_table"], prefix_len=case["prefix"], draft_mask=s["mask"],
                             lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _rows(s):
    """Of every new token: its sequence, its place among the new ones, and its place in the sequence's cache."""
    n = s["q"].shape[0]
    token = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["indptr"][1:].long(), token, right=True)
    local = token - s["indptr"].long()[seq]
    q_len = (s["indptr"][1:] - s["indptr"][:-1]).long()
    return seq, local, s["kv_len"].long()[seq] - q_len[seq] + local


def _plain_append(s):
    case = s["case"]
    seq, _, slot = _rows(s)
    if s["positions"] is None:
        pos = (case["prefix"] + slot)[:, None].expand(-1, case["rot"] // 2)
    else:
        pos = s["positions"].long()[s["axis"].long()].T
    angle = pos.double() * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotated(x):
        x = x.float()
        head, rest = x[..., : case["rot"]], x[..., case["rot"] :]
        if case["interleaved"]:
            a, b = head[..., 0::2], head[..., 1::2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        else:
            a, b = head.chunk(2, dim=-1)
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        return torch.cat([turned, rest], dim=-1).to(s["q"].dtype)

    page = s["table"].long()[seq, slot // case["page"]]
    s["k_pages"][page, slot % case["page"]] = rotated(s["k"])
    s["v_pages"][page, slot % case["page"]] = s["v"]
    return {"q": rotated(s["q"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _plain_attend(s):
    case = s["case"]
    B, Hk, D, Q, P = case["B"], case["Hk"], case["D"], s["q_max"], case["prefix"]
    group = case["Hq"] // Hk
    seq, local, slot = _rows(s)
    width = s["table"].shape[1] * case["page"]
    q = torch.zeros((B, Q, Hk, group, D), dtype=torch.float32, device="cuda")
    q[seq, local] = s["q"].float().unflatten(1, (Hk, group))
    # the prefix once for all, the sequences' pages one batch entry each
    pk, pv = (p[s["prefix_table"].long()].flatten(0, 1)[:P].float() for p in (s["k_pages"], s["v_pages"]))
    ok, ov = (p[s["table"].long().flatten()].unflatten(0, s["table"].shape).flatten(1, 2).float() for p in (s["k_pages"], s["v_pages"]))
    q_len = (s["indptr"][1:] - s["indptr"][:-1]).long()[:, None, None]
    key = torch.arange(width, device="cuda")[None, None]
    new = key - (s["kv_len"].long()[:, None, None] - q_len)  # the key's place among the new tokens, negative: older
    if s["mask"] is None:
        seen = new <= torch.arange(Q, device="cuda")[None, :, None]
    else:
        bits = torch.zeros((B, Q), dtype=torch.int64, device="cuda")
        bits[seq, local] = s["mask"]
        seen = (new < 0) | (((bits[:, :, None] >> new.clamp(0, 63)) & 1 == 1) & (new < 64))
    live = key < s["kv_len"].long()[:, None, None]
    seen = seen & live
    ov = torch.where(live[:, 0, :, None, None], ov, 0.0)
    q = q * (1.0 / math.sqrt(D))
    shared = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(Hk, B * Q * group, D), pk.permute(1, 2, 0))
    shared = shared.reshape(Hk, B, Q, group, P).permute(1, 0, 2, 3, 4).reshape(B, Hk, Q * group, P)
    each = torch.matmul(q.transpose(1, 2).reshape(B, Hk, Q * group, D), ok.permute(0, 2, 3, 1)).unflatten(2, (Q, group))
    each = each.masked_fill(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    score = torch.cat([shared, each], dim=-1)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    lse = (torch.log(total) + top)[..., 0]
    p = p / torch.where(total == 0, 1.0, total)
    left = p[..., :P].permute(1, 0, 2, 3).reshape(Hk, B * Q * group, P)
    out = torch.matmul(left, pv.permute(1, 0, 2)).reshape(Hk, B, Q * group, D).transpose(0, 1)
    out = out + torch.matmul(p[..., P:], ov.permute(0, 2, 1, 3))
    out = out.unflatten(2, (Q, group)).permute(0, 2, 1, 3, 4)[seq, local].flatten(1, 2)
    lse = lse.unflatten(2, (Q, group)).permute(0, 2, 1, 3)[seq, local].flatten(1, 2)
    return {"out": out.to(s["q"].dtype), "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if work(case)["flops"] > 1.5e12:
        return None
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    """Each pair is a complex number times e^(i angle), sequence by sequence."""
    case = s["case"]
    half, page = case["rot"] // 2, case["page"]
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    starts, lens, table = s["indptr"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
    turned_q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    even = list(range(0, case["rot"], 2)) if case["interleaved"] else list(range(half))
    odd = list(range(1, case["rot"], 2)) if case["interleaved"] else list(range(half, case["rot"]))

    def turn(x, unit):
        y = x.double().clone()
        z = torch.complex(y[..., even], y[..., odd]) * unit[:, None]
        y[..., even], y[..., odd] = z.real, z.imag
        return y

    for b, total in enumerate(lens):
        a, e = starts[b], starts[b + 1]
        first = total - (e - a)
        at = np.arange(first, total)
        angle = torch.empty((e - a, half), dtype=torch.float64, device="cuda")
        for i, f in enumerate(s["inv_freq"].tolist()):
            p = torch.from_numpy(at).cuda() + case["prefix"] if s["positions"] is None else s["positions"][int(s["axis"][i]), a:e]
            angle[:, i] = p * f
        unit = torch.polar(torch.ones_like(angle), angle)
        turned_q[a:e] = turn(s["q"][a:e], unit)
        pages = torch.tensor([table[b][i // page] for i in at.tolist()], device="cuda")
        slots = torch.from_numpy(at % page).cuda()
        k_pages[pages, slots] = turn(s["k"][a:e], unit)
        v_pages[pages, slots] = s["v"][a:e].double()
    return {"q": turned_q, "k_pages": k_pages, "v_pages": v_pages}


def _exact_attend(s):
    """One sequence and one key head at a time: the keys that a query may see, gathered into one line."""
    case = s["case"]
    page, P, group = case["page"], case["prefix"], case["Hq"] // case["Hk"]
    starts, lens = s["indptr"].tolist(), s["kv_len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    shared = torch.arange(P, device="cuda")
    shared = s["prefix_table"].long()[shared // page] * page + shared % page

    for b, total in enumerate(lens):
        a, e = starts[b], starts[b + 1]
        n = e - a
        line = torch.arange(total, device="cuda")
        line = torch.cat([shared, s["table"][b].long()[line // page] * page + line % page])
        seen = torch.ones((n, P + total), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            seen[:, P + total - n :] = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
        else:
            words = s["mask"][a:e].tolist()
            rows = [[(w >> j) & 1 == 1 if j < 64 else False for j in range(n)] for w in words]
            seen[:, P + total - n :] = torch.tensor(rows, device="cuda")
        for h in range(case["Hk"]):
            keys = s["k_pages"][line // page, line % page, h].double()
            values = s["v_pages"][line // page, line % page, h].double()
            for g in range(h * group, (h + 1) * group):
                score = s["q"][a:e, g].double() @ keys.T / math.sqrt(case["D"])
                score[~seen] = -math.inf
                norm = torch.logsumexp(score, dim=1)
                lse[a:e, g] = norm
                weight = torch.exp(score - norm[:, None])
                out[a:e, g] = torch.where((norm > -math.inf)[:, None], weight @ values, 0.0)
    return {"out": out, "lse": lse}
