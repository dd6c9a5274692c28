"""Cases of the 8-bit paged cache and of the append with norms, their plain forms, and their calls.

A target model verifies gamma + 1 drafted positions of every sequence in one
forward pass.  Where it normalises each head of its queries and keys, that is
done in the pass that rotates and appends them (spec_kv_append_norm).  A cache
of codes in 8 bits (e4m3, a power-of-two scale for each block of entries and
head) holds twice the entries and is read in half the time: spec_kv_append8
fills it, spec_prefix_attention8 attends to it, spec_kv_read8 gives entries
back in 16 bits.

``own`` selects between the plain form (elementary torch operations in 32
bits, angles in 64) and the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# exponents of a block's scale: what a code stands for is a number of the type
_EXPONENTS = {"bf16": (-100, 120), "fp16": (-15, 8)}


def _case(op, name, **kw):
    case = dict(name=name, op=op, dtype="bf16", B=1, q=1, ragged=False, Hq=32, Hk=8, D=128, page=16, heads_first=False,
                suffix=64, prefix=0)
    if op != "norm":
        case["block"] = 16
    if op in ("norm", "append"):
        case.update(rot=case["D"], axes=1, interleaved=False)
    if op == "append":
        case["norm"] = True
    if op == "attend":
        case["mask"] = False
    case.update(kw)
    return case


def listed():
    return [
        # the verify pass of a served batch: 32 sequences x (gamma = 4) + 1, a 16-bit cache
        _case("norm", "norm_verify_b32", B=32, q=5, page=64, suffix=1024, prefix=8192),
        # prompts entering a 16-bit cache: bandwidth
        _case("norm", "norm_prompts_d256", B=8, q=4096, Hq=16, Hk=8, D=256, rot=256, page=64, heads_first=True, suffix=4096),
        # one user's plain decode step: one token, a launch's latency
        _case("append", "append8_one", suffix=1000, prefix=512),
        # drafts of different lengths, seven query heads a key head, a part of
        # each head rotated in neighbouring pairs, pages of no power of two, no norms
        _case("append", "append8_ragged_d64", dtype="fp16", B=48, q=9, ragged=True, Hq=28, Hk=4, D=64, rot=32,
              interleaved=True, page=24, block=8, suffix=777, norm=False),
        # prompts entering the cache: bandwidth
        _case("append", "append8_prompts", B=8, q=4097, ragged=True, Hq=32, Hk=8, page=64, heads_first=True, suffix=4500),
        # one sequence's entries for a cache of 16 bits
        _case("read", "read8_one_d64", dtype="fp16", q=0, Hq=4, Hk=4, D=64, page=24, block=8, suffix=777),
        # a batch's caches taken out: bandwidth
        _case("read", "read8_batch", B=16, q=0, ragged=True, Hq=8, page=64, block=32, heads_first=True, suffix=32768),
        # one user's plain decode step behind a system prompt: latency
        _case("attend", "attend8_one", prefix=512, suffix=37),
        # the verify pass of a served batch behind a shared system prompt
        _case("attend", "attend8_verify_b32", B=32, q=5, ragged=True, prefix=8192, suffix=1024),
        # long conversations with nothing shared: the cache's bytes bound it
        _case("attend", "attend8_long_caches", B=16, q=5, ragged=True, page=64, heads_first=True, suffix=32768),
        # long drafts and a long shared document: matrix products bound it
        _case("attend", "attend8_longdraft_b128", B=128, q=9, ragged=True, page=64, block=64, prefix=32768, suffix=2048),
        # several draft candidates a sequence in one pass, told apart by the mask
        _case("attend", "attend8_candidates_d64", dtype="fp16", B=24, q=12, Hq=28, Hk=4, D=64, page=24, block=8,
              prefix=2051, suffix=611, ragged=True, mask=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_OPS = ("norm", "append", "read", "attend")


def draw(rng):
    largest = {op: [max(_cost(c)[k] for c in listed() if c["op"] == op) for k in range(3)] for op in _OPS}
    while True:
        op = rng.choice(["norm", "append", "append", "read", "attend", "attend", "attend"])
        hk = rng.choice([1, 2, 3, 4, 5, 8, 16])
        group = 1 if op == "read" else rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), B=_log_int(rng, 1, 128), Hk=hk, Hq=hk * group,
                    ragged=rng.random() < 0.75, heads_first=rng.random() < 0.4, D=rng.choice([64, 128]),
                    page=rng.choice([8, 16, 24, 32, 40, 64, 128, 256]), prefix=0)
        if op != "norm":
            case["block"] = rng.choice([b for b in (8, 16, 32, 64) if case["page"] % b == 0])
        if op in ("norm", "append"):
            if rng.random() < 0.25:
                case["D"] = 256
            case.update(axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4, q=_log_int(rng, 1, 4096),
                        prefix=rng.choice([0, 0, _log_int(rng, 1, 100000)]))
            case["rot"] = rng.choice([case["D"], case["D"] // 2, 2 * rng.randint(1, case["D"] // 2)])
            case["suffix"] = case["q"] + _log_int(rng, 1, 4096) - 1
            if op == "append":
                case["norm"] = rng.random() < 0.7
        elif op == "read":
            case.update(q=0, suffix=_log_int(rng, 1, 32768))
        else:
            case["mask"] = rng.random() < 0.3
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
    q = [rng.randint(min(1, case["q"]), case["q"]) for _ in range(case["B"])]
    return q, [rng.randint(max(1, n), case["suffix"]) for n in q]


def work(case):
    q, kv = _lengths(case)
    n, Hq, Hk, D = sum(q), case["Hq"], case["Hk"], case["D"]
    if case["op"] in ("norm", "append"):
        # q in and out in 16 bits, k and v in 16, out in 16 or in 8 with their blocks' scales
        size = 2 if case["op"] == "norm" else 1
        scales = 0 if case["op"] == "norm" else 2 * Hk * sum(-(-x // case["block"]) for x in q)
        moved = n * (Hq * 4 + 2 * Hk * (2 + size)) * D + scales + n * 4 * (case["axes"] if case["axes"] > 1 else 0)
        norm = 4 * n * (Hq + Hk) * D if case.get("norm", True) else 0
        return {"bytes": moved, "flops": 6 * n * (Hq + Hk) * (case["rot"] // 2) + norm}
    blocks = sum(-(-x // case["block"]) for x in kv) + -(-case["prefix"] // case["block"])
    cached = ((case["prefix"] + sum(kv)) * D + blocks) * Hk * 2
    if case["op"] == "read":
        return {"bytes": cached + sum(kv) * Hk * D * 2 * 2, "flops": sum(kv) * Hk * D * 2}
    # new positions see every older one; among themselves the causal half, or
    # under a mask at most that
    pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, kv)) + n * case["prefix"]
    return {"bytes": cached + 2 * n * Hq * D * 2 + 4 * n * Hq, "flops": 4 * pairs * Hq * D}


def _cost(case):
    """What bounds a drawn case: bytes, operations, and the plain form's largest table of scores (padded to the longest sequence)."""
    w = work(case)
    q, kv = _lengths(case)
    table = {"attend": case["B"] * max(q) * case["Hq"] * (case["prefix"] + max(kv)), "read": case["B"] * max(kv)}.get(case["op"], sum(q))
    return w["bytes"], w["flops"], table


def _two(exponent):
    """2^exponent exactly, which a power function on the GPU may miss: fp32 by its bits."""
    return ((exponent.int() + 127) << 23).view(torch.float32)


def _codes(x, exponent):
    """e4m3 codes of x at scales 2^exponent; what has no finite value is NaN."""
    return (x * _two(-exponent)).to(torch.float8_e4m3fn)


def _pages(case, gen):
    """Pages dealt in random order: the pools of 16 bits, or of codes and their scales; the sequences' table and the prefix's."""
    _, kv = _lengths(case)
    page, Hk, D = case["page"], case["Hk"], case["D"]
    width = max(-(-n // page) for n in kv)
    shared = -(-case["prefix"] // page) if case["op"] == "attend" else 0
    total = case["B"] * width + shared + 3
    order = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int32)
    shape = (total, Hk, page, D) if case["heads_first"] else (total, page, Hk, D)
    state = {}
    for x in "kv":
        pool = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        if case["op"] == "norm":
            pool = pool.to(_DTYPES[case["dtype"]])
        else:
            # an entry's length differs from its neighbours'
            entry = torch.exp2(torch.rand(shape[:3] + (1,), generator=gen, device="cuda") * 3 - 2)
            pool = (pool * entry).transpose(1, 2) if case["heads_first"] else pool * entry
            pool = pool.unflatten(1, (page // case["block"], case["block"]))
            top = torch.frexp(pool.abs().amax(dim=(2, 4)))[1] - 8  # [pages, blocks, heads]
            state[x + "_scales"] = (top + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
            pool = _codes(pool, top[:, :, None, :, None]).flatten(1, 2)
            pool = pool.transpose(1, 2).contiguous() if case["heads_first"] else pool.contiguous()
        state[x + "_pages"] = pool.transpose(1, 2) if case["heads_first"] else pool  # seen as [pages, slots, heads, D] either way
    return dict(state, table=order[: case["B"] * width].reshape(case["B"], width).contiguous(),
                prefix_table=order[total - shared :].contiguous())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q_len, kv_len = _lengths(case)
    n, Hq, Hk, D, dt = sum(q_len), case["Hq"], case["Hk"], case["D"], _DTYPES[case["dtype"]]
    indptr = torch.tensor([0] + q_len, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
    lens = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    state = dict(_pages(case, gen), case=case, indptr=indptr, kv_len=lens, q_max=max(q_len), kept={})
    if case["op"] == "read":
        rows = sum(kv_len)
        state["out_indptr"] = torch.tensor([0] + kv_len, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        state["k_out"] = torch.empty((rows, Hk, D), dtype=dt, device="cuda")
        state["v_out"] = torch.empty((rows, Hk, D), dtype=dt, device="cuda")
        return state
    if case["op"] != "attend":
        # q, k and v lie side by side in the output of one projection
        qkv = 3 * torch.randn((n, (Hq + 2 * Hk) * D), generator=gen, device="cuda")
        qkv = (qkv * torch.exp2(torch.rand((n, 1), generator=gen, device="cuda") * 3 - 2)).to(dt)
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
        state["q_weight"] = state["k_weight"] = None
        if case.get("norm", True):
            state["q_weight"], state["k_weight"] = (0.5 + torch.rand(D, generator=gen, device="cuda") for _ in "qk")
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


_EPS = 1e-6


def run(state):
    if own:
        return _call(state)
    return {"norm": _plain_append, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[state["case"]["op"]](state)


def _call(s):
    import speculative_decoding_verification_54_gb300 as sv

    case, kept = s["case"], s["kept"]
    if not kept:  # what a program makes once for its cache
        if case["op"] == "norm":
            kept["cache"] = sv.make_kv_cache(s["k_pages"], s["v_pages"])
        else:
            kept["cache"] = sv.make_kv_cache8(s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], _DTYPES[case["dtype"]])
        kept["ws"] = (sv.make_attention_workspace(case["B"], s["q"].shape[0], case["Hq"], case["D"]) if case["op"] == "attend"
                      else sv.make_append_workspace())
    if case["op"] in ("norm", "append"):
        call = sv.spec_kv_append_norm if case["op"] == "norm" else sv.spec_kv_append8
        call(kept["cache"], s["q"], s["k"], s["v"], s["q_out"], s["indptr"], s["table"], s["kv_len"], kept["ws"],
             inv_freq=s["inv_freq"], positions=s["positions"], axis=s["axis"], interleaved=case["interleaved"],
             position_base=case["prefix"], q_weight=s["q_weight"], k_weight=s["k_weight"], norm_eps=_EPS)
        return _filled(s, s["q_out"])
    if case["op"] == "read":
        sv.spec_kv_read8(kept["cache"], s["k_out"], s["v_out"], s["out_indptr"], s["table"], kept["ws"])
        return {"k": s["k_out"], "v": s["v_out"]}
    sv.spec_prefix_attention8(kept["cache"], s["q"], s["out"], s["indptr"], s["table"], s["kv_len"], kept["ws"],
                              prefix_table=s["prefix_table"], prefix_len=case["prefix"], draft_mask=s["mask"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _filled(s, q):
    names = ["k_pages", "v_pages"] + (["k_scales", "v_scales"] if "k_scales" in s else [])
    return {"q": q, **{name: s[name] for name in names}}


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

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + _EPS) * weight
        head, rest = x[..., : case["rot"]], x[..., case["rot"] :]
        if case["interleaved"]:
            a, b = head[..., 0::2], head[..., 1::2]
            new = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
        else:
            a, b = head.chunk(2, dim=-1)
            new = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
        return torch.cat([new, rest], dim=-1)

    q = turned(s["q"], s["q_weight"]).to(s["q"].dtype)
    page = s["table"].long()[seq, slot // case["page"]]
    if case["op"] == "norm":
        s["k_pages"][page, slot % case["page"]] = turned(s["k"], s["k_weight"]).to(s["q"].dtype)
        s["v_pages"][page, slot % case["page"]] = s["v"]
    else:
        _plain_quantise(s, "k", turned(s["k"], s["k_weight"]), page, slot)
        _plain_quantise(s, "v", s["v"].float(), page, slot)
    return _filled(s, q)


def _plain_quantise(s, name, x, page, slot):
    """x [n, heads, D] into the codes at (page, slot); the blocks' scales; older entries of the blocks that get a larger scale."""
    case, block, (low, high) = s["case"], s["case"]["block"], _EXPONENTS[s["case"]["dtype"]]
    codes, scales = s[name + "_pages"].view(torch.uint8), s[name + "_scales"].view(torch.uint8)
    most = math.ldexp(240.0, high)
    finite = torch.isfinite(x)
    top = torch.where(finite, x, 0.0).abs().amax(dim=-1).clamp(max=most)  # [n, heads]
    per_page = scales.shape[1]
    where = page * per_page + slot % case["page"] // block
    new = torch.zeros((scales.shape[0] * per_page, scales.shape[2]), device="cuda")
    new = new.scatter_reduce(0, where[:, None].expand(top.shape), top, "amax")
    exponent = torch.where(new > 0, torch.frexp(new)[1] - 8, low).clamp(low, high).int().reshape(scales.shape)
    # a sequence's first new entry may stand behind older ones of its block
    q_len = (s["indptr"][1:] - s["indptr"][:-1]).long()
    first = s["kv_len"].long() - q_len
    behind = ((first % block) != 0) & (q_len > 0)
    at_page = s["table"].long().gather(1, (first // case["page"]).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    at_block = first % case["page"] // block
    was = scales[at_page, at_block].int() - 127  # [B, heads]
    now = torch.where(behind[:, None], torch.maximum(was, exponent[at_page, at_block]), exponent[at_page, at_block])
    lanes = torch.arange(block, device="cuda")
    in_page = at_block[:, None] * block + lanes  # [B, block]
    old = codes[at_page[:, None], in_page]  # [B, block, heads, D]
    less = _codes(old.view(torch.float8_e4m3fn).float(), (now - was)[:, None, :, None]).view(torch.uint8)
    older = (behind[:, None] & (lanes < (first % block)[:, None]))[:, :, None, None] & (now > was)[:, None, :, None]
    touched = q_len > 0
    codes[at_page[touched][:, None], in_page[touched]] = torch.where(older, less, old)[touched]
    exponent[at_page[touched], at_block[touched]] = now[touched]
    scales.view(-1, scales.shape[2])[where] = (exponent.view(-1, scales.shape[2])[where] + 127).to(torch.uint8)
    x = torch.where(finite, x.clamp(-most, most), math.nan)
    codes[page, slot % case["page"]] = _codes(x, exponent.view(-1, scales.shape[2])[where][:, :, None]).view(torch.uint8)


def _values(s, name, pages):
    """The values of whole pages [..., page, heads, D] in 32 bits."""
    codes = s[name + "_pages"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float()
    exponent = s[name + "_scales"].view(torch.uint8)[pages].int() - 127
    return codes * _two(exponent.repeat_interleave(s["case"]["block"], dim=-2)[..., None])


def _plain_read(s):
    live = torch.arange(s["table"].shape[1] * s["case"]["page"], device="cuda")[None] < s["kv_len"][:, None]
    return {x: _values(s, x, s["table"].long()).flatten(1, 2)[live].to(s[x + "_out"].dtype) for x in "kv"}


def _plain_attend(s):
    case = s["case"]
    B, Hk, D, Q, P = case["B"], case["Hk"], case["D"], s["q_max"], case["prefix"]
    group = case["Hq"] // Hk
    seq, local, slot = _rows(s)
    width = s["table"].shape[1] * case["page"]
    q = torch.zeros((B, Q, Hk, group, D), dtype=torch.float32, device="cuda")
    q[seq, local] = s["q"].float().unflatten(1, (Hk, group))
    # the prefix once for all, the sequences' pages one batch entry each
    pk, pv = (_values(s, x, s["prefix_table"].long()).flatten(0, 1)[:P] for x in "kv")
    ok, ov = (_values(s, x, s["table"].long()).flatten(1, 2) for x in "kv")
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
    return {"norm": _exact_append, "append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _code_values():
    """The finite values of e4m3 that are not negative, in order of their codes: 3 bits of fraction, 4 of exponent, a bias of 7."""
    return torch.tensor([(i % 8 / 8 + (i >= 8)) * 2.0 ** (max(i // 8, 1) - 7) for i in range(127)], dtype=torch.float64, device="cuda")


def _nearest_code(x):
    """x in 64 bits to the nearest value of e4m3, ties to the even code."""
    grid = _code_values()
    between = (grid[1:] + grid[:-1]) / 2
    above = torch.bucketize(x.abs(), between, right=False)  # a tie goes down ...
    tie = (x.abs() == between[above.clamp(max=125)]) & (above % 2 == 1)
    return torch.where(torch.isfinite(x), torch.copysign(grid[(above + tie.long()).clamp(max=126)], x), math.nan)


def _power(exponent):
    """2^exponent exactly, in 64 bits."""
    return ((exponent.long() + 1023) << 52).view(torch.float64)


def _exponent(x):
    """The exponent of positive numbers in 64 bits."""
    return (x.contiguous().view(torch.int64) >> 52) - 1023


def _exact_append(s):
    """Each pair is a complex number times e^(i angle), sequence by sequence."""
    case = s["case"]
    half, page = case["rot"] // 2, case["page"]
    starts, lens, table = s["indptr"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
    turned_q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    even = list(range(0, case["rot"], 2)) if case["interleaved"] else list(range(half))
    odd = list(range(1, case["rot"], 2)) if case["interleaved"] else list(range(half, case["rot"]))
    pools = {x: s[x + "_pages"].double() for x in "kv"}
    scales = {x: _power(s[x + "_scales"].view(torch.uint8).long() - 127) for x in "kv" if x + "_scales" in s}

    def turn(x, unit, weight):
        y = x.double().clone()
        if weight is not None:
            y = y / (y.square().mean(-1, keepdim=True) + _EPS).sqrt() * weight.double()
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
        turned_q[a:e] = turn(s["q"][a:e], unit, s["q_weight"])
        pages = torch.tensor([table[b][i // page] for i in at.tolist()], device="cuda")
        slots = torch.from_numpy(at % page).cuda()
        new = {"k": turn(s["k"][a:e], unit, s["k_weight"]), "v": s["v"][a:e].double()}
        for x in "kv":
            if case["op"] == "norm":
                pools[x][pages, slots] = new[x]
            else:
                _exact_blocks(case, pools[x], scales[x], new[x], table[b], first)
    out = {"q": turned_q, **{x + "_pages": pools[x] for x in "kv"}}
    return {**out, **{x + "_scales": scales[x] for x in scales}}


def _exact_blocks(case, pool, scales, new, pages, first):
    """One sequence's new entries, its blocks side by side: the block that the first of them falls into is filled up with older ones."""
    block, (low, high) = case["block"], _EXPONENTS[case["dtype"]]
    lead, total = first % block, first + len(new)
    count = -(-(lead + len(new)) // block)
    x = torch.zeros((count * block,) + new.shape[1:], dtype=torch.float64, device="cuda")
    x[lead : lead + len(new)] = new
    x = x.unflatten(0, (count, block))
    top = x.abs().amax(dim=(1, 3))
    exponent = torch.where(top > 0, _exponent(top) - 7, low).clamp(low, high)
    entry = first - lead + torch.arange(count * block, device="cuda")
    page = torch.tensor(pages, device="cuda")[(entry // case["page"]).clamp(max=len(pages) - 1)].unflatten(0, (count, block))
    slot = (entry % case["page"]).unflatten(0, (count, block))
    if lead:
        was = scales[page[0, 0], slot[0, 0] // block]
        exponent[0] = torch.maximum(exponent[0], _exponent(was))
        older = pool[page[0, :lead], slot[0, :lead]]
        pool[page[0, :lead], slot[0, :lead]] = _nearest_code(older * (was / _power(exponent[0]))[None, :, None])
    scales[page[:, 0], slot[:, 0] // block] = _power(exponent)
    code = _nearest_code(x / _power(exponent)[:, None, :, None]).flatten(0, 1)[lead : lead + len(new)]
    pool[page.flatten()[lead : total - first + lead], slot.flatten()[lead : total - first + lead]] = code


def _entries(s, name, pages, line, head):
    """Entries of one key head in 64 bits: line [n] of places in `pages`."""
    page, block = s["case"]["page"], s["case"]["block"]
    code = s[name + "_pages"][pages[line // page], line % page, head].double()
    scale = s[name + "_scales"].view(torch.uint8)[pages[line // page], line % page // block, head].long()
    return code * _power(scale - 127)[:, None]


def _exact_read(s):
    case = s["case"]
    out = {x: torch.empty(s["k_out"].shape, dtype=torch.float64, device="cuda") for x in "kv"}
    starts = s["out_indptr"].tolist()
    for b, total in enumerate(s["kv_len"].tolist()):
        line = torch.arange(total, device="cuda")
        for h in range(case["Hk"]):
            for x in "kv":
                out[x][starts[b] : starts[b + 1], h] = _entries(s, x, s["table"][b].long(), line, h)
    return out


def _exact_attend(s):
    """One sequence and one key head at a time: the keys that a query may see, gathered into one line."""
    case = s["case"]
    page, P, group = case["page"], case["prefix"], case["Hq"] // case["Hk"]
    starts, lens = s["indptr"].tolist(), s["kv_len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    whole = -(-P // page)

    for b, total in enumerate(lens):
        a, e = starts[b], starts[b + 1]
        n = e - a
        pages = torch.cat([s["prefix_table"].long(), s["table"][b].long()])
        line = torch.cat([torch.arange(P, device="cuda"), whole * page + torch.arange(total, device="cuda")])
        seen = torch.ones((n, P + total), dtype=torch.bool, device="cuda")
        if s["mask"] is None:
            seen[:, P + total - n :] = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()
        else:
            words = s["mask"][a:e].tolist()
            rows = [[(w >> j) & 1 == 1 if j < 64 else False for j in range(n)] for w in words]
            seen[:, P + total - n :] = torch.tensor(rows, device="cuda")
        for h in range(case["Hk"]):
            keys, values = _entries(s, "k", pages, line, h), _entries(s, "v", pages, line, h)
            for g in range(h * group, (h + 1) * group):
                score = s["q"][a:e, g].double() @ keys.T / math.sqrt(case["D"])
                score[~seen] = -math.inf
                norm = torch.logsumexp(score, dim=1)
                lse[a:e, g] = norm
                weight = torch.exp(score - norm[:, None])
                out[a:e, g] = torch.where((norm > -math.inf)[:, None], weight @ values, 0.0)
    return {"out": out, "lse": lse}
