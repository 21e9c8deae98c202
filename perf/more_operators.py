"""Cases of a decoder layer's attention: norms and rotation of the heads (rope), writing keys and values into a paged cache
in 8 bits (append), attention of a few query rows over that cache (cached) and causal attention over packed prompts (prompt).

Each case runs in a plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the package's
entry points. ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step of a 32-head model: the latency of rotating its heads, nothing else
        _rope("rope one token", tokens=1, hq=32, hkv=32, dim=128, dtype="f16"),
        # a decode batch, normed heads of which a part is rotated, neighbouring values paired
        _rope("rope decode batch, normed", tokens=96, hq=64, hkv=8, dim=128, rot=64, dtype="bf16", normed=True, interleaved=True),
        # a large prefill of images and text: positions in time, height and width, heads normed
        _rope("rope prefill, three axes", tokens=16384, hq=64, hkv=8, dim=128, dtype="bf16", normed=True, axes=3),
        # a decode step of 32 requests: a token each, most of them into pages that hold some already
        _append("append one token each", batch=32, new=1, held=2000, hkv=8, dim=128, page=64, dtype="bf16", ragged=True),
        # pieces of prompts of unlike lengths behind what the cache holds; heads of 48 values
        _append("append ragged pieces", batch=21, new=700, held=300, hkv=6, dim=48, page=16, dtype="f16", ragged=True),
        # whole prompts into an empty cache
        _append("append prompts", batch=4, new=4096, held=0, hkv=32, dim=128, page=64, dtype="bf16"),
        # one request of a 32-head model without shared heads: latency
        _cached("cached one request", batch=1, held=1003, n=1, hq=32, hkv=32, dim=128, page=64, dtype="f16"),
        # requests of unlike lengths, four tokens each that a draft proposed, eight query heads a key head
        _cached("cached ragged, four tokens", batch=48, held=8000, n=4, hq=64, hkv=8, dim=128, page=16, dtype="bf16", ragged=True),
        # a full decode batch of long requests: bound by reading the cache
        _cached("cached long batch", batch=128, held=8192, n=1, hq=64, hkv=8, dim=128, page=64, dtype="bf16"),
        # one short prompt: latency
        _prompt("prompt short", batch=1, longest=37, hq=32, hkv=32, dim=128, dtype="f16"),
        # prompts of unlike lengths packed into one batch, small heads
        _prompt("prompt packed, ragged", batch=9, longest=1900, hq=24, hkv=8, dim=64, dtype="bf16", ragged=True),
        # a long prompt: bound by the products
        _prompt("prompt long", batch=1, longest=8192, hq=64, hkv=8, dim=128, dtype="bf16"),
    ]


def _rope(name, tokens, hq, hkv, dim, dtype, rot=0, normed=False, interleaved=False, axes=1):
    return dict(name=name, op="rope", tokens=tokens, hq=hq, hkv=hkv, dim=dim, rot=rot or dim, dtype=dtype, normed=normed,
                interleaved=interleaved, axes=axes)


def _append(name, batch, new, held, hkv, dim, page, dtype, ragged=False, lens=1):
    return dict(name=name, op="append", batch=batch, new=new, held=held, hkv=hkv, dim=dim, page=page, dtype=dtype, ragged=ragged,
                lens=lens)


def _cached(name, batch, held, n, hq, hkv, dim, page, dtype, ragged=False, lens=1):
    return dict(name=name, op="cached", batch=batch, held=held, n=n, hq=hq, hkv=hkv, dim=dim, page=page, dtype=dtype, ragged=ragged,
                lens=lens)


def _prompt(name, batch, longest, hq, hkv, dim, dtype, ragged=False, lens=1):
    return dict(name=name, op="prompt", batch=batch, longest=longest, hq=hq, hkv=hkv, dim=dim, dtype=dtype, ragged=ragged, lens=lens)


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lengths(case, longest):
    """A length for each sequence, `longest` at most: alike, or spread over the logarithm with one of them the longest."""
    if not case["ragged"] or longest < 2:
        return [longest] * case["batch"]
    rng = random.Random(case["lens"])
    lens = [_spread(rng, 1, longest) for _ in range(case["batch"])]
    lens[rng.randrange(len(lens))] = longest
    return lens


def _held(case):
    """(tokens that the cache holds before, new tokens) of each sequence."""
    new = _lengths(case, case["new"])
    rng = random.Random(case["lens"] + 1)
    held = [_spread(rng, 1, case["held"]) if case["held"] else 0 for _ in new]
    return held, new


def draw(rng):
    op = rng.choice(("rope", "append", "cached", "prompt"))
    dtype = rng.choice(("f16", "bf16"))
    dim = rng.choice((48, 64, 80, 96, 128, 128))
    hkv = rng.choice((1, 2, 4, 6, 8, 8, 32))
    hq = hkv * rng.choice((1, 2, 3, 4, 8) if hkv <= 8 else (1, 2))
    page = rng.choice((16, 32, 64, 64, 128))
    ragged, lens = rng.random() < 0.6, rng.randrange(1 << 20)
    if op == "rope":
        case = _rope("", tokens=_spread(rng, 1, 16384 * 72 // max(72, hq + hkv)), hq=hq, hkv=hkv, dim=dim, rot=dim if rng.random() < 0.6 else 32,
                     dtype=dtype, normed=rng.random() < 0.6, interleaved=rng.random() < 0.3, axes=rng.choice((1, 1, 3)))
    elif op == "append":
        batch = _spread(rng, 1, 64)
        new = 1 if rng.random() < 0.3 else _spread(rng, 1, 4096 * 4 * 32 // (batch * max(hkv, 8)))
        case = _append("", batch=batch, new=new, held=rng.choice((0, 100, 2000)), hkv=hkv, dim=dim, page=page, dtype=dtype, ragged=ragged,
                       lens=lens)
    elif op == "cached":
        batch = _spread(rng, 1, 128)
        most = 128 * 8192 * 8 // (batch * hkv)  # no dearer than the largest listed case
        n = rng.choice((1, 1, 1, 2, 5))
        case = _cached("", batch=batch, held=_spread(rng, 16, max(16, min(65536, most))), n=n, hq=hq, hkv=hkv, dim=dim, page=page,
                       dtype=dtype, ragged=ragged, lens=lens)
    else:
        batch = _spread(rng, 1, 24)
        longest = _spread(rng, 1, 8192)
        longest = max(1, min(longest, int(math.sqrt(8192 * 8192 * 64 / (batch * max(hq, 8))))))
        case = _prompt("", batch=batch, longest=longest, hq=hq, hkv=hkv, dim=dim, dtype=dtype, ragged=ragged, lens=lens)
    del case["name"]
    return case


# ----------------------------------------------------------------------------------------------------------- inputs

def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _ints(values):
    return torch.tensor(values, device="cuda", dtype=torch.int32)


def _starts(lens):
    return _ints([sum(lens[:i]) for i in range(len(lens) + 1)])


def _heads(gen, tokens, heads, dim, dtype, std=1.0):
    """Keys or queries as a projection gives them: a few channels of each head stand out."""
    loud = 1 + 4 * (torch.rand((heads, dim), generator=gen, device="cuda") < 0.05)
    return (_normal(gen, (tokens, heads, dim), std) * loud).to(dtype)


def _pages(gen, lens, page):
    """The table of each sequence's pages, from a cache with a few pages to spare, and the cache's number of pages."""
    need = [-(-l // page) for l in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, device="cuda", dtype=torch.int32)
    live = torch.arange(table.shape[1], device="cuda") < _ints(need)[:, None]
    table[live] = order[: sum(need)]
    return table, total


def _cache(gen, total, case):
    """Codes and scales of a cache in use: values of normal distribution, scales within a factor of four."""
    shape = (total, case["hkv"], case["page"], case["dim"])
    codes = (_normal(gen, shape) * 100).clamp(-448, 448).to(F8)
    scale = torch.exp2(torch.randint(-8, -5, shape[:2], generator=gen, device="cuda").float())
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dtype, hkv, dim = DTYPES[case["dtype"]], case["hkv"], case["dim"]
    if case["op"] == "rope":
        T, half = case["tokens"], case["rot"] // 2
        # the fused projection's output, as the call takes it: queries and keys side by side in a row
        both = _heads(gen, T, case["hq"] + hkv, dim, dtype)
        s["q"], s["k"] = both[:, : case["hq"]], both[:, case["hq"]:]
        start = int(torch.randint(0, 100000, (1,), generator=gen, device="cuda"))
        p = start + torch.arange(T, device="cuda", dtype=torch.int32)
        if case["axes"] > 1:  # rows of a picture: time stands still, height and width go on
            p = torch.stack([torch.full_like(p, start), start + (p - start) // 96, start + (p - start) % 96])
        s["positions"] = p
        s["freqs"] = (10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        s["sections"] = _sections(case)
        for name in ("q", "k"):
            s[name + "_weight"] = (1 + _normal(gen, (dim,), 0.2)).to(dtype) if case["normed"] else None
    elif case["op"] == "append":
        held, new = _held(case)
        s["pages"], total = _pages(gen, [h + n for h, n in zip(held, new)], case["page"])
        s["k_cache"], s["k_scale"] = _cache(gen, total, case)
        s["v_cache"], s["v_scale"] = _cache(gen, total, case)
        s["k"], s["v"] = _heads(gen, sum(new), hkv, dim, dtype), _heads(gen, sum(new), hkv, dim, dtype, 0.5)
        s["cu"], s["held_lens"] = _starts(new), _ints(held)
    elif case["op"] == "cached":
        lens = [max(l, case["n"]) for l in _lengths(case, case["held"])]
        s["pages"], total = _pages(gen, lens, case["page"])
        s["k_cache"], s["k_scale"] = _cache(gen, total, case)
        s["v_cache"], s["v_scale"] = _cache(gen, total, case)
        s["q"] = _heads(gen, case["batch"] * case["n"], case["hq"], dim, dtype).view(case["batch"], case["n"], case["hq"], dim)
        s["kv_lens"] = _ints(lens)
    else:
        lens = _lengths(case, case["longest"])
        T = sum(lens)
        s["q"], s["k"] = _heads(gen, T, case["hq"], dim, dtype), _heads(gen, T, hkv, dim, dtype)
        s["v"] = _normal(gen, (T, hkv, dim)).to(dtype)
        s["cu"] = _starts(lens)
    return s


def _sections(case):
    """How many of the rotation's frequencies go by each axis: the first the fewest, the others alike."""
    half = case["rot"] // 2
    if case["axes"] == 1:
        return None
    part = 3 * half // 8
    return (half - 2 * part, part, part)


# -------------------------------------------------------------------------------------------------------- the passes

def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["op"]](s)


def _rope_own(s):
    import w4a16_group_quantized_gb300 as w4

    return w4.w4_qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6,
                              sections=s["sections"], interleaved=s["interleaved"])


def _append_own(s):
    import w4a16_group_quantized_gb300 as w4

    w4.w4_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["pages"], s["cu"], s["held_lens"])
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _cached_own(s):
    import w4a16_group_quantized_gb300 as w4

    if "workspace" not in s:  # a program keeps one for all its calls
        s["workspace"] = w4.Workspace("cuda")
    return w4.w4_kv_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["pages"], s["kv_lens"],
                              workspace=s["workspace"])


def _prompt_own(s):
    import w4a16_group_quantized_gb300 as w4

    return w4.w4_prompt_attention(s["q"], s["k"], s["v"], s["cu"])


def _rope_plain(s):
    rot, half = s["rot"], s["rot"] // 2
    p = s["positions"].view(s["axes"], -1)
    of = torch.arange(half, device="cuda")
    axis = torch.zeros_like(of) if s["axes"] == 1 else (of >= s["sections"][0]).long() + (of >= s["sections"][0] + s["sections"][1]).long()
    angle = p.t()[:, axis].double() * s["freqs"].double()  # far positions need the angle in 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    return _rotated(s["q"], s["q_weight"], cos, sin, rot, s["interleaved"]), _rotated(s["k"], s["k_weight"], cos, sin, rot, s["interleaved"])


def _rotated(x, weight, cos, sin, rot, interleaved):
    u = x.float()
    if weight is not None:
        u = u * torch.rsqrt((u * u).mean(dim=-1, keepdim=True) + 1e-6) * weight.float()
    part, rest = u[..., :rot], u[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = part[..., : rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, rest], dim=-1).to(x.dtype)


def _append_plain(s):
    page, B = s["page"], s["batch"]
    cu, held = s["cu"].long(), s["held_lens"].long()
    T = s["k"].shape[0]
    row = torch.arange(T, device="cuda")
    seq = torch.searchsorted(cu[1:], row, right=True)
    pos = held[seq] + row - cu[seq]
    at, slot = s["pages"][seq, pos // page].long(), pos % page
    # the page that each sequence goes on in, and how many rows of it stay
    kept = held % page
    last = s["pages"].gather(1, (held // page).clamp(max=s["pages"].shape[1] - 1)[:, None])[:, 0].long()
    going = (kept > 0) & (cu[1:] > cu[:-1])
    last = last.clamp(min=0)
    for x, codes, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        f = x.float()
        most = torch.zeros_like(scale).index_reduce_(0, at, f.abs().amax(dim=-1), "amax")
        m, e = torch.frexp(most)
        e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-100, 120)
        need = torch.exp2(torch.where(most > 0, e, torch.full_like(e, -100)).float())
        touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, at, True)
        old = torch.zeros_like(scale)
        old[last[going]] = scale[last[going]]
        new = torch.maximum(old, need)
        # rows that stay, in the page's new scale
        lg = last[going]
        stay = (torch.arange(page, device="cuda") < kept[going][:, None])[:, None, :, None]
        before = codes[lg].float()
        after = torch.where(stay, before * (old[lg] / new[lg])[:, :, None, None], before).to(F8)
        codes.view(torch.uint8)[lg] = after.view(torch.uint8)
        codes.view(torch.uint8)[at, :, slot] = (f / new[at][:, :, None]).to(F8).view(torch.uint8)
        scale[touched] = new[touched]
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _cached_plain(s):
    B, n, hkv, dim, page = s["batch"], s["n"], s["hkv"], s["dim"], s["page"]
    r = s["hq"] // hkv
    pages = s["pages"].long().clamp(min=0)
    L = pages.shape[1] * page

    def values(codes, scale):  # [B, hkv, L, dim]
        return (codes[pages].float() * scale[pages][..., None, None]).transpose(1, 2).reshape(B, hkv, L, dim)

    q = s["q"].float().view(B, n, hkv, r, dim).permute(0, 2, 1, 3, 4).reshape(B, hkv, n * r, dim)
    w = torch.matmul(q, values(s["k_cache"], s["k_scale"]).transpose(2, 3)) / math.sqrt(dim)
    last = s["kv_lens"][:, None] - n + torch.arange(n, device="cuda")
    seen = torch.arange(L, device="cuda") <= last[:, :, None]  # [B, n, L]
    w = w.masked_fill(~seen[:, None, :, None].expand(B, 1, n, r, L).reshape(B, 1, n * r, L), -math.inf)
    w = torch.exp(w - w.amax(dim=-1, keepdim=True))
    v = values(s["v_cache"], s["v_scale"]).masked_fill((torch.arange(L, device="cuda") >= s["kv_lens"][:, None])[:, None, :, None], 0)
    o = torch.matmul(w, v) / w.sum(dim=-1, keepdim=True)
    return o.view(B, hkv, n, r, dim).permute(0, 2, 1, 3, 4).reshape(B, n, s["hq"], dim).to(s["q"].dtype)


def _prompt_plain(s):
    hkv, dim, B = s["hkv"], s["dim"], s["batch"]
    r = s["hq"] // hkv
    T = s["q"].shape[0]
    L = s["longest"]
    cu = s["cu"].long()
    i = torch.arange(L, device="cuda")
    live = i < (cu[1:] - cu[:-1])[:, None]  # [B, L]
    rows = (cu[:-1, None] + i).clamp(max=T - 1)
    q = s["q"].float()[rows].view(B, L, hkv, r, dim).permute(0, 2, 3, 1, 4).reshape(B, hkv, r * L, dim)
    k, v = s["k"].float()[rows].transpose(1, 2), s["v"].float()[rows].transpose(1, 2)
    w = torch.matmul(q, k.transpose(2, 3)).mul_(1 / math.sqrt(dim)).view(B, hkv, r, L, L)
    w.masked_fill_(i[None, :] > i[:, None], -math.inf)
    w.sub_(w.amax(dim=-1, keepdim=True)).exp_()
    l = w.sum(dim=-1)
    o = torch.matmul(w.view(B, hkv, r * L, L), v).view(B, hkv, r, L, dim) / l[..., None]
    return o.permute(0, 3, 1, 2, 4).reshape(B, L, s["hq"], dim)[live].to(s["q"].dtype)


_RUN_OWN = {"rope": _rope_own, "append": _append_own, "cached": _cached_own, "prompt": _prompt_own}
_RUN_PLAIN = {"rope": _rope_plain, "append": _append_plain, "cached": _cached_plain, "prompt": _prompt_plain}


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    hkv, dim = case["hkv"], case["dim"]
    if case["op"] == "rope":
        values = case["tokens"] * (case["hq"] + hkv) * dim
        return {"bytes": 4 * values + 4 * case["axes"] * case["tokens"], "flops": 9 * values}
    if case["op"] == "append":
        held, new = _held(case)
        values = 2 * sum(new) * hkv * dim
        pages = sum(-(-(h % case["page"] + n) // case["page"]) for h, n in zip(held, new))
        return {"bytes": 3 * values + 8 * pages * hkv, "flops": 3 * values}
    if case["op"] == "cached":
        lens = [max(l, case["n"]) for l in _lengths(case, case["held"])]
        rows = case["batch"] * case["n"] * case["hq"] * dim
        scales = 8 * sum(-(-l // case["page"]) for l in lens) * hkv
        return {"bytes": 2 * sum(lens) * hkv * dim + scales + 4 * rows, "flops": 4 * sum(lens) * case["n"] * case["hq"] * dim}
    lens = _lengths(case, case["longest"])
    return {"bytes": 4 * sum(lens) * (case["hq"] + hkv) * dim, "flops": 2 * dim * case["hq"] * sum(l * (l + 1) for l in lens)}


# ---------------------------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope_exact, "append": _append_exact, "cached": _cached_exact, "prompt": _prompt_exact}[case["op"]](s)


def _rope_exact(s):
    half = s["rot"] // 2
    p = s["positions"].reshape(s["axes"], -1).double()
    parts, start = [], 0
    for axis, count in enumerate(s["sections"] or (half,)):
        parts.append(p[axis][:, None] * s["freqs"][start:start + count].double())
        start += count
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), torch.cat(parts, dim=1))[:, None]
    outs = []
    for name in ("q", "k"):
        x = s[name].double()
        if s[name + "_weight"] is not None:
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s[name + "_weight"].double()
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.complex(x[..., first], x[..., second]) * turn
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _append_exact(s):
    held, new = _held(s)
    page, start = s["page"], 0
    cut = {}
    table = s["pages"].tolist()
    for b, (h, n) in enumerate(zip(held, new)):
        while n > 0:
            take = min(n, page - h % page)
            cut[table[b][h // page]] = (h % page, start, take)
            start, h, n = start + take, h + take, n - take
    at = torch.tensor(list(cut), device="cuda")
    off, first, take = (torch.tensor(c, device="cuda")[:, None] for c in zip(*cut.values()))
    slot = torch.arange(page, device="cuda")
    fresh, stay = (slot >= off) & (slot < off + take), slot < off
    rows = (first + slot - off).clamp(0, s["k"].shape[0] - 1)
    powers = torch.tensor([2.0 ** e for e in range(-100, 121)], device="cuda", dtype=torch.float64)
    outs = []
    for name in ("k", "v"):
        codes, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        x = torch.where(fresh[..., None, None], s[name][rows].double(), 0.0).transpose(1, 2)  # [pages, heads, page, dim]
        most = x.abs().amax(dim=(2, 3))
        need = powers[torch.searchsorted(448 * powers, most).clamp(max=220)]
        new_scale = torch.where(off > 0, torch.maximum(scale[at], need), need)
        moved = (codes[at] * (scale[at] / new_scale)[..., None, None]).float().to(F8).double()
        filled = (x / new_scale[..., None, None]).float().to(F8).double()
        mine = torch.where(fresh[:, None, :, None], filled, torch.where(stay[:, None, :, None], moved, codes[at]))
        codes[at], scale[at] = mine, new_scale
        outs.append((codes, scale))
    return outs[0][0], outs[1][0], outs[0][1], outs[1][1]


def _softmax_rows(q, k, v, seen):
    """Each row of q [h, rows, d] over the keys that it sees."""
    w = torch.einsum("hrd,hkd->hrk", q, k) / math.sqrt(q.shape[-1])
    w = torch.softmax(w.masked_fill(~seen, -math.inf), dim=-1)
    return torch.einsum("hrk,hkd->hrd", w, v)


def _cached_exact(s):
    hkv, n, page = s["hkv"], s["n"], s["page"]
    r = s["hq"] // hkv
    y = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    for b, length in enumerate(s["kv_lens"].tolist()):
        at = s["pages"][b, : -(-length // page)].long()
        k, v = ((s[m + "_cache"][at].double() * s[m + "_scale"][at].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :length]
                for m in ("k", "v"))
        q = s["q"][b].double().reshape(n, hkv, r, -1).permute(1, 0, 2, 3).flatten(1, 2)
        j = torch.arange(n, device="cuda").repeat_interleave(r)[:, None]
        o = _softmax_rows(q, k, v, torch.arange(length, device="cuda") <= length - n + j)
        y[b] = o.view(hkv, n, r, -1).permute(1, 0, 2, 3).flatten(1, 2)
    return y


def _prompt_exact(s):
    y = torch.zeros(s["q"].shape, device="cuda", dtype=torch.float64)
    r = s["hq"] // s["hkv"]
    cu = s["cu"].tolist()
    for a, z in zip(cu[:-1], cu[1:]):
        seen = torch.ones((z - a, z - a), dtype=torch.bool, device="cuda").tril()
        for h in range(s["hkv"]):
            q = s["q"][a:z, h * r:(h + 1) * r].double().transpose(0, 1)
            k, v = (s[m][a:z, h].double().expand(r, -1, -1) for m in ("k", "v"))
            y[a:z, h * r:(h + 1) * r] = _softmax_rows(q, k, v, seen).transpose(0, 1)
    return y
