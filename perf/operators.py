"""Cases of the operators whose weights are chosen row by row: the router of a mixture of experts (route), the experts'
W4A16 products (experts) and the low-rank adapters of many requests beside a shared projection (lora).

Each case runs in a plain form (elementary torch operations in 32 bits) or, with ``own`` set, through the package's
entry points. ``exact`` is the definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a decode step: the router's latency, nothing else
        _route("route one token", tokens=1, experts=64, k=8, dtype="bf16"),
        # a decode batch: sigmoid scores, a balance bias, 4 of 8 groups kept by the sum of their two best
        _route("route decode batch, groups", tokens=64, experts=256, k=8, dtype="f32", sigmoid=True, bias=True, groups=8,
               top_groups=4, group_top=2, scale=2.5),
        # a ragged prefill chunk: an expert count that is no power of two, some experts masked, weights left as they are
        _route("route ragged, masked", tokens=5003, experts=60, k=6, dtype="f16", renormalize=False, masked=True),
        # a large prefill: the most rows and scores
        _route("route prefill, groups", tokens=16384, experts=256, k=8, dtype="bf16", sigmoid=True, bias=True, groups=8,
               top_groups=4, group_top=2),
        # one request with an adapter on a 4096 x 4096 projection
        _lora("lora one token", tokens=1, k=4096, n=4096, rank=16, adapters=16, dtype="f16"),
        # a decode batch of many requests on the fused 12288 x 4096 projection, adapters of unlike ranks
        _lora("lora decode batch, mixed ranks", tokens=96, k=4096, n=12288, rank=64, adapters=32, dtype="bf16", mixed=True),
        # a ragged mixture of prefill pieces; some rows have no adapter; odd output width
        _lora("lora ragged", tokens=1501, k=4000, n=4099, rank=24, adapters=7, dtype="bf16", none=0.2, runs=True),
        # a large prefill of a few requests on the 10240 x 8192 projection
        _lora("lora prefill", tokens=8192, k=8192, n=10240, rank=32, adapters=8, dtype="bf16", runs=True),
        # one token of a decode step through many small experts: 8 experts' weights
        _experts("experts one token", tokens=1, hidden=2048, inter=1024, experts=64, k=8, g=128, dtype="bf16"),
        # a decode batch through a few large experts: every expert's weights, a handful of rows each
        _experts("experts decode batch, large", tokens=16, hidden=4096, inter=11008, experts=8, k=2, g=128, dtype="f16"),
        # a ragged batch: sizes that end inside tiles and groups, some choices dropped (id -1)
        _experts("experts ragged, dropped", tokens=333, hidden=4000, inter=1352, experts=60, k=6, g=64, dtype="bf16", none=0.05),
        # a large prefill: bound by the products
        _experts("experts prefill", tokens=4096, hidden=2048, inter=1024, experts=64, k=8, g=128, dtype="bf16"),
    ]


def _route(name, tokens, experts, k, dtype, sigmoid=False, bias=False, groups=1, top_groups=1, group_top=1, renormalize=True,
           scale=1.0, masked=False):
    return dict(name=name, op="route", tokens=tokens, experts=experts, k=k, dtype=dtype, sigmoid=sigmoid, bias=bias, groups=groups,
                top_groups=top_groups, group_top=group_top, renormalize=renormalize, scale=scale, masked=masked)


def _lora(name, tokens, k, n, rank, adapters, dtype, mixed=False, none=0.0, runs=False):
    return dict(name=name, op="lora", tokens=tokens, k=k, n=n, rank=rank, adapters=adapters, dtype=dtype, mixed=mixed, none=none,
                runs=runs)


def _experts(name, tokens, hidden, inter, experts, k, g, dtype, none=0.0):
    return dict(name=name, op="experts", tokens=tokens, hidden=hidden, inter=inter, experts=experts, k=k, g=g, dtype=dtype, none=none)


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("route", "lora", "experts"))
    if op == "route":
        sigmoid = rng.random() < 0.5
        groups = rng.choice((1, 4, 8)) if sigmoid else rng.choice((1, 1, 4))
        experts = groups * rng.randint(2, 256 // groups) if groups > 1 else rng.randint(4, 256)
        group_top = rng.choice((1, 2)) if sigmoid and groups > 1 else 1
        top_groups = rng.randint(1, groups - 1) if groups > 1 else 1
        k = rng.randint(1, min(8, top_groups * (experts // groups)))
        case = _route("", tokens=_spread(rng, 1, 16384), experts=experts, k=k, dtype=rng.choice(("f16", "bf16", "f32")),
                      sigmoid=sigmoid, bias=sigmoid and rng.random() < 0.7, groups=groups, top_groups=top_groups,
                      group_top=group_top, renormalize=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)),
                      masked=groups == 1 and k < experts // 2 and rng.random() < 0.3)
    elif op == "lora":
        case = _lora("", tokens=_spread(rng, 1, 8192), k=8 * _spread(rng, 36, 1024), n=_spread(rng, 288, 10240),
                     rank=8 * rng.randint(1, 4) if rng.random() < 0.7 else 64, adapters=_spread(rng, 1, 32),
                     dtype=rng.choice(("f16", "bf16")), mixed=rng.random() < 0.3, none=rng.choice((0.0, 0.0, 0.2)),
                     runs=rng.random() < 0.5)
        case["tokens"] = min(case["tokens"], max(1, 8192 * 32 // case["rank"]))
    else:
        experts = _spread(rng, 4, 64)
        case = _experts("", tokens=_spread(rng, 1, 4096), hidden=8 * _spread(rng, 36, 512), inter=8 * _spread(rng, 36, 512),
                        experts=experts, k=rng.randint(1, min(8, experts)), g=rng.choice((32, 64, 128, 128, 256)),
                        dtype=rng.choice(("f16", "bf16")), none=rng.choice((0.0, 0.0, 0.05)))
        # no dearer than the largest listed case, in its products and in the weights it holds
        most, weight = 4096 * 8 * 2048 * 1024, case["hidden"] * case["inter"]
        case["tokens"] = max(1, min(case["tokens"], most // (case["k"] * weight)))
        if experts * weight > 8 * 4096 * 11008:
            case["inter"] = max(288, 8 * 4096 * 11008 // (experts * case["hidden"]) // 8 * 8)
    del case["name"]
    return case


# ----------------------------------------------------------------------------------------------------------- inputs

def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _packed_weights(gen, experts, n, k, g, dtype):
    """Random weights in the canonical packed form, `experts` matrices [n, k] with 0.9 / sqrt(k) as their values' deviation."""
    groups = -(-k // g)
    words, zwords = -(-k // 8), -(-groups // 8)
    qw = torch.randint(-2**31, 2**31, (experts, n, words), generator=gen, device="cuda", dtype=torch.int32)
    scales = (0.7 + 0.6 * torch.rand((experts, n, groups), generator=gen, device="cuda")) * (0.2 / math.sqrt(k))
    zeros = torch.zeros((experts, n, zwords), device="cuda", dtype=torch.int32)
    z = torch.randint(6, 10, (experts, n, zwords * 8), generator=gen, device="cuda", dtype=torch.int32)
    z[..., groups:] = 0
    for i in range(8):
        zeros |= z[..., i::8] << (4 * i)
    return qw, scales.to(dtype), zeros


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "route":
        T, E = case["tokens"], case["experts"]
        logits = _normal(gen, (T, E), 1.5) + _normal(gen, (E,), 0.5)
        if case["masked"]:  # an eighth of the experts is away for each token
            away = torch.rand((T, E), generator=gen, device="cuda") < 0.125
            logits = logits.masked_fill(away, -math.inf)
        s["logits"] = logits.to(dtype)
        s["bias_values"] = _normal(gen, (E,), 0.1) if case["bias"] else None
    elif case["op"] == "lora":
        T, K, N, r, R = (case[n] for n in ("tokens", "k", "n", "rank", "adapters"))
        s["x"] = _normal(gen, (T, K)).to(dtype)
        s["base"] = _normal(gen, (T, N)).to(dtype)
        s["A"] = _normal(gen, (R, r, K), 1 / math.sqrt(K)).to(dtype)
        s["B"] = _normal(gen, (R, N, r), 0.5 / math.sqrt(r)).to(dtype)
        adapter = torch.randint(0, R, (T,), generator=gen, device="cuda", dtype=torch.int32)
        if case["runs"]:  # prefill: a request's rows follow one another
            adapter = adapter[torch.arange(T, device="cuda") // 64 * 64]
        none = torch.rand((T,), generator=gen, device="cuda") < case["none"]
        s["adapter"] = adapter.masked_fill(none, -1)
        s["scaling"] = 0.5 + torch.rand((R,), generator=gen, device="cuda")
        s["rank_of"] = torch.tensor(_ranks(case), device="cuda", dtype=torch.int32) if case["mixed"] else None
    else:
        T, K, I, E, k, g = (case[n] for n in ("tokens", "hidden", "inter", "experts", "k", "g"))
        s["x"] = _normal(gen, (T, K)).to(dtype)
        scores = _normal(gen, (T, E)) + _normal(gen, (E,), 0.5)
        top = torch.topk(scores, k, dim=1)
        ids = top.indices.to(torch.int32)
        none = torch.rand((T, k), generator=gen, device="cuda") < case["none"]
        s["ids"] = ids.masked_fill(none, -1)
        s["weights"] = torch.softmax(top.values, dim=1)
        s["gate_up"] = _packed_weights(gen, E, 2 * I, K, g, dtype)
        s["down"] = _packed_weights(gen, E, K, I, g, dtype)
    if own:
        import w4a16_group_quantized_gb300 as w4

        s["workspace"] = w4.Workspace("cuda")
        if case["op"] == "experts":  # laid out once, as a program does when it loads the model
            for name, n, k in (("gate_up", 2 * s["inter"], s["hidden"]), ("down", s["hidden"], s["inter"])):
                laid = torch.empty((s["experts"], w4.w4_repacked_bytes(n, k, s["g"])), device="cuda", dtype=torch.uint8)
                for e, (qw, sc, zw) in enumerate(zip(*s[name])):
                    w4.w4_repack(qw, sc, zw, n, k, s["g"], out=laid[e])
                s[name] = laid
    return s


def _ranks(case):
    """The ranks of adapters of unlike ranks: the largest, half of it and a quarter in turn."""
    return [max(1, case["rank"] >> (i % 3)) for i in range(case["adapters"])]


# -------------------------------------------------------------------------------------------------------- the passes

def run(s):
    return (_RUN_OWN if own else _RUN_PLAIN)[s["op"]](s)


def _route_own(s):
    import w4a16_group_quantized_gb300 as w4

    return w4.w4_route(s["logits"], s["k"], sigmoid=s["sigmoid"], bias=s["bias_values"], groups=s["groups"],
                       top_groups=s["top_groups"], group_top=s["group_top"], renormalize=s["renormalize"], scale=s["scale"])


def _lora_own(s):
    import w4a16_group_quantized_gb300 as w4

    return w4.w4_lora_add(s["base"], s["x"], s["A"], s["B"], s["adapter"], scaling=s["scaling"], ranks=s["rank_of"],
                          workspace=s["workspace"])


def _experts_own(s):
    import w4a16_group_quantized_gb300 as w4

    return w4.w4a16_experts(s["x"], s["gate_up"], s["down"], s["ids"], s["weights"], s["inter"], s["g"],
                            workspace=s["workspace"])


def _best(v, n):
    """The places of the n largest values of each row, largest first, the lowest place first among equal ones."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[..., :n]


def _route_plain(s):
    l = s["logits"].float()
    T, E = l.shape
    away = l == -math.inf
    if s["sigmoid"]:
        score = 1 / (1 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(dim=1, keepdim=True)).masked_fill(away, 0)
        score = e / e.sum(dim=1, keepdim=True).clamp(min=1e-37)  # zeros for a row with every expert masked
    # without a bias the order of the scores is that of the logits
    key = l if s["bias_values"] is None else (score + s["bias_values"]).masked_fill(away, -math.inf)
    if s["groups"] > 1:
        of_group = (key if s["group_top"] == 1 else score if s["bias_values"] is None else key).view(T, s["groups"], -1)
        of_group = torch.sort(of_group, dim=-1, descending=True).values[..., : s["group_top"]].sum(dim=-1)
        kept = torch.zeros_like(of_group, dtype=torch.bool).scatter_(1, _best(of_group, s["top_groups"]), True)
        kept = kept.repeat_interleave(E // s["groups"], dim=1)
        ids = _best(kept, E)[:, : s["top_groups"] * (E // s["groups"])]  # places in the kept groups, in order
        ids = ids.gather(1, _best(key.gather(1, ids), s["k"]))
    else:
        ids = _best(key, s["k"])
    w = score.gather(1, ids)
    if s["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-37)
    return w * s["scale"], ids.to(torch.int32)


def _lora_plain(s):
    x, A, B = s["x"].float(), s["A"].float(), s["B"].float()
    R, r, K = A.shape
    N, T = B.shape[1], x.shape[0]
    adapter = s["adapter"].long()
    some = (adapter >= 0).float()
    adapter = adapter.clamp(min=0)
    scale = s["scaling"][adapter] * some
    rank = torch.full((R,), r, device="cuda") if s["rank_of"] is None else s["rank_of"]
    live = torch.arange(r, device="cuda") < rank[adapter][:, None]  # [T, r]
    if T <= R:  # few rows: their adapters alone
        v = torch.matmul(A[adapter], x[:, :, None])[:, :, 0] * live * scale[:, None]
        d = torch.matmul(B[adapter], v[:, :, None])[:, :, 0]
    else:  # every adapter on every row, and each row keeps its own
        v = torch.matmul(x, A.view(R * r, K).t()).view(T, R, r)
        mine = adapter[:, None] == torch.arange(R, device="cuda")
        v = v * (mine[:, :, None] & live[:, None, :]) * scale[:, None, None]
        d = torch.matmul(v.view(T, R * r), B.permute(0, 2, 1).reshape(R * r, N))
    return (s["base"].float() + d).to(s["base"].dtype)


def _dequant(packed, k, g):
    """[.., n, k] weights in 32 bits of a canonical packed form."""
    qw, scales, zeros = packed
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    group = torch.arange(k, device="cuda") // g
    q = ((qw[..., None] >> shift) & 15).flatten(-2)[..., :k].float()
    z = ((zeros[..., None] >> shift) & 15).flatten(-2)[..., : scales.shape[-1]].float()
    return (q - z[..., group]) * scales.float()[..., group]


def _experts_plain(s):
    T, k, K = s["tokens"], s["k"], s["hidden"]
    ids = s["ids"].flatten().long()
    pair = torch.sort(ids, stable=True).indices  # pairs (row, choice) by expert, the dropped ones first
    pair = pair[(ids < 0).sum():]
    y = torch.zeros((T * k, K), device="cuda")
    if pair.numel():
        expert, count = torch.unique_consecutive(ids[pair], return_counts=True)
        slot = torch.repeat_interleave(torch.arange(expert.numel(), device="cuda"), count)
        place = torch.arange(pair.numel(), device="cuda") - (count.cumsum(0) - count)[slot]
        x = torch.zeros((expert.numel(), int(count.max()), K), device="cuda")
        x[slot, place] = s["x"].float()[pair // k]
        both = torch.bmm(x, _dequant([p[expert] for p in s["gate_up"]], K, s["g"]).transpose(1, 2))
        gate, up = both[..., 0::2], both[..., 1::2]
        h = gate / (1 + torch.exp(-gate)) * up
        out = torch.bmm(h, _dequant([p[expert] for p in s["down"]], s["inter"], s["g"]).transpose(1, 2))
        y[pair] = out[slot, place] * s["weights"].flatten()[pair][:, None]
    return y.view(T, k, K).sum(dim=1).to(s["x"].dtype)


_RUN_OWN = {"route": _route_own, "lora": _lora_own, "experts": _experts_own}
_RUN_PLAIN = {"route": _route_plain, "lora": _lora_plain, "experts": _experts_plain}


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    if case["op"] == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": T * E * size + T * k * 8 + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    if case["op"] == "lora":
        T, K, N, R = (case[n] for n in ("tokens", "k", "n", "adapters"))
        rank = sum(_ranks(case)) / R if case["mixed"] else case["rank"]
        rows = T * (1 - case["none"])
        draws = max(1.0, rows / 64) if case["runs"] else rows
        used = R * (1 - (1 - 1 / R) ** draws)  # adapters that some row has, on average
        return {"bytes": 2 * T * K + 4 * T * N + 4 * T + used * rank * (K + N) * 2, "flops": 2 * rows * rank * (K + N)}
    T, K, I, E, k, g = (case[n] for n in ("tokens", "hidden", "inter", "experts", "k", "g"))
    live = 1 - case["none"]
    used = E * (1 - (1 - k * live / E) ** T)  # experts that some row has, on average
    weights = 1.5 * K * I + 2.5 * (2 * I * -(-K // g) + K * -(-I // g))  # codes, and a scale and half a byte of zero a group
    return {"bytes": 4 * T * K + 8 * T * k + used * weights, "flops": 6 * T * k * live * K * I}


# ---------------------------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"route": _route_exact, "lora": _lora_exact, "experts": _experts_exact}[case["op"]](s)


def _route_exact(s):
    l = s["logits"].double()
    T, E = l.shape
    score = torch.sigmoid(l) if s["sigmoid"] else torch.softmax(l, dim=1)
    choice = l if s["bias_values"] is None else score + s["bias_values"].double()
    choice = torch.where(torch.isinf(l), torch.full_like(l, -math.inf), choice)
    if s["groups"] > 1:
        per = choice if s["group_top"] == 1 or s["bias_values"] is not None else score
        worth = torch.topk(per.reshape(T, s["groups"], E // s["groups"]), s["group_top"], dim=2).values.sum(2)
        order = torch.argsort(worth, dim=1, descending=True, stable=True)
        out = order[:, s["top_groups"]:]
        places = (out[:, :, None] * (E // s["groups"]) + torch.arange(E // s["groups"], device="cuda")).reshape(T, -1)
        # what is left out lies below even the masked places of the groups that are kept
        choice = choice.clamp(min=-1e300).scatter(1, places, -math.inf)
    ids = torch.argsort(choice, dim=1, descending=True, stable=True)[:, : s["k"]]
    w = torch.gather(score, 1, ids)
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return torch.nan_to_num(w * s["scale"]), None  # a row with every expert masked: zeros


def _lora_exact(s):
    y = s["base"].double()
    for a in range(s["adapters"]):
        rows = torch.nonzero(s["adapter"] == a)[:, 0]
        r = s["rank"] if s["rank_of"] is None else int(s["rank_of"][a])
        v = s["x"][rows].double() @ s["A"][a, :r].double().T
        y[rows] += float(s["scaling"][a]) * (v @ s["B"][a, :, :r].double().T)
    return y


def _experts_exact(s):
    def weight(packed, e, k):
        qw, scales, zeros = (p[e].cpu() if p.numel() < 4096 else p[e] for p in packed)
        cols = torch.arange(k, device=qw.device)
        q = (qw[:, cols // 8] >> (4 * (cols % 8)).int()) & 15
        j = cols // s["g"]
        z = (zeros[:, j // 8] >> (4 * (j % 8)).int()) & 15
        return ((q - z).double() * scales[:, j].double()).cuda()

    y = torch.zeros((s["tokens"], s["hidden"]), device="cuda", dtype=torch.float64)
    for e in range(s["experts"]):
        row, choice = torch.nonzero(s["ids"] == e, as_tuple=True)
        if row.numel() == 0:
            continue
        t = s["x"][row].double() @ weight(s["gate_up"], e, s["hidden"]).T
        h = torch.nn.functional.silu(t[:, 0::2]) * t[:, 1::2]
        o = h @ weight(s["down"], e, s["inter"]).T
        y.index_add_(0, row, o * s["weights"][row, choice].double()[:, None])
    return y
