"""The operators around the quantised decode step, as measured cases.

Four operators of layers whose weights stay in 16 bits (a shared expert, the
projections around the step, experts that a checkpoint leaves unquantised) and
of routers other than the built-in softmax top-k:

  linear   out = act(x W^T + bias) [* (x Wup^T + bias_up)] [+ residual]
  grouped  the same product with one weight matrix per expert, over rows
           grouped by expert at ragged offsets, optionally gathered by token
  slots    top-k expert ids -> rows grouped by expert (a stable counting sort)
  combine  out[t] = sum_j w[t, j] y[slot_of[t, j]] [+ residual[t]]

run() takes the plain form (elementary torch operations in 32 bits, one
rounding at the end) or, with `own` set, the library's operators.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _linear(name, n, K, N, dtype, act="none", gated=False, bias=False, residual=False):
    return dict(name=name, op="linear", n=n, K=K, N=N, dtype=dtype, act=act, gated=gated, bias=bias,
                residual=residual)


def _grouped(name, n, k, E, K, N, dtype, act="none", gated=False, bias=False, gather=False, skew=0.0):
    return dict(name=name, op="grouped", n=n, k=k, E=E, K=K, N=N, dtype=dtype, act=act, gated=gated,
                bias=bias, gather=gather, skew=skew)


def _slots(name, n, k, E, begin, end, skew=0.0):
    return dict(name=name, op="slots", n=n, k=k, E=E, begin=begin, end=end, skew=skew)


def _combine(name, n, k, E, N, dtype, residual):
    return dict(name=name, op="combine", n=n, k=k, E=E, N=N, dtype=dtype, residual=residual)


def listed():
    return [
        # one token through a hidden-size projection that adds the residual stream:
        # the smallest product, once or more per layer of every decode tick
        _linear("linear_1_token", 1, 2048, 2048, "bf16", residual=True),
        # the gate and up product of a shared expert for a decode cohort
        _linear("linear_shared_8_tokens", 8, 2048, 768, "bf16", act="silu", gated=True),
        # a chunk of a prompt through a biased layer, at sizes that fill no tile
        _linear("linear_chunk_317", 317, 2040, 4104, "f16", act="gelu", bias=True, residual=True),
        # a whole prompt through the wide layer's gate and up product
        _linear("linear_prompt_8192", 8192, 4096, 2048, "bf16", act="silu", gated=True),
        # one token's eight experts, gate and up: each weight row is read for one row
        _grouped("grouped_1_token_gate_up", 1, 8, 128, 2048, 768, "bf16", act="silu", gated=True, gather=True),
        # the down product of a decode cohort of 64: most experts with a few rows each
        _grouped("grouped_64_tokens_down", 64, 8, 128, 768, 2048, "bf16"),
        # a prompt through the 256-expert layer under a skewed router: groups from
        # none to hundreds of rows, biased experts
        _grouped("grouped_skewed_1024", 1024, 6, 256, 4096, 2048, "f16", act="gelu_tanh", gated=True,
                 bias=True, gather=True, skew=1.1),
        # the largest prompt's gate and up product
        _grouped("grouped_8192_tokens_gate_up", 8192, 8, 128, 2048, 768, "bf16", act="silu", gated=True,
                 gather=True),
        # the grouping of a decode cohort: latency alone
        _slots("slots_8_tokens", 8, 8, 128, 0, 128),
        # the grouping of the largest prompt on one of four expert-parallel shards
        _slots("slots_8192_tokens_shard", 8192, 6, 256, 64, 128, skew=1.1),
        # the weighted sum of a decode cohort
        _combine("combine_8_tokens", 8, 8, 128, 2048, "bf16", True),
        # the weighted sum of the largest prompt
        _combine("combine_8192_tokens", 8192, 8, 128, 2048, "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: every operator, both types, odd sizes."""
    op = rng.choice(["linear", "linear", "grouped", "grouped", "slots", "combine"])
    dtype = rng.choice(["bf16", "f16"])
    act = rng.choice(["none", "silu", "gelu", "gelu_tanh"])
    gated, bias, flag = rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.5
    if op == "linear":
        n, K, N = _log(rng, 1, 8192), 8 * _log(rng, 16, 512), _log(rng, 100, 4096)
        if gated:
            N = max(64, N // 2)
        c = _linear("", n, K, N, dtype, act, gated, bias, flag)
    elif op == "grouped":
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        K, N = 8 * _log(rng, 16, 256), _log(rng, 100, 1024)
        c = _grouped("", _log(rng, 1, 4096), k, E, K, N, dtype, act, gated, bias, flag, rng.choice([0.0, 0.0, 1.1]))
    elif op == "slots":
        E = _log(rng, 4, 1024)
        b = rng.choice([0, 0, rng.randrange(E)])
        c = _slots("", _log(rng, 1, 8192), rng.randint(1, min(8, E)), E, b, rng.randint(b + 1, E) if b else E,
                   rng.choice([0.0, 1.1]))
    else:
        E = _log(rng, 8, 256)
        c = _combine("", _log(rng, 1, 8192), rng.randint(1, 8), E, _log(rng, 100, 4096), dtype, flag)
    del c["name"]
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, std, generator=g)


def _route(g, n, k, E, skew):
    """Distinct expert ids per token by descending logit, and their weights."""
    logits = torch.randn((n, E), generator=g, device="cuda")
    if skew:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
        logits = logits - skew * torch.log(rank)
    top, idx = torch.topk(logits, k, dim=1)
    return idx.to(torch.int32).contiguous(), torch.softmax(top, dim=1).contiguous()


def _weights(case, g, lead):
    dt = _DT[case["dtype"]]
    N, K = case["N"], case["K"]
    w = {"w": _normal(g, lead + (N, K), K ** -0.5, dt)}
    if case["gated"]:
        w["w_up"] = _normal(g, lead + (N, K), K ** -0.5, dt)
    if case["bias"]:
        w["bias"] = _normal(g, lead + (N,), 0.5, dt)
        if case["gated"]:
            w["bias_up"] = _normal(g, lead + (N,), 0.5, dt)
    return w


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("linear", "grouped"):
        dt = _DT[case["dtype"]]
        lead = () if op == "linear" else (case["E"],)
        s["x"] = _normal(g, (case["n"], case["K"]), 1.0, dt)
        s.update(_weights(case, g, lead))
        if own:
            import quantized_moe_decode_softmax_gb300 as q

            s["handle"] = q.LinearWeights(s["w"], w_up=s.get("w_up"), bias=s.get("bias"), bias_up=s.get("bias_up"),
                                          activation=case["act"])
    if op == "linear" and case["residual"]:
        s["residual"] = _normal(g, (case["n"], case["N"]), 1.0, _DT[case["dtype"]])
    if op == "linear":
        return s
    n, k, E = case["n"], case["k"], case["E"]
    idx, wt = _route(g, n, k, E, case.get("skew", 0.0))
    if op == "slots":
        s["topk_idx"] = idx
        return s
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    if op == "combine":
        s["slot_of"] = torch.argsort(order, stable=True).to(torch.int32).reshape(n, k).contiguous()
        s["topk_w"] = wt
        s["y"] = _normal(g, (n * k, case["N"]), 1.0, _DT[case["dtype"]])
        if case["residual"]:
            s["residual"] = _normal(g, (n, case["N"]), 1.0, _DT[case["dtype"]])
        return s
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    s["offsets"] = offsets
    token = torch.div(order, k, rounding_mode="floor").to(torch.int32)
    if case["gather"]:
        s["row_token"] = token
    else:  # the rows are in hand in grouped order, as the gate and up product left them
        s["x"] = s["x"][token.long()].contiguous()
    # what a plain program would also keep: the experts in use and the largest group
    s["used"] = torch.nonzero(counts).reshape(-1)
    s["most"] = int(counts.max())
    return s


def _act(v, kind):
    if kind == "silu":
        return v * torch.sigmoid(v)
    if kind == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.7071067811865476))
    if kind == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    return v


def _plain_linear(s, c):
    x = s["x"].float()
    v = x @ s["w"].float().t()
    if "bias" in s:
        v = v + s["bias"].float()
    v = _act(v, c["act"])
    if c["gated"]:
        u = x @ s["w_up"].float().t()
        v = v * (u + s["bias_up"].float() if "bias_up" in s else u)
    if "residual" in s:
        v = v + s["residual"].float()
    return v.to(_DT[c["dtype"]])


def _plain_grouped(s, c):
    used, offsets = s["used"], s["offsets"].long()
    rows = torch.arange(c["n"] * c["k"], device="cuda")
    x = s["x"][s["row_token"].long()] if c["gather"] else s["x"]
    e = torch.searchsorted(offsets[1:], rows, right=True)  # the expert of each row
    at = torch.searchsorted(used, e)
    pos = rows - offsets[e]
    xp = torch.zeros((used.numel(), s["most"], c["K"]), dtype=torch.float32, device="cuda")
    xp[at, pos] = x.float()
    v = torch.bmm(xp, s["w"][used].float().transpose(1, 2))[at, pos]
    if "bias" in s:
        v = v + s["bias"].float()[e]
    v = _act(v, c["act"])
    if c["gated"]:
        u = torch.bmm(xp, s["w_up"][used].float().transpose(1, 2))[at, pos]
        v = v * (u + s["bias_up"].float()[e] if "bias_up" in s else u)
    return v.to(_DT[c["dtype"]])


def _plain_slots(s, c):
    n, k, E, b, end = c["n"], c["k"], c["E"], c["begin"], c["end"]
    flat = s["topk_idx"].reshape(-1).long()
    owned = (flat >= b) & (flat < end)
    key = torch.where(owned, flat, torch.full_like(flat, E))
    ranked, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ranked, torch.arange(E + 1, device="cuda")).to(torch.int32)
    live = owned[order]
    none = torch.full_like(order, -1)
    place = torch.empty_like(order)
    place[order] = torch.arange(n * k, device="cuda")
    return {"offsets": offsets,
            "slot_token": torch.where(live, torch.div(order, k, rounding_mode="floor"), none).to(torch.int32),
            "slot_k": torch.where(live, order % k, none).to(torch.int32),
            "slot_of": torch.where(owned, place, none).to(torch.int32).reshape(n, k)}


def _plain_combine(s, c):
    v = (s["y"][s["slot_of"].long()].float() * s["topk_w"].unsqueeze(-1)).sum(1)
    if "residual" in s:
        v = v + s["residual"].float()
    return v.to(_DT[c["dtype"]])


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import quantized_moe_decode_softmax_gb300 as q

        if op == "linear":
            return q.moe_linear(s["x"], s["handle"], residual=s.get("residual"))
        if op == "grouped":
            return q.moe_grouped_linear(s["x"], s["handle"], s["offsets"], row_token=s.get("row_token"))
        if op == "slots":
            g = q.moe_group_slots(s["topk_idx"], c["E"], experts=(c["begin"], c["end"]))
            return {"offsets": g.offsets, "slot_token": g.slot_token, "slot_k": g.slot_k, "slot_of": g.slot_of}
        return q.moe_combine_slots(s["y"], s["slot_of"], s["topk_w"], residual=s.get("residual"))
    return {"linear": _plain_linear, "grouped": _plain_grouped, "slots": _plain_slots,
            "combine": _plain_combine}[op](s, c)


def work(case):
    """Each input read once and each output written once; two operations per
    product and sum of the contraction."""
    op, n = case["op"], case["n"]
    if op == "slots":
        s = n * case["k"]
        return {"bytes": 4.0 * (s + 3 * s + case["E"] + 1), "flops": 0.0}
    N = case["N"]
    if op == "combine":
        s = n * case["k"]
        return {"bytes": 2.0 * s * N + 8.0 * s + 2.0 * n * N * (2 if case["residual"] else 1),
                "flops": 2.0 * s * N}
    K, mats = case["K"], 2 if case["gated"] else 1
    if op == "linear":
        return {"bytes": 2.0 * (n * K + mats * N * (K + (1 if case["bias"] else 0))
                                + n * N * (2 if case["residual"] else 1)),
                "flops": 2.0 * n * K * N * mats}
    s, E = n * case["k"], case["E"]
    if case["skew"]:  # the chance that an expert is in use, from the mean softmax of the skewed logits
        p = [r ** -case["skew"] for r in range(1, E + 1)]
        t = sum(p)
        used = sum(1.0 - (1.0 - min(1.0, case["k"] * v / t)) ** n for v in p)
    else:
        used = E * (1.0 - (1.0 - case["k"] / E) ** n)
    return {"bytes": 2.0 * ((n if case["gather"] else s) * K + used * mats * N * (K + (1 if case["bias"] else 0)) + s * N)
            + 4.0 * (E + 1) + (4.0 * s if case["gather"] else 0.0),
            "flops": 2.0 * s * K * N * mats}


def _act64(v, kind):
    if kind == "silu":
        return v / (1.0 + torch.exp(-v))
    if kind == "gelu":
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
    if kind == "gelu_tanh":
        z = math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)
        return v / (1.0 + torch.exp(-2.0 * z))
    return v


def exact(case, seed):
    """The same from the definitions in 64 bits: one expert (or one rank of the
    sum) at a time. The grouping has whole numbers only."""
    op = case["op"]
    if op == "slots":
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if op == "combine":
        out = torch.zeros((case["n"], case["N"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            rows = torch.index_select(s["y"], 0, s["slot_of"][:, j].long())
            out.addcmul_(rows.double(), s["topk_w"][:, j:j + 1].double())
        return out + s["residual"].double() if case["residual"] else out

    def product(x, pick):
        z = torch.einsum("rk,nk->rn", x.double(), pick(s["w"]).double())
        z = _act64(z + pick(s["bias"]).double() if case["bias"] else z, case["act"])
        if case["gated"]:
            u = torch.einsum("rk,nk->rn", x.double(), pick(s["w_up"]).double())
            z = z * (u + pick(s["bias_up"]).double() if case["bias"] else u)
        return z

    if op == "linear":
        z = product(s["x"], lambda t: t)
        return z + s["residual"].double() if case["residual"] else z
    ends = s["offsets"].tolist()
    out = torch.empty((case["n"] * case["k"], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            rows = s["x"].index_select(0, s["row_token"][a:b].long()) if case["gather"] else s["x"][a:b]
            out[a:b] = product(rows, lambda t: t[e])
    return out
