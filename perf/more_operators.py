"""Routing to experts and products in 8-bit integers, as measured cases.

Four operators of a layer whose router is not the step's softmax top-k and whose
experts (or shared expert, or projections) are kept in 8-bit integers:

  route      router logits -> expert ids and weights: softmax or sigmoid scores, a
             bias that only steers the choice, groups of experts of which some are
             kept, top-k, renormalised and scaled weights
  quantize   rows of 16-bit values -> 8-bit codes with one scale per row
  linear     out = act(sx sw (x W^T) + bias) [* the up product] [+ residual], x and W
             in 8-bit codes with a scale per row of x and per row of W
  grouped    the same product with one weight matrix per expert, over rows grouped
             by expert at ragged offsets, optionally gathered by token

run() takes the plain form (elementary torch operations in 32 bits, one rounding at
the end; the router's scores in 64, because its choice compares values that may lie
next to one another) or, with `own` set, the library's operators.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _route(name, n, E, k, dtype, score="softmax", bias=False, groups=1, top_groups=1, group_score="max",
           renormalize=True, scale=1.0, masked=False):
    return dict(name=name, op="route", n=n, E=E, k=k, dtype=dtype, score=score, bias=bias, groups=groups,
                top_groups=top_groups, group_score=group_score, renormalize=renormalize, scale=scale, masked=masked)


def _quantize(name, n, K, dtype):
    return dict(name=name, op="quantize", n=n, K=K, dtype=dtype)


def _linear(name, n, K, N, dtype, act="none", gated=False, bias=False, residual=False):
    return dict(name=name, op="linear", n=n, K=K, N=N, dtype=dtype, act=act, gated=gated, bias=bias,
                residual=residual)


def _grouped(name, n, k, E, K, N, dtype, act="none", gated=False, bias=False, gather=False, skew=0.0):
    return dict(name=name, op="grouped", n=n, k=k, E=E, K=K, N=N, dtype=dtype, act=act, gated=gated, bias=bias,
                gather=gather, skew=skew)


def listed():
    return [
        # the router of one decoded token, once per layer of every tick: latency alone
        _route("route_1_token", 1, 128, 8, "bf16"),
        # a decode cohort through a balanced router with limited groups
        _route("route_64_tokens_groups", 64, 256, 8, "f32", score="sigmoid", bias=True, groups=8, top_groups=4,
               group_score="top2", scale=2.5),
        # a chunk of a prompt, few groups kept by their best expert, some experts switched
        # off, weights as the softmax gives them
        _route("route_chunk_317", 317, 160, 6, "f16", groups=8, top_groups=3, renormalize=False, scale=16.0,
               masked=True),
        # the largest prompt through the 256-expert layer's router, balanced by a bias
        _route("route_8192_tokens", 8192, 256, 6, "bf16", score="sigmoid", bias=True, scale=2.5),
        # one token's activations before a projection: latency alone
        _quantize("quantize_1_token", 1, 2048, "bf16"),
        # the largest prompt's activations
        _quantize("quantize_8192_tokens", 8192, 4096, "bf16"),
        # one token through a hidden-size projection that adds the residual stream
        _linear("linear_1_token", 1, 2048, 2048, "bf16", residual=True),
        # a chunk of a prompt through a biased layer, at sizes that fill no tile
        _linear("linear_chunk_317", 317, 2032, 4104, "f16", act="gelu", bias=True, residual=True),
        # a whole prompt through the wide layer's gate and up product
        _linear("linear_prompt_8192", 8192, 4096, 2048, "bf16", act="silu", gated=True),
        # one token's eight experts, gate and up: each weight row is read for one row
        _grouped("grouped_1_token_gate_up", 1, 8, 128, 2048, 768, "bf16", act="silu", gated=True, gather=True),
        # the down product of a decode cohort of 64: most experts with a few rows each
        _grouped("grouped_64_tokens_down", 64, 8, 128, 768, 2048, "bf16"),
        # the largest prompt's gate and up product
        _grouped("grouped_8192_tokens_gate_up", 8192, 8, 128, 2048, 768, "bf16", act="silu", gated=True,
                 gather=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: every operator, every type, odd sizes."""
    op = rng.choice(["route", "route", "quantize", "linear", "linear", "grouped", "grouped"])
    dtype = rng.choice(["bf16", "f16"])
    act = rng.choice(["none", "silu", "gelu", "gelu_tanh"])
    gated, bias, flag = rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.5
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 1024 // groups)
        top = rng.randint(1, groups)
        # as many experts as the kept groups have at least
        k = rng.randint(1, min(16, top * (E // groups)))
        c = _route("", _log(rng, 1, 8192), E, k, rng.choice(["bf16", "f16", "f32"]), rng.choice(["softmax", "sigmoid"]),
                   bias, groups, top, rng.choice(["max", "top2"]), flag, rng.choice([1.0, 2.5]), rng.random() < 0.2)
    elif op == "quantize":
        c = _quantize("", _log(rng, 1, 8192), _log(rng, 64, 4096), dtype)
    elif op == "linear":
        n, K, N = _log(rng, 1, 8192), 16 * _log(rng, 8, 256), _log(rng, 100, 4096)
        if gated:
            N = max(64, N // 2)
        c = _linear("", n, K, N, dtype, act, gated, bias, flag)
    else:
        E = _log(rng, 4, 256)
        k = rng.randint(1, min(8, E))
        K, N = 16 * _log(rng, 8, 128), _log(rng, 100, 1024)
        if gated:
            N = min(N, 768)
        c = _grouped("", _log(rng, 1, 4096), k, E, K, N, dtype, act, gated, bias, flag, rng.choice([0.0, 0.0, 1.1]))
    del c["name"]
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, std, dtype):
    t = torch.empty(shape, dtype=dtype, device="cuda")
    return t.normal_(0.0, std, generator=g)


def _codes(g, lead, N, K):
    """Weights in 8-bit codes, as rounding normal weights by their row's largest leaves
    them (the largest near four deviations), and the scale of each row."""
    q = _normal(g, lead + (N, K), 32.0, torch.bfloat16).round_().clamp_(-127.0, 127.0).to(torch.int8)
    return q, (1.0 + 0.2 * torch.rand(lead + (N,), generator=g, device="cuda")) * (K ** -0.5 / 32.0)


def _quantized(x):
    """Codes and scales of the rows of x: round(127 x / max|x|), halves to even. In 64
    bits, where the quotient of two 16-bit values next to a half stays on its side of it."""
    z = x.double()
    most = z.abs().amax(1, keepdim=True)
    codes = torch.where(most > 0, torch.round(z * 127.0 / most), torch.zeros_like(z)).to(torch.int8)
    return codes, (most / 127.0).float().squeeze(1)


def _weights(case, g, lead):
    dt, N, K = _DT[case["dtype"]], case["N"], case["K"]
    w = {}
    w["w"], w["w_scale"] = _codes(g, lead, N, K)
    if case["gated"]:
        w["w_up"], w["w_up_scale"] = _codes(g, lead, N, K)
    if case["bias"]:
        w["bias"] = _normal(g, lead + (N,), 0.5, dt)
        if case["gated"]:
            w["bias_up"] = _normal(g, lead + (N,), 0.5, dt)
    return w


def _topk_of_random_logits(g, n, k, E, skew):
    """Distinct expert ids per token by descending logit."""
    logits = torch.randn((n, E), generator=g, device="cuda")
    if skew:
        rank = torch.randperm(E, generator=g, device="cuda").float() + 1.0
        logits = logits - skew * torch.log(rank)
    return torch.topk(logits, k, dim=1).indices


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    s = {"case": case}
    if op == "route":
        n, E = case["n"], case["E"]
        # the logits of a trained router: a spread of a few units, some experts preferred
        z = 1.5 * torch.randn((n, E), generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
        if case["masked"]:  # experts that are switched off for these tokens
            z = torch.where(torch.rand((n, E), generator=g, device="cuda") < 0.1, -math.inf, z)
        s["logits"] = z.to(dt)
        if case["bias"]:  # what balancing the load has added up for each expert
            s["bias"] = 0.1 * torch.randn(E, generator=g, device="cuda")
        if own:
            import quantized_moe_decode_softmax_gb300 as q

            s["router"] = q.Router(E, case["k"], score=case["score"], bias=s.get("bias"), groups=case["groups"],
                                   top_groups=case["top_groups"], group_score=case["group_score"],
                                   renormalize=case["renormalize"], scale=case["scale"])
        return s
    if op == "quantize":
        s["x"] = _normal(g, (case["n"], case["K"]), 1.0, dt)
        return s
    lead = () if op == "linear" else (case["E"],)
    s["x"], s["x_scale"] = _quantized(_normal(g, (case["n"], case["K"]), 1.0, dt))
    s.update(_weights(case, g, lead))
    if own:
        import quantized_moe_decode_softmax_gb300 as q

        s["handle"] = q.LinearWeightsQ8(s["w"], s["w_scale"], w_up=s.get("w_up"), scale_up=s.get("w_up_scale"),
                                        bias=s.get("bias"), bias_up=s.get("bias_up"), activation=case["act"], dtype=dt)
    if op == "linear":
        if case["residual"]:
            s["residual"] = _normal(g, (case["n"], case["N"]), 1.0, dt)
        return s
    n, k, E = case["n"], case["k"], case["E"]
    flat = _topk_of_random_logits(g, n, k, E, case["skew"]).reshape(-1)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    s["offsets"] = offsets
    token = torch.div(order, k, rounding_mode="floor")
    if case["gather"]:
        s["row_token"] = token.to(torch.int32)
    else:  # the rows are in hand in grouped order, as the gate and up product left them
        s["x"], s["x_scale"] = s["x"][token].contiguous(), s["x_scale"][token].contiguous()
    # what a plain program would also keep: the experts in use and the largest group
    s["used"] = torch.nonzero(counts).reshape(-1)
    s["most"] = int(counts.max())
    return s


def _plain_route(s, c):
    n, E, k, G = c["n"], c["E"], c["k"], c["groups"]
    z = s["logits"].double()
    if c["score"] == "softmax":
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
    key = p + s["bias"].double() if "bias" in s else p
    key = torch.where(torch.isneginf(z), -math.inf, key)
    if G > 1:
        best = torch.sort(key.reshape(n, G, E // G), dim=2, descending=True).values
        of_group = best[:, :, 0]
        if c["group_score"] == "top2" and E // G > 1:  # the second of a group counts where there is one
            of_group = of_group + torch.where(torch.isneginf(best[:, :, 1]), 0.0, best[:, :, 1])
        kept = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        mask = torch.zeros((n, G), dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        key = torch.where(mask.repeat_interleave(E // G, dim=1), key, -math.inf)
    ranked = torch.sort(key, dim=1, descending=True, stable=True)
    idx, live = ranked.indices[:, :k], ~torch.isneginf(ranked.values[:, :k])
    w = torch.where(live, torch.gather(p, 1, idx), 0.0)
    if c["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"topk_idx": torch.where(live, idx, -1).to(torch.int32), "topk_w": (w * c["scale"]).float()}


def _act(v, kind):
    if kind == "silu":
        return v * torch.sigmoid(v)
    if kind == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.7071067811865476))
    if kind == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(0.7978845608028654 * (v + 0.044715 * v * v * v)))
    return v


def _plain_linear(s, c):
    x, sx = s["x"].float(), s["x_scale"].unsqueeze(1)
    v = (x @ s["w"].float().t()) * sx * s["w_scale"]
    if "bias" in s:
        v = v + s["bias"].float()
    v = _act(v, c["act"])
    if c["gated"]:
        u = (x @ s["w_up"].float().t()) * sx * s["w_up_scale"]
        v = v * (u + s["bias_up"].float() if "bias_up" in s else u)
    if "residual" in s:
        v = v + s["residual"].float()
    return v.to(_DT[c["dtype"]])


def _plain_grouped(s, c):
    used, offsets = s["used"], s["offsets"].long()
    rows = torch.arange(c["n"] * c["k"], device="cuda")
    x, sx = s["x"], s["x_scale"]
    if c["gather"]:
        x, sx = x[s["row_token"].long()], sx[s["row_token"].long()]
    sx = sx.unsqueeze(1)
    e = torch.searchsorted(offsets[1:], rows, right=True)  # the expert of each row
    at = torch.searchsorted(used, e)
    pos = rows - offsets[e]
    xp = torch.zeros((used.numel(), s["most"], c["K"]), dtype=torch.float32, device="cuda")
    xp[at, pos] = x.float()
    v = torch.bmm(xp, s["w"][used].float().transpose(1, 2))[at, pos] * sx * s["w_scale"][e]
    if "bias" in s:
        v = v + s["bias"].float()[e]
    v = _act(v, c["act"])
    if c["gated"]:
        u = torch.bmm(xp, s["w_up"][used].float().transpose(1, 2))[at, pos] * sx * s["w_up_scale"][e]
        v = v * (u + s["bias_up"].float()[e] if "bias_up" in s else u)
    return v.to(_DT[c["dtype"]])


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        import quantized_moe_decode_softmax_gb300 as q

        if op == "route":
            r = q.moe_route(s["logits"], s["router"])
            return {"topk_idx": r.topk_idx, "topk_w": r.topk_w}
        if op == "quantize":
            r = q.moe_quantize_rows(s["x"])
            return {"codes": r.codes, "scale": r.scale}
        if op == "linear":
            return q.moe_linear_q8((s["x"], s["x_scale"]), s["handle"], residual=s.get("residual"))
        return q.moe_grouped_linear_q8((s["x"], s["x_scale"]), s["handle"], s["offsets"],
                                       row_token=s.get("row_token"))
    if op == "quantize":
        codes, scale = _quantized(s["x"])
        return {"codes": codes, "scale": scale}
    return {"route": _plain_route, "linear": _plain_linear, "grouped": _plain_grouped}[op](s, c)


def work(case):
    """Each input read once and each output written once; two operations per product
    and sum of the contraction."""
    op, n = case["op"], case["n"]
    if op == "route":
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": float(n * case["E"] * size + 8 * n * case["k"] + (4 * case["E"] if case["bias"] else 0)),
                "flops": 0.0}
    K = case["K"]
    if op == "quantize":
        return {"bytes": 3.0 * n * K + 4.0 * n, "flops": 0.0}
    N, mats = case["N"], 2 if case["gated"] else 1
    per_row = K + 4 + (2 if case["bias"] else 0)  # of a weight matrix
    if op == "linear":
        return {"bytes": float(n * (K + 4) + mats * N * per_row + 2 * n * N * (2 if case["residual"] else 1)),
                "flops": 2.0 * n * K * N * mats}
    s, E = n * case["k"], case["E"]
    if case["skew"]:  # the chance that an expert is in use, from the mean softmax of the skewed logits
        p = [r ** -case["skew"] for r in range(1, E + 1)]
        t = sum(p)
        used = sum(1.0 - (1.0 - min(1.0, case["k"] * v / t)) ** n for v in p)
    else:
        used = E * (1.0 - (1.0 - case["k"] / E) ** n)
    return {"bytes": (n if case["gather"] else s) * (K + 4.0) + used * mats * N * per_row + 2.0 * s * N
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


def _exact_route(s, c):
    """The weights, token by token in blocks: an expert's rank is the number of experts
    that come before it, a group's rank the number of groups before it."""
    E, k, G = c["E"], c["k"], c["groups"]
    at = torch.arange(E, device="cuda")
    parts = []
    for z in s["logits"].double().split(max(1, (1 << 25) // (E * E))):
        if c["score"] == "softmax":
            p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        else:
            t = torch.exp(-z.abs())
            p = torch.where(z >= 0, 1.0 / (1.0 + t), t / (1.0 + t))
        key = p + (s["bias"].double() if c["bias"] else 0.0)
        ok = z > -math.inf
        if G > 1:
            gk = torch.where(ok, key, -math.inf).unflatten(1, (G, E // G))
            score = gk.max(2).values
            if c["group_score"] == "top2":
                gk = gk.scatter(2, gk.argmax(2, keepdim=True), -math.inf)
                second = gk.max(2).values
                score = score + torch.where(second > -math.inf, second, torch.zeros_like(second))
            a, b, j = score.unsqueeze(2), score.unsqueeze(1), torch.arange(G, device="cuda")
            before = ((b > a) | ((b == a) & (j[None, :] < j[:, None]))).sum(2)
            ok = ok & (before < c["top_groups"])[:, at // (E // G)]
        a, b = key.unsqueeze(2), key.unsqueeze(1)
        rank = (ok.unsqueeze(1) & ((b > a) | ((b == a) & (at[None, :] < at[:, None])))).sum(2)
        rank = torch.where(ok & (rank < k), rank, k)
        w = torch.zeros((z.shape[0], k + 1), dtype=torch.float64, device="cuda").scatter_(1, rank, p)[:, :k]
        if c["renormalize"]:
            w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
        parts.append(w * c["scale"])
    return {"topk_idx": None, "topk_w": torch.cat(parts)}


def exact(case, seed):
    """The same from the definitions in 64 bits: one expert at a time. The ids and the
    codes are whole numbers."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "route":
        return _exact_route(s, case)
    if op == "quantize":
        x = s["x"]
        return {"codes": None, "scale": torch.maximum(x.max(1).values, -x.min(1).values).double() / 127.0}

    def product(x, sx, pick):
        z = torch.einsum("rk,nk->rn", x.double(), pick(s["w"]).double())
        z = z * torch.outer(sx.double(), pick(s["w_scale"]).double())
        z = _act64(z + pick(s["bias"]).double() if case["bias"] else z, case["act"])
        if case["gated"]:
            u = torch.einsum("rk,nk->rn", x.double(), pick(s["w_up"]).double())
            u = u * torch.outer(sx.double(), pick(s["w_up_scale"]).double())
            z = z * (u + pick(s["bias_up"]).double() if case["bias"] else u)
        return z

    if op == "linear":
        z = product(s["x"], s["x_scale"], lambda t: t)
        return z + s["residual"].double() if case["residual"] else z
    ends = s["offsets"].tolist()
    out = torch.empty((case["n"] * case["k"], case["N"]), dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if b > a:
            if case["gather"]:
                t = s["row_token"][a:b].long()
                rows, scales = s["x"].index_select(0, t), s["x_scale"].index_select(0, t)
            else:
                rows, scales = s["x"][a:b], s["x_scale"][a:b]
            out[a:b] = product(rows, scales, lambda t: t[e])
    return out
