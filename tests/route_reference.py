"""Routing to experts in plain 64-bit Python, one row at a time, with the error a
weight may have."""
import math

import torch

# Relative error of one f32 score. Sigmoid: expf (2 ulp), 1 + e, the division, each at most
# 2^-23 of the result. Softmax: l - max rounds (2^-24 |l - max|, below), expf, up to 37
# additions of positive terms in the divisor, its reciprocal and the product.
SCORE_ERR = {"sigmoid": 5 * 2.0 ** -23, "softmax": 43 * 2.0 ** -24}


def scores(row, kind):
    """s of one row of logits (floats); NaN where the logit takes no part."""
    part = [v for v in row if v > -math.inf]
    if kind == "sigmoid":
        # 1 / (1 + e^-v) without overflow
        return [math.nan if not v > -math.inf else 1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v))
                for v in row]
    if not part:
        return [math.nan] * len(row)
    m = max(part)
    e = [math.nan if not v > -math.inf else 1.0 if v == m else math.exp(v - m) for v in row]
    total = math.fsum(v for v in e if v == v)
    return [v / total for v in e]


def route_row(row, k, kind, bias, groups, top_groups, group_score, renormalize, scale):
    E = len(row)
    s = scores(row, kind)
    size = E // groups
    ok = [s[e] == s[e] and (bias is None or bias[e] > -math.inf) for e in range(E)]
    # without a bias the order is that of the logits, wherever their scores round to the same
    key = [(s[e] + bias[e] if bias is not None else row[e]) if ok[e] else -math.inf for e in range(E)]
    kept = list(range(groups))
    if top_groups < groups:
        def of_group(g):
            own = sorted((e for e in range(g * size, (g + 1) * size) if ok[e]), key=lambda e: (-key[e], e))
            if not own:
                return -math.inf
            if group_score == "max":
                return key[own[0]]
            return math.fsum((s[e] + bias[e] if bias is not None else s[e]) for e in own[:2])
        value = [of_group(g) for g in range(groups)]
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
    ranked = sorted((e for e in range(E) if ok[e] and e // size in kept), key=lambda e: (-key[e], e))[:k]
    w = [s[e] for e in ranked]
    rel = [SCORE_ERR[kind]] * len(w)
    if kind == "softmax" and w:
        top = max(v for v in row if v > -math.inf)
        if math.isfinite(top):
            rel = [r + 2.0 ** -24 * (top - row[e]) for r, e in zip(rel, ranked)]
    if renormalize:
        if kind == "sigmoid" and ranked and max(row[e] for e in ranked) < -40:
            t = max(row[e] for e in ranked)  # (their ratios, where they themselves underflow)
            w = [math.exp(row[e] - t) for e in ranked]
            rel = [r + 2.0 ** -24 * (t - row[e]) for r, e in zip(rel, ranked)]
        total = math.fsum(w)
        worst = max(rel, default=0.0)
        w = [v / total if total > 0 else 0.0 for v in w]
        rel = [r + worst + 8 * 2.0 ** -24 for r in rel]
    pad = k - len(ranked)
    return (ranked + [-1] * pad, [v * scale for v in w] + [0.0] * pad,
            [abs(v * scale) * (r + 2 * 2.0 ** -24) + 2.0 ** -140 for v, r in zip(w, rel)] + [0.0] * pad)


def check(routing, logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_score="max", renormalize=True,
          scale=1.0):
    """Ids are equal, weights within their error."""
    b = None if bias is None else bias.double().tolist()
    rows = [route_row(r, k, score, b, groups, top_groups, group_score, renormalize, scale)
            for r in logits.double().tolist()]
    got_i, got_w = routing.topk_idx.tolist(), routing.topk_w.double().tolist()
    assert routing.topk_idx.dtype == torch.int32 and routing.topk_w.dtype == torch.float32
    assert len(got_i) == len(rows)
    for t, (ids, w, err) in enumerate(rows):
        assert got_i[t] == ids, f"row {t}: {got_i[t]} instead of {ids}"
        for j in range(k):
            assert abs(got_w[t][j] - w[j]) <= err[j], f"row {t} rank {j}: {got_w[t][j]} instead of {w[j]} +- {err[j]:.2e}"
