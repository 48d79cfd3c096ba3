"""Plain 64-bit forms of the operators of moe_ops.h, with the error each output
may have.

The bound of a product is derived, not fitted. With S = sum_k |x w| (+ |bias|):
the K additions of f32 partials lose at most one unit in the last place, 2^-23 of
the partial, each (rounding or truncating), so |z - z_ref| <= (K + 16) 2^-23 S =
d. An activation's slope is at most 1.13, its own error at most 2^-19 |z| + 2^-22.
A gated product of a and u adds |a| d_u + |u| d_a + d_a d_u. The result is
rounded once: half a step of the output type, plus half its smallest step."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def act64(kind, z):
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def product(x, w, bias=None, w_up=None, bias_up=None, act="none", limit=0.0, residual=None):
    """(exact result, bound of its error before the last rounding), f64."""
    def sums(m, b):
        xd, md = x.double(), m.double()
        z, s = xd @ md.t(), xd.abs() @ md.abs().t()
        if b is not None:
            z, s = z + b.double(), s + b.double().abs()
        return z, s * (m.shape[1] + 16) * 2.0 ** -23

    z, d = sums(w, bias)
    if w_up is not None:
        u, du = sums(w_up, bias_up)
        if limit > 0:
            z, u = z.clamp(max=limit), u.clamp(-limit, limit)
    a = act64(act, z)
    da = d if act == "none" else 1.13 * d + z.abs() * 2.0 ** -19 + 2.0 ** -22
    if w_up is not None:
        da = a.abs() * du + u.abs() * da + da * du
        a = a * u
    if residual is not None:
        a = a + residual.double()
        da = da + a.abs() * 2.0 ** -23
    return a, da


def check(out, ref, bound):
    """Every element within half a step of the rounded type, beyond the bound."""
    h = HALF_STEP[out.dtype]
    err = (out.double() - ref).abs()
    allowed = bound * (1 + h) + ref.abs() * h * (1 + 2.0 ** -10) + TINY[out.dtype]
    bad = ~(err <= allowed)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {out.numel()} values are off, the worst by "
                                 f"{float((err - allowed).max()):.3e} more than allowed, first at "
                                 f"{torch.nonzero(bad)[0].tolist()}")




def slot_tables(rows, ids, n, k, E):
    """offsets, slot_token, slot_k, slot_of of the (token, rank) list `rows`."""
    offsets = [0] * (E + 1)
    for t, j in rows:
        offsets[ids[t][j] + 1] += 1
    for e in range(E):
        offsets[e + 1] += offsets[e]
    of = [[-1] * k for _ in range(n)]
    for r, (t, j) in enumerate(rows):
        of[t][j] = r
    pad = [-1] * (n * k - len(rows))
    return offsets, [t for t, _ in rows] + pad, [j for _, j in rows] + pad, of
