"""Plain 64-bit forms of the products of 8-bit codes, with the error each output may have.

A sum of products of whole numbers is exact in f32 while no partial leaves 2^24, which
S = sum_k |x w| bounds; above, K additions lose at most 2^-23 of a partial each, as for the
products of 16-bit values. Scaling it is two products (2 x 2^-24), the bias one addition."""
import torch

import ops_reference as ref


def quantized(x):
    """Codes and scale of rows: the exact quotient, halves to even (in 64 bits a quotient of
    two 16-bit values is off by 2^-53 of itself and at least 1e-6 away from a half, or on it)."""
    z = x.double()
    m = z.abs().amax(1, keepdim=True)
    codes = torch.where(m > 0, torch.round(z * 127 / m), torch.zeros_like(z))
    return codes.to(torch.int8), (m[:, 0] / 127).float()


def product(x, sx, w, scale, bias=None, w_up=None, scale_up=None, bias_up=None, act="none", limit=0.0, residual=None):
    """(exact result, bound of its error before the last rounding), f64."""
    def sums(m, sw, b):
        xd, md = x.double(), m.double()
        s = xd.abs() @ md.abs().t()
        d = torch.where(s < 2.0 ** 24, torch.zeros_like(s), s * (m.shape[1] + 16) * 2.0 ** -23)
        by = sx.double()[:, None] * sw.double()[None, :]
        z = (xd @ md.t()) * by
        d = d * by.abs() + z.abs() * 2.0 ** -23
        if b is not None:
            z = z + b.double()
            d = d + z.abs() * 2.0 ** -24
        return z, d

    z, d = sums(w, scale, bias)
    if w_up is not None:
        u, du = sums(w_up, scale_up, bias_up)
        if limit > 0:
            z, u = z.clamp(max=limit), u.clamp(-limit, limit)
    a = ref.act64(act, z)
    da = d if act == "none" else 1.13 * d + z.abs() * 2.0 ** -19 + 2.0 ** -22
    if w_up is not None:
        da = a.abs() * du + u.abs() * da + da * du + (a * u).abs() * 2.0 ** -24
        a = a * u
    if residual is not None:
        a = a + residual.double()
        da = da + a.abs() * 2.0 ** -23
    return a, da
