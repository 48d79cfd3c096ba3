"""The operators of include/moe_ops.h on the GPU: ranges and refusals beside test_gpu_ops.py."""
import math

import pytest
import torch

import ops_reference as ref
import quantized_moe_decode_softmax_gb300 as q
from test_gpu_ops import check_grouped, combine_ref, gen, normal, offsets_of, weights

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def relative_error(act, z):
    """Bound of the activation's own relative error, from its roundings: the hardware's
    2^x (2^-22) and 1/x (2^-23), three more roundings of 2^-24, the fit of the exact
    GELU (1e-6), and the rounding of the exponent t, an absolute error of at most
    |t| 2^-24 per operation that makes it (SiLU 1, tanh GELU 3, GELU 2, and half of
    one for the constant), after a shift by 16 for SiLU and tanh GELU; times ln 2."""
    if act == "none":
        return torch.zeros_like(z)
    if act == "gelu":
        return 2.0 ** -18 + z ** 2 * 2.0 ** -23
    t = z.abs() if act == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3).abs()
    return 2.0 ** -18 + t * 2.0 ** -22


def act_exact(act, z):
    """The activation in 64 bits without cancellation or overflow in the negative tail."""
    if act == "none":
        return z
    if act == "gelu":
        return z * torch.exp(torch.special.log_ndtr(z))
    t = z if act == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    return torch.where(t < -1, z * torch.exp(t) / (1 + torch.exp(t.clamp(max=0))), z / (1 + torch.exp(-t.clamp(min=-1))))


@pytest.mark.parametrize("n", [2, 90])
@pytest.mark.parametrize("up", [None, 1.0, 1000.0], ids=["plain", "gated", "gated_1000"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
def test_activations_keep_their_relative_error(act, dtype, up, n):
    """The tail of every activation, down to the smallest numbers of the type: through
    an identity product, each result within half a step of the type and the
    activation's relative error. `up` multiplies it (a constant second product)."""
    z = torch.cat([-torch.linspace(0, 16, 1500), -torch.linspace(16, 104, 600), torch.linspace(0, 20, 300),
                   torch.logspace(-6, 0, 50), -torch.logspace(-6, 0, 50)]).cuda().to(dtype)
    w = torch.zeros(8, 8, dtype=dtype, device="cuda")
    w[0, 0] = 1
    bias = torch.zeros(8, dtype=dtype, device="cuda")
    lw = q.LinearWeights(w, w_up=None if up is None else torch.zeros_like(w),
                         bias_up=None if up is None else bias.fill_(up), activation=act)
    out = []
    for part in z.split(n):
        x = torch.zeros(part.numel(), 8, dtype=dtype, device="cuda")
        x[:, 0] = part
        out.append(q.moe_linear(x, lw)[:, 0])
    d = z.double()
    r = act_exact(act, d) * (1.0 if up is None else up)
    out = torch.cat(out)
    # f16: from 65520 = 65504 + half a step on, a value rounds to infinity (here for act "none" only, where r is exact)
    over = r.abs() >= 65520 if dtype == F16 else torch.zeros_like(r, dtype=torch.bool)
    assert torch.equal(out[over].double(), r[over].sign() * math.inf)
    # below 2^-135, half the smallest subnormal of bf16, the activation may be zero
    ref.check(out[~over], r[~over], (r.abs() * relative_error(act, d) + 2.0 ** -135 * (up or 1.0))[~over])


def many(E, sizes):
    """Rows per expert: `sizes` in turn at both ends and around every 416th expert (the
    tcgen05 products number their work for so many experts at a time), none elsewhere."""
    counts, at = [0] * E, 0
    for e in sorted({e for b in range(0, E + 1, 416) for e in range(b - 2, b + 2) if e != b - 1} | {7, E // 2, E - 1}):
        if 0 <= e < E:
            counts[e] = sizes[at % len(sizes)]
            at += 1
    return counts


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("sizes", [(1, 2, 3), (40, 1, 150, 9)], ids=["streamed", "tcgen05"])
@pytest.mark.parametrize("E", [415, 416, 417, 832, 833, 1024])
def test_grouped_over_many_experts(E, sizes, gated, gather):
    counts = many(E, sizes)
    rows, (N, K) = sum(counts), (40, 72)
    assert (rows <= 64) == (sizes[0] == 1)
    g = gen(E + gated)
    t = weights(g, (E,), N, K, BF16, gated, True)
    x = normal(g, (rows, K))
    token = torch.randperm(rows, device="cuda", generator=g).to(torch.int32) if gather else None
    out = q.moe_grouped_linear(x, q.LinearWeights(**t, activation="silu"), offsets_of(counts), row_token=token)
    check_grouped(x, t, counts, "silu", out, token)
    q.moe_ops_check()


@pytest.mark.parametrize("n", [5, 300])
def test_grouped_with_every_expert_in_use(n):
    """1024 experts that all hold rows, or nearly all, in the order that the grouping gives."""
    E, k, N, K = 1024, 8, 24, 64
    g = gen(n)
    idx = torch.randint(0, E, (n, k), device="cuda", generator=g).to(torch.int32)
    t = weights(g, (E,), N, K, F16, False, False)
    x = normal(g, (n, K), 1.0, F16)
    s = q.moe_group_slots(idx, E)
    counts = torch.bincount(idx.reshape(-1).long(), minlength=E).tolist()
    check_grouped(x, t, counts, "none", q.moe_grouped_linear(x, q.LinearWeights(**t), s.offsets, row_token=s.slot_token),
                  s.slot_token)


# the widest, the longest and the most rows, through both kernels
@pytest.mark.parametrize("n,N,K", [(1, 150001, 512), (66, 150001, 64), (1, 1 << 20, 8), (66, 1 << 20, 8), (3, 24, 65536),
                                   (70, 24, 65536), (100000, 16, 16), (70001, 7, 8)])
def test_linear_far_sizes(n, N, K):
    g = gen(n + N)
    t = weights(g, (), N, K, BF16, False, True)
    x = normal(g, (n, K))
    ref.check(q.moe_linear(x, q.LinearWeights(**t)), *ref.product(x, **t))


@pytest.mark.parametrize("N", [8, 5])
def test_combine_more_tokens_than_a_grid_has_rows(N):
    n, k = 70001, 2
    g = gen(N)
    y = normal(g, (n, N))
    of = torch.randint(-1, n, (n, k), device="cuda", generator=g).to(torch.int32)
    w = torch.rand((n, k), device="cuda", generator=g)
    res = normal(g, (n, N))
    ref.check(q.moe_combine_slots(y, of, w, residual=res), *combine_ref(y, of, w, res))
