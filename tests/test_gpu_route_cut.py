"""moe_route with a bias where the last place is a matter of roundings: what is behind the
cut may belong before it."""
import math

import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
import route_reference as ref
from test_gpu_route import both

pytestmark = pytest.mark.gpu

F32, F64 = torch.float32, torch.float64


def row(*values):
    return torch.tensor([values], dtype=F32).cuda()


@pytest.mark.parametrize("z,b,want", [
    ([0.0, 0.0, 0.0], [0.0, 0.0, 2.0 ** -26], 2),
    ([0.0, 0.0, 0.0], [0.1, 0.1, math.nextafter(float(torch.tensor(0.1)), 1) + 2.0 ** -27], 2),
    ([20.0, 20.0, 21.0], [0.0, 0.0, 0.0], 2),
    ([21.0, 21.0, 20.0], [0.0, 0.0, 0.0], 0),
    ([20.0, 20.0, 21.0, 21.0, 20.5], [0.0] * 5, 2),
], ids=["bias", "next bias", "saturated", "settled", "two ties"])
def test_an_expert_behind_a_tie_at_the_cut(z, b, want):
    """Keys alike in f32: two experts tie exactly, one behind them is larger."""
    r = both(row(*z), 1, score="sigmoid", bias=row(*b)[0])
    assert r.topk_idx.tolist() == [[want]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [7, 40, 128, 200, 256, 300, 1000])
def test_experts_behind_many_ties(E, score):
    """More exact ties than places, at any ids, and one or two experts that are larger by less than
    an f32 step of a key; the cut before, among and behind the ties; few rows and many."""
    for seed in range(3):
        g = torch.Generator().manual_seed(10 * E + seed)
        order = torch.randperm(E, generator=g)
        tied, larger = order[:E // 2 + 1], order[-2:]
        z = torch.full((E,), -1.0)
        b = torch.full((E,), 0.5)
        z[tied] = 18.0 if score == "sigmoid" else 1.0
        z[larger] = 18.5 if score == "sigmoid" else 1.0 + 2.0 ** -23
        z[order[E // 2 + 1:-2]] += torch.rand(E - E // 2 - 3, generator=g)
        for k in sorted({1, 2, 3, E // 2, min(64, E // 2 + 2)}):
            both(z[None].cuda(), min(k, 64), score=score, bias=b.cuda(), renormalize=seed % 2 == 0)
    both(z[None].repeat(900, 1).cuda(), 2, score=score, bias=b.cuda())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_saturated_16_bit_logits_with_a_bias_of_zeros(dtype):
    """A bias that training has not moved yet, and logits of few different values."""
    g = torch.Generator().manual_seed(3)
    z = (16.0 + torch.randint(0, 8, (60, 64), generator=g) / 8).to(dtype).cuda()
    for k in (1, 2, 6):
        both(z, k, score="sigmoid", bias=torch.zeros(64, device="cuda"))
        both(z, k, score="sigmoid", bias=torch.zeros(64, device="cuda"), groups=8, top_groups=3)


def test_a_large_score_behind_the_cut():
    """Softmax: two small scores, whose own errors tell them apart, and a large one with a bias that
    brings it next to them."""
    z = row(-13.8, -13.9, -9.0, -9.0, -9.0, -0.37806016, -10.0, 0.0)
    b = row(0.0, 0.0, -2.0, -2.0, -2.0, -0.4064935, -2.0, -2.0)[0]
    assert both(z, 1, bias=b).topk_idx.tolist() == [[5]]


def cancelled(E, n, seed):
    """Rows of E logits and a bias: expert `big` has a score of about 0.85 and a bias that leaves
    about 3e-6 of it; experts 3 and 4 have such scores, 1e-8 to 6e-8 apart; the others are far below."""
    g = torch.Generator().manual_seed(seed)
    big = E - 2
    bias = torch.full((E,), -2.0, dtype=F64)
    bias[big] = -0.84
    bias[3] = bias[4] = 0.0
    bias = bias.to(F32)
    u = torch.rand((n, 3), generator=g, dtype=F64)
    small = 3e-6 + 1e-6 * u[:, 0]
    next_small = small - (1e-8 + 5e-8 * u[:, 1])
    p = -float(bias[big]) + small + 2e-7 * (2 * u[:, 2] - 1)
    z = torch.log((1 - p - small - next_small) / (E - 3))[:, None].repeat(1, E)
    z[:, 3], z[:, 4], z[:, big] = torch.log(small), torch.log(next_small), torch.log(p)
    return z.to(F32).cuda(), bias.cuda()


@pytest.mark.parametrize("E", [40, 64, 250, 500])
def test_rows_with_a_large_score_behind_the_cut(E):
    z, b = cancelled(E, 1500, E)
    both(z[:60].contiguous(), 1, bias=b)
    both(z[:700].contiguous(), 1, bias=b)
    both(z, 1, bias=b)
    z, b = cancelled(E, 4200, E + 1)
    both(z, 1, bias=b)
    both(z, 2, bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [64, 65, 128, 129, 256])
def test_64_places_and_the_one_left_out(E, score):
    """The most places, by lanes that rank in their registers (few rows) and in shared memory."""
    g = torch.Generator(device="cuda").manual_seed(E)
    z = 2 * torch.randn((70, E), generator=g, device="cuda")
    b = 0.2 * torch.randn(E, generator=g, device="cuda")
    for rows in (z[:9], z):
        both(rows, 64, score=score, bias=b)
    if E % 8 == 0:
        both(z[:9], 64 if E > 64 else 32, score=score, bias=b, groups=8, top_groups=4 + (E == 64), group_score="top2")


@pytest.mark.parametrize("E,n", [(64, 40), (250, 900), (256, 4200), (1000, 300)])
def test_rows_of_one_large_score_and_rows_of_equal_logits(E, n):
    """Softmax rows in which nearly all scores are next to zero, 16-bit logits that tie, rows of zeros as
    padded batches have them; biases of zeros, of one sign, of a few steps."""
    g = torch.Generator().manual_seed(E)
    z = 6 * torch.randn((n, E), generator=g)
    z[::3, 5] = 40.0
    z[1::7] = 0.0
    z = z.to(torch.bfloat16).cuda()
    for b in (torch.zeros(E), -0.25 * torch.rand(E, generator=g), 2.0 ** -20 * torch.randint(0, 3, (E,), generator=g)):
        for score in ("softmax", "sigmoid"):
            both(z, 6, score=score, bias=b.to(F32).cuda(), renormalize=False)
