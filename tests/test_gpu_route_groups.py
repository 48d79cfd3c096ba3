"""moe_route by groups whose best two nearly cancel: the rounding of the terms decides."""
import pytest
import torch

from test_gpu_route import INF, both

pytestmark = pytest.mark.gpu

F32, F64 = torch.float32, torch.float64


def cancelling(groups, n, seed, size):
    """Sigmoid logits and a bias of `groups` pairs: each pair's biases are +-`size`, its two scores
    add up to the row's sum but for less than an f32 step of `size`."""
    g = torch.Generator().manual_seed(seed)
    bias = torch.tensor([size, -size] * groups, dtype=F32)
    step = float(torch.nextafter(bias[0], torch.tensor(INF)) - bias[0])
    s = 0.3 + 0.4 * torch.rand((n, 2 * groups), generator=g, dtype=F64)
    total = (s[:, 0] + s[:, 1])[:, None]
    s[:, 1::2] = total - s[:, ::2] + step * (2 * torch.rand((n, groups), generator=g, dtype=F64) - 1)
    s = s[((s > 0.02) & (s < 0.98)).all(1)]
    return torch.log(s / (1 - s)).to(F32).cuda(), bias.cuda()


@pytest.mark.parametrize("size", [30.0, 1000.0, 20000.0])
@pytest.mark.parametrize("groups,top,n", [(2, 1, 800), (3, 1, 3000), (4, 2, 1500), (8, 3, 40000), (16, 5, 60000)])
def test_biases_that_cancel(groups, top, n, size):
    z, b = cancelling(groups, n, groups, size)
    z = z[:5000].contiguous()
    assert z.shape[0] >= 50
    for rows in (z[:60].contiguous(), z):
        both(rows, 2 * top, score="sigmoid", bias=b, groups=groups, top_groups=top, group_score="top2")
        both(rows, 1, score="sigmoid", bias=b, groups=groups, top_groups=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_kept_out_by_a_large_negative_bias(score):
    """A bias far below every score, instead of -inf, in some groups, in all, and the largest numbers."""
    g = torch.Generator().manual_seed(4)
    z = torch.randn((50, 24), generator=g).cuda()
    for off in (-1e4, -1e9, -3e38):
        for out in ([0, 1, 2, 3], [1, 5, 9, 13, 17, 21], list(range(0, 24, 2)), list(range(24))):
            b = 0.1 * torch.randn(24, generator=g)
            b[out] = off
            for best in ("max", "top2"):
                both(z, 4, score=score, bias=b.cuda(), groups=6, top_groups=2, group_score=best)
