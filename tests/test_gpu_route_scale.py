"""moe_route with factors at the ends of f32."""
import pytest
import torch

from test_gpu_route import both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [3e38, -3e38, 1e37, 1e-37, 0.0])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scales_near_the_largest_and_smallest(score, renormalize, scale):
    """A weight divided by the sum of all is at most 1: the factor on it stays in range, whatever the
    sum is."""
    g = torch.Generator(device="cuda").manual_seed(1)
    z = 3 * torch.randn((20, 12), generator=g, device="cuda")
    z[0], z[1], z[2] = 0.0, -30.0, -60.0
    for k in (1, 3, 12):
        both(z, k, score=score, renormalize=renormalize, scale=scale)
        both(z, k, score=score, renormalize=renormalize, scale=scale, bias=torch.zeros(12, device="cuda"))
