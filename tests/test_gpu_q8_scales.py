"""Products of 8-bit codes whose scales are far from 1: the result is in range, whatever the sum
times one of the scales would be."""
import pytest
import torch

import ops_reference as ref
import q8_reference as ref8
import quantized_moe_decode_softmax_gb300 as q
from test_gpu_q8 import codes, gen, normal, offsets_of, scales

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16

# (rows, columns, inputs): a handful of rows, some, many
SIZES = [(1, 256, 512), (3, 72, 48), (12, 2048, 2048), (300, 256, 512), (700, 130, 2064)]
# x_scale, scale: row scales at both ends of what rows of bf16 values have; the largest of weights
SCALES = [(2e36, 1e-10), (2e36, 1e-36), (1e-42, 1e12), (2.0 ** -140, 2.0 ** 90), (1e-25, 1e29)]


@pytest.mark.parametrize("sx,sw", SCALES, ids=lambda v: f"{v:.0e}")
@pytest.mark.parametrize("n,N,K", SIZES)
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
def test_linear(n, N, K, sx, sw, gated):
    g = gen(n)
    t = {"w": codes(g, (N, K)), "scale": scales(g, (N,), sw)}
    if gated:  # (the up product at 1, or less)
        t.update(w_up=codes(g, (N, K)), scale_up=scales(g, (N,), min(5e28, 1 / (sx * K ** 0.5 * 5000))))
    x, xs = codes(g, (n, K)), scales(g, (n,), sx)
    x[0], t["w"][0], t["w"][1] = 127, 127, -128
    r, d = ref8.product(x, xs, **t)
    ref.check(q.moe_linear_q8((x, xs), q.LinearWeightsQ8(**t)), r, d)


@pytest.mark.parametrize("sx,sw", SCALES, ids=lambda v: f"{v:.0e}")
@pytest.mark.parametrize("counts", [[2, 1, 0, 1], [9, 0, 20, 11], [300, 0, 77, 5]], ids=lambda c: str(sum(c)))
def test_grouped(counts, sx, sw):
    E, N, K, n = len(counts), 72, 512, sum(counts)
    g = gen(n)
    t = {"w": codes(g, (E, N, K)), "scale": scales(g, (E, N), sw)}
    x, xs = codes(g, (n, K)), scales(g, (n,), sx)
    t["w"][:, 0], x[:] = 127, x.abs()
    out = q.moe_grouped_linear_q8((x, xs), q.LinearWeightsQ8(**t), offsets_of(counts))
    at = 0
    for e, c in enumerate(counts):
        r, d = ref8.product(x[at:at + c], xs[at:at + c], t["w"][e], t["scale"][e])
        ref.check(out[at:at + c], r, d)
        at += c


@pytest.mark.parametrize("n", [1, 12, 300])
def test_a_row_of_the_largest_values(n):
    """Rows of bf16 values around 3e38, as the quantiser takes them, through small weights."""
    g = gen(n)
    N, K = 2048, 2048
    x = (normal(g, (n, K), 0.2, torch.float32).clamp(-1, 1) * 3e38).to(BF16)
    x[:, 0] = 3e38
    w = normal(g, (N, K), 1e-5)
    lw, xq = q.LinearWeightsQ8.quantize(w), q.moe_quantize_rows(x)
    r, d = ref8.product(*xq, lw.tensors[0], lw.tensors[2])
    out = q.moe_linear_q8(xq, lw)
    assert bool(torch.isfinite(out).all())
    ref.check(out, r, d)
