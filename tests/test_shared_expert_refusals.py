"""A shared expert that cannot run is refused before the step is launched, not after."""
import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
from quantized_moe_decode_softmax_gb300 import _abi, layer, ops
from test_ops_layers import BF16, step_layer

I8 = torch.int8


def weights16(F, D, dtype=BF16):
    return [torch.zeros(*s, dtype=dtype) for s in ((F, D), (F, D), (D, F))]


def shared8(F, D, pad=0):
    codes = lambda n, k: torch.zeros(n, k + pad, dtype=I8)[:, :k]  # noqa: E731
    return q.SharedExpertQ8(q.LinearWeightsQ8(codes(F, D), torch.ones(F), w_up=codes(F, D), scale_up=torch.ones(F), activation="silu"),
                            q.LinearWeightsQ8(codes(D, F), torch.ones(D)))


@pytest.fixture
def step(monkeypatch):
    ops._lib()
    lay = step_layer(monkeypatch)
    w = layer.DeviceLayer.__new__(layer.DeviceLayer)
    w.D, w.router_w, w.router_bias, w.c_planes = 512, None, None, None

    def run(shared, launched):
        seen = []
        monkeypatch.setattr(_abi, "moe_decode_forward", lambda *a: seen.append(1))
        try:
            lay.forward(torch.zeros(2, 512, dtype=BF16), w, out=torch.zeros(2, 512, dtype=BF16), stream=77, shared=shared)
        finally:
            assert bool(seen) == launched
    return run


@pytest.mark.parametrize("F,status", [(24, "MOE_ERR_UNSUPPORTED"), (8, "MOE_ERR_UNSUPPORTED"), (1000, "MOE_ERR_UNSUPPORTED")])
def test_widths_that_the_8_bit_products_do_not_take(step, F, status):
    with pytest.raises(q.MoeError) as e:
        step(shared8(F, 512), launched=False)
    assert e.value.status == getattr(q, status)


def test_row_distances_that_the_8_bit_products_do_not_take(step):
    with pytest.raises(q.MoeError) as e:
        step(shared8(32, 512, pad=8), launched=False)
    assert e.value.status == q.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("F", [12, 7])
def test_widths_that_the_16_bit_products_do_not_take(step, F):
    with pytest.raises(q.MoeError) as e:
        step(q.SharedExpert(*weights16(F, 512)), launched=False)
    assert e.value.status == q.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("make", [lambda: q.SharedExpert(*weights16(24, 512)), lambda: shared8(32, 512)], ids=["16", "8"])
def test_what_fits_reaches_the_step(step, make):
    """(The expert itself then asks for a CUDA device.)"""
    with pytest.raises(ValueError, match="CUDA"):
        step(make(), launched=True)


def test_statuses_of_weights():
    ops._lib()
    g = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    for w, status in ((q.LinearWeights(g(16, 32)), q.MOE_OK), (q.LinearWeights(g(3, 16, 24)), q.MOE_OK),
                      (q.LinearWeights(g(16, 12)), q.MOE_ERR_UNSUPPORTED), (q.LinearWeights(g(3, 16, 12)), q.MOE_ERR_UNSUPPORTED),
                      (q.LinearWeights(g(16, 32), act_limit=1.0), q.MOE_ERR_INVALID_ARG),
                      (q.LinearWeightsQ8(g(16, 32, dtype=I8), torch.ones(16)), q.MOE_OK),
                      (q.LinearWeightsQ8(g(3, 16, 32, dtype=I8), torch.ones(3, 16)), q.MOE_OK),
                      (q.LinearWeightsQ8(g(3, 16, 24, dtype=I8), torch.ones(3, 16)), q.MOE_ERR_UNSUPPORTED)):
        assert w.status == status


def test_matrices_of_two_types():
    ops._lib()
    gate, up, _ = weights16(24, 512, torch.float16)
    with pytest.raises(TypeError):
        q.SharedExpert(gate, up, weights16(24, 512)[2])


@pytest.mark.gpu
def test_another_device_than_the_steps(step):
    t = [w.cuda() for w in weights16(32, 512)]
    with pytest.raises(ValueError, match="is on cuda"):
        step(q.SharedExpert(*t), launched=False)
