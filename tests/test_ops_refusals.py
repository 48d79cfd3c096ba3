"""Calls of the operators that are refused before any CUDA work, with and without the torch_calls module."""
import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
from quantized_moe_decode_softmax_gb300 import build as qbuild
from quantized_moe_decode_softmax_gb300 import ops

BF16 = torch.bfloat16


@pytest.fixture(params=[True, False], ids=["module", "ctypes"])
def module(request, monkeypatch):
    qbuild.build()
    ops._lib()
    if not request.param:
        monkeypatch.setattr(ops, "_calls", None)
    return request.param


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request):
    return request.param


def tensors(device):
    t = lambda *s: torch.zeros(*s, dtype=BF16, device=device)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=device)  # noqa: E731
    return dict(x=t(4, 24), w=t(16, 24), w_up=t(16, 24), bias=t(16), bias_up=t(16), residual=t(4, 16), out=t(4, 16),
                gw=t(3, 16, 24), gbias=t(3, 16), topk_w=torch.zeros(2, 2, device=device), y=t(4, 16), of=i(2, 2), off=i(4))


def calls(t):
    """Every operator that takes floating-point tensors, with the names of those."""
    linear = lambda: q.moe_linear(t["x"], q.LinearWeights(t["w"], w_up=t["w_up"], bias=t["bias"], bias_up=t["bias_up"]),  # noqa: E731
                                  residual=t["residual"], out=t["out"])
    grouped = lambda: q.moe_grouped_linear(t["x"], q.LinearWeights(t["gw"], bias=t["gbias"]), t["off"], out=t["out"])  # noqa: E731
    combine = lambda: q.moe_combine_slots(t["y"], t["of"], t["topk_w"], residual=t["residual"][:2], out=t["out"][:2])  # noqa: E731
    return [(linear, ("x", "w", "w_up", "bias", "bias_up", "residual", "out")), (grouped, ("x", "gw", "gbias", "out")),
            (combine, ("y", "topk_w", "residual", "out"))]


def passes(call, device):
    """The checks let the call through: it runs, or has no GPU to run on."""
    if device == "cuda":
        call()
    else:
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_no_gradient_is_dropped(module, device):
    """Whatever asks for a gradient is refused where gradients are enabled, and not under no_grad."""
    for i, (call, names) in enumerate(calls(tensors(device))):
        passes(call, device)
        for name in names:
            t = tensors(device)
            t[name] = torch.nn.Parameter(t[name])
            call = calls(t)[i][0]
            with pytest.raises(RuntimeError, match="requires a gradient"):
                call()
            with torch.no_grad():
                passes(call, device)


def test_no_tangent_is_dropped(module, device):
    fw = torch.autograd.forward_ad
    for i, (_, names) in enumerate(calls(tensors(device))):
        for name in names:
            t = tensors(device)
            with fw.dual_level():
                t[name] = fw.make_dual(t[name], torch.ones_like(t[name]))
                call = calls(t)[i][0]
                with pytest.raises(RuntimeError, match="forward-mode tangent"):
                    call()
                with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode tangent"):
                    call()


def test_module_hands_back_what_is_not_usual():
    qbuild.build()
    ops._lib()
    c = ops._calls
    assert c is not None
    w = torch.zeros(16, 24, dtype=BF16)
    lw, x, i = q.LinearWeights(w), torch.zeros(2, 24, dtype=BF16), torch.zeros(2, 2, dtype=torch.int32)
    for dev in (lw.device_index, 0):
        for bad in (x, None, "x", torch.nn.Parameter(x), x.to_sparse()):
            assert c.linear(lw.ref, dev, bad, None, None, lw.tensors) is None
    for bad in ((), None, (w,), (w, "w", None, None), (torch.nn.Parameter(w), None, None, None)):
        assert c.linear(lw.ref, 0, x, None, None, bad) is None
        assert c.grouped(lw.ref, 0, x, i, None, None, bad) is None
    assert c.grouped(lw.ref, 0, x, i, None, None, lw.tensors) is None
    assert c.grouped(lw.ref, 0, x, None, None, None, lw.tensors) is None
