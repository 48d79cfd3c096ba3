"""SharedExpert and RoutedExperts beside the step: what they report and refuse."""
import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
from quantized_moe_decode_softmax_gb300 import _abi, layer, ops

BF16 = torch.bfloat16


class FakeLib:
    """The C functions that a check calls, with the statuses that they answer."""

    def __init__(self, *statuses):
        self.statuses, self.streams = list(statuses), []

    def moe_ops_check(self, stream):
        self.streams.append(stream)
        return self.statuses.pop(0)


class FakeShared:
    dtype = BF16

    def refuse(self, x, out, width):
        pass

    def forward(self, x, residual, out, stream):
        return out.add_(1)


def step_layer(monkeypatch):
    """A MoeDecodeLayer whose step does nothing and whose plan never fails."""
    monkeypatch.setattr(_abi, "moe_decode_forward", lambda *a: None)
    monkeypatch.setattr(_abi, "moe_plan_check", lambda plan: None)
    monkeypatch.setattr(_abi, "moe_plan_create", lambda cfg: 0)  # 0: nothing to free
    return layer.MoeDecodeLayer(8, 2, 512, 256)


def test_check_reports_a_wait_of_the_shared_expert(monkeypatch):
    lay = step_layer(monkeypatch)
    fake = FakeLib(q.MOE_ERR_TIMEOUT, q.MOE_OK, q.MOE_OK)
    monkeypatch.setattr(ops, "_c", fake)
    weights = layer.DeviceLayer.__new__(layer.DeviceLayer)
    weights.D, weights.router_w, weights.router_bias, weights.c_planes = 512, None, None, None
    x, out = torch.zeros(2, 512, dtype=BF16), torch.zeros(2, 512, dtype=BF16)
    lay.check()
    lay.forward(x, weights, out=out, stream=77)
    lay.check()
    assert fake.streams == []  # no shared expert, nothing to ask
    lay.forward(x, weights, out=out, stream=77, shared=FakeShared())
    with pytest.raises(q.MoeError) as e:
        lay.check()
    assert e.value.status == q.MOE_ERR_TIMEOUT and fake.streams == [77]
    lay.check()
    lay.forward(x, weights, out=out, stream=78, shared=FakeShared())
    lay.check()
    assert fake.streams == [77, 77, 78]


def test_experts_have_a_check(monkeypatch):
    ops._lib()
    g, d = torch.zeros(3, 16, 24, dtype=BF16), torch.zeros(3, 24, 16, dtype=BF16)
    for e in (q.SharedExpert(g[0], g[0], d[0]), q.RoutedExperts(g, g, d)):
        monkeypatch.setattr(ops, "_c", FakeLib(q.MOE_OK, q.MOE_ERR_TIMEOUT))
        e.check(stream=5)
        with pytest.raises(q.MoeError):
            e.check(stream=5)


def test_shared_expert_of_another_width_is_refused_before_the_step(monkeypatch):
    ops._lib()
    lay = step_layer(monkeypatch)
    weights = layer.DeviceLayer.__new__(layer.DeviceLayer)
    weights.D, weights.router_w, weights.router_bias, weights.c_planes = 512, None, None, None
    monkeypatch.setattr(_abi, "moe_decode_forward", lambda *a: pytest.fail("launched"))
    g, d = torch.zeros(16, 256, dtype=BF16), torch.zeros(256, 16, dtype=BF16)
    x, out = torch.zeros(2, 512, dtype=BF16), torch.zeros(2, 512, dtype=BF16)
    with pytest.raises(ValueError, match="wide"):
        lay.forward(x, weights, out=out, stream=77, shared=q.SharedExpert(g, g, d))


def test_shared_expert_that_asks_for_gradients_is_refused_before_the_step(monkeypatch):
    ops._lib()
    lay = step_layer(monkeypatch)
    weights = layer.DeviceLayer.__new__(layer.DeviceLayer)
    weights.D, weights.router_w, weights.router_bias, weights.c_planes = 512, None, None, None
    monkeypatch.setattr(_abi, "moe_decode_forward", lambda *a: pytest.fail("launched"))
    t = lambda *s: torch.zeros(*s, dtype=BF16)  # noqa: E731
    for i in range(4):
        given = [t(16, 512), t(16, 512), t(512, 16), t(2, 512)]
        given[i] = torch.nn.Parameter(given[i])
        with pytest.raises(RuntimeError, match="requires a gradient"):
            lay.forward(given[3], weights, out=t(2, 512), stream=77, shared=q.SharedExpert(*given[:3]))


def test_routed_experts_refuse_ids_of_other_tokens(monkeypatch):
    """One row of ids per token: ids of more tokens would be read as ids of the last one."""
    ops._lib()
    g, d = torch.zeros(3, 16, 24, dtype=BF16), torch.zeros(3, 24, 16, dtype=BF16)
    e = q.RoutedExperts(g, g, d)
    monkeypatch.setattr(layer, "moe_group_slots", lambda *a, **k: pytest.fail("launched"))
    ids = lambda n: torch.zeros(n, 2, dtype=torch.int32)  # noqa: E731
    for x, idx in ((torch.zeros(4, 24, dtype=BF16), ids(5)), (torch.zeros(4, 24, dtype=BF16), ids(3)),
                   (torch.zeros(24, dtype=BF16), ids(1)), (torch.zeros(4, 24, dtype=BF16), ids(4)[:, 0])):
        with pytest.raises(ValueError, match="topk_idx"):
            e.forward(x, idx, torch.zeros(idx.shape))


@pytest.mark.gpu
def test_checks_on_the_gpu(monkeypatch):
    """The same on a device and a stream: nothing to report, then a status from a fake of
    the failing call."""
    from gpu_cases import case, device_layer, make_plan, x_tensor
    lay, x = case("qwen3", 2, 4)
    dl, xt = device_layer(lay), x_tensor(lay.shape, x)
    D, F = lay.shape.D, lay.shape.F
    t = lambda *s: torch.zeros(*s, dtype=BF16, device="cuda")  # noqa: E731
    shared, plan, side = q.SharedExpert(t(F, D), t(F, D), t(D, F)), make_plan(lay.shape), torch.cuda.Stream()
    plan.forward(xt, dl, shared=shared)
    plan.check()
    torch.cuda.synchronize()
    out = t(xt.shape[0], D)
    side.wait_stream(torch.cuda.current_stream())
    plan.forward(xt, dl, out=out, stream=side, shared=shared)
    shared.check(side)
    shared.check()
    q.moe_ops_check(side.cuda_stream)
    fake = FakeLib(q.MOE_ERR_TIMEOUT)
    monkeypatch.setattr(ops, "_c", fake)
    with pytest.raises(q.MoeError):
        plan.check()
    assert fake.streams == [side.cuda_stream]
