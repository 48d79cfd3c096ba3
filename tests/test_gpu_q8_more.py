"""The 8-bit layers in the places that the package names for them, and what the torch_calls module
hands back to Python."""
import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
from quantized_moe_decode_softmax_gb300 import ops
from test_gpu_q8 import BF16, F16, codes, gen, layer, normal, offsets_of, routed64, scales

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 7, 64])
def test_shared_expert_beside_the_step(n):
    """The step, then the expert on the step's output as residual: bit for bit as the two by
    themselves, on the current stream, another one and in a graph."""
    from gpu_cases import case, device_layer, make_plan, x_tensor
    lay, x = case("qwen3", 2, n)
    dl, xt, plan = device_layer(lay), x_tensor(lay.shape, x), make_plan(lay.shape)
    g, D, F = gen(n), lay.shape.D, lay.shape.F
    shared = q.SharedExpertQ8.quantize(normal(g, (F, D), D ** -0.5), normal(g, (F, D), D ** -0.5), normal(g, (D, F), F ** -0.5))
    step = plan.forward(xt, dl)
    want = shared.forward(xt, residual=step)
    assert not torch.equal(want, step)
    assert torch.equal(plan.forward(xt, dl, shared=shared), want)
    side, out = torch.cuda.Stream(), torch.empty_like(want)
    side.wait_stream(torch.cuda.current_stream())
    plan.forward(xt, dl, out=out, stream=side, shared=shared)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(xt, dl, out=out, shared=shared)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    plan.check()


@pytest.mark.parametrize("n,E,k", [(1, 16, 4), (9, 16, 4), (130, 8, 2), (600, 8, 2)])
def test_shards_of_the_experts(n, E, k):
    """A range of the experts: the slots of the others (and dropped ones) belong to no group, the rows
    behind the last group stay unset, and nothing of them reaches a result."""
    g = gen(n)
    D, F = 256, 128
    w16 = layer(g, E, D, F)
    x, res = normal(g, (n, D)), normal(g, (n, D))
    idx = torch.stack([torch.randperm(E, generator=g, device="cuda")[:k] for _ in range(n)]).int()
    idx[0, 0] = -1
    w = torch.rand((n, k), generator=g, device="cuda")
    whole = q.RoutedExpertsQ8.quantize(*w16)
    for lo, hi in ((0, E), (0, 3), (3, E), (5, 6), (4, 4)):
        shard = q.RoutedExpertsQ8(whole.gate_up, whole.down, experts=(lo, hi))
        only = torch.where((idx >= lo) & (idx < hi), idx, torch.full_like(idx, -1))
        nans = torch.full((n * k, D), float("nan"), dtype=BF16, device="cuda")
        del nans  # (memory that the rows between the products may get)
        got = shard.forward(x, idx, w, residual=res)
        assert bool(torch.isfinite(got).all())
        assert torch.equal(got, whole.forward(x, only, w, residual=res))
        if lo == hi:
            assert torch.equal(got, res)
        if n <= 9:
            want = routed64(x, only, w, whole) + res.double()
            assert float((got.double() - want).norm() / want.norm()) < 0.02


def test_module_takes_the_usual_call_and_hands_back_any_other():
    """One usual call of each operator returns a result; with any one argument changed the module
    returns None, for the checks in Python."""
    c = ops._calls
    assert c is not None
    g = gen(1)
    n, N, K = 5, 48, 64
    lw = q.LinearWeightsQ8(codes(g, (N, K)), scales(g, (N,), 1.0), bias=normal(g, (N,)))
    lg = q.LinearWeightsQ8(codes(g, (2, N, K)), scales(g, (2, N), 1.0))
    l16 = q.LinearWeights(normal(g, (N, K)))
    x, sx, off = codes(g, (n, K)), scales(g, (n,), 1.0), offsets_of([2, 3])
    tok, res, out = torch.arange(n, device="cuda").int(), normal(g, (n, N)), normal(g, (n, N))
    x16, z = normal(g, (n, K)), torch.randn((n, K), generator=g, device="cuda")
    r = q.Router(K, 4, bias=torch.zeros(K, device="cuda"))
    grad = lambda t: t.clone().requires_grad_()  # noqa: E731
    wide = torch.zeros(n, 2 * K, dtype=torch.int8, device="cuda")

    class Sub(torch.Tensor):
        pass

    bad16 = [None, "x", x16.cpu(), x16.float(), x16[:, :K - 8], x16[0], grad(x16), x16.as_subclass(Sub), x16.to_sparse(), x16[:0]]
    bad_x = [None, 1, (x,), (x, sx, sx), [x, sx], (x, None), (None, sx), (x.cpu(), sx), (x, sx.cpu()), (x, sx[:4]), (x, sx.double()),
             (x, sx[:, None]), (x, grad(sx)), (x16, sx), (wide[:, ::2], sx), (x[:, :K - 16], sx), (x[:0], sx[:0]), (x.as_subclass(Sub), sx)]
    bad_out = [1, res.cpu(), res.to(F16), res[:4], res[:, :N - 1], grad(res), res.t().contiguous().t()]
    usual = {
        "linear_q8": ([lw.ref, lw.device_index, (x, sx), res, out, lw.tensors],
                      {0: [0], 1: [-1, 99], 2: bad_x, 3: bad_out, 4: bad_out,
                       5: [None, lw.tensors[:5], lw.tensors[:4], (x,) + lw.tensors[1:], lw.tensors[:4] + (None, None)]}),
        "grouped_q8": ([lg.ref, lg.device_index, (x, sx), off, tok, out, lg.tensors],
                       {0: [0], 1: [-1, 99], 2: bad_x, 3: [None, off[:2], off.long(), off.cpu(), off[:, None]],
                        4: [1, tok.long(), tok.cpu(), tok[:, None], tok[:0]], 5: bad_out, 6: [None, lg.tensors[:4], lw.tensors]}),
        "quantize": ([x16, q.QuantizedRows], {0: [b for b in bad16 if not (torch.is_tensor(b) and b.shape == x16[:, :K - 8].shape)],
                                              1: [None, list, 1]}),
        "route": ([r.ref, z, r.tensors, q.Routing],
                  {0: [0], 1: [None, z.cpu(), z.double(), z[:, :60], z[0], grad(z), z.as_subclass(Sub), z[:0], z.t().contiguous().t()],
                   2: [None, (), (None,), (z[0].clone(),), (r.tensors[0].double(),), [r.tensors[0]]], 3: [None, list, 1]}),
        "linear": ([l16.ref, l16.device_index, x16, res, out, l16.tensors], {2: bad16, 5: [lw.tensors]}),
    }
    for name, (args, others) in usual.items():
        call = getattr(c, name)
        got = call(*args)
        assert torch.is_tensor(got) or isinstance(got, tuple), (name, got)
        for i, values in others.items():
            for v in values:
                assert call(*args[:i], v, *args[i + 1:]) is None, (name, i, v)
        assert call(*args[:-1]) is None and call(*args, None) is None and call() is None
    torch.cuda.synchronize()
