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


def test_weights_follow_their_tensors():
    """A weight that is given another storage is found at its new address; one that has
    become another shape or type is refused."""
    w, b = torch.zeros(16, 24, dtype=BF16), torch.zeros(16, dtype=BF16)
    lw = q.LinearWeights(w, w_up=torch.zeros_like(w), bias=b, activation="silu")
    ref = lw.ref
    for t, field in ((w, "w"), (lw.tensors[1], "w_up"), (b, "bias")):
        old = t.data  # keeps the old storage, so that its address is not given out again
        t.data = torch.ones_like(t)
        c = lw.current()
        assert getattr(c, field) == t.data_ptr() == getattr(lw.c, field) and t.data_ptr() != old.data_ptr()
        assert lw.ref == ref and (c.N, c.K, c.ldw, c.activation) == (16, 24, 24, q.MOE_EPI_SILU)
    for t in lw.tensors[:2]:
        t.data = torch.zeros(16, 32, dtype=BF16)[:, :24]
    with pytest.raises(ValueError):  # w_up would have followed w: their strides have to agree
        w.data = torch.zeros(16, 24, dtype=BF16)
        lw.current()
    w.data = lw.tensors[1].data
    assert lw.current().ldw == 32
    x = torch.zeros(2, 24, dtype=BF16)
    for bad in (torch.zeros(8, 24, dtype=BF16), torch.zeros(16, 24, dtype=torch.float16), torch.zeros(24, 16, dtype=BF16).t()):
        keep, w.data = w.data, bad
        with pytest.raises(ValueError):
            lw.current()
        with pytest.raises(ValueError):
            q.moe_linear(x, lw)
        w.data = keep


@pytest.mark.gpu
def test_calls_follow_weights_that_move(module):
    """The same handle before and after its weights get other storages, other strides,
    a trip to the host and back; a graph keeps what it was captured with."""
    g = torch.Generator(device="cuda").manual_seed(5)
    t = lambda *s: torch.empty(s, dtype=BF16, device="cuda").normal_(generator=g)  # noqa: E731
    x, off = t(5, 64), torch.tensor([0, 2, 2, 5], dtype=torch.int32, device="cuda")
    w, b, gw = t(16, 64), t(16), t(3, 16, 64)
    lw, lg = q.LinearWeights(w, bias=b), q.LinearWeights(gw)
    kept = []  # the old storages stay alive: a call that used them would give the old answer

    def fresh():
        return q.moe_linear(x, q.LinearWeights(w, bias=b)), q.moe_grouped_linear(x, q.LinearWeights(gw), off)

    def same():
        want, got = fresh(), (q.moe_linear(x, lw), q.moe_grouped_linear(x, lg, off))
        return all(torch.equal(a, c) for a, c in zip(want, got))

    assert same()
    for new in ((t(16, 64), t(16), t(3, 16, 64)), (t(16, 80)[:, :64], t(32)[:16], t(16, 3, 64).transpose(0, 1)),
                (t(32, 64)[::2], t(16), t(1, 16, 64).expand(3, 16, 64))):
        for p, n in zip((w, b, gw), new):
            kept.append(p.data)
            p.data = n
        assert same() and same()
    before = q.moe_linear(x, lw)
    for p in (w, b, gw):
        kept.append(p.data)
        p.data = p.data.cpu()
    for call in (lambda: q.moe_linear(x, lw), lambda: q.moe_grouped_linear(x, lg, off)):
        with pytest.raises(ValueError):
            call()
    for p in (w, b, gw):
        p.data = p.data.cuda()
    assert same() and torch.equal(q.moe_linear(x, lw), before)
    kept.append(w.data)
    w.data = w.data[:8]  # the same address, fewer rows
    with pytest.raises(ValueError):
        q.moe_linear(x, lw)
    w.data = t(16, 64)
    assert same()
    size = b.untyped_storage().nbytes()
    b.untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        q.moe_linear(x, lw)
    b.untyped_storage().resize_(size)
    b.zero_()
    assert same()
