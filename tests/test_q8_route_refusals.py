"""Calls of the router and of the 8-bit products that are refused before any CUDA work, from C
and from Python, with and without the torch_calls module."""
import ctypes
import re

import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
from quantized_moe_decode_softmax_gb300 import build as qbuild
from quantized_moe_decode_softmax_gb300 import ops
from test_ops_cpu import header

BF16, I8 = torch.bfloat16, torch.int8
P = 1 << 20  # a 16-byte aligned address; no refused call reads it
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return ops._lib()


@pytest.fixture(params=[True, False], ids=["module", "ctypes"])
def module(request, monkeypatch, lib):
    if not request.param:
        monkeypatch.setattr(ops, "_calls", None)
    return request.param


def test_header_and_binding_agree(lib):
    for name in ("moe_product_q8", "moe_router"):
        body = re.search(r"typedef struct \{([^}]*)\}\s*%s;" % name, header()).group(1)
        assert re.findall(r"(\w+)\s*;", body) == [f for f, _ in getattr(q, name)._fields_]
    for name, value in re.findall(r"(MOE_SCORE_\w+)\s*=\s*(\d+)", header()):
        assert getattr(q, name) == int(value)


def product(**over):
    f = dict(dtype=q.MOE_DTYPE_BF16, E=1, N=64, K=128, w=P, w_up=None, ldw=128, stride_e=64 * 128, scale=P, scale_up=None,
             bias=None, bias_up=None, activation=0, act_limit=0.0)
    f.update(over)
    return q.moe_product_q8(**f)


UP = dict(w_up=P, scale_up=P)
BAD_PRODUCT = [
    (dict(w=None), 1), (dict(w=P + 8), 1), (dict(scale=None), 1), (dict(scale=P + 2), 1), (dict(w_up=P), 1),
    (dict(scale_up=P), 1), (dict(UP, w_up=P + 8), 1), (dict(UP, scale_up=P + 1), 1), (dict(bias=P + 1), 1), (dict(dtype=0), 2),
    (dict(dtype=3), 1), (dict(E=0), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(K=-16), 1), (dict(K=120), 2),
    (dict(K=65552, ldw=65552), 2), (dict(N=(1 << 20) + 1), 2), (dict(ldw=112), 1), (dict(ldw=136), 1), (dict(bias_up=P), 1),
    (dict(activation=4), 1), (dict(activation=-1), 1), (dict(act_limit=1.0), 1), (dict(UP, act_limit=-1.0), 1),
    (dict(UP, act_limit=NAN), 1), (dict(UP, act_limit=INF), 1),
]


@pytest.mark.parametrize("over,status", BAD_PRODUCT, ids=[str(o) for o, _ in BAD_PRODUCT])
def test_products_refuse_bad_weights(lib, over, status):
    p = product(**over)
    at = ctypes.addressof(p)
    assert lib.moe_linear_q8(at, P, 65552, P, 1, None, 0, P + 4096, 1 << 21, None) == status
    assert lib.moe_grouped_linear_q8(at, P, None, P, 65552, P, 4, 4, P + 4096, 1 << 21, None) == status


def test_linear_refuses_bad_calls(lib):
    p, two = product(), product(E=2)
    good = dict(p=ctypes.addressof(p), x=P, ldx=128, s=4 * P, n=3, res=None, ldr=0, out=2 * P, ldo=64)
    for over, status in [(dict(p=None), 1), (dict(x=None), 1), (dict(s=None), 1), (dict(out=None), 1), (dict(n=-1), 1),
                         (dict(ldx=112), 1), (dict(ldx=136), 1), (dict(ldo=63), 1), (dict(x=P + 8), 1), (dict(s=4 * P + 2), 1),
                         (dict(out=2 * P + 1), 1), (dict(out=P), 1), (dict(s=2 * P), 1), (dict(res=3 * P, ldr=63), 1),
                         (dict(res=3 * P + 1, ldr=64), 1), (dict(res=2 * P, ldr=72), 1), (dict(n=(1 << 24) + 1), 2),
                         (dict(p=ctypes.addressof(two)), 1)]:
        a = dict(good, **over)
        st = lib.moe_linear_q8(a["p"], a["x"], a["ldx"], a["s"], a["n"], a["res"], a["ldr"], a["out"], a["ldo"], None)
        assert st == status, over
    assert lib.moe_linear_q8(good["p"], P, 128, P, 0, None, 0, 2 * P, 64, None) == q.MOE_OK


def test_grouped_refuses_bad_calls(lib):
    p = product(E=4)
    good = dict(p=ctypes.addressof(p), off=P, tok=None, x=2 * P, ldx=128, s=4 * P, x_rows=9, rows=9, out=3 * P, ldo=64)
    for over, status in [(dict(off=None), 1), (dict(off=P + 2), 1), (dict(x=None), 1), (dict(s=None), 1), (dict(out=None), 1),
                         (dict(rows=-1), 1), (dict(x_rows=-1), 1), (dict(x_rows=8), 1), (dict(tok=P, x_rows=0), 1),
                         (dict(tok=P + 1), 1), (dict(ldx=64), 1), (dict(ldx=136), 1), (dict(ldo=10), 1),
                         (dict(rows=(1 << 24) + 1), 2)]:
        a = dict(good, **over)
        st = lib.moe_grouped_linear_q8(a["p"], a["off"], a["tok"], a["x"], a["ldx"], a["s"], a["x_rows"], a["rows"],
                                       a["out"], a["ldo"], None)
        assert st == status, over
    for over, status in [(dict(E=1025), 2), (dict(stride_e=8), 1), (dict(stride_e=-16), 1)]:
        b = product(**dict(dict(E=4), **over))
        assert lib.moe_grouped_linear_q8(ctypes.addressof(b), P, None, 2 * P, 128, P, 9, 9, 3 * P, 64, None) == status, over
    assert lib.moe_grouped_linear_q8(good["p"], P, None, 2 * P, 128, P, 0, 0, 3 * P, 64, None) == q.MOE_OK


def test_quantize_refuses_bad_calls(lib):
    good = dict(dt=1, x=P, ldx=64, n=3, K=64, c=2 * P, ldc=64, s=3 * P)
    for over, status in [(dict(dt=0), 2), (dict(dt=9), 2), (dict(x=None), 1), (dict(c=None), 1), (dict(s=None), 1),
                         (dict(n=-1), 1), (dict(K=0), 1), (dict(ldx=63), 1), (dict(ldc=63), 1), (dict(x=P + 1), 1),
                         (dict(s=3 * P + 2), 1), (dict(c=P), 1), (dict(s=P), 1), (dict(s=2 * P), 1), (dict(n=(1 << 24) + 1), 2),
                         (dict(K=(1 << 20) + 1, ldx=1 << 21, ldc=1 << 21), 2)]:
        a = dict(good, **over)
        st = lib.moe_quantize_rows(a["dt"], a["x"], a["ldx"], a["n"], a["K"], a["c"], a["ldc"], a["s"], None)
        assert st == status, over
    assert lib.moe_quantize_rows(1, P, 64, 0, 64, 2 * P, 64, 3 * P, None) == q.MOE_OK


def rule(**over):
    f = dict(E=64, top_k=4, score=0, groups=1, top_groups=1, group_best=1, renormalize=1, scale=1.0, bias=None)
    f.update(over)
    return q.moe_router(**f)


BAD_RULE = [(dict(E=0), 1), (dict(top_k=0), 1), (dict(top_k=65), 1), (dict(score=2), 1), (dict(score=-1), 1), (dict(groups=0), 1),
            (dict(groups=7), 1), (dict(groups=8, top_groups=9), 1), (dict(top_groups=0), 1), (dict(top_groups=2), 1),
            (dict(group_best=0), 1), (dict(group_best=3), 1), (dict(groups=16, top_groups=1, top_k=5), 1), (dict(scale=NAN), 1),
            (dict(scale=INF), 1), (dict(scale=-INF), 1), (dict(bias=P + 2), 1), (dict(E=1025), 2), (dict(groups=64, top_groups=4), 2),
            (dict(E=128, top_k=65), 2)]


@pytest.mark.parametrize("over,status", BAD_RULE, ids=[str(o) for o, _ in BAD_RULE])
def test_route_refuses_bad_rules(lib, over, status):
    r = rule(**over)
    assert lib.moe_route(ctypes.addressof(r), 0, P, 4096, 3, 2 * P, 3 * P, None) == status


def test_route_refuses_bad_calls(lib):
    r = rule()
    good = dict(r=ctypes.addressof(r), dt=0, l=P, ldl=64, n=3, i=2 * P, w=3 * P)
    for over, status in [(dict(r=None), 1), (dict(l=None), 1), (dict(i=None), 1), (dict(w=None), 1), (dict(n=-1), 1), (dict(dt=3), 1),
                         (dict(dt=-1), 1), (dict(ldl=63), 1), (dict(l=P + 2), 1), (dict(dt=1, l=P + 1), 1), (dict(i=2 * P + 1), 1),
                         (dict(w=3 * P + 2), 1), (dict(w=2 * P), 1), (dict(i=P), 1), (dict(w=P), 1), (dict(n=(1 << 24) + 1), 2),
                         (dict(n=(1 << 22) + 1), 2)]:
        a = dict(good, **over)
        assert lib.moe_route(a["r"], a["dt"], a["l"], a["ldl"], a["n"], a["i"], a["w"], None) == status, over
    assert lib.moe_route(good["r"], 0, P, 64, 0, 2 * P, 3 * P, None) == q.MOE_OK


def zeros(*s, dtype=BF16):
    return torch.zeros(*s, dtype=dtype)


def test_python_checks_of_the_weights(lib):
    w, s = zeros(16, 32, dtype=I8), torch.ones(16)
    lw = q.LinearWeightsQ8(w, s, bias=zeros(16))
    assert (lw.N, lw.K, lw.E, lw.grouped, lw.dtype) == (16, 32, 1, False, BF16)
    for bad in (lambda: q.LinearWeightsQ8(zeros(16, 32), s), lambda: q.LinearWeightsQ8(w, s.double()),
                lambda: q.LinearWeightsQ8(w, s[:15]), lambda: q.LinearWeightsQ8(w, torch.ones(32)[::2]),
                lambda: q.LinearWeightsQ8(w.t(), torch.ones(32)), lambda: q.LinearWeightsQ8(w, s, w_up=w),
                lambda: q.LinearWeightsQ8(w, s, scale_up=s), lambda: q.LinearWeightsQ8(w, s, activation="swish"),
                lambda: q.LinearWeightsQ8(w, s, bias=zeros(16, dtype=torch.float16)), lambda: q.LinearWeightsQ8(w[0], s),
                lambda: q.LinearWeightsQ8(w, s, w_up=zeros(16, 48, dtype=I8)[:, :32], scale_up=s),
                lambda: q.LinearWeightsQ8(w[:0], s[:0])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        q.LinearWeightsQ8(w, s, dtype=torch.float32)


def test_python_checks_of_the_products(module):
    lw = q.LinearWeightsQ8(zeros(16, 32, dtype=I8), torch.ones(16))
    lg = q.LinearWeightsQ8(zeros(3, 16, 32, dtype=I8), torch.ones(3, 16))
    x = (zeros(4, 32, dtype=I8), torch.ones(4))
    off = torch.zeros(4, dtype=torch.int32)
    for bad, kind in ((lambda: q.moe_linear_q8(x[0], lw), TypeError), (lambda: q.moe_linear_q8([*x], lw), TypeError),
                      (lambda: q.moe_linear_q8(x + (1,), lw), TypeError), (lambda: q.moe_linear_q8((x[0][:, :16], x[1]), lw), ValueError),
                      (lambda: q.moe_linear_q8((zeros(4, 32), x[1]), lw), TypeError),
                      (lambda: q.moe_linear_q8((x[0], x[1][:3]), lw), ValueError),
                      (lambda: q.moe_linear_q8((x[0], x[1].double()), lw), ValueError),
                      (lambda: q.moe_linear_q8(x, lw), ValueError),  # no CUDA tensors
                      (lambda: q.moe_linear_q8(x, lw, residual=zeros(4, 15)), ValueError),
                      (lambda: q.moe_linear_q8(x, lw, out=zeros(4, 16, dtype=torch.float16)), TypeError),
                      (lambda: q.moe_linear_q8(x, lg), ValueError), (lambda: q.moe_grouped_linear_q8(x, lw, off), ValueError),
                      (lambda: q.moe_grouped_linear_q8(x, lg, off[:3]), ValueError),
                      (lambda: q.moe_grouped_linear_q8(x, lg, off.long()), TypeError),
                      (lambda: q.moe_grouped_linear_q8((x[0][:0], x[1][:0]), lg, off, row_token=off), ValueError),
                      (lambda: q.moe_quantize_rows(zeros(4, 32)), ValueError), (lambda: q.moe_quantize_rows(zeros(32)), ValueError),
                      (lambda: q.moe_quantize_rows(torch.zeros(4, 32)), TypeError)):
        with pytest.raises(kind):
            bad()


def test_weights_of_the_other_kind_are_refused(module):
    l16 = q.LinearWeights(zeros(16, 32))
    g16 = q.LinearWeights(zeros(3, 16, 32))
    l8 = q.LinearWeightsQ8(zeros(16, 32, dtype=I8), torch.ones(16))
    g8 = q.LinearWeightsQ8(zeros(3, 16, 32, dtype=I8), torch.ones(3, 16))
    x, x8, off = zeros(4, 32), (zeros(4, 32, dtype=I8), torch.ones(4)), torch.zeros(4, dtype=torch.int32)
    for bad in (lambda: q.moe_linear(x, l8), lambda: q.moe_linear_q8(x8, l16), lambda: q.moe_grouped_linear(x, g8, off),
                lambda: q.moe_grouped_linear_q8(x8, g16, off), lambda: q.moe_route(x, l16), lambda: q.RoutedExpertsQ8(g16, g16),
                lambda: q.SharedExpertQ8(l16, l16)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        q.SharedExpertQ8(g8, g8)
    with pytest.raises(ValueError):
        q.RoutedExpertsQ8(l8, l8)
    with pytest.raises(ValueError):
        q.RouterLayer(zeros(16, 32), q.Router(8, 2))


def test_python_checks_of_the_router(module):
    for bad in (dict(score="relu"), dict(group_score="mean"), dict(bias=torch.zeros(7)), dict(bias=zeros(8)),
                dict(bias=torch.zeros(16)[::2])):
        with pytest.raises(ValueError):
            q.Router(8, 2, **bad)
    r = q.Router(8, 2, bias=torch.zeros(8))
    for bad, kind in ((torch.zeros(3, 7), ValueError), (torch.zeros(3, 8, dtype=torch.float64), TypeError),
                      (torch.zeros(8), ValueError), (torch.zeros(3, 8), ValueError), (torch.zeros(3, 16)[:, ::2], ValueError)):
        with pytest.raises(kind):
            q.moe_route(bad, r)


def test_no_gradient_is_dropped(module):
    """Whatever asks for a gradient, or carries a tangent, is refused where it would be dropped."""
    def tensors():
        return dict(logits=torch.zeros(3, 8), bias=torch.zeros(8), x=zeros(4, 32), scale=torch.ones(4), w_scale=torch.ones(16),
                    up_scale=torch.ones(16), w_bias=zeros(16), up_bias=zeros(16), residual=zeros(4, 16), out=zeros(4, 16),
                    g_scale=torch.ones(3, 16))

    c, w, gw, off = zeros(4, 32, dtype=I8), zeros(16, 32, dtype=I8), zeros(3, 16, 32, dtype=I8), torch.zeros(4, dtype=torch.int32)
    calls = [
        (lambda t: q.moe_route(t["logits"], q.Router(8, 2, bias=t["bias"])), ("logits", "bias")),
        (lambda t: q.moe_quantize_rows(t["x"]), ("x",)),
        (lambda t: q.moe_linear_q8((c, t["scale"]), q.LinearWeightsQ8(w, t["w_scale"], w_up=w, scale_up=t["up_scale"],
                                                                      bias=t["w_bias"], bias_up=t["up_bias"]),
                                   residual=t["residual"], out=t["out"]),
         ("scale", "w_scale", "up_scale", "w_bias", "up_bias", "residual", "out")),
        (lambda t: q.moe_grouped_linear_q8((c, t["scale"]), q.LinearWeightsQ8(gw, t["g_scale"]), off, out=t["out"]),
         ("scale", "g_scale", "out")),
    ]
    fw = torch.autograd.forward_ad
    for call, names in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call(tensors())
        for name in names:
            t = tensors()
            t[name] = torch.nn.Parameter(t[name])
            with pytest.raises(RuntimeError, match="requires a gradient"):
                call(t)
            with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
                call(t)
            with fw.dual_level():
                t = tensors()
                t[name] = fw.make_dual(t[name], torch.ones_like(t[name]))
                with pytest.raises(RuntimeError, match="forward-mode tangent"):
                    call(t)


def test_module_hands_back_what_is_not_usual(lib):
    c = ops._calls
    assert c is not None
    lw = q.LinearWeightsQ8(zeros(16, 32, dtype=I8), torch.ones(16))
    r = q.Router(8, 2)
    x, s, l = zeros(4, 32, dtype=I8), torch.ones(4), torch.zeros(3, 8)
    for bad in (x, None, "x", x.to_sparse(), x.float().requires_grad_()):
        assert c.linear_q8(lw.ref, 0, bad, s, None, None, lw.tensors) is None
        assert c.grouped_q8(lw.ref, 0, bad, s, bad, None, None, lw.tensors) is None
        assert c.quantize(bad) is None and c.route(r.ref, bad, r.tensors) is None
    assert c.route(r.ref, l, ()) is None and c.route(r.ref, l, None) is None and c.route(0, l, r.tensors) is None
    assert c.route(r.ref, l, (l,)) is None
    assert c.linear_q8(lw.ref, 0, x, s, None, None, lw.tensors[:4]) is None
    assert c.linear_q8(1) is None and c.grouped_q8(1) is None and c.quantize() is None
    l16 = q.LinearWeights(zeros(16, 32))
    assert c.linear_q8(l16.ref, 0, x, s, None, None, l16.tensors) is None
    assert c.linear(lw.ref, 0, zeros(4, 32), None, None, lw.tensors) is None


def test_weights_and_router_follow_their_tensors(lib):
    w, s = zeros(16, 32, dtype=I8), torch.ones(16)
    lw = q.LinearWeightsQ8(w, s)
    keep = [w.data, s.data]
    w.data, s.data = zeros(16, 48, dtype=I8)[:, :32], torch.zeros(16)
    c = lw.current()
    assert (c.w, c.scale, c.ldw) == (w.data_ptr(), s.data_ptr(), 48) and c.w != keep[0].data_ptr()
    w.data = zeros(16, 32)
    with pytest.raises(ValueError):
        lw.current()
    b = torch.zeros(8)
    r = q.Router(8, 2, bias=b)
    old, b.data = b.data, torch.ones(8)
    assert r.current().bias == b.data_ptr() != old.data_ptr()
