"""The operators of include/moe_ops.h on the host: declarations, structs and
argument checks (every call here is refused before any CUDA work)."""
import ctypes
import os
import re

import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
from quantized_moe_decode_softmax_gb300 import build as qbuild
from quantized_moe_decode_softmax_gb300 import ops

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_ops.h")
P = 1 << 20  # a 16-byte aligned address; no refused call reads it


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return ops._lib()


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_and_binding_agree(lib):
    names = set(re.findall(r"^\s*moe_status\s+(moe_\w+)\s*\(", header(), re.M))
    assert names == set(q.OPS_EXPORTED)
    assert all(hasattr(lib, n) for n in names)
    body = re.search(r"typedef struct \{([^}]*)\}\s*moe_product;", header()).group(1)
    assert re.findall(r"(\w+)\s*;", body) == [f for f, _ in q.moe_product._fields_]
    for name, value in re.findall(r"(MOE_(?:EPI|DTYPE)_\w+)\s*=\s*(\d+)", header()):
        assert getattr(q, name) == int(value)


def product(**over):
    f = dict(dtype=q.MOE_DTYPE_BF16, E=1, N=64, K=128, w=P, w_up=None, ldw=128, stride_e=64 * 128, bias=None,
             bias_up=None, activation=0, act_limit=0.0)
    f.update(over)
    return q.moe_product(**f)


BAD_PRODUCT = [
    (dict(w=None), 1), (dict(w=P + 8), 1), (dict(w_up=P + 2), 1), (dict(bias=P + 1), 1), (dict(dtype=0), 2),
    (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(E=0), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(K=-8), 1),
    (dict(K=132), 2), (dict(K=65544, ldw=65544), 2), (dict(N=(1 << 20) + 1), 2), (dict(ldw=120), 1),
    (dict(ldw=132), 1), (dict(bias_up=P), 1), (dict(activation=4), 1), (dict(activation=-1), 1),
    (dict(act_limit=1.0), 1), (dict(act_limit=-1.0, w_up=P), 1), (dict(act_limit=float("nan"), w_up=P), 1),
    (dict(act_limit=float("inf"), w_up=P), 1),
]


@pytest.mark.parametrize("over,status", BAD_PRODUCT, ids=[str(o) for o, _ in BAD_PRODUCT])
def test_products_refuse_bad_weights(lib, over, status):
    p = product(**over)
    ref = ctypes.addressof(p)
    assert lib.moe_linear(ref, P, 65544, 1, None, 0, P + 4096, 1 << 21, None) == status
    assert lib.moe_grouped_linear(ref, P, None, P, 65544, 4, 4, P + 4096, 1 << 21, None) == status


def test_linear_refuses_bad_calls(lib):
    p = product()
    ref = ctypes.addressof(p)
    good = dict(p=ref, x=P, ldx=128, n=3, res=None, ldr=0, out=2 * P, ldo=64)
    for over, status in [(dict(p=None), 1), (dict(x=None), 1), (dict(out=None), 1), (dict(n=-1), 1), (dict(ldx=120), 1),
                         (dict(ldx=132), 1), (dict(ldo=63), 1), (dict(x=P + 8), 1), (dict(out=2 * P + 1), 1),
                         (dict(out=P), 1), (dict(res=3 * P, ldr=63), 1), (dict(res=3 * P + 1, ldr=64), 1),
                         (dict(res=2 * P, ldr=72), 1), (dict(n=(1 << 24) + 1), 2)]:
        a = dict(good, **over)
        st = lib.moe_linear(a["p"], a["x"], a["ldx"], a["n"], a["res"], a["ldr"], a["out"], a["ldo"], None)
        assert st == status, over
    assert lib.moe_linear(ref, P, 128, 0, None, 0, 2 * P, 64, None) == q.MOE_OK  # no rows: nothing launched
    two = product(E=2)
    assert lib.moe_linear(ctypes.addressof(two), P, 128, 1, None, 0, 2 * P, 64, None) == q.MOE_ERR_INVALID_ARG


def test_grouped_refuses_bad_calls(lib):
    p = product(E=4)
    good = dict(p=ctypes.addressof(p), off=P, tok=None, x=2 * P, ldx=128, x_rows=9, rows=9, out=3 * P, ldo=64)
    for over, status in [(dict(off=None), 1), (dict(off=P + 2), 1), (dict(x=None), 1), (dict(out=None), 1),
                         (dict(rows=-1), 1), (dict(x_rows=-1), 1), (dict(x_rows=8), 1), (dict(tok=P, x_rows=0), 1),
                         (dict(tok=P + 1), 1), (dict(ldx=64), 1), (dict(ldo=10), 1), (dict(rows=(1 << 24) + 1), 2)]:
        a = dict(good, **over)
        st = lib.moe_grouped_linear(a["p"], a["off"], a["tok"], a["x"], a["ldx"], a["x_rows"], a["rows"], a["out"],
                                    a["ldo"], None)
        assert st == status, over
    for over, status in [(dict(E=1025), 2), (dict(stride_e=4), 1), (dict(stride_e=-8), 1)]:
        b = product(**dict(dict(E=4), **over))
        assert lib.moe_grouped_linear(ctypes.addressof(b), P, None, 2 * P, 128, 9, 9, 3 * P, 64, None) == status, over
    assert lib.moe_grouped_linear(good["p"], P, None, 2 * P, 128, 0, 0, 3 * P, 64, None) == q.MOE_OK


def test_slots_and_combine_refuse_bad_calls(lib):
    good = dict(i=P, n=4, k=2, E=8, lo=0, hi=8, a=P, b=P, c=None, d=P)
    for over, status in [(dict(i=None), 1), (dict(a=None), 1), (dict(b=None), 1), (dict(d=None), 1), (dict(n=-1), 1),
                         (dict(k=0), 1), (dict(E=0), 1), (dict(lo=-1), 1), (dict(lo=5, hi=4), 1), (dict(hi=9), 1),
                         (dict(i=P + 2), 1), (dict(c=P + 1), 1), (dict(E=1025, hi=9), 2), (dict(k=65), 2),
                         (dict(n=1 << 24, k=2), 2)]:
        a = dict(good, **over)
        assert lib.moe_group_slots(a["i"], a["n"], a["k"], a["E"], a["lo"], a["hi"], a["a"], a["b"], a["c"], a["d"],
                                   None) == status, over
    good = dict(dt=1, y=P, ldy=64, rows=8, of=P, w=P, n=4, k=2, N=64, res=None, ldr=0, out=2 * P, ldo=64)
    for over, status in [(dict(dt=0), 2), (dict(dt=7), 2), (dict(y=None), 1), (dict(of=None), 1), (dict(w=None), 1),
                         (dict(out=None), 1), (dict(rows=-1), 1), (dict(n=-1), 1), (dict(k=0), 1), (dict(N=0), 1),
                         (dict(ldy=63), 1), (dict(ldo=63), 1), (dict(res=3 * P, ldr=1), 1), (dict(out=P), 1),
                         (dict(of=P + 2), 1), (dict(w=P + 1), 1), (dict(k=65), 2), (dict(res=2 * P, ldr=80), 1)]:
        a = dict(good, **over)
        st = lib.moe_combine_slots(a["dt"], a["y"], a["ldy"], a["rows"], a["of"], a["w"], a["n"], a["k"], a["N"],
                                   a["res"], a["ldr"], a["out"], a["ldo"], None)
        assert st == status, over


def test_torch_calls_module_leaves_what_is_not_usual(lib):
    """The module is built with the library, and answers None (never an exception)
    to a call that its caller has to look at."""
    c = ops._calls
    assert c is not None and os.path.samefile(c.__file__, qbuild.calls_path())
    w = torch.zeros(16, 24, dtype=torch.bfloat16)
    lw, x, i = q.LinearWeights(w), torch.zeros(2, 24, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    assert c.linear(lw.ref, lw.device_index, x, None, None) is None  # not on a GPU
    assert c.linear(lw.ref, 0, x, None, None) is None
    assert c.linear(lw.ref, 0, None, None, None) is None
    assert c.linear(lw.ref, 0, "x", None, None) is None
    assert c.linear(lw.ref, 0, torch.nn.Parameter(x), None, None) is None
    assert c.linear(lw.ref, 0, x.to_sparse(), None, None) is None
    assert c.linear(1, 2) is None
    assert c.grouped(lw.ref, 0, x, i, None, None) is None and c.grouped(lw.ref, 0, x, None, None, None) is None
    assert c.slots(i, 4, 0, 4) is None and c.slots(i, "4", 0, 4) is None and c.slots(i, 1 << 70, 0, 4) is None
    assert c.combine(x, i, i, None, None) is None and c.combine(x, None, i, None, None) is None


def test_python_checks():
    w = torch.zeros(16, 24, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.LinearWeights(w, activation="swish")
    with pytest.raises(TypeError):
        q.LinearWeights(w.float())
    with pytest.raises(ValueError):
        q.LinearWeights(w.t())
    with pytest.raises(ValueError):
        q.LinearWeights(w, w_up=torch.zeros(16, 32, dtype=torch.bfloat16)[:, :24])
    with pytest.raises(ValueError):
        q.LinearWeights(w, bias=torch.zeros(15, dtype=torch.bfloat16))
    lw = q.LinearWeights(w)
    x = torch.zeros(2, 24, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.moe_linear(x[:, :16], lw)
    with pytest.raises(TypeError):
        q.moe_linear(x.half(), lw)
    with pytest.raises(ValueError):  # no CUDA tensors
        q.moe_linear(x, lw)
    with pytest.raises(ValueError):
        q.moe_linear(x, lw, residual=torch.zeros(2, 15, dtype=torch.bfloat16))
    with pytest.raises(RuntimeError):
        q.moe_linear(x.clone().requires_grad_(), lw)
    with pytest.raises(ValueError):
        q.moe_grouped_linear(x, lw, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        q.moe_group_slots(torch.zeros(2, 2, dtype=torch.int64), 4)
    with pytest.raises(ValueError):
        q.moe_combine_slots(x, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(2, 1))
    g = torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.RoutedExperts(g, g, g)
    with pytest.raises(ValueError):
        q.SharedExpert(g[0], g[0], g[0])
