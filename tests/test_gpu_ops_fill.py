"""Outputs of the operators under torch.use_deterministic_algorithms."""
import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
from quantized_moe_decode_softmax_gb300 import ops
from test_gpu_q8 import BF16, codes, gen, normal, offsets_of, scales

pytestmark = pytest.mark.gpu


@pytest.fixture
def deterministic():
    before = torch.are_deterministic_algorithms_enabled(), torch.utils.deterministic.fill_uninitialized_memory
    yield
    torch.use_deterministic_algorithms(before[0])
    torch.utils.deterministic.fill_uninitialized_memory = before[1]


def calls():
    """name -> (call, the row from which on its output is unset; None: it sets all of them)."""
    g = gen(1)
    n, N, K = 40, 48, 64
    x, off, off_q8 = normal(g, (n, K)), offsets_of([3, 9]), offsets_of([0, 5])
    lw, lg = q.LinearWeights(normal(g, (N, K))), q.LinearWeights(normal(g, (2, N, K)))
    x8 = (codes(g, (n, K)), scales(g, (n,), 0.01))
    l8 = q.LinearWeightsQ8(codes(g, (N, K)), scales(g, (N,), 0.01))
    g8 = q.LinearWeightsQ8(codes(g, (2, N, K)), scales(g, (2, N), 0.01))
    idx = torch.randint(0, 4, (n, 2), generator=g, device="cuda").int()
    of, w = torch.zeros((n, 2), dtype=torch.int32, device="cuda"), torch.ones((n, 2), device="cuda")
    return {"linear": (lambda: (q.moe_linear(x, lw),), None), "grouped": (lambda: (q.moe_grouped_linear(x, lg, off),), 12),
            "linear_q8": (lambda: (q.moe_linear_q8(x8, l8),), None), "grouped_q8": (lambda: (q.moe_grouped_linear_q8(x8, g8, off_q8),), 5),
            "slots": (lambda: tuple(q.moe_group_slots(idx, 4)), None), "combine": (lambda: (q.moe_combine_slots(x, of, w),), None),
            "route": (lambda: tuple(q.moe_route(x, q.Router(K, 2))), None), "quantize": (lambda: tuple(q.moe_quantize_rows(x)), None)}


@pytest.mark.parametrize("module", [True, False], ids=["module", "ctypes"])
@pytest.mark.parametrize("name", ["linear", "grouped", "linear_q8", "grouped_q8", "slots", "combine", "route", "quantize"])
def test_new_outputs_are_filled_as_torch_fills_them(name, module, deterministic, monkeypatch):
    """Rows outside every group hold NaN, as torch.empty's memory does; everything else is as ever."""
    call, rows = calls()[name]
    want = [t.clone() for t in call()]
    assert ops._calls is not None
    if not module:
        monkeypatch.setattr(ops, "_calls", None)
    for fill in (True, False):
        torch.use_deterministic_algorithms(True)
        torch.utils.deterministic.fill_uninitialized_memory = fill
        for _ in range(3):
            zeros = torch.zeros(40, 48, dtype=BF16, device="cuda")
            del zeros  # (memory that the next output may get)
            got = call()
            for a, b in zip(got, want):
                assert torch.equal(a[:rows], b[:rows])
                assert not fill or rows is None or bool(torch.isnan(a[rows:]).all())


def test_an_output_that_was_given_is_not_filled(deterministic):
    g = gen(2)
    lg = q.LinearWeights(normal(g, (2, 48, 64)))
    x, off, out = normal(g, (40, 64)), offsets_of([3, 9]), normal(g, (40, 48))
    before = out.clone()
    torch.use_deterministic_algorithms(True)
    torch.utils.deterministic.fill_uninitialized_memory = True
    q.moe_grouped_linear(x, lg, off, out=out)
    assert torch.equal(out[12:], before[12:]) and not torch.equal(out[:12], before[:12])
