"""Calls of the operators on another stream than the tensors' own."""
import types

import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
from quantized_moe_decode_softmax_gb300 import ops

BF16 = torch.bfloat16


def test_a_stream_of_another_device_is_refused():
    ops._lib()
    with pytest.raises(ValueError, match="cuda:1"):
        ops._Elsewhere(0, types.SimpleNamespace(device=torch.device("cuda:1")))


def operands(op, g):
    """The tensors of a call, none of which anything else holds, and the call."""
    n, N, K, E, k = 256, 512, 256, 8, 2
    t = lambda *s: torch.empty(s, dtype=BF16, device="cuda").normal_(generator=g)  # noqa: E731
    idx = torch.randint(0, E, (n, k), device="cuda", generator=g).to(torch.int32)
    if op == "linear":
        return [t(n, K), t(N, K), t(n, N)], lambda a, st: q.moe_linear(a[0], q.LinearWeights(a[1]), residual=a[2], stream=st)
    if op == "grouped":
        s = q.moe_group_slots(idx, E)
        return ([t(n, K), t(E, N, K), s.offsets.clone(), s.slot_token.clone()],
                lambda a, st: q.moe_grouped_linear(a[0], q.LinearWeights(a[1]), a[2], row_token=a[3], stream=st))
    if op == "slots":
        return [idx], lambda a, st: q.moe_group_slots(a[0], E, stream=st).slot_of
    of = torch.arange(n * k, dtype=torch.int32, device="cuda").reshape(n, k)
    return [t(n * k, N), of, torch.rand(n, k, device="cuda", generator=g)], \
        lambda a, st: q.moe_combine_slots(a[0], a[1], a[2], stream=st)


@pytest.mark.gpu
@pytest.mark.parametrize("op", ["linear", "grouped", "slots", "combine"])
def test_memory_let_go_of_after_the_call_is_not_reused_before_it_ran(op):
    """The inputs of a call on a busy side stream are dropped right after it, and their
    memory asked for again and overwritten at once from the current stream."""
    g = torch.Generator(device="cuda").manual_seed(3)
    tensors, call = operands(op, g)
    want = call(tensors, None).clone()
    shapes = [(t.shape, t.dtype) for t in tensors]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms: the call below waits behind it
    got = call(tensors, side)
    del tensors
    again = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes for _ in range(2)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del again


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 200])
@pytest.mark.parametrize("before", ["nothing", "copy", "memset", "join", "join_of_operators", "fork"])
def test_captured_behind_every_kind_of_node(before, n):
    """A captured call whose dependencies are no kernel, several nodes or none; replayed
    on new inputs it gives the bits of the eager call."""
    g = torch.Generator(device="cuda").manual_seed(n)
    t = lambda *s: torch.empty(s, dtype=BF16, device="cuda").normal_(generator=g)  # noqa: E731
    lw, x, src, y = q.LinearWeights(t(256, 128), activation="silu"), t(n, 128), t(n, 128), t(n, 128)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    q.moe_linear(x, lw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        if before == "copy":
            x.copy_(src)
        elif before == "memset":
            x.zero_()
        elif before.startswith("join"):
            for st, buf in ((side, x), (other, y)):
                st.wait_stream(main)
                with torch.cuda.stream(st):
                    if before == "join":
                        buf.copy_(src)
                    else:
                        buf.copy_(q.moe_linear(src, lw)[:, :128])
            main.wait_stream(side)
            main.wait_stream(other)
        if before == "fork":
            side.wait_stream(main)
            with torch.cuda.stream(side):
                b = q.moe_linear(y, lw)
            a = q.moe_linear(x, lw)
            main.wait_stream(side)
            out = torch.cat([a, b, q.moe_linear(x, lw)])
        else:
            out = torch.cat([q.moe_linear(x, lw), q.moe_linear(y, lw)])
    for _ in range(3):
        for buf in (src, x, y):
            buf.copy_(t(n, 128))
        graph.replay()
        torch.cuda.synchronize()
        tail = [x] if before == "fork" else []
        assert torch.equal(out, torch.cat([q.moe_linear(v, lw) for v in [x, y] + tail]))
    q.moe_ops_check()


@pytest.mark.gpu
def test_an_output_counts_as_written():
    """Autograd notices that a buffer which it keeps for a backward pass was the output of
    a call, as after an in-place operation of torch, with and without the module."""
    t = lambda *s: torch.ones(s, dtype=BF16, device="cuda")  # noqa: E731
    lw, lg, off = q.LinearWeights(t(16, 24)), q.LinearWeights(t(1, 16, 24)), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    of, w = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, 1, device="cuda")
    keep = q.ops._calls
    try:
        for module in (keep, None):
            q.ops._calls = module
            for call in (lambda o: q.moe_linear(t(4, 24), lw, out=o), lambda o: q.moe_grouped_linear(t(4, 24), lg, off, out=o),
                         lambda o: q.moe_combine_slots(t(4, 16), of, w, out=o)):
                p, out = torch.nn.Parameter(t(16)), t(4, 16)
                loss = (p * out).sum()
                call(out)
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    loss.backward()
                with torch.inference_mode():
                    inner = t(4, 16)
                    call(inner)
                call(inner)
    finally:
        q.ops._calls = keep
