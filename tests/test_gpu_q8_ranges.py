"""The 8-bit products, the quantiser and the router on the GPU: ranges beside test_gpu_q8.py and
test_gpu_route.py."""
import pytest
import torch

import ops_reference as ref
import q8_reference as ref8
import quantized_moe_decode_softmax_gb300 as q
import route_reference
from test_gpu_q8 import codes, gen, normal, offsets_of, rows_of, scales, weights

pytestmark = pytest.mark.gpu

BF16, F16, I8 = torch.bfloat16, torch.float16, torch.int8


def sampled(out, x, t, rows, act="none"):
    """Check some rows of a linear product."""
    r = torch.as_tensor(rows, device="cuda")
    ref.check(out[r], *ref8.product(x.codes[r], x.scale[r], act=act, **t))


@pytest.mark.parametrize("n", [1, 3, 40, 100])
def test_a_million_columns(n):
    g = gen(n)
    N, K = 1 << 20, 32
    t = weights(g, (), N, K, BF16, False, True)
    x = rows_of(g, n, K)
    sampled(q.moe_linear_q8(x, q.LinearWeightsQ8(**t)), x, t, [0, n - 1])


@pytest.mark.parametrize("n", [1, 20, 70])
def test_65536_inputs(n):
    g = gen(n)
    t = weights(g, (), 270, 65536, BF16, False, False)
    x = rows_of(g, n, 65536)
    sampled(q.moe_linear_q8(x, q.LinearWeightsQ8(**t)), x, t, list(range(n)))


def test_100000_rows():
    g = gen(4)
    t = weights(g, (), 264, 48, F16, True, True)
    x = rows_of(g, 100000, 48)
    out = q.moe_linear_q8(x, q.LinearWeightsQ8(**t, activation="silu", dtype=F16))
    sampled(out, x, t, list(range(0, 100000, 997)) + [99999], act="silu")
    q.moe_ops_check()


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("n,N,K", [(250, 40, 4096), (256, 128, 2048), (129, 70, 528), (65, 200, 1040), (33, 500, 2064), (18, 1000, 4112),
                                   (100, 33, 16), (64, 256, 8192), (40, 1100, 2048)])
def test_narrow_layers(n, N, K, gated):
    """Many rows by few columns: the kernels for few rows take them too."""
    g = gen(n)
    t = weights(g, (), N, K, BF16, gated, n % 2 == 0)
    x, res = rows_of(g, n, K), normal(g, (n, N))
    out = q.moe_linear_q8(x, q.LinearWeightsQ8(**t, activation="gelu_tanh"), residual=res)
    ref.check(out, *ref8.product(*x, act="gelu_tanh", residual=res, **t))


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("n,N,K", [(7, 3000, 1040), (8, 2048, 784), (12, 4100, 528), (16, 2050, 2064), (17, 2056, 16), (20, 2048, 2048),
                                   (31, 2500, 1104), (40, 2064, 1040), (64, 2051, 2064), (24, 8200, 272), (64, 12290, 144)])
def test_wide_layers(n, N, K, gated):
    g = gen(n + N)
    t = weights(g, (), N, K, BF16, gated, n % 2 == 0)
    x, res = rows_of(g, n, K), normal(g, (n, N))
    out = q.moe_linear_q8(x, q.LinearWeightsQ8(**t, activation="silu"), residual=res)
    ref.check(out, *ref8.product(*x, act="silu", residual=res, **t))


@pytest.mark.parametrize("rows", [60, 1500, 20000])
def test_1024_experts(rows):
    g = gen(rows)
    E, N, K = 1024, 72, 64
    t = weights(g, (E,), N, K, BF16, True, False)
    x = rows_of(g, rows, K)
    e = torch.randint(0, E, (rows,), generator=g, device="cuda").sort().values
    off = offsets_of(torch.bincount(e, minlength=E).tolist())
    out = q.moe_grouped_linear_q8(x, q.LinearWeightsQ8(**t, activation="gelu"), off)
    for r in list(range(0, rows, max(1, rows // 60))) + [rows - 1]:
        at = int(e[r])
        ref.check(out[r:r + 1], *ref8.product(x.codes[r:r + 1], x.scale[r:r + 1], act="gelu", **{k: v[at] for k, v in t.items()}))


@pytest.mark.parametrize("E,mean", [(300, 80), (1024, 90), (1024, 60), (1000, 200)])
def test_many_experts_and_rows(E, mean):
    """The table of the groups next to tiles of each length."""
    g = gen(E + mean)
    N, K, rows = 136, 272, E * mean
    t = weights(g, (E,), N, K, BF16, False, True)
    x = rows_of(g, rows, K)
    e = torch.randint(0, E, (rows,), generator=g, device="cuda").sort().values
    out = q.moe_grouped_linear_q8(x, q.LinearWeightsQ8(**t), offsets_of(torch.bincount(e, minlength=E).tolist()))
    for r in list(range(0, rows, rows // 60)) + [rows - 1]:
        at = int(e[r])
        ref.check(out[r:r + 1], *ref8.product(x.codes[r:r + 1], x.scale[r:r + 1], **{k: v[at] for k, v in t.items()}))
    q.moe_ops_check()


@pytest.mark.parametrize("rows", [3, 100, 1000])
def test_weights_and_rows_past_32_bits(rows):
    """Experts that begin more than 2^32 bytes into the weights, rows of x and of out that lie far
    apart."""
    g = gen(rows)
    E, N, K = 5, 48, 80
    far = 1 << 30
    buf = torch.empty(E * far, dtype=I8, device="cuda")
    w = buf.as_strided((E, N, K), (far, 96, 1))
    w.copy_(codes(g, (E, N, K)))
    s = scales(g, (E, N), 1e-3)
    wide = 1 << 23
    xb = torch.empty(rows * wide, dtype=I8, device="cuda")
    x = xb.as_strided((rows, K), (wide, 1))
    x.copy_(codes(g, (rows, K)))
    sx = scales(g, (rows,), 1e-2)
    counts = [0, rows // 3, 0, rows - rows // 3 - 1, 1]
    ob = torch.empty(rows * (1 << 22), dtype=BF16, device="cuda")
    out = ob.as_strided((rows, N), (1 << 22, 1))
    q.moe_grouped_linear_q8((x, sx), q.LinearWeightsQ8(w, s), offsets_of(counts), out=out)
    at = 0
    for e, c in enumerate(counts):
        if c:
            ref.check(out[at:at + c], *ref8.product(x[at:at + c], sx[at:at + c], w[e], s[e]))
        at += c


def test_quantize_past_32_bits():
    x = torch.empty(600 * (1 << 23), dtype=BF16, device="cuda").as_strided((600, 100), (1 << 23, 1))
    x.copy_(normal(gen(1), (600, 100)))
    assert torch.equal(q.moe_quantize_rows(x).codes, ref8.quantized(x)[0])
    big = normal(gen(2), (300000, 16384 // 4))
    r = q.moe_quantize_rows(big)
    at = [0, 1, 150000, 299999]
    assert torch.equal(r.codes[at], ref8.quantized(big[at])[0])


MOST = 1 << 24  # rows of a call


def test_the_longest_rows_to_quantize():
    for dtype in (BF16, F16):
        x = normal(gen(5), (3, 1 << 20), dtype=dtype)
        r = q.moe_quantize_rows(x)
        codes_, scale = ref8.quantized(x)[:2]
        assert torch.equal(r.codes, codes_) and torch.equal(r.scale, scale.float())


def test_the_most_rows():
    g = gen(6)
    x = normal(g, (MOST, 3))
    r = q.moe_quantize_rows(x)
    at = torch.cat([torch.arange(0, MOST, 99991, device="cuda"), torch.arange(MOST - 300, MOST, device="cuda")])
    assert torch.equal(r.codes[at], ref8.quantized(x[at])[0])
    del x, r
    z = torch.randn((MOST, 2), generator=g, device="cuda")
    r = q.moe_route(z, q.Router(2, 1, score="sigmoid", bias=torch.tensor([0.25, 0.0], device="cuda"), renormalize=False))
    assert torch.equal(r.topk_idx[:, 0].long(), ((torch.sigmoid(z.double()) + torch.tensor([0.25, 0.0], device="cuda")).argmax(1)))
    del z, r
    t = weights(g, (), 3, 16, BF16, True, True)
    x = q.QuantizedRows(codes(g, (MOST, 16)), scales(g, (MOST,), 1e-2))
    out = q.moe_linear_q8(x, q.LinearWeightsQ8(**t, activation="silu"))
    ref.check(out[at], *ref8.product(x.codes[at], x.scale[at], act="silu", **t))
    with pytest.raises(q.MoeError):
        q.moe_quantize_rows(normal(g, (MOST + 1, 1)))
    q.moe_ops_check()


def test_route_past_32_bits():
    z = torch.empty(4200 * (1 << 20), dtype=BF16, device="cuda").as_strided((4200, 100), (1 << 20, 1))
    z.copy_(normal(gen(3), (4200, 100)))
    rule = dict(score="sigmoid", bias=0.1 * torch.randn(100, device="cuda"))
    for part in (z[:50], z[-50:]):
        route_reference.check(q.moe_route(part, q.Router(100, 5, **rule)), part, 5, **rule)
    r = q.moe_route(z, q.Router(100, 5, **rule))
    route_reference.check(q.Routing(r.topk_idx[-50:], r.topk_w[-50:]), z[-50:], 5, **rule)


def test_another_stream_and_memory_let_go_of():
    """Inputs of a call on a busy side stream that are dropped right after it, their memory asked
    for again and overwritten."""
    g = gen(9)

    def operands():
        z = torch.randn(300, 64, generator=g, device="cuda")
        x = normal(g, (300, 256))
        w = codes(g, (128, 256))
        return z, x, w, torch.full((128,), 1e-3, device="cuda")

    def run(o, st):
        r = q.moe_route(o[0], q.Router(64, 4), stream=st)
        out = q.moe_linear_q8(q.moe_quantize_rows(o[1], stream=st), q.LinearWeightsQ8(o[2], o[3]), stream=st)
        return r.topk_idx, r.topk_w, out

    o = operands()
    want = [t.clone() for t in run(o, None)]
    shapes = [(t.shape, t.dtype) for t in o]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    got = run(o, side)
    del o
    again = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del again


def test_two_graphs_of_one_layer_on_two_streams():
    """Calls keep no workspace: two captured graphs of the same weights replay side by side."""
    g = gen(10)
    lw = q.LinearWeightsQ8(**weights(g, (), 512, 1024, BF16, True, False), activation="silu")
    xs, outs, graphs = [normal(g, (200, 1024)) for _ in range(2)], [], []
    q.moe_linear_q8(q.moe_quantize_rows(xs[0]), lw)
    torch.cuda.synchronize()
    for x in xs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = q.moe_linear_q8(q.moe_quantize_rows(x), lw)
        outs.append(out)
        graphs.append(graph)
    want = [q.moe_linear_q8(q.moe_quantize_rows(x), lw) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    q.moe_ops_check()


def test_an_output_counts_as_written():
    t = lambda *s: torch.ones(s, dtype=BF16, device="cuda")  # noqa: E731
    lw = q.LinearWeightsQ8(torch.ones(16, 32, dtype=I8, device="cuda"), torch.ones(16, device="cuda"))
    lg = q.LinearWeightsQ8(torch.ones(1, 16, 32, dtype=I8, device="cuda"), torch.ones(1, 16, device="cuda"))
    x, off = (torch.ones(4, 32, dtype=I8, device="cuda"), torch.ones(4, device="cuda")), offsets_of([4])
    keep = q.ops._calls
    try:
        for module in (keep, None):
            q.ops._calls = module
            for call in (lambda o: q.moe_linear_q8(x, lw, out=o), lambda o: q.moe_grouped_linear_q8(x, lg, off, out=o)):
                p, out = torch.nn.Parameter(t(16)), t(4, 16)
                loss = (p * out).sum()
                call(out)
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    loss.backward()
    finally:
        q.ops._calls = keep


@pytest.mark.parametrize("mode", [torch.enable_grad, torch.no_grad, torch.inference_mode])
def test_results_are_ordinary_tensors(mode):
    """Outputs made by a call are what torch.empty makes: their dispatch keys, version counters,
    autograd, storages."""
    x, off = normal(gen(1), (6, 32)), offsets_of([6])
    lw = q.LinearWeightsQ8(torch.ones(16, 32, dtype=I8, device="cuda"), torch.ones(16, device="cuda"))
    lg = q.LinearWeightsQ8(torch.ones(1, 16, 32, dtype=I8, device="cuda"), torch.ones(1, 16, device="cuda"))
    l16, idx = q.LinearWeights(normal(gen(2), (16, 32))), torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    with mode():
        made = [*q.moe_quantize_rows(x), *q.moe_route(x, q.Router(32, 4)), *q.moe_group_slots(idx, 4), q.moe_linear(x, l16)]
        made += [q.moe_linear_q8(q.moe_quantize_rows(x), lw), q.moe_grouped_linear_q8(q.moe_quantize_rows(x), lg, off)]
        for t in made:
            like = torch.empty(t.shape, dtype=t.dtype, device="cuda")
            assert torch._C._dispatch_keys(t) == torch._C._dispatch_keys(like)
            assert t.is_inference() == like.is_inference() and t.device == like.device and t.layout == like.layout
            assert t.is_contiguous() and not t.requires_grad and t.is_leaf
            if not t.is_inference():
                assert t._version == 0
                t.add_(1)
                assert t._version == 1
    if mode is not torch.inference_mode:
        out = made[-1].detach().requires_grad_()
        (3 * out).sum().backward()
        assert bool((out.grad == 3).all())
        alone = made[-1]
        alone.resize_(0)
        assert alone.numel() == 0


def test_results_give_their_memory_back():
    x = normal(gen(3), (4096, 1024))
    r = q.Router(1024, 8)
    for call in (lambda: q.moe_quantize_rows(x), lambda: q.moe_route(x, r)):
        call()
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        first, second = call()
        more = torch.cuda.memory_allocated() - before
        assert more >= first.nbytes + second.nbytes
        keep = second.clone()
        del first
        assert torch.cuda.memory_allocated() - before >= more
        assert torch.equal(keep, second)
        del second, keep
        assert torch.cuda.memory_allocated() == before
