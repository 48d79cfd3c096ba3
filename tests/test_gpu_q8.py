"""moe_quantize_rows, moe_linear_q8 and moe_grouped_linear_q8 on the GPU against their 64-bit forms."""
import pytest
import torch

import ops_reference as ref
import q8_reference as ref8
import quantized_moe_decode_softmax_gb300 as q

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
INF, NAN = float("inf"), float("nan")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, std=1.0, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def codes(g, shape, lo=-128):
    return torch.randint(lo, 128, shape, generator=g, device="cuda").to(torch.int8)


def scales(g, shape, size):
    return (0.5 + torch.rand(shape, generator=g, device="cuda")) * size


def weights(g, lead, N, K, dtype, gated, bias):
    size = K ** -0.5 / 74
    t = {"w": codes(g, lead + (N, K)), "scale": scales(g, lead + (N,), size)}
    if gated:
        t.update(w_up=codes(g, lead + (N, K)), scale_up=scales(g, lead + (N,), size))
    if bias:
        t["bias"] = normal(g, lead + (N,), 0.5, dtype)
        if gated:
            t["bias_up"] = normal(g, lead + (N,), 0.5, dtype)
    return t


def rows_of(g, n, K):
    return q.QuantizedRows(codes(g, (n, K)), scales(g, (n,), 1 / 74))


def offsets_of(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.cumsum(torch.tensor(counts), 0)
    return o.cuda()


# ---- quantisation -----------------------------------------------------------------

QUANTIZE = [(1, 1), (3, 7), (1, 8), (5, 40), (2, 256), (4, 264), (9, 512), (3, 1000), (7, 1024), (5, 2048), (6, 2056), (3, 4096),
            (2, 4104), (3, 8192), (2, 8200), (2, 16384), (1, 20000), (2, 32768), (1, 32776), (1, 65536), (513, 96), (1000, 24)]


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("n,K", QUANTIZE)
def test_quantize(n, K, dtype):
    x = normal(gen(n + K), (n, K), 3.0, dtype)
    r = q.moe_quantize_rows(x)
    c, s = ref8.quantized(x)
    assert r.codes.dtype == torch.int8 and r.scale.dtype == torch.float32
    assert torch.equal(r.codes, c)
    assert float(((r.scale.double() - s.double()) / s.double()).abs().max()) <= 2.0 ** -23  # both are one rounding away
    keep, q.ops._calls = q.ops._calls, None
    try:
        again = q.moe_quantize_rows(x)
    finally:
        q.ops._calls = keep
    assert torch.equal(again.codes, c) and torch.equal(again.scale, r.scale)


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("aligned", [True, False], ids=["wide", "single"])
def test_quantize_halves_and_all_ratios(dtype, aligned):
    """Every value of one binade against every largest value: all halves and all quotients
    next to one."""
    bits = 7 if dtype == BF16 else 10
    m = torch.arange(2 ** bits, 2 ** (bits + 1), device="cuda")
    if dtype == F16:
        m = m[::7]
    for shift in (0, 1, 3, 6):
        x = torch.arange(2 ** bits, 2 ** (bits + 1), device="cuda").double() * 2.0 ** -shift
        rows = torch.where(x[None, :] <= m[:, None], x[None, :], torch.zeros(1, device="cuda").double())
        rows = torch.cat([rows, -rows, m[:, None].double().expand(-1, 8)], 1).to(dtype)
        buf = torch.zeros((rows.shape[0], rows.shape[1] + 8), dtype=dtype, device="cuda")
        at = 0 if aligned else 1
        buf[:, at:at + rows.shape[1]] = rows
        r = q.moe_quantize_rows(buf[:, at:at + rows.shape[1]])
        assert torch.equal(r.codes, ref8.quantized(rows)[0])


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("K", [16, 1024, 19])
def test_quantize_extremes(K, dtype):
    """Zeros, the largest and smallest values, subnormals, and rows with infinities or NaN,
    which leave the other rows alone."""
    big, small = (3.3e38, 9.2e-41) if dtype == BF16 else (65504.0, 5.97e-8)
    x = normal(gen(5), (10, K), 1.0, dtype)
    x[0] = 0
    x[1, 3], x[2, 0] = INF, NAN
    x[3] = normal(gen(6), (K,), 1.0).float().clamp(-1, 1).mul(big).to(dtype)
    x[3, 5] = big
    x[4] = 0
    x[4, 2], x[4, 9] = small, -2 * small
    x[5, 7], x[5, 8] = -INF, NAN
    x[6] = -0.0
    x[7] = (x[7].float() * (1e-30 if dtype == BF16 else 1e-4)).to(dtype)
    r = q.moe_quantize_rows(x)
    fine = [0, 3, 4, 6, 7, 8, 9]
    c, s = ref8.quantized(x[fine])
    assert torch.equal(r.codes[fine], c)
    # (the scale of the smallest is itself subnormal: a step of 2^-149)
    assert bool(((r.scale[fine].double() - s.double()).abs() <= s.double().abs() * 2.0 ** -23 + 2.0 ** -149).all())
    assert r.scale[0].item() == 0 and r.scale[1].item() == INF and r.scale[2].isnan() and r.scale[5].isnan()
    assert not bool(r.codes[[0, 1, 2, 5, 6]].any())
    w = q.LinearWeightsQ8(torch.ones(4, (K + 15) // 16 * 16, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda"))
    if K % 16 == 0:
        out = q.moe_linear_q8(r, w)
        assert bool(out[[1, 2, 5]].isnan().all()) and bool(out[fine].isfinite().all() if dtype == F16 else ~out[fine].isnan().any())


@pytest.mark.parametrize("off,pad", [(0, 8), (8, 8), (1, 0), (3, 5), (0, 1)])
def test_quantize_strides(off, pad):
    n, K = 37, 136
    buf = normal(gen(off + pad), (n, off + K + pad))
    x = buf[:, off:off + K]
    r = q.moe_quantize_rows(x)
    assert torch.equal(r.codes, ref8.quantized(x)[0])
    assert q.moe_quantize_rows(buf[:0]).codes.shape == (0, buf.shape[1])


def test_quantize_writes_only_its_rows():
    """From C, into rows wider than K: what lies between them stays."""
    lib = q.ops._lib()
    for dtype, K, ld in ((BF16, 64, 80), (F16, 33, 47), (BF16, 4096, 4104)):
        n = 6
        x = normal(gen(3), (n, K), 1.0, dtype)
        buf = torch.full((n + 2, ld), 77, dtype=torch.int8, device="cuda")
        sc = torch.full((n + 2,), 5.0, device="cuda")
        st = lib.moe_quantize_rows(q.ops._dtype_code(dtype), x.data_ptr(), K, n, K, buf[1].data_ptr(), ld,
                                   sc[1:].data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == q.MOE_OK
        assert torch.equal(buf[1:n + 1, :K], ref8.quantized(x)[0])
        assert bool((buf[1:n + 1, K:] == 77).all()) and bool((buf[[0, n + 1]] == 77).all())
        assert sc[0].item() == 5 and sc[n + 1].item() == 5


# ---- products ---------------------------------------------------------------------

# rows x columns x inputs at and around every tile border, the smallest and odd ones
LINEAR = [(1, 1, 16), (1, 2048, 2048), (2, 7, 32), (7, 17, 80), (8, 768, 2048), (9, 256, 144), (16, 100, 1040),
          (17, 33, 64), (31, 64, 48), (32, 130, 528), (33, 257, 2032), (64, 16, 128), (65, 511, 208), (127, 129, 192),
          (128, 128, 64), (129, 384, 320), (200, 1000, 1104), (256, 256, 256), (257, 256, 272), (317, 520, 2032),
          (513, 1031, 784), (1000, 40, 4096), (1024, 768, 768), (70, 300, 8192),
          # a handful of rows of more than 1024 inputs; many row tiles of each length
          (2, 2048, 2048), (3, 33, 1040), (4, 130, 4112), (4, 8, 20000), (5, 100, 2064), (4096, 1030, 144), (2500, 2000, 80)]


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("n,N,K", LINEAR)
def test_linear(n, N, K, dtype, gated):
    g = gen(1000 * n + N + K)
    i = LINEAR.index((n, N, K)) + (5 if gated else 0) + (2 if dtype == F16 else 0)
    act = ("none", "silu", "gelu", "gelu_tanh")[i % 4]
    t = weights(g, (), N, K, dtype, gated, i % 3 != 0)
    x = rows_of(g, n, K)
    res = normal(g, (n, N), 1.0, dtype) if i % 2 else None
    out = q.moe_linear_q8(x, q.LinearWeightsQ8(**t, activation=act, dtype=dtype), residual=res)
    ref.check(out, *ref8.product(*x, act=act, residual=res, **t))


@pytest.mark.parametrize("n", [1, 5, 40, 300])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
def test_linear_clamp(n, act):
    g = gen(n)
    t = weights(g, (), 264, 256, BF16, True, True)
    x = rows_of(g, n, 256)
    out = q.moe_linear_q8(x, q.LinearWeightsQ8(**t, activation=act, act_limit=0.75))
    ref.check(out, *ref8.product(*x, act=act, limit=0.75, **t))


@pytest.mark.parametrize("n", [1, 20, 90, 400])
@pytest.mark.parametrize("K", [1024, 2048, 65536])
def test_linear_sums_of_the_largest_codes(n, K):
    """All codes at the ends of their range: exact to 2^24 and an f32 sum above it. Then all
    products of one sign and one of the other."""
    g = gen(n + K)
    N = 40
    x = torch.full((n, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[::2] = 127
    w[5] = codes(g, (K,))
    w[7, :] = 0
    w[7, K - 1] = 1
    one, s = torch.ones(n, device="cuda"), torch.full((N,), 2.0 ** -20, device="cuda")
    out = q.moe_linear_q8((x, one), q.LinearWeightsQ8(w, s))
    ref.check(out, *ref8.product(x, one, w, s))
    if K == 1024:  # exact, as a power of two scales it: one rounding
        assert torch.equal(out, ((x.double() @ w.double().t()) * 2.0 ** -20).to(BF16))


@pytest.mark.parametrize("n", [3, 20, 150, 600])
def test_linear_strides_alignment_and_in_place_residual(n):
    g = gen(7 + n)
    N, K = 200, 336
    wide = codes(g, (n, K + 48))
    fused = codes(g, (2 * N, K + 16))
    x, w, w_up = wide[:, 16:16 + K], fused[:N, :K], fused[N:, :K]
    sx, s = scales(g, (n,), 1 / 74), scales(g, (2 * N,), K ** -0.5 / 74)
    lw = q.LinearWeightsQ8(w, s[:N], w_up=w_up, scale_up=s[N:], activation="silu")
    for off, pad in ((0, 0), (1, 3), (8, 16), (4, 4)):
        buf = normal(g, (n, N + off + pad))
        before = buf.clone()
        out = buf[:, off:off + N]
        r, d = ref8.product(x, sx, w, s[:N], w_up=w_up, scale_up=s[N:], act="silu", residual=out)
        got = q.moe_linear_q8((x, sx), lw, residual=out, out=out)
        assert got.data_ptr() == out.data_ptr()
        ref.check(out, r, d)
        assert torch.equal(buf[:, :off], before[:, :off]) and torch.equal(buf[:, off + N:], before[:, off + N:])


@pytest.mark.parametrize("n", [4, 24, 130, 700])
def test_linear_keeps_scales_that_are_no_numbers_to_their_rows_and_columns(n):
    g = gen(11)
    N, K = 272, 208
    x, t = rows_of(g, n, K), weights(g, (), N, K, BF16, False, False)
    x.scale[1], x.scale[n - 1] = NAN, INF
    t["scale"][5], t["scale"][N - 1] = INF, NAN
    out = q.moe_linear_q8(x, q.LinearWeightsQ8(**t))
    clean = torch.ones((n, N), dtype=torch.bool, device="cuda")
    clean[1], clean[n - 1], clean[:, 5], clean[:, N - 1] = False, False, False, False
    r, d = ref8.product(*x, **t)
    assert torch.equal(torch.isfinite(out), torch.isfinite(r)) and torch.equal(torch.isnan(out), torch.isnan(r))
    ref.check(out[clean], r[clean], d[clean])


# counts of rows per expert: none, one, ragged, all on one, many experts
COUNTS = [[1], [0, 0, 1], [3, 0, 9, 1], [40, 0, 7, 33, 64], [0, 300, 1, 0, 130], [1] * 64, [2, 0] * 50 + [200],
          [129, 257, 511], [0] * 200 + [5] * 3, [17] * 24, [256, 255], [700]]


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_grouped(counts, gated):
    i = COUNTS.index(counts) + (2 if gated else 0)
    g = gen(i)
    E, rows = len(counts), sum(counts)
    dtype = (BF16, F16)[i % 2]
    N, K = [(130, 208), (64, 512), (257, 96)][i % 3]
    act = ("silu", "none", "gelu", "gelu_tanh")[i % 4]
    t = weights(g, (E,), N, K, dtype, gated, i % 2 == 0)
    tokens = max(1, rows // 2)
    gather = i % 3 != 1
    x = rows_of(g, tokens if gather else rows + 3, K)
    token = torch.randint(0, tokens, (rows + 5,), generator=g, device="cuda").to(torch.int32) if gather else None
    total = rows + (5 if gather else 3)  # rows behind the last group stay as they were
    out = normal(g, (total, N), 1.0, dtype)
    before = out.clone()
    lw = q.LinearWeightsQ8(**t, activation=act, dtype=dtype)
    q.moe_grouped_linear_q8(x, lw, offsets_of(counts), row_token=token, out=out)
    assert torch.equal(out[rows:], before[rows:])
    at = 0
    for e, c in enumerate(counts):
        if c:
            xs = [v[token[at:at + c].long()] if gather else v[at:at + c] for v in x]
            r, d = ref8.product(*xs, act=act, **{k: v[e] for k, v in t.items()})
            ref.check(out[at:at + c], r, d)
        at += c


# a handful of rows per expert: runs of one, two and four of them, short and long rows of inputs
FEW = [[1], [1] * 8, [2, 2, 1, 3], [0, 5, 0, 0, 1, 0, 0, 0, 2], [4] * 3 + [0] * 300, [1] * 128, [2] * 64, [9] + [1] * 40, [64] + [0] * 63,
       [0] * 500 + [3, 1], [1, 0] * 512]


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("K", [16, 528, 1024, 1040, 2048, 4112])
@pytest.mark.parametrize("counts", FEW, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_grouped_few_rows(counts, K, gated):
    i = FEW.index(counts) + K // 16
    g = gen(i)
    E, rows, N = len(counts), sum(counts), (40, 37, 8)[i % 3]
    t = weights(g, (E,), N, K, BF16, gated, i % 2 == 0)
    x = rows_of(g, rows, K)
    token = torch.randperm(rows, generator=g, device="cuda").to(torch.int32) if i % 3 else None
    out = normal(g, (rows + 2, N))
    before = out.clone()
    q.moe_grouped_linear_q8(q.QuantizedRows(*x), q.LinearWeightsQ8(**t, activation="silu" if gated else "none"), offsets_of(counts),
                            row_token=token, out=out[:rows])
    assert torch.equal(out[rows:], before[rows:])
    at = 0
    for e, c in enumerate(counts):
        if c:
            xs = [v[token[at:at + c].long()] if token is not None else v[at:at + c] for v in x]
            ref.check(out[at:at + c], *ref8.product(*xs, act="silu" if gated else "none", **{k: v[e] for k, v in t.items()}))
        at += c


@pytest.mark.parametrize("rows", [5, 40, 300])
def test_grouped_reads_and_writes_nothing_out_of_range(rows):
    """Offsets and tokens that mean nothing: what is outside the buffers' rows is not touched."""
    g = gen(rows)
    E, N, K = 5, 96, 64
    x, t = rows_of(g, rows, K), weights(g, (E,), N, K, BF16, False, False)
    lw = q.LinearWeightsQ8(**t)
    buf = normal(g, (rows + 64, N))
    before = buf.clone()
    big = 2 ** 31 - 1
    for wild in ([0, -5, 10, big, 7, rows + 9], [big, -big, 3, 2, 1, 0], [-1, -2, -3, -4, -5, -6], [0, 3, 3, 3, 3, big]):
        off = torch.tensor(wild, dtype=torch.int32, device="cuda")
        token = torch.randint(-big, big, (rows,), generator=g, device="cuda").to(torch.int32)
        q.moe_grouped_linear_q8(x, lw, off, out=buf[32:32 + rows])
        q.moe_grouped_linear_q8(x, lw, off, row_token=token, out=buf[32:32 + rows])
    torch.cuda.synchronize()
    q.moe_ops_check()
    assert torch.equal(buf[:32], before[:32]) and torch.equal(buf[32 + rows:], before[32 + rows:])


def test_experts_that_share_one_matrix_and_lie_apart():
    g = gen(4)
    E, N, K, counts = 4, 80, 96, [30, 0, 5, 100]
    x = rows_of(g, sum(counts), K)
    one, s = codes(g, (N, K)), scales(g, (E, N), 1e-3)
    apart = codes(g, (E, N + 7, K + 32))
    for w in (one.expand(E, N, K), apart[:, 3:3 + N, 16:16 + K]):
        out = q.moe_grouped_linear_q8(x, q.LinearWeightsQ8(w, s), offsets_of(counts))
        at = 0
        for e, c in enumerate(counts):
            ref.check(out[at:at + c], *ref8.product(x.codes[at:at + c], x.scale[at:at + c], w[e], s[e]))
            at += c


def test_results_do_not_depend_on_the_run():
    g = gen(8)
    for n in (3, 30, 500):
        x, t = rows_of(g, n, 4096), weights(g, (), 300, 4096, BF16, True, True)
        lw = q.LinearWeightsQ8(**t, activation="silu")
        first = q.moe_linear_q8(x, lw)
        assert all(torch.equal(first, q.moe_linear_q8(x, lw)) for _ in range(5))


def test_no_rows():
    lw = q.LinearWeightsQ8(torch.zeros(16, 32, dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda"))
    e = (torch.zeros(0, 32, dtype=torch.int8, device="cuda"), torch.zeros(0, device="cuda"))
    assert q.moe_linear_q8(e, lw).shape == (0, 16)
    lg = q.LinearWeightsQ8(torch.zeros(2, 16, 32, dtype=torch.int8, device="cuda"), torch.ones(2, 16, device="cuda"))
    assert q.moe_grouped_linear_q8(e, lg, offsets_of([0, 0])).shape == (0, 16)


# ---- together ---------------------------------------------------------------------

def layer(g, E, D, F):
    return normal(g, (E, F, D), D ** -0.5), normal(g, (E, F, D), D ** -0.5), normal(g, (E, D, F), F ** -0.5)


def routed64(x, idx, w, experts, act="silu"):
    """The layer in 64 bits on the same codes, the activations between the products rounded
    and quantised as the layer does."""
    up, down = experts.gate_up.tensors, experts.down.tensors
    xq, sx = ref8.quantized(x)
    out = torch.zeros(x.shape[0], down[0].shape[1], dtype=torch.float64, device="cuda")
    for t in range(x.shape[0]):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if e >= 0:
                h, _ = ref8.product(xq[t:t + 1], sx[t:t + 1], up[0][e], up[2][e], w_up=up[1][e], scale_up=up[3][e], act=act)
                hq, hs = ref8.quantized(h.to(x.dtype))
                y, _ = ref8.product(hq, hs, down[0][e], down[2][e])
                out[t] += w[t, j].double() * y.to(x.dtype).double()[0]
    return out


@pytest.mark.parametrize("n", [1, 9, 130])
def test_router_and_experts_together(n):
    """Router, grouping, quantised experts and combine as one layer. The activations in between
    may round, and then quantise, one step apart from the 64-bit form's (2^-8 of a value, 1 / 127 of
    a row's largest): a few such steps over the row's sum stay below 2 % of its size."""
    g = gen(n)
    E, D, F, k = 16, 256, 128, 4
    experts = q.RoutedExpertsQ8.quantize(*layer(g, E, D, F))
    router = q.RouterLayer(normal(g, (E, D), D ** -0.5), q.Router(E, k, score="sigmoid", bias=0.1 * torch.randn(E, device="cuda"),
                                                                  groups=4, top_groups=2, group_score="top2", scale=2.5))
    x, res = normal(g, (n, D)), normal(g, (n, D))
    r = router.forward(x)
    out = experts.forward(x, r.topk_idx, r.topk_w, residual=res)
    want = routed64(x, r.topk_idx, r.topk_w, experts) + res.double()
    assert float((out.double() - want).norm() / want.norm()) < 0.02
    shared = q.SharedExpertQ8.quantize(*[t[0] for t in layer(g, 1, D, F)])
    both = shared.forward(x, residual=out)
    alone = shared.forward(x)
    assert float((both.double() - out.double() - alone.double()).norm() / both.double().norm()) < 2.0 ** -7
    experts.check()


def test_layer_captured_and_replayed_on_new_inputs():
    g = gen(12)
    E, D, F, k, n = 8, 128, 64, 2, 40
    experts = q.RoutedExpertsQ8.quantize(*layer(g, E, D, F))
    router = q.RouterLayer(normal(g, (E, D)), q.Router(E, k))
    x = normal(g, (n, D))

    def run():
        r = router.forward(x)
        return experts.forward(x, r.topk_idx, r.topk_w, residual=x)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(4):
        x.copy_(normal(g, (n, D)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, run())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = router.forward(x, stream=side)
    got = experts.forward(x, r.topk_idx, r.topk_w, residual=x, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, run())
    experts.check()


def test_weights_quantised_from_16_bits():
    g = gen(2)
    w, up = normal(g, (3, 40, 64)), normal(g, (3, 40, 64))
    lw = q.LinearWeightsQ8.quantize(w, w_up=up, activation="silu")
    c, s = ref8.quantized(up.reshape(-1, 64))
    assert torch.equal(lw.tensors[1].reshape(-1, 64), c) and lw.dtype == BF16 and lw.tensors[3].shape == (3, 40)
    x = q.moe_quantize_rows(normal(g, (9, 64)))
    out = q.moe_grouped_linear_q8(x, lw, offsets_of([4, 0, 5]))
    t = lw.tensors
    ref.check(out[:4], *ref8.product(x.codes[:4], x.scale[:4], t[0][0], t[2][0], w_up=t[1][0], scale_up=t[3][0], act="silu"))
