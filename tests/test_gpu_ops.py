"""The operators of include/moe_ops.h on the GPU against their 64-bit forms."""
import pytest
import torch

import ops_reference as ref
import quantized_moe_decode_softmax_gb300 as q

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, shape, std=1.0, dtype=BF16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def weights(g, lead, N, K, dtype, gated, bias):
    t = {"w": normal(g, lead + (N, K), K ** -0.5, dtype)}
    if gated:
        t["w_up"] = normal(g, lead + (N, K), K ** -0.5, dtype)
    if bias:
        t["bias"] = normal(g, lead + (N,), 0.5, dtype)
        if gated:
            t["bias_up"] = normal(g, lead + (N,), 0.5, dtype)
    return t


# rows x columns x inputs at and around every tile border, the smallest and odd ones
LINEAR = [(1, 1, 8), (1, 2048, 2048), (2, 7, 16), (7, 17, 72), (8, 768, 2048), (9, 256, 136), (16, 100, 1032),
          (17, 33, 64), (31, 64, 40), (32, 130, 520), (33, 257, 2040), (64, 16, 128), (65, 511, 200), (127, 129, 192),
          (128, 128, 64), (129, 384, 320), (200, 1000, 1096), (256, 256, 256), (317, 520, 2040), (513, 1031, 776),
          (1000, 40, 4096), (1024, 768, 768)]


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("n,N,K", LINEAR)
def test_linear(n, N, K, dtype, gated):
    g = gen(1000 * n + N + K)
    # activation, bias and residual vary with the case so that all meet all
    i = LINEAR.index((n, N, K)) + (5 if gated else 0) + (2 if dtype == F16 else 0)
    act = ("none", "silu", "gelu", "gelu_tanh")[i % 4]
    t = weights(g, (), N, K, dtype, gated, i % 3 != 0)
    x = normal(g, (n, K), 1.0, dtype)
    res = normal(g, (n, N), 1.0, dtype) if i % 2 else None
    out = q.moe_linear(x, q.LinearWeights(**t, activation=act), residual=res)
    ref.check(out, *ref.product(x, act=act, residual=res, **t))


@pytest.mark.parametrize("n", [1, 5, 40, 300])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
def test_linear_clamp(n, act):
    g = gen(n)
    t = weights(g, (), 264, 256, BF16, True, True)
    x = normal(g, (n, 256), 2.0)
    out = q.moe_linear(x, q.LinearWeights(**t, activation=act, act_limit=0.75))
    r, d = ref.product(x, act=act, limit=0.75, **t)
    ref.check(out, r, d)


@pytest.mark.parametrize("n", [3, 20, 150, 600])
def test_linear_strides_alignment_and_in_place_residual(n):
    """Rows of wider buffers, outputs off the 16-byte boundaries, the halves of a
    fused weight, a residual that the output replaces; nothing else is written."""
    g = gen(7 + n)
    N, K = 200, 328
    wide = normal(g, (n, K + 24))
    fused = normal(g, (2 * N, K + 8), K ** -0.5)
    x, w, w_up = wide[:, 8:8 + K], fused[:N, :K], fused[N:, :K]
    lw = q.LinearWeights(w, w_up=w_up, activation="silu")
    for off, pad in ((0, 0), (1, 3), (8, 16), (4, 4)):
        buf = normal(g, (n, N + off + pad))
        before = buf.clone()
        out = buf[:, off:off + N]
        r, d = ref.product(x, w, w_up=w_up, act="silu", residual=out)
        got = q.moe_linear(x, lw, residual=out, out=out)
        assert got.data_ptr() == out.data_ptr()
        ref.check(out, r, d)
        assert torch.equal(buf[:, :off], before[:, :off]) and torch.equal(buf[:, off + N:], before[:, off + N:])


@pytest.mark.parametrize("n", [4, 24, 130, 700])
def test_linear_keeps_nan_and_inf_to_their_rows_and_columns(n):
    g = gen(11)
    N, K = 272, 200  # the last K step is cut
    x, w = normal(g, (n, K)), normal(g, (N, K), K ** -0.5)
    x[1, 3], x[n - 1, K - 1] = float("nan"), float("inf")
    w[5, 0], w[N - 1, K - 1] = float("inf"), float("nan")
    out = q.moe_linear(x, q.LinearWeights(w))
    clean = torch.ones((n, N), dtype=torch.bool, device="cuda")
    clean[1], clean[n - 1], clean[:, 5], clean[:, N - 1] = False, False, False, False
    r, d = ref.product(x, w)
    assert torch.equal(torch.isfinite(out), torch.isfinite(r))
    assert torch.equal(torch.isnan(out), torch.isnan(r))
    ref.check(out[clean], r[clean], d[clean])


@pytest.mark.parametrize("n", [2, 40, 100])
def test_linear_extreme_values(n):
    """The largest and smallest 16-bit values, subnormals among them, pass through an
    identity product; f16 overflows to infinity as a cast does."""
    for dtype, values in ((BF16, [3.0e38, 1e-38, 1e-40, -1e-20]), (F16, [65504.0, 6e-5, 6e-8, -1e-7])):
        x = torch.tensor(values, device="cuda").to(dtype).repeat(n, 2)
        assert bool((x != 0).all())
        assert torch.equal(q.moe_linear(x, q.LinearWeights(torch.eye(8, device="cuda").to(dtype))), x)
    x = torch.full((n, 64), 60000.0, device="cuda").to(F16)
    out = q.moe_linear(x, q.LinearWeights(torch.ones(16, 64, dtype=F16, device="cuda")))
    assert bool(torch.isinf(out).all())


@pytest.mark.parametrize("n", [2, 90])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
def test_activations_over_the_whole_range(act, gated, n):
    """Each activation from -inf to inf through an identity product: the values and
    signs of infinities and NaN as the formula gives them."""
    z = torch.cat([torch.linspace(-30, 30, 400), torch.tensor([0.0, -0.0, 1e-6, -1e-6, 90.0, -90.0, 1e4, -1e4])]).cuda()
    for dtype, far in ((BF16, 3e38), (F16, 6e4)):
        v = torch.cat([z, torch.tensor([far, -far], device="cuda")]).to(dtype)
        w = torch.zeros(8, 8, dtype=dtype, device="cuda")
        w[0, 0] = 1
        one = torch.zeros(8, dtype=dtype, device="cuda")
        one[0] = 1
        for start in range(0, v.numel(), n):
            part = v[start:start + n]
            x = torch.zeros(part.numel(), 8, dtype=dtype, device="cuda")
            x[:, 0] = part
            lw = q.LinearWeights(w, w_up=torch.zeros_like(w) if gated else None, bias_up=one if gated else None,
                                 activation=act)
            d = part.double()
            r = ref.act64(act, d)
            r = torch.where(d < -1e3, torch.zeros_like(r) if act != "none" else r, r)  # exp overflows f64 there
            ref.check(q.moe_linear(x, lw)[:, 0], r, d.abs() * 2.0 ** -19 + 2.0 ** -22)
    # an infinite sum: bias of the type's infinity
    x, w = torch.zeros(n, 8, dtype=BF16, device="cuda"), torch.zeros(2, 8, dtype=BF16, device="cuda")
    b = torch.tensor([float("inf"), float("nan")], dtype=BF16, device="cuda")
    out = q.moe_linear(x, q.LinearWeights(w, bias=b, activation=act))
    assert bool((out[:, 0] == float("inf")).all()) and bool(torch.isnan(out[:, 1]).all())
    out = q.moe_linear(x, q.LinearWeights(w, bias=b, w_up=w, bias_up=torch.ones_like(b), activation=act, act_limit=2.0))
    r = ref.act64(act, torch.tensor(2.0, dtype=torch.float64))
    assert float((out[:, 0].double() - r.cuda()).abs().max()) <= 2.0 * 2.0 ** -8
    assert bool(torch.isnan(out[:, 1]).all())  # a clamp keeps a NaN


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("n,N,K", [(70, 256, 4096), (100, 300, 1000), (128, 128, 8192), (257, 512, 2056), (300, 40, 16384),
                                   (640, 768, 2048), (1500, 256, 8000)])
def test_linear_long_inputs_and_few_tiles(n, N, K, dtype, gated):
    """Fewer tiles than the GPU has SMs to run them, each over a long K."""
    g = gen(n + K)
    t = weights(g, (), N, K, dtype, gated, True)
    x, res = normal(g, (n, K), 1.0, dtype), normal(g, (n, N), 1.0, dtype)
    lw = q.LinearWeights(**t, activation="gelu")
    out = q.moe_linear(x, lw, residual=res)
    ref.check(out, *ref.product(x, act="gelu", residual=res, **t))
    for _ in range(5):
        assert torch.equal(q.moe_linear(x, lw, residual=res), out)
    q.moe_ops_check()


@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("n,N,K", [(100, 7, 8), (70, 1, 24), (333, 300, 16), (5000, 9, 72), (90, 2050, 1000)])
def test_linear_thin_products(n, N, K, gated):
    """Many rows with a few columns or inputs, far below a tile."""
    g = gen(n)
    t = weights(g, (), N, K, BF16, gated, True)
    x = normal(g, (n, K))
    ref.check(q.moe_linear(x, q.LinearWeights(**t, activation="silu")), *ref.product(x, act="silu", **t))


@pytest.mark.parametrize("rows", [3, 200])
def test_grouped_weights_in_other_layouts(rows):
    """One matrix for all experts, and experts inside the rows ([N, E, K])."""
    g = gen(rows)
    E, N, K = 3, 72, 136
    counts = [rows, 0, rows + 1]
    x = normal(g, (sum(counts), K))
    one = normal(g, (1, N, K), K ** -0.5).expand(E, N, K)
    mixed = normal(g, (N, E, K), K ** -0.5).transpose(0, 1)
    for w in (one, mixed):
        out = q.moe_grouped_linear(x, q.LinearWeights(w), offsets_of(counts))
        check_grouped(x, {"w": w}, counts, "none", out)


def test_empty_calls():
    lw = q.LinearWeights(torch.zeros(16, 24, dtype=BF16, device="cuda"))
    assert q.moe_linear(torch.zeros(0, 24, dtype=BF16, device="cuda"), lw).shape == (0, 16)
    gw = q.LinearWeights(torch.zeros(3, 16, 24, dtype=BF16, device="cuda"))
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert q.moe_grouped_linear(torch.zeros(0, 24, dtype=BF16, device="cuda"), gw, off).shape == (0, 16)
    g = q.moe_group_slots(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 5)
    assert g.offsets.tolist() == [0] * 6 and g.slot_of.shape == (0, 4)
    y = torch.zeros(0, 16, dtype=BF16, device="cuda")
    of, w = torch.full((3, 2), -1, dtype=torch.int32, device="cuda"), torch.ones(3, 2, device="cuda")
    assert torch.equal(q.moe_combine_slots(y, of, w), torch.zeros(3, 16, dtype=BF16, device="cuda"))
    assert q.moe_combine_slots(y, of[:0], w[:0]).shape == (0, 16)


def offsets_of(counts):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def check_grouped(x, t, counts, act, out, token=None, limit=0.0):
    at = 0
    for e, c in enumerate(counts):
        if c:
            rows = x[token[at:at + c].long()] if token is not None else x[at:at + c]
            r, d = ref.product(rows, act=act, limit=limit, **{k: v[e] for k, v in t.items()})
            ref.check(out[at:at + c], r, d)
        at += c


# rows per expert: none, one, tile borders, one expert with everything
GROUPS = [[1], [0, 3, 0], [1] * 8 + [0] * 56, [0] * 9 + [40] + [0] * 4, [5, 0, 17, 8, 0, 9, 1, 33],
          [128, 0, 127, 129, 1, 64, 63, 65], [300, 0, 2], [0, 0, 700], [16] * 40, [100, 3, 0, 260, 31, 0, 0, 5] * 4]


@pytest.mark.parametrize("gather", [False, True], ids=["rows", "gather"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped(case, dtype, gated, gather):
    counts = GROUPS[case]
    g = gen(50 + case)
    E, rows = len(counts), sum(counts)
    N, K = ((7, 8), (200, 136), (768, 512), (264, 1032))[(case + gated) % 4]
    act = ("none", "silu", "gelu", "gelu_tanh")[(case + 2 * gather) % 4]
    t = weights(g, (E,), N, K, dtype, gated, case % 2 == 0)
    tokens = max(1, rows // 3)
    x = normal(g, (tokens if gather else rows + 2, K), 1.0, dtype)
    token = torch.randint(0, tokens, (rows,), device="cuda", generator=g).to(torch.int32) if gather else None
    out = torch.full((rows if gather else rows + 2, N), 7.0, dtype=dtype, device="cuda")
    q.moe_grouped_linear(x, q.LinearWeights(**t, activation=act), offsets_of(counts), row_token=token, out=out)
    check_grouped(x, t, counts, act, out, token)
    assert bool((out[rows:] == 7).all())  # rows outside every group are left as they were


def test_grouped_fused_weights_and_strided_rows():
    """Gate and up as the halves of [E, 2 N, K], x and out as columns of wider rows."""
    g = gen(77)
    for counts in ([3, 0, 1, 6], [150, 0, 290, 40]):
        E, N, K, rows = 4, 136, 264, sum(counts)
        fused = normal(g, (E, 2 * N, K), K ** -0.5)
        x = normal(g, (rows, K + 16))[:, 16:]
        buf = normal(g, (rows, N + 5))
        before = buf.clone()
        t = {"w": fused[:, :N], "w_up": fused[:, N:]}
        q.moe_grouped_linear(x, q.LinearWeights(**t, activation="silu", act_limit=1.5), offsets_of(counts),
                             out=buf[:, 2:2 + N])
        check_grouped(x, t, counts, "silu", buf[:, 2:2 + N], limit=1.5)
        assert torch.equal(buf[:, :2], before[:, :2]) and torch.equal(buf[:, 2 + N:], before[:, 2 + N:])


@pytest.mark.parametrize("counts", [[4, 0, 3, 1], [70, 200, 0, 31]])
def test_grouped_keeps_nan_to_its_group(counts):
    """NaN in an unused expert's weights, in one row, and in the rows behind the last group."""
    g = gen(5)
    E, N, K, rows = 4, 72, 200, sum(counts)
    w = normal(g, (E, N, K), K ** -0.5)
    w[counts.index(0)] = float("nan")
    x = normal(g, (rows + 3, K))
    x[rows:] = float("nan")
    x[2] = float("nan")
    out = torch.zeros((rows + 3, N), dtype=BF16, device="cuda")
    q.moe_grouped_linear(x, q.LinearWeights(w), offsets_of(counts), out=out)
    assert bool(torch.isnan(out[2]).all())
    out[2], x[2] = 0, 0
    assert bool((out[rows:] == 0).all())
    check_grouped(x, {"w": w}, counts, "none", out)


@pytest.mark.parametrize("rows", [12, 700])
def test_grouped_bounds_offsets_and_tokens(rows):
    """Offsets and tokens outside their documented ranges touch nothing out of
    range: in-range groups are right and the bytes around the buffers stay."""
    g = gen(3)
    E, N, K = 3, 40, 64
    w = normal(g, (E, N, K), K ** -0.5)
    x = normal(g, (rows, K))
    buf = torch.full((rows + 64, N), 7.0, dtype=BF16, device="cuda")
    half = rows // 2
    if rows > 100:  # offsets that go back and forth: nothing is promised but that nothing else is touched
        wild = torch.tensor([rows, -9, 1 << 30, 5], dtype=torch.int32, device="cuda")
        q.moe_grouped_linear(x, q.LinearWeights(w), wild, out=buf[32:32 + rows])
        q.moe_ops_check()
        assert bool((buf[:32] == 7).all()) and bool((buf[32 + rows:] == 7).all())
    off = torch.tensor([-5, half, 1 << 30, -7], dtype=torch.int32, device="cuda")
    token = torch.arange(rows, dtype=torch.int32, device="cuda")
    token[-1], token[-2] = 1 << 30, -3
    q.moe_grouped_linear(x, q.LinearWeights(w), off, row_token=token, out=buf[32:32 + rows])
    out = buf[32:32 + rows]
    check_grouped(x, {"w": w}, [half, rows - half - 2], "none", out[:rows - 2])
    assert bool((buf[:32] == 7).all()) and bool((buf[32 + rows:] == 7).all())
    q.moe_ops_check()


SLOTS = [(1, 1, 1, 0, 1), (1, 8, 128, 0, 128), (3, 2, 5, 1, 4), (8, 8, 128, 0, 128), (33, 4, 16, 0, 16),
         (64, 6, 256, 64, 128), (200, 3, 1024, 0, 1024), (511, 8, 7, 0, 7), (600, 7, 33, 5, 5), (1100, 4, 64, 0, 64),
         (5000, 2, 300, 17, 250)]


@pytest.mark.parametrize("n,k,E,lo,hi", SLOTS)
def test_group_slots(n, k, E, lo, hi):
    """Against a loop over the slots; ids repeat inside a token, some are -1 or
    outside the experts."""
    g = gen(n + k)
    idx = torch.randint(-1, E + 1, (n, k), device="cuda", generator=g).to(torch.int32)
    got = q.moe_group_slots(idx, E, experts=(lo, hi))
    by = {}
    for i, e in enumerate(idx.reshape(-1).tolist()):
        if lo <= e < hi:
            by.setdefault(e, []).append((i // k, i % k))
    rows = [s for e in sorted(by) for s in by[e]]
    want = ref.slot_tables(rows, idx.tolist(), n, k, E)
    for name, w in zip(("offsets", "slot_token", "slot_k", "slot_of"), want):
        assert getattr(got, name).cpu().tolist() == w, name


@pytest.mark.parametrize("n,k,E", [(1, 1, 1), (3, 3, 5), (8, 8, 128)])
def test_group_slots_outputs_stand_alone(n, k, E):
    """Each of the four tensors can be written, moved to another type and outlive
    the others without a change in them; a call within inference mode gives the same."""
    idx = torch.randint(0, E, (n, k), device="cuda", generator=gen(n)).to(torch.int32)
    want = [t.tolist() for t in q.moe_group_slots(idx, E)]
    with torch.inference_mode():
        assert [t.tolist() for t in q.moe_group_slots(idx, E)] == want
    for i in range(4):
        got = list(q.moe_group_slots(idx, E))
        got[i].fill_(-77)
        assert [t.tolist() for j, t in enumerate(got) if j != i] == [w for j, w in enumerate(want) if j != i]
        last, got = got[3 - i], None
        other = torch.full((4096,), 5, dtype=torch.int32, device="cuda")  # may take freed memory
        assert last.add(0).tolist() == want[3 - i] and last.is_contiguous() and int(other[0]) == 5


def test_group_slots_without_ranks_and_long():
    """slot_k left out; a million slots, against a stable sort."""
    n, k, E = 131072, 8, 1000
    g = gen(9)
    idx = torch.randint(0, E, (n, k), device="cuda", generator=g).to(torch.int32)
    idx[: n // 2] = 3  # half of all slots on one expert
    a = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    token, of = torch.empty(n * k, dtype=torch.int32, device="cuda"), torch.empty(n, k, dtype=torch.int32, device="cuda")
    lib = q.ops._lib()
    st = torch.cuda.current_stream().cuda_stream
    assert lib.moe_group_slots(idx.data_ptr(), n, k, E, 0, E, a.data_ptr(), token.data_ptr(), None, of.data_ptr(),
                               st) == q.MOE_OK
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    assert torch.equal(token.long(), order // k)
    assert torch.equal(of.reshape(-1)[order].long(), torch.arange(n * k, device="cuda"))
    assert torch.equal(a[1:].long(), torch.cumsum(torch.bincount(flat, minlength=E), 0)) and int(a[0]) == 0


def combine_ref(y, of, w, residual):
    n, k = of.shape
    acc = torch.zeros((n, y.shape[1]), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(acc)
    for j in range(k):
        live = (of[:, j] >= 0) & (of[:, j] < y.shape[0])
        rows = y.double()[of[:, j].long().clamp(0, max(0, y.shape[0] - 1))] * w[:, j:j + 1].double()
        rows = torch.where(live[:, None], rows, torch.zeros_like(rows))
        acc, mag = acc + rows, mag + rows.abs()
    if residual is not None:
        acc, mag = acc + residual.double(), mag + residual.double().abs()
    return acc, mag * (2 * k + 2) * 2.0 ** -24  # a rounding per product and per sum


@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("n,k,N,rows", [(1, 1, 1, 1), (1, 8, 2048, 8), (5, 3, 7, 9), (8, 8, 2048, 64), (33, 6, 129, 100),
                                        (64, 16, 264, 900), (700, 8, 1000, 5600), (9, 64, 40, 300)])
def test_combine(n, k, N, rows, dtype):
    g = gen(n + N)
    y = normal(g, (rows, N), 1.0, dtype)
    of = torch.randint(-2, rows + 2, (n, k), device="cuda", generator=g).to(torch.int32)  # some slots add nothing
    w = torch.rand((n, k), device="cuda", generator=g)
    w[of < 0] = float("nan")  # the weight of a slot that adds nothing does not matter
    for residual in (None, normal(g, (n, N), 1.0, dtype)):
        r, d = combine_ref(y, of, torch.nan_to_num(w), residual)
        ref.check(q.moe_combine_slots(y, of, w, residual=residual), r, d)
    # strided, unaligned, in place
    wide = normal(g, (rows, N + 3), 1.0, dtype)
    buf = normal(g, (n, N + 4), 1.0, dtype)
    before = buf.clone()
    r, d = combine_ref(wide[:, 3:], of, torch.nan_to_num(w), buf[:, 1:N + 1])
    q.moe_combine_slots(wide[:, 3:], of, w, residual=buf[:, 1:N + 1], out=buf[:, 1:N + 1])
    ref.check(buf[:, 1:N + 1], r, d)
    assert torch.equal(buf[:, 0], before[:, 0]) and torch.equal(buf[:, N + 1:], before[:, N + 1:])


def layer_tensors(g, E, D, F, dtype=BF16):
    lead = (E,) if E else ()
    return (normal(g, lead + (F, D), D ** -0.5, dtype), normal(g, lead + (F, D), D ** -0.5, dtype),
            normal(g, lead + (D, F), F ** -0.5, dtype))


def route(g, n, k, E):
    top, idx = torch.topk(torch.randn((n, E), device="cuda", generator=g), k, dim=1)
    return idx.to(torch.int32), torch.softmax(top, 1)


@pytest.mark.parametrize("n,k,E,D,F", [(1, 8, 128, 256, 128), (8, 2, 8, 256, 128), (64, 8, 32, 512, 256),
                                       (500, 6, 16, 264, 136)])
def test_routed_and_shared_experts_together(n, k, E, D, F):
    """Group, gate and up, down, combine onto the shared expert's output: as a
    layer runs them, against the same with every intermediate rounded alike."""
    g = gen(n + E)
    gate, up, down = layer_tensors(g, E, D, F)
    sg, su, sd = layer_tensors(g, 0, D, F)
    x, res = normal(g, (n, D)), normal(g, (n, D))
    idx, w = route(g, n, k, E)
    shared = q.SharedExpert(sg, su, sd).forward(x, residual=res)
    out = q.RoutedExperts(gate, up, down).forward(x, idx, w, residual=shared)
    # two shards of the experts: the second adds to the first
    half = q.RoutedExperts(gate, up, down, experts=(0, E // 2)).forward(x, idx, w, residual=shared)
    parts = q.RoutedExperts(gate, up, down, experts=(E // 2, E)).forward(x, idx, w, residual=half)
    r = res.double()
    mlp = lambda a, b, c: (ref.product(x, a, w_up=b, act="silu")[0].to(BF16).double() @ c.double().t())  # noqa: E731
    r = (r + mlp(sg, su, sd)).to(BF16).double()
    scale = r.abs()
    for j in range(k):
        for e in idx[:, j].unique().tolist():
            at = idx[:, j] == e
            y = mlp(gate[e], up[e], down[e])[at] * w[at, j:j + 1].double()
            r[at] += y
            scale[at] += y.abs()
    # a step (2^-7) of h, weighted by the size of y's terms, a step of y and of the
    # sums: each value passes at most four roundings that may fall the other way
    root = float(scale.square().mean().sqrt())
    for got in (out, parts):
        err = (got.double() - r).abs()
        assert float(err.max()) <= 4 * 2.0 ** -7 * (float(scale.max()) + root), float(err.max())
        assert float(err.square().mean().sqrt()) <= 2.0 ** -8 * 2 * root


def test_shared_expert_beside_the_quantised_step():
    """MoeDecodeLayer.forward(shared=...) is the step plus the shared expert."""
    from gpu_cases import case, device_layer, make_plan, x_tensor
    lay, x = case("qwen3", 2, 4)
    dl, xt = device_layer(lay), x_tensor(lay.shape, x)
    shared = q.SharedExpert(*layer_tensors(gen(1), 0, lay.shape.D, lay.shape.F))
    plan = make_plan(lay.shape)
    step = plan.forward(xt, dl).clone()
    both = plan.forward(xt, dl, shared=shared)
    assert torch.equal(both, shared.forward(xt, residual=step))
    plan.check()
    with pytest.raises(TypeError):
        make_plan(lay.shape, out_dtype="f32").forward(xt, dl, shared=shared)


def run_all(x, t, tg, idx, w):
    a = q.moe_linear(x, t)
    g = q.moe_group_slots(idx, tg.E)
    b = q.moe_grouped_linear(x, tg, g.offsets, row_token=g.slot_token)
    return a, b, q.moe_combine_slots(b, g.slot_of, w, residual=a), g.slot_of


@pytest.mark.parametrize("n", [2, 40, 600])
def test_graphs_streams_and_repeats(n):
    """The same bits from eager calls, a side stream, and two captured graphs
    replayed in turn on new inputs."""
    E, k, N, K = 16, 4, 264, 200
    g = gen(n)
    t = q.LinearWeights(normal(g, (N, K), K ** -0.5), activation="silu")
    tg = q.LinearWeights(normal(g, (E, N, K), K ** -0.5), w_up=normal(g, (E, N, K), K ** -0.5), activation="gelu")
    x = normal(g, (n, K))
    idx, w = route(g, n, k, E)
    want = [v.clone() for v in run_all(x, t, tg, idx, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run_all(x, t, tg, idx, w)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    given = q.moe_linear(x, t, stream=side)
    side.synchronize()
    assert torch.equal(given, want[0])
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(run_all(x, t, tg, idx, w))
        graphs.append(gr)
    x2 = normal(g, (n, K))
    idx2, w2 = route(g, n, k, E)
    want2 = [v.clone() for v in run_all(x2, t, tg, idx2, w2)]
    old = [v.clone() for v in (x, idx, w)]
    for first in (True, False, True):
        for dst, src in zip((x, idx, w), old if first else (x2, idx2, w2)):
            dst.copy_(src)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for o in outs:
            for a, b in zip(want if first else want2, o):
                assert torch.equal(a, b)


@pytest.mark.parametrize("n", [1, 90])
def test_calls_with_and_without_the_torch_module(n, monkeypatch):
    """The same bits and the same refusals with the torch_calls module and without."""
    g = gen(n)
    t = q.LinearWeights(normal(g, (72, 136), 0.1), activation="silu")
    tg = q.LinearWeights(normal(g, (6, 72, 136), 0.1))
    x, res = normal(g, (n, 136)), normal(g, (n, 72))
    idx, w = route(g, n, 2, 6)

    def every():
        out = normal(gen(1), (n, 80))[:, 3:75]
        yield q.moe_linear(x, t, residual=res)
        yield q.moe_linear(x, t, residual=out, out=out)
        s = q.moe_group_slots(idx, 6, experts=(1, 5))
        yield from s
        y = torch.zeros(2 * n, 72, dtype=BF16, device="cuda")
        yield q.moe_grouped_linear(x, tg, s.offsets, row_token=s.slot_token, out=y)
        yield q.moe_combine_slots(y, s.slot_of, w, residual=res)
        yield q.moe_combine_slots(y[:, 1:], s.slot_of, w)

    def refused():
        for call in (lambda: q.moe_linear(x[:, :128], t), lambda: q.moe_linear(x.half(), t),
                     lambda: q.moe_linear(x, tg), lambda: q.moe_linear(x.cpu(), t),
                     lambda: q.moe_linear(x.t().contiguous().t() if n > 1 else x[:, ::2], t),
                     lambda: q.moe_linear(x, t, residual=res[:, :71]), lambda: q.moe_linear(x, t, out=x),
                     lambda: q.moe_linear(x.clone().requires_grad_(), t),
                     lambda: q.moe_linear(x, t, residual=res.clone().requires_grad_()),
                     lambda: q.moe_linear(x[:1].expand(9, 136), t), lambda: q.moe_linear(None, t),
                     lambda: q.moe_grouped_linear(x, tg, torch.zeros(6, dtype=torch.int32, device="cuda")),
                     lambda: q.moe_grouped_linear(x, tg, torch.zeros(7, device="cuda")),
                     lambda: q.moe_grouped_linear(x, t, torch.zeros(2, dtype=torch.int32, device="cuda")),
                     lambda: q.moe_group_slots(idx, 2000), lambda: q.moe_group_slots(idx, 6, experts=(4, 2)),
                     lambda: q.moe_group_slots(idx.long(), 6), lambda: q.moe_group_slots(idx, 0),
                     lambda: q.moe_combine_slots(x, idx, w.double()), lambda: q.moe_combine_slots(x.float(), idx, w),
                     lambda: q.moe_combine_slots(x, idx[:, :1], w)):
            try:
                call()
                yield "nothing"
            except Exception as e:
                yield type(e).__name__

    assert q.ops._calls is not None
    with_module, refusals = [v.clone() for v in every()], list(refused())
    monkeypatch.setattr(q.ops, "_calls", None)
    for a, b in zip(with_module, every()):
        assert torch.equal(a, b)
    assert list(refused()) == refusals and "nothing" not in refusals


@pytest.mark.parametrize("n", [1, 8, 40, 130])
def test_back_to_back_calls_see_each_other(n):
    """A chain that reads what the call before has just written, in place and out of
    place, the kernels overlapping at their ends: the same bits as with a wait after
    every call."""
    g = gen(n)
    D, F, E, k = 512, 264, 8, 2
    up, down = q.LinearWeights(normal(g, (F, D), D ** -0.5)), q.LinearWeights(normal(g, (D, F), F ** -0.5))
    tg = q.LinearWeights(normal(g, (E, D, D), D ** -0.5), activation="silu")
    start, ids = normal(g, (n, D)), [route(g, n, k, E) for _ in range(4)]

    def chain(wait):
        x, h = start.clone(), torch.empty((n, F), dtype=BF16, device="cuda")
        torch.cuda.synchronize()
        for i in range(40):
            calls = [lambda: q.moe_linear(x, up, out=h), lambda: q.moe_linear(h, down, residual=x, out=x)]
            for c in calls:
                c()
                if wait:
                    torch.cuda.synchronize()
            idx, w = ids[i % 4]
            s = q.moe_group_slots(idx, E)
            if wait:
                torch.cuda.synchronize()
            y = q.moe_grouped_linear(x, tg, s.offsets, row_token=s.slot_token)
            if wait:
                torch.cuda.synchronize()
            q.moe_combine_slots(y, s.slot_of, w, residual=x, out=x)
            x.mul_(0.5)  # another library's kernel in between
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return x

    want = chain(True)
    assert bool(torch.isfinite(want).all())
    for _ in range(5):
        assert torch.equal(chain(False), want)


def test_two_streams_at_once():
    """Independent calls that overlap on the device do not disturb one another."""
    g = gen(21)
    sets = []
    for i in range(2):
        n, N, K, E, k = (700, 264, 776, 8, 3) if i else (9, 768, 512, 32, 4)
        idx, w = route(g, n, k, E)
        sets.append((normal(g, (n, K)), q.LinearWeights(normal(g, (N, K), K ** -0.5)),
                     q.LinearWeights(normal(g, (E, N, K), K ** -0.5)), idx, w))
    want = [[v.clone() for v in run_all(*s)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(run_all(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for a, b in zip(want[i], run):
                assert torch.equal(a, b)
