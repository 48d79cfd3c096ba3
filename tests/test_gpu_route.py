"""moe_route on the GPU against plain 64-bit routing."""
import itertools
import math

import pytest
import torch

import quantized_moe_decode_softmax_gb300 as q
import route_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
INF, NAN = float("inf"), float("nan")


def logits(seed, n, E, dtype=F32, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = std * torch.randn((n, E), generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    return z.to(dtype), 0.1 * torch.randn(E, generator=g, device="cuda")


def both(z, k, **rule):
    """The call against the reference, with and without the torch_calls module, and with the
    rows many times over (from 4096 on, eight lanes take a row instead of a warp)."""
    router = q.Router(z.shape[1], k, **rule)
    r = q.moe_route(z, router)
    ref.check(r, z, k, **rule)
    keep, q.ops._calls = q.ops._calls, None
    try:
        again = q.moe_route(z, router)
    finally:
        q.ops._calls = keep
    assert torch.equal(r.topk_idx, again.topk_idx) and torch.equal(r.topk_w, again.topk_w)
    n = z.shape[0]
    if n <= 64:
        times = 4100 // n + 1
        many = q.moe_route(z.repeat(times, 1), router)
        ids, w = many.topk_idx.view(times, n, k), many.topk_w.view(times, n, k)
        assert bool((ids == r.topk_idx).all())
        assert torch.equal(w.view(torch.int32), w[:1].expand_as(w).contiguous().view(torch.int32))
        ref.check(q.Routing(ids[0], w[0]), z, k, **rule)
    return r


# experts at and around what a lane holds (4, 8, 16, 32 for 128, 256, 512, 1024) and odd ones
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
@pytest.mark.parametrize("n,E,k", [(1, 1, 1), (1, 2, 2), (3, 5, 5), (1, 128, 8), (7, 64, 6), (5, 127, 1), (4, 129, 9),
                                   (64, 256, 8), (9, 257, 33), (6, 300, 64), (3, 512, 31), (2, 513, 32), (5, 1023, 10),
                                   (33, 1024, 64)])
def test_route(n, E, k, biased, score):
    i = n + E + k + (1 if biased else 0)
    z, b = logits(i, n, E, (F32, BF16, F16)[i % 3])
    both(z, k, score=score, bias=b if biased else None, renormalize=i % 2 == 0, scale=(1.0, 2.5)[i % 2])


GROUPED = [(1, 256, 8, 8, 4), (40, 160, 6, 8, 3), (3, 32, 1, 32, 1), (5, 64, 7, 32, 31), (9, 12, 4, 3, 2), (4, 33, 3, 11, 1),
           (4, 1024, 8, 2, 1), (6, 1000, 16, 20, 5), (2, 16, 8, 8, 4), (2, 8, 2, 8, 2), (3, 96, 12, 24, 3)]


@pytest.mark.parametrize("score,biased,best", list(itertools.product(["softmax", "sigmoid"], [False, True], ["max", "top2"])))
@pytest.mark.parametrize("n,E,k,groups,top", GROUPED)
def test_groups(n, E, k, groups, top, score, biased, best):
    z, b = logits(n + E, n, E, (F32, BF16)[n % 2])
    both(z, k, score=score, bias=b if biased else None, groups=groups, top_groups=top, group_score=best,
         renormalize=best == "max")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
def test_ties_go_to_the_lower_id(score, biased):
    """Rows of equal logits, of a few values each, zeros of both signs, equal groups."""
    E = 96
    z = torch.zeros(6, E, device="cuda")
    z[1] = torch.arange(E, device="cuda") % 3
    z[2, ::2] = -0.0
    z[3, 50:] = 1.0
    z[4] = 2.0
    z[5, 17], z[5, 80] = 3.0, 3.0
    b = torch.full((E,), 0.25, device="cuda") if biased else None
    for k in (1, 7, 40):
        r = both(z, k, score=score, bias=b)
        assert r.topk_idx[0].tolist() == list(range(k)) and r.topk_idx[2].tolist() == list(range(k))
    for best in ("max", "top2"):
        r = both(z, 12, score=score, bias=b, groups=8, top_groups=3, group_score=best)
        assert r.topk_idx[0].tolist() == list(range(12))


def test_scores_next_to_each_other_are_told_apart():
    """Keys whose f32 forms are equal or in the wrong order: the ids are those of c in f64."""
    E = 64
    g = torch.Generator().manual_seed(5)
    z = 15 + 2 * torch.rand((50, E), generator=g)  # s = 1 - 1e-7 .. : f32 holds one or two values
    b = torch.zeros(E)
    both(z.cuda(), 8, score="sigmoid", bias=b.cuda())
    b = torch.randint(0, 3, (E,), generator=g) * 2.0 ** -24
    both(z.cuda(), 8, score="sigmoid", bias=b.cuda())
    both(z.cuda(), 8, score="sigmoid", bias=b.cuda(), groups=8, top_groups=3, group_score="top2")
    # logits one f32 step apart
    z = torch.full((20, E), 0.7)
    z = (z.view(torch.int32) + torch.randint(-3, 4, (20, E), generator=g, dtype=torch.int32)).view(F32)
    for score in ("sigmoid", "softmax"):
        both(z.cuda(), 9, score=score, bias=torch.full((E,), 0.5).cuda())
        both(z.cuda(), 9, score=score, groups=16, top_groups=5, group_score="top2")
        both(z.cuda(), 9, score=score, bias=torch.full((E,), 0.5).cuda(), groups=16, top_groups=5, group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,tied,target", [(40, 6, 0.75), (200, 25, 0.5), (256, 31, 1.0), (128, 90, 0.3), (1000, 20, 2.0), (64, 33, -3.0)])
def test_scores_that_tie_but_for_the_rounding_of_their_bias(E, tied, target, score):
    """Score + bias is `target` for some experts, but for the bias's rounding to f32: their ranks lie
    2^-26 |target| and less from each other."""
    for seed in range(4):
        g = torch.Generator().manual_seed(100 * E + seed)
        z = (2.5 * torch.randn(E, generator=g)).to(F32)
        s = torch.tensor(ref.scores(z.double().tolist(), score), dtype=torch.float64)
        b = torch.full((E,), target - 1.5, dtype=torch.float64)
        chosen = torch.randperm(E, generator=g)[:tied]
        b[chosen] = target - s[chosen]
        both(z[None].cuda(), min(8, tied), score=score, bias=b.to(F32).cuda(), scale=1.5)


@pytest.mark.parametrize("n", [3000, 5001])
def test_many_rows_with_a_bias(n):
    """Enough rows that some are ranked again; a warp or eight lanes a row."""
    z, b = logits(77, n, 256, BF16)
    both(z, 8, score="sigmoid", bias=b, groups=8, top_groups=4, group_score="top2")
    both(z[:, :200], 6, score="softmax", bias=0.01 * b[:200].contiguous(), scale=2.5)
    both(z[:, :60].float(), 9, score="sigmoid", groups=4, top_groups=2, group_score="top2")


def test_close_rows_side_by_side():
    """Rows that are ranked again next to rows that are not, in every place of a warp, with more
    ranks than lanes have a row: all lanes vote, whatever their row has found."""
    g = torch.Generator().manual_seed(8)
    E = 250
    z, b = logits(78, 4500, E)
    close = torch.rand(4500, generator=g) < 0.3
    z[close.cuda()] = (17 + 2 * torch.rand((int(close.sum()), E), generator=g)).cuda()
    b = (torch.randint(0, 2, (E,), generator=g) * 2.0 ** -24).cuda()
    for k in (3, 8, 20):
        both(z, k, score="sigmoid", bias=b)
        both(z, k, score="sigmoid", bias=b, groups=5, top_groups=2, group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top", [(1, 1), (4, 2)])
def test_experts_that_take_no_part(score, groups, top):
    """-inf and NaN logits or biases: never chosen; a row that has too few experts ends in
    -1, one that has none is all -1; the rows beside it do not change."""
    E, k = 40, 6
    z, b = logits(3, 8, E)
    z[0, :] = -INF
    z[1, :] = NAN
    z[2, 1:] = -INF
    z[3, 5:] = -INF
    z[4, ::2] = NAN
    z[5, 10:38] = -INF
    r = both(z, k, score=score, groups=groups, top_groups=top, group_score="top2")
    assert r.topk_idx[0].tolist() == [-1] * k and r.topk_idx[1].tolist() == [-1] * k
    assert r.topk_idx[2].tolist() == [0] + [-1] * (k - 1)
    assert r.topk_w[:2].abs().max().item() == 0
    off = b.clone()
    off[::3] = -INF
    off[1] = NAN
    r = both(z, k, score=score, bias=off, groups=groups, top_groups=top)
    live = r.topk_idx[r.topk_idx >= 0]
    assert bool((live % 3 != 0).all()) and not bool((live == 1).any())


@pytest.mark.parametrize("biased", [False, True], ids=["plain", "biased"])
def test_infinite_logits_and_biases(biased):
    E = 24
    z, b = logits(4, 4, E)
    z[0, 3], z[0, 20] = INF, INF
    z[1, 0] = INF
    bias = b if biased else None
    for renormalize in (True, False):
        r = q.moe_route(z, q.Router(E, 4, bias=bias, renormalize=renormalize))
        if not biased:
            assert r.topk_idx[0, :2].tolist() == [3, 20] and r.topk_idx[1, 0].item() == 0
        got = dict(zip(r.topk_idx[0].tolist(), r.topk_w[0].tolist()))
        assert got[3] == 0.5 and got[20] == 0.5 and sum(got.values()) == 1.0
        ref.check(q.Routing(r.topk_idx[2:], r.topk_w[2:]), z[2:], 4, bias=bias, renormalize=renormalize)
    r = q.moe_route(z, q.Router(E, 4, score="sigmoid", bias=bias, renormalize=False))
    got = dict(zip(r.topk_idx[0].tolist(), r.topk_w[0].tolist()))
    assert (biased or {3, 20} <= set(got)) and got.get(3, 1.0) == 1.0 and got.get(20, 1.0) == 1.0
    force = b.clone()
    force[[2, 9, 11]] = INF
    r = q.moe_route(z, q.Router(E, 4, score="sigmoid", bias=force))
    assert r.topk_idx[:, :3].tolist() == [[2, 9, 11]] * 4
    force[:] = INF
    r = q.moe_route(z, q.Router(E, 4, score="sigmoid", bias=force, groups=6, top_groups=2, group_score="top2"))
    assert r.topk_idx.tolist() == [[0, 1, 2, 3]] * 4


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(score):
    """Scores that underflow: their ratios are kept where they are renormalised."""
    z = torch.tensor([[-200.0, -201.0, -202.5, -300.0], [100.0, 99.0, -100.0, -104.0], [3e38, -3e38, 0.0, 1e38],
                      [-1e30, -2e30, -3e30, -3.4e38], [-87.0, -88.0, -90.0, -95.0], [-39.0, -41.0, -60.0, -80.0]],
                     device="cuda")
    for renormalize in (True, False):
        both(z, 3, score=score, renormalize=renormalize)
    # groups and a bias that choose experts far below the largest logit
    both(z.repeat(1, 3), 2, score=score, bias=torch.tensor([0.0] * 8 + [3.0] * 4, device="cuda"), groups=3, top_groups=1)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("E", [8, 100, 256, 1000])
def test_strides_and_alignment(E, dtype):
    n = 5
    buf, _ = logits(E, n, E + 24, dtype)
    for off, width in ((0, E + 24), (1, E + 24), (8, E + 24), (3, E + 24)):
        z = buf[:, off:off + E]
        both(z, min(E, 5))
    column = buf.t()[:E, :n]
    with pytest.raises(ValueError):
        q.moe_route(column.t()[:, ::2], q.Router((E + 1) // 2, 1))


def test_no_rows_and_many_rows():
    r = q.moe_route(torch.zeros(0, 16, device="cuda"), q.Router(16, 4))
    assert r.topk_idx.shape == (0, 4) and r.topk_w.shape == (0, 4)
    n = 70001
    z = torch.randn(n, 8, device="cuda")
    r = q.moe_route(z, q.Router(8, 2))
    top = torch.topk(z, 2)
    assert torch.equal(r.topk_idx.long(), top.indices)
    assert float((r.topk_w - torch.softmax(top.values, 1)).abs().max()) < 1e-6


def test_captured_and_replayed_on_new_logits():
    z, b = logits(9, 17, 256)
    router = q.Router(256, 8, score="sigmoid", bias=b, groups=8, top_groups=4, group_score="top2")
    q.moe_route(z, router)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = q.moe_route(z, router)
    for seed in range(3):
        z.copy_(logits(100 + seed, 17, 256)[0])
        b.copy_(logits(200 + seed, 17, 256)[1])
        graph.replay()
        torch.cuda.synchronize()
        ref.check(r, z, 8, score="sigmoid", bias=b, groups=8, top_groups=4, group_score="top2")


def test_on_another_stream_and_two_at_once():
    z, b = logits(10, 2000, 256)
    router = q.Router(256, 8, score="sigmoid", bias=b)
    want = q.moe_route(z, router)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [q.moe_route(z, router, stream=s) for s in streams] + [q.moe_route(z, router, stream=streams[0].cuda_stream)]
    torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r.topk_idx, want.topk_idx) and torch.equal(r.topk_w, want.topk_w)


def test_bias_follows_its_tensor():
    z = torch.zeros(2, 8, device="cuda")
    b = torch.arange(8.0, device="cuda")
    router = q.Router(8, 2, bias=b)
    assert q.moe_route(z, router).topk_idx.tolist() == [[7, 6]] * 2
    old = b.data
    b.data = -torch.arange(8.0, device="cuda")
    assert q.moe_route(z, router).topk_idx.tolist() == [[0, 1]] * 2
    b.data = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        q.moe_route(z, router)
    del old


def test_feeds_the_grouping_and_the_combine():
    """Ids of -1 from a row without experts belong to no group, and the row's output is its
    residual."""
    z = torch.randn(6, 16, device="cuda")
    z[2] = -INF
    r = q.moe_route(z, q.Router(16, 4))
    g = q.moe_group_slots(r.topk_idx, 16)
    assert g.offsets[-1].item() == 20 and g.slot_of[2].tolist() == [-1] * 4
    y = torch.randn(24, 32, device="cuda").to(BF16)
    res = torch.randn(6, 32, device="cuda").to(BF16)
    out = q.moe_combine_slots(y, g.slot_of, r.topk_w, residual=res)
    assert torch.equal(out[2], res[2]) and math.isfinite(out.float().sum().item())
