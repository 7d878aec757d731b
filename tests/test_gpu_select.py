"""Routing by scores and its gradient on the GPU against plain 64-bit forms."""
import math

import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref, select_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(T, E, dtype, seed):
    """Random logits; from row 8 on (where there are so many) rows that are special."""
    l = torch.randn(T, E, generator=gen(seed), device="cuda") * 2
    special = [
        lambda r: r.fill_(-INF), lambda r: r.fill_(0.25), lambda r: r.fill_(NAN), lambda r: r[: E - 1].fill_(-INF),
        lambda r: r[::2].fill_(NAN), lambda r: r[E // 2:].fill_(INF), lambda r: r.mul_(1e37), lambda r: r.mul_(1e-38),
        lambda r: r.sub_(400.0), lambda r: r.add_(60.0), lambda r: r[1:].fill_(-3e38), lambda r: r.copy_(r.sign() * 0.0),
        lambda r: r[: E // 2].fill_(-INF), lambda r: r.sub_(2000.0), lambda r: r[0].fill_(INF),
    ]
    for i, f in enumerate(special):
        if 8 + i < T:
            f(l[8 + i])
    return l.to(dtype)


def run(l, k, spare=True, **kw):
    """ids, weights and scores of a call, all between guards."""
    T, E = l.shape
    ids, ib = ops_ref.guarded(torch.full((T, k), -7, dtype=torch.int32, device="cuda"), 16, -7)
    w, wb = ops_ref.guarded(torch.full((T, k), 7.0, device="cuda"), 16, 7.0)
    s, sb = ops_ref.guarded(torch.full((T, E), 7.0, device="cuda"), 16, 7.0)
    moe.moe_select(l, ids, w, scores=s if spare else None, **kw)
    for big, v in ((ib, -7), (wb, 7.0), (sb, 7.0)):
        assert ops_ref.guards_intact(big, 16, v)
    return ids, w, s


def score_bound(l, want, score):
    """fp32 scores. Sigmoid: e^-|l| 4 half steps, 1 + it 3 more, the reciprocal 2, the product 1. Softmax: logit - maximum rounds
    by half a step of itself, which the exponential turns into a relative error; the exponential 4, the sum of up to 256
    terms 16 + 4 and the terms' own errors 8, the quotient and the product 2. Subnormal results: a few times 2^-149."""
    if score == "sigmoid":
        return 10 * U * want + 2.0 ** -146
    x = l.cpu().double().nan_to_num(nan=-INF)
    far = (x.amax(1, keepdim=True) - x).nan_to_num(nan=0.0).clamp(max=110.0)
    return (far + 36) * U * want + 2.0 ** -146


def check(l, k, **kw):
    ids, w, s = run(l, k, **kw)
    wi, ww, ws = ref.select(l.cpu(), k, **kw)
    assert torch.equal(ids.cpu(), wi)
    assert bool(((s.cpu().double() - ws).abs() <= score_bound(l, ws, kw["score"])).all())
    # weights are rounded once (half a step, or half of the smallest subnormal), but for the softmax's fp32 sum
    halves = 36 if kw["score"] == "softmax" and not kw["renorm"] else 1.0001
    assert bool(((w.cpu().double() - ww).abs() <= halves * U * ww.abs() + 2.0 ** -149).all())
    again = run(l, k, spare=False, **kw)
    assert torch.equal(ids, again[0]) and torch.equal(w, again[1]) and bool((again[2] == 7.0).all())


# (T, E, k, groups, group_k, group_top)
SHAPES = [
    (1, 1, 1, 1, 1, 1), (1, 256, 8, 8, 4, 2), (40, 256, 8, 1, 1, 1), (33, 256, 8, 8, 4, 2), (40, 256, 8, 8, 3, 1),
    (40, 160, 6, 8, 3, 2), (40, 160, 6, 8, 3, 1), (23, 64, 6, 1, 1, 1), (40, 60, 2, 4, 2, 2), (40, 7, 7, 7, 7, 2),
    (40, 7, 3, 1, 1, 1), (40, 255, 8, 5, 2, 2), (40, 255, 5, 51, 20, 2), (40, 128, 8, 64, 9, 1), (40, 64, 4, 64, 64, 2),
    (40, 128, 8, 64, 40, 2), (30, 130, 1, 1, 1, 1), (30, 130, 3, 10, 1, 2), (30, 193, 4, 1, 1, 1), (40, 2, 2, 2, 2, 2),
    (40, 200, 8, 40, 33, 2), (17, 96, 8, 3, 2, 2), (40, 8, 8, 1, 1, 1), (15, 68, 8, 17, 16, 1),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_select(shape, score, renorm, dtype):
    T, E, k, groups, group_k, group_top = shape
    l, _ = ops_ref.guarded(rows(T, E, dtype, E + k), 16, NAN)
    kw = dict(score=score, renorm=renorm, scale=2.5, groups=groups, group_k=group_k, group_top=group_top)
    check(l, k, **kw)
    bias = torch.randn(E, generator=gen(1), device="cuda") * 0.2
    check(l, k, bias=bias, **kw)
    bias[::5] = -INF
    bias[3::7] = NAN
    bias[1::11] = INF
    check(l, k, bias=bias, **kw)
    check(l, k, bias=torch.zeros(E, device="cuda"), **kw)


def test_order_of_near_logits_and_choices():
    """Without a bias the order is that of the logits, however close their scores; with one, differences of 2^-40 count."""
    l = torch.full((2, 200), -1.0, device="cuda")
    l[0, 10], l[0, 150] = 60.0, 60.5
    l[1, 10], l[1, 150] = 1.0, torch.nextafter(torch.tensor(1.0), torch.tensor(2.0))
    for score in ("softmax", "sigmoid"):
        ids, _, _ = run(l, 2, score=score)
        assert ids.tolist() == [[150, 10]] * 2
    # the least fp32 step of a logit moves its score by 2^-23 s (1 - s)
    ids, _, _ = run(l[1:], 2, score="sigmoid", bias=torch.full((200,), 0.5, device="cuda"))
    assert ids.tolist() == [[150, 10]]
    # -0 and 0 are equal: the lowest id first
    z = torch.zeros(1, 40, device="cuda")
    z[0, :20] = -0.0
    z[0, 3] = 0.0
    assert run(z, 8, score="sigmoid")[0].tolist() == [list(range(8))]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("groups,group_k", [(1, 1), (8, 3), (16, 5)])
def test_close_choices(score, dtype, groups, group_k):
    """Choices a few steps of fp32 apart, on both sides of what fp32 can tell, in rows beside ordinary ones; ranges that
    32-bit keys do not hold (logits and biases far apart or large)."""
    T, E, k = 48, 64, 8
    g = gen(groups)
    base = torch.randn(T, E, generator=g, device="cuda")
    steps = torch.randint(-3, 4, (T, E), generator=g, device="cuda").float()
    l = torch.where(torch.arange(T, device="cuda")[:, None] % 3 == 0, 1.0 + steps * 2.0 ** -23, base)
    l[1::6] *= 200
    l[2::6] += 1000
    l = l.to(dtype)
    tiny = steps[0] * 2.0 ** -24
    for bias in (None, tiny, 0.5 + tiny, torch.randn(E, generator=g, device="cuda"), 3 + tiny, 1e4 * tiny, 100 + 10 * steps[1],
                 torch.where(steps[2] > 0, -1e9, 0.25)):
        for top in (1, 2):
            check(l, k, score=score, renorm=True, scale=1.0, bias=bias, groups=groups, group_k=group_k, group_top=top)


GRADS = [(1, 1, 1), (1, 256, 8), (40, 256, 8), (40, 64, 6), (33, 160, 6), (40, 7, 7), (23, 255, 8), (40, 130, 1),
         (17, 193, 4), (40, 2, 2), (30, 128, 3)]


@pytest.mark.parametrize("shape", GRADS)
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("dtype,dl_dtype,dense", [(F32, F32, True), (F32, BF, False), (BF, F32, False), (BF, BF, True)])
def test_select_backward(shape, score, renorm, dtype, dl_dtype, dense):
    T, E, k = shape
    l, _ = ops_ref.guarded(rows(T, E, dtype, 3 * E + k), 16, NAN)
    g = gen(E)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    if T > 8:
        ids[3] = int(ids[3, 0])  # one expert in every slot
        ids[4, 0], ids[5, -1], ids[6, 0] = -1, E, -2 ** 31
        ids[7] = -1
    dw = torch.randn(T, k, generator=g, device="cuda")
    dw[ids < 0] = NAN  # the gradient of a slot without an expert is not looked at
    ds = torch.randn(T, E, generator=g, device="cuda") * 0.1 if dense else None
    dl, big = ops_ref.guarded(torch.full((T, E), 7.0, device="cuda", dtype=dl_dtype), 16, 7.0)
    moe.moe_select_backward(l, ids, dw, dl, score=score, renorm=renorm, scale=2.5, dscores=ds)
    want, bound = ref.backward(l.cpu(), ids.cpu(), dw.cpu(), score, renorm, 2.5, None if ds is None else ds.cpu())
    err = (dl.cpu().double() - want).abs()
    assert not err.isnan().any()
    bound = bound + ops_ref.HALF[dl_dtype] * (want.abs() + bound)
    assert bool((err <= bound).all()), (err / bound.clamp(min=1e-300)).max()
    assert ops_ref.guards_intact(big, 16, 7.0)
    again = torch.empty_like(dl)
    moe.moe_select_backward(l, ids, dw, again, score=score, renorm=renorm, scale=2.5, dscores=ds)
    assert torch.equal(again, dl)


@pytest.mark.parametrize("level", [-2000.0, -300.0, -20.0, 5.0, 20.0, 300.0, 900.0, 1e5])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [dict(), dict(groups=8, group_k=3, group_top=2), dict(groups=8, group_k=3)])
def test_bias_of_any_level(level, score, groups):
    """A common level in the bias costs the choices their last bits in fp32: they are ordered as in fp64, some of them
    a few fp32 steps of that level apart, and so are groups whose largest choices cancel."""
    T, E, k = 48, 64, 6
    g = gen(int(abs(level)))
    l = torch.randn(T, E, generator=g, device="cuda")
    l[::2] = l[::2, :1] + torch.randn(T // 2, E, generator=g, device="cuda") * abs(level) * 2.0 ** -23
    bias = level + torch.randn(E, generator=g, device="cuda") * 0.1
    bias[::4] = level
    check(l, k, score=score, renorm=True, bias=bias, **groups)
    bias[::8] = -level
    check(l, k, score=score, renorm=True, bias=bias, **groups)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Directional differences of the kernel's own weights and scores (the choice held: no near ties move it)."""
    T, E, k = 64, 96, 4
    g = gen(2)
    l = torch.randn(T, E, generator=g, device="cuda")
    l[:, :k] += 8.0  # the chosen ones stand clear
    dw, ds = torch.randn(T, k, generator=g, device="cuda"), torch.randn(T, E, generator=g, device="cuda")
    step = torch.randn(T, E, generator=g, device="cuda")

    def loss(x):
        ids, w, s = run(x, k, score=score, renorm=renorm)
        at = torch.zeros(T, E, device="cuda", dtype=torch.float64).scatter_(1, ids.long(), w.double())
        return (at[:, :k] * dw).sum(1) + (s.double() * ds).sum(1)

    ids = torch.arange(k, device="cuda", dtype=torch.int32).repeat(T, 1)
    dl = torch.empty(T, E, device="cuda")
    moe.moe_select_backward(l, ids, dw, dl, score=score, renorm=renorm, dscores=ds)
    h = 2.0 ** -6
    num = (loss(l + h * step) - loss(l - h * step)) / (2 * h)
    # fp32 results: up to 100 terms of size <= 4 off by 2^-24 each, over h; third derivative times h^2 / 6
    assert (num - (dl.double() * step).sum(1)).abs().max() < 400 * U / h + 60 * h * h


def test_large_batch_and_empty():
    """More tokens than one dimension of blocks is wide elsewhere, the last block partly filled; and none."""
    T, E, k = 300007, 64, 6
    l = torch.randn(T, E, generator=gen(4), device="cuda")
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.moe_select(l, ids, w)
    top = torch.sort(l, dim=1, descending=True, stable=True)
    assert torch.equal(ids, top.indices[:, :k].int())
    want = torch.softmax(top.values[:, :k].double(), 1)
    assert bool(((w.double() - want).abs() <= 1.0001 * U * want).all())
    moe.moe_select(l[:0], ids[:0], w[:0])
    moe.moe_select_backward(l[:0], ids[:0], w[:0], l[:0].clone())


def test_past_32_bit_offsets():
    """Rows behind 4 GiB of logits, scores and gradients."""
    T, E, k = (1 << 24) - 1, 256, 2
    tail = 40
    l = torch.zeros(T, E, dtype=BF, device="cuda")
    l[-tail:] = rows(tail, E, BF, 9)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    s = torch.empty(T, E, device="cuda")
    moe.moe_select(l, ids, w, score="sigmoid", scores=s)
    wi, ww, ws = ref.select(l[-tail:].cpu(), k, "sigmoid")
    assert torch.equal(ids[-tail:].cpu(), wi) and bool((ids[:-tail] == torch.arange(k, device="cuda")).all())
    assert bool(((s[-tail:].cpu().double() - ws).abs() <= score_bound(l[-tail:], ws, "sigmoid")).all())
    assert bool((s[:-tail] == 0.5).all())
    dl = torch.empty(T, E, device="cuda")
    moe.moe_select_backward(l, ids, w, dl, score="sigmoid", renorm=False, dscores=s)
    want, bound = ref.backward(l[-tail:].cpu(), wi, w[-tail:].cpu(), "sigmoid", False, 1.0, s[-tail:].cpu())
    assert bool(((dl[-tail:].cpu().double() - want).abs() <= bound + U * want.abs()).all())


def test_streams_and_graphs():
    """Two streams at once and a graph replayed among eager work: the results of one call after the other."""
    T, E, k = 500, 256, 8
    kw = dict(score="sigmoid", groups=8, group_k=4, group_top=2, scale=2.5)
    bias = torch.randn(E, generator=gen(6), device="cuda") * 0.1
    ls = [torch.randn(T, E, generator=gen(7 + i), device="cuda") for i in range(3)]
    dw = torch.randn(T, k, generator=gen(11), device="cuda")

    def outs():
        return (torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"),
                torch.empty(T, E, device="cuda"))

    def both(l, o, stream=None):
        moe.moe_select(l, o[0], o[1], bias=bias, stream=stream, **kw)
        moe.moe_select_backward(l, o[0], dw, o[2], score="sigmoid", scale=2.5, stream=stream)

    want = [outs() for _ in ls]
    for l, o in zip(ls, want):
        both(l, o)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ls], [outs() for _ in ls]
    for l, o, st in zip(ls, got, streams):
        both(l, o, st)
    torch.cuda.synchronize()
    for o, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    x, o = ls[0].clone(), outs()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both(x, o)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        both(x, o)
    for l, w in list(zip(ls, want)) * 2:
        x.copy_(l)
        graph.replay()
        eager = outs()
        both(ls[1], eager)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, w)) and torch.equal(eager[1], want[1][1])


@pytest.mark.parametrize("E,k,first", [(2, 1, 0), (2, 1, 1), (7, 3, 0), (64, 1, 0), (64, 8, 1), (200, 8, 0), (256, 2, 0)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
@pytest.mark.parametrize("dense", [False, True])
def test_gradient_of_sure_tokens(E, k, first, score, renorm, dense):
    """Tokens whose largest score is nearly all of the sum: the gradients are its small rest, to the digits that the rest
    has. first 0: the largest is the first slot, 1: it is not among the slots (k = 1) or is the second."""
    gaps = torch.tensor([8.0, 12.0, 16.0, 17.0, 20.0, 25.0, 33.0, 40.0, 60.0], device="cuda").repeat(2)
    T, g = len(gaps), gen(E + k)
    l = torch.randn(T, E, generator=g, device="cuda") * 0.5
    top = torch.randint(0, E, (T,), generator=g, device="cuda")
    at = torch.arange(T, device="cuda")
    # by gap over all others' sum
    l[at, top] = gaps + l.amax(1) + math.log(E)
    if score == "sigmoid":  # scores far below 1 are in the ratios of a softmax
        l -= l.amax(1, keepdim=True) + 1
    others = torch.rand(T, E, generator=g, device="cuda")
    others[at, top] = 2.0
    order = others.argsort(1, descending=True)
    if first:
        order = torch.cat((order[:, 1:2], order[:, :1], order[:, 2:]), 1)
    ids = order[:, :k].to(torch.int32).contiguous()
    dw = torch.randn(T, k, generator=g, device="cuda")
    dw[T // 2:] = 1 + dw[T // 2:] * 2.0 ** -12  # nearly equal ones
    ds = torch.randn(T, E, generator=g, device="cuda") * 0.1 if dense else None
    for dl_dtype in (F32, BF):
        dl = torch.empty(T, E, device="cuda", dtype=dl_dtype)
        moe.moe_select_backward(l, ids, dw, dl, score=score, renorm=renorm, scale=2.5, dscores=ds)
        want, bound = ref.backward_sure(l.cpu(), ids.cpu(), dw.cpu(), score, renorm, 2.5, None if ds is None else ds.cpu())
        err = (dl.cpu().double() - want).abs()
        bound = bound + ops_ref.HALF[dl_dtype] * (want.abs() + bound)
        assert bool((err <= bound).all()), (err / bound).max()
