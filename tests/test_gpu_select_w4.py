"""Routing by scores and 4-bit integer weights as one layer: served, and trained through frozen weights."""
import math

import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref, select_ref, w4_ref

pytestmark = pytest.mark.gpu
BF, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
INF, NAN = float("inf"), float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def empty(*shape, t=F32):
    return torch.empty(*shape, dtype=t, device="cuda")


def quantised(w, group, zeros, sdtype):
    """Codes of weights [E, K, N] along K: [E, N, K/2]."""
    E, K, N = w.shape
    q = dict(codes=empty(E, N, K // 2, t=U8), scales=empty(E, N, K // group, t=sdtype),
             zeros=empty(E, N, K // group, t=U8) if zeros else None)
    moe.moe_w4_quantize(w, q["codes"], q["scales"], zeros=q["zeros"], trans=True)
    return q


def weights64(q):
    return w4_ref.weights64(q["codes"], q["scales"], q["zeros"])


def layer(seed, T, k, E, H, I, group=64, zeros=True, sdtype=BF, masked=True, **route):
    g = gen(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    L = dict(T=T, k=k, E=E, H=H, I=I, x=r(T, H).to(BF), logits=r(T, E), bias=r(E) * 0.1, dout=r(T, H).to(BF),
             dscores=r(T, E), route=route,
             up=quantised((r(E, H, 2 * I) * H ** -0.5).to(BF), group, zeros, sdtype),
             down=quantised((r(E, I, H) * I ** -0.5).to(BF), group, zeros, sdtype))
    if masked and T > 2:
        L["logits"][1] = -INF                    # a padded token: no expert at all
        L["logits"][2, k - 1:] = NAN             # fewer experts than slots
    return L


def buffers(L):
    T, k, E, H, I = (L[n] for n in ("T", "k", "E", "H", "I"))
    P, i32 = T * k, torch.int32
    return dict(ids=empty(T, k, t=i32), w=empty(T, k), s=empty(T, E), counts=empty(E, t=i32), off=empty(E + 1, t=i32),
                sp=empty(P, t=i32), pp=empty(P, t=i32), a=torch.full((P, 2 * I), 7.0, dtype=BF, device="cuda"),
                h=empty(P, I, t=BF), y=torch.full((P, H), 7.0, device="cuda"), out=empty(T, H, t=BF), out32=empty(T, H),
                dy=empty(P, H, t=BF), dw=empty(T, k), dh=torch.zeros(P, I, dtype=BF, device="cuda"), da=empty(P, 2 * I, t=BF),
                dxs=empty(P, H), dx=empty(T, H, t=BF), dx32=empty(T, H), dl=empty(T, E), ones=torch.ones(T, k, device="cuda"),
                wu=empty(E, 2 * I, H, t=BF), wd=empty(E, H, I, t=BF))


def serve(L, b, stream=None):
    st = dict(stream=stream)
    moe.moe_select(L["logits"], b["ids"], b["w"], bias=L["bias"], scores=b["s"], **L["route"], **st)
    moe.moe_permute(b["ids"], L["E"], b["counts"], b["off"], b["sp"], b["pp"], **st)
    up, down = L["up"], L["down"]
    moe.moe_w4_grouped_gemm(L["x"], up["codes"], up["scales"], b["off"], b["a"], zeros=up["zeros"], row_index=b["sp"],
                            row_div=L["k"], **st)
    moe.moe_swiglu(b["a"], b["h"], **st)
    moe.moe_w4_grouped_gemm(b["h"], down["codes"], down["scales"], b["off"], b["y"], zeros=down["zeros"], **st)
    moe.moe_finalize(b["y"], b["pp"], b["w"], b["out"], out_f32=b["out32"], **st)


def train(L, b, stream=None):
    """serve, then the gradients of x and of the logits through frozen weights."""
    st = dict(stream=stream)
    serve(L, b, stream)
    up, down, kind = L["up"], L["down"], {n: v for n, v in L["route"].items() if n in ("score", "renorm", "scale")}
    moe.moe_finalize_backward(L["dout"], b["y"], b["pp"], b["w"], b["dy"], b["dw"], **st)
    moe.moe_select_backward(L["logits"], b["ids"], b["dw"], b["dl"], dscores=L["dscores"], **kind, **st)
    moe.moe_w4_dequantize(down["codes"], down["scales"], b["wd"], zeros=down["zeros"], **st)
    moe.moe_grouped_gemm(b["dy"], b["wd"], b["off"], b["dh"], **st)
    moe.moe_swiglu_backward(b["a"], b["dh"], b["da"], **st)
    moe.moe_w4_dequantize(up["codes"], up["scales"], b["wu"], zeros=up["zeros"], **st)
    moe.moe_grouped_gemm(b["da"], b["wu"], b["off"], b["dxs"], **st)
    moe.moe_finalize(b["dxs"], b["pp"], b["ones"], b["dx"], out_f32=b["dx32"], **st)


def close(got, want, bound):
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (err / bound.clamp(min=1e-300)).max().item()


GROUPED = dict(score="sigmoid", groups=4, group_k=2, group_top=2, scale=2.5)
PLAIN = dict(score="softmax")
WHOLE = dict(score="softmax", renorm=False, groups=4, group_k=3)


@pytest.mark.parametrize("T,k,E,H,I,route", [(1, 2, 8, 64, 64, GROUPED), (45, 4, 16, 320, 192, GROUPED), (90, 6, 64, 256, 64, PLAIN),
                                             (333, 3, 8, 192, 128, WHOLE), (3000, 4, 8, 512, 320, GROUPED)])
@pytest.mark.parametrize("group,zeros,sdtype", [(32, True, F32), (64, False, BF)])
def test_serving_pass(T, k, E, H, I, route, group, zeros, sdtype):
    """Each stage against 64 bits, from what the stage before it wrote."""
    L = layer(T, T, k, E, H, I, group, zeros, sdtype, **route)
    b = buffers(L)
    serve(L, b)
    some = min(T, 64)
    want, ww, _ = select_ref.select(L["logits"][:some].cpu(), k, bias=L["bias"].cpu(), **route)
    assert torch.equal(b["ids"][:some].cpu(), want)
    # one rounding, and 36 half steps of 2^-24 by a softmax's fp32 sum
    close(b["w"][:some].cpu(), ww, 37 * 2.0 ** -24 * ww.abs() + 2.0 ** -149)
    counts = b["counts"].tolist()
    used = sum(counts)
    assert used == int((b["ids"] >= 0).sum()) and (used < T * k) == (T > 2)
    assert bool((b["a"][used:] == 7.0).all()) and bool((b["y"][used:] == 7.0).all())
    for rows, q, got, depth in ((ops_ref.gather64(L["x"], T * k, b["sp"], k), L["up"], b["a"], H), (b["h"].double(), L["down"], b["y"], I)):
        ref, _ = ops_ref.product64(rows, weights64(q), counts, True)
        mag = ops_ref.product64(rows.abs(), w4_ref.spread64(q["codes"], q["scales"], q["zeros"]), counts, True)[0]
        close(got[:used], ref, ops_ref.sum_bound(ref, mag, depth + 8, got.dtype))
    pos = b["pp"].long().view(T, k)
    terms = torch.where(pos[..., None] >= 0, b["y"].double()[pos.clamp(min=0)], 0.0) * b["w"].double()[..., None]
    close(b["out"], terms.sum(1), ops_ref.sum_bound(terms.sum(1), terms.abs().sum(1), k + 1, BF))
    if T > 2:
        assert not b["out"][1].any()


def scores64(l, score):
    dead = l.isnan() | (l == -INF)
    l = torch.where(dead, -INF, l)
    if score == "sigmoid":
        return torch.where(dead, 0.0, torch.sigmoid(torch.where(dead, 0.0, l)))
    m = l.amax(1, keepdim=True)
    e = torch.where(dead, 0.0, (torch.where(dead, 0.0, l) - torch.where(m == -INF, 0.0, m)).exp())
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def loss64(L, ids, x, l, wu, wd):
    """<out, dout> + <scores, dscores> in fp64 for the choice ids."""
    T, k, route = L["T"], L["k"], L["route"]
    s = scores64(l, route["score"])
    w = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0)), 0.0)
    if route.get("renorm", True):
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    w = w * route.get("scale", 1.0)
    out = torch.zeros(T, L["H"], dtype=torch.float64)
    for e in range(L["E"]):
        t, j = (ids == e).nonzero(as_tuple=True)
        a = x[t] @ wu[e].t()
        h = torch.nn.functional.silu(a[:, :L["I"]]) * a[:, L["I"]:]
        out = out.index_add(0, t, w[t, j].unsqueeze(1) * (h @ wd[e].t()))
    return (out * L["dout"].double().cpu()).sum() + (s * L["dscores"].double().cpu()).sum()


@pytest.mark.parametrize("route", [GROUPED, PLAIN, WHOLE])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 64, 64), (37, 3, 8, 128, 64), (150, 2, 4, 192, 128)])
def test_training_pass(T, k, E, H, I, route):
    """Gradients of x and of the logits through the whole layer against fp64 and its differences.

    dx: seven results are rounded to bf16 on the longest way (a, h, dy, dh, da and the two sets of weights), each by at
    most 2^-8 of its value: 7 * 2^-8 of its norm. dw: a and h, then sums of H fp32 products of y with dout: 3 * 2^-8 of
    |y| |dout|, whose norm is at least that of dw. The logits' gradient takes dw through scale r (1 - r), whose norm is
    at most scale (1 + sqrt k), and its fp32 roundings are far below."""
    L = layer(T + 1, T, k, E, H, I, **route)
    b = buffers(L)
    train(L, b)
    ids = b["ids"].cpu().long()
    wu, wd = (weights64(L[n]).cpu() for n in ("up", "down"))
    x, l = L["x"].double().cpu().requires_grad_(), L["logits"].double().cpu().requires_grad_()
    dx, dl = torch.autograd.grad(loss64(L, ids, x, l, wu, wd), (x, l))
    dl = torch.nan_to_num(dl)
    assert (b["dx32"].double().cpu() - dx).norm() <= 7 * 2.0 ** -8 * dx.norm()
    pos = b["pp"].cpu().long()
    y = torch.where(pos[:, None] >= 0, b["y"].double().cpu()[pos.clamp(min=0)], 0.0).view(T, k, H)
    size = (y.norm(dim=2) * L["dout"].double().cpu().norm(dim=1, keepdim=True)).norm()
    allowed = 3 * 2.0 ** -8 * size * route.get("scale", 1.0) * (1 + math.sqrt(k)) + 1e-4
    assert (b["dl"].double().cpu() - dl).norm() <= allowed
    # a difference along a random direction, the choice held
    gc = torch.Generator().manual_seed(T)
    ux, ul = (torch.randn(t.shape, generator=gc, dtype=torch.float64) for t in (x, l))
    h = 1e-6
    with torch.no_grad():
        up, down = (loss64(L, ids, x + c * h * ux, l + c * h * ul, wu, wd) for c in (1, -1))
    slope = ((up - down) / (2 * h)).item()
    got = ((b["dx32"].double().cpu() * ux).sum() + (b["dl"].double().cpu() * ul).sum()).item()
    assert abs(got - slope) <= 7 * 2.0 ** -8 * (dx.norm() * ux.norm()).item() + (allowed * ul.norm()).item() + 1e-6 * abs(slope)
    if T > 2:
        assert not b["dx"][1].any() and not b["dl"][1].any()


@pytest.mark.parametrize("T,k,E,H,I", [(5, 4, 16, 256, 128), (900, 4, 16, 320, 192)])
def test_streams_and_graphs(T, k, E, H, I):
    """Two passes side by side on streams given by the caller, both captured and replayed among eager work."""
    Ls = [layer(seed, T, k, E, H, I, **GROUPED) for seed in (1, 2)]
    want = [buffers(L) for L in Ls]
    for L, b in zip(Ls, want):
        train(L, b)
    torch.cuda.synchronize()
    names = [n for n in want[0] if n not in ("h", "dy", "da", "dh", "dxs", "a", "y")]  # the others hold rows nobody writes
    got, streams = [buffers(L) for L in Ls], [torch.cuda.Stream() for _ in Ls]
    torch.cuda.synchronize()
    for L, b, st in zip(Ls, got, streams):
        with torch.cuda.stream(st):
            train(L, b, st)
    torch.cuda.synchronize()
    cap, graphs = [buffers(L) for L in Ls], []
    for L, b in zip(Ls, cap):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            train(L, b)
        graphs.append(graph)
    for _ in range(3):
        for b in cap:
            for n in ("ids", "w", "off", "out", "dx", "dl"):
                b[n].fill_(3)
        for graph in graphs:
            graph.replay()
        train(Ls[1], got[1])
        torch.cuda.synchronize()
        for b, v in list(zip(cap, want)) + list(zip(got, want)):
            for n in names:
                assert torch.equal(b[n], v[n]), n


def test_logits_that_arrive_late():
    """The call waits for what its stream still has to write."""
    T, k, E, H, I = 64, 4, 16, 256, 128
    L = layer(3, T, k, E, H, I, **GROUPED)
    want = buffers(L)
    serve(L, want)
    st, b = torch.cuda.Stream(), buffers(L)
    late = dict(L, logits=torch.zeros_like(L["logits"]), x=torch.zeros_like(L["x"]))
    busy = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(4):
            busy = busy @ busy * 1e-2
        late["logits"].copy_(L["logits"])
        late["x"].copy_(L["x"])
    serve(late, b, st)
    st.synchronize()
    assert torch.equal(b["ids"], want["ids"]) and torch.equal(b["out"], want["out"])


def test_choice_of_moe_route():
    """On moe_route's own logits, softmax scores choose what it chooses."""
    T, H, E, k = 130, 256, 64, 6
    g = gen(8)
    x, wr = torch.randn(T, H, generator=g, device="cuda"), torch.randn(H, E, generator=g, device="cuda") * H ** -0.5
    logits, ids, w = empty(T, E), empty(T, k, t=torch.int32), empty(T, k)
    need = moe.moe_route_workspace_size(T, H, E)
    moe.moe_route(x, wr, None, k, moe.MOE_F32, logits, None, ids, w, moe.workspace(need) if need else None)
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    moe.moe_select(logits, ids2, w2)
    assert torch.equal(ids2, ids)
    # both are softmaxes over the chosen logits; moe_route's in fp32: differences (far) 2^-24 of at most 16, an
    # exponential, a sum of six, a quotient
    assert bool(((w2 - w).abs() <= 40 * 2.0 ** -24 * w2).all())


@pytest.mark.parametrize("route", [GROUPED, PLAIN, WHOLE])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 64, 64), (37, 3, 8, 128, 64), (150, 2, 4, 192, 128), (60, 4, 16, 320, 192)])
def test_training_pass_logits_step_by_step(T, k, E, H, I, route):
    """The weights' and the logits' gradients, each against 64 bits from what the step before it wrote, to fp32 roundings."""
    L = layer(T + 5, T, k, E, H, I, **route)
    b = buffers(L)
    train(L, b)
    c = {n: v.cpu() for n, v in dict(b, **{n: L[n] for n in ("dout", "logits", "dscores")}).items()}
    kind = {n: v for n, v in route.items() if n in ("score", "renorm", "scale")}
    dw, dl, share = select_ref.gradient_chain(c["y"], c["dout"], c["pp"].view(T, k), c["dw"], c["logits"], c["ids"], c["dl"],
                                              c["dscores"], **kind)
    assert dw <= 1 and dl <= 1 and share < 1e-3
