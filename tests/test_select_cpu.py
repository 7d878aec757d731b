"""Routing by scores on the host: the plain form against hand-made rows, and every refusal before anything is enqueued."""
import math
import subprocess

import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from sparse_moe_layer_gemm_amd import build as pkg_build
from tests import select_ref as ref

OK, INVAL, UNSUP = 0, 1, 2
GB = 1 << 30
A, B, C, D, F = (i * (GB << 8) for i in range(1, 6))
MIS, NAN, INF = A + 4, float("nan"), float("inf")
SEL = dict(l=A, dt=0, T=64, E=32, k=4, score=1, bias=None, groups=1, gk=1, gt=1, renorm=1, scale=1.0, ids=B, w=C,
           scores=None, st=None)
BWD = dict(l=A, dt=1, T=64, E=32, k=4, score=0, renorm=1, scale=1.0, ids=B, dw=C, ds=None, ddt=0, dl=D, st=None)


def call(fn, defaults, **kw):
    assert not set(kw) - set(defaults)
    return getattr(moe.load_library(), fn)(*{**defaults, **kw}.values())


def test_select_refusals():
    f = lambda **kw: call("moe_select", SEL, **kw)  # noqa: E731
    assert f(T=0, l=None, ids=None, w=None) == OK
    for bad in (dict(l=None), dict(ids=None), dict(w=None), dict(l=MIS), dict(ids=MIS), dict(w=MIS), dict(bias=MIS),
                dict(scores=MIS), dict(dt=2), dict(score=2), dict(score=-1), dict(renorm=2), dict(scale=NAN),
                dict(scale=INF), dict(T=-1), dict(E=0), dict(k=0), dict(E=3), dict(groups=0), dict(groups=5),
                dict(groups=-4), dict(groups=4, gk=5), dict(groups=4, gk=0), dict(gt=0), dict(gt=3),
                dict(groups=16, gk=1), dict(groups=64, E=128, gk=1), dict(ids=A), dict(w=A), dict(w=B), dict(scores=A),
                dict(scores=B), dict(scores=C), dict(bias=F, ids=F), dict(bias=F, w=F), dict(bias=F, scores=F)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(E=257), dict(k=9), dict(T=1 << 24), dict(E=256, groups=128, gk=128)):
        assert f(**bad) == UNSUP, bad


def test_select_backward_refusals():
    f = lambda **kw: call("moe_select_backward", BWD, **kw)  # noqa: E731
    assert f(T=0, l=None, ids=None, dw=None, dl=None) == OK
    for bad in (dict(l=None), dict(ids=None), dict(dw=None), dict(dl=None), dict(l=MIS), dict(ids=MIS), dict(dw=MIS),
                dict(dl=MIS), dict(ds=MIS), dict(dt=3), dict(ddt=2), dict(score=5), dict(renorm=-1), dict(scale=NAN),
                dict(T=-2), dict(E=0), dict(k=0), dict(k=5, E=4), dict(dl=A), dict(dl=B), dict(dl=C), dict(ds=D)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(E=300), dict(k=9), dict(T=1 << 24)):
        assert f(**bad) == UNSUP, bad


def test_binding_refusals():
    l, ids, w = torch.zeros(6, 16), torch.zeros(6, 4, dtype=torch.int32), torch.zeros(6, 4)
    bad = [
        lambda: moe.moe_select(l, ids, w),  # host tensors
        lambda: moe.moe_select(l[0], ids, w),
        lambda: moe.moe_select(l, ids[:5], w[:5]),
        lambda: moe.moe_select(l, ids.long(), w),
        lambda: moe.moe_select(l, ids, w[:, :3]),
        lambda: moe.moe_select(l, ids, w.bfloat16()),
        lambda: moe.moe_select(l, ids, w, score="tanh"),
        lambda: moe.moe_select(l, ids, w, bias=torch.zeros(15)),
        lambda: moe.moe_select(l, ids, w, bias=torch.zeros(16, dtype=torch.bfloat16)),
        lambda: moe.moe_select(l, ids, w, scores=torch.zeros(6, 15)),
        lambda: moe.moe_select(l, ids, w, groups=1 << 32),
        lambda: moe.moe_select_backward(l, ids, w, l[:, :8]),
        lambda: moe.moe_select_backward(l, ids, w.double(), l),
        lambda: moe.moe_select_backward(l, ids, w, l, dscores=l.bfloat16()),
        lambda: moe.moe_select_backward(l, ids, w, l, score=None),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(TypeError):
        moe.moe_select(l.half(), ids, w)


def test_plain_form():
    """By hand: ties, experts left out, groups by one and two choices, weights."""
    l = torch.tensor([[0.0, 1.0, 1.0, -1.0], [-INF, NAN, 2.0, -INF], [-INF] * 4, [INF, 0.0, INF, 1.0]])
    ids, w, s = ref.select(l, 2)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [0, 2]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [0.5, 0.5]]
    assert s[3].tolist() == [0.5, 0.0, 0.5, 0.0] and s[2].tolist() == [0.0] * 4
    ids, w, _ = ref.select(l[:1], 2, "sigmoid", renorm=False, scale=2.0)
    assert w[0].tolist() == [2 / (1 + math.exp(-1.0))] * 2
    b = torch.tensor([0.0, -INF, 0.0, 10.0])
    assert ref.select(l[:1], 3, "sigmoid", bias=b)[0].tolist() == [[3, 2, 0]]
    # groups (0, 1) and (2, 3): the largest is in the second, the larger pair in the first
    v = torch.tensor([[2.0, 2.0, 2.1, -9.0]])
    assert ref.select(v, 2, "sigmoid", groups=2, group_top=1)[0].tolist() == [[2, 3]]
    assert ref.select(v, 2, "sigmoid", groups=2, group_top=2)[0].tolist() == [[0, 1]]
    assert ref.select(torch.zeros(1, 4), 1, groups=2)[0].tolist() == [[0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_plain_gradient_is_that_of_the_plain_form(score, renorm):
    """Against differences of the weights and scores in fp64."""
    g = torch.Generator().manual_seed(5)
    l = torch.randn(3, 9, generator=g, dtype=torch.float64)
    l[1, 4] = -INF
    dw, ds = torch.randn(3, 4, generator=g, dtype=torch.float64), torch.randn(3, 9, generator=g, dtype=torch.float64)
    ids = ref.select(l, 4, score, renorm=renorm, scale=1.5)[0]
    got, _ = ref.backward(l, ids, dw, score, renorm, 1.5, ds)

    def loss(x):
        _, _, s = ref.select(x, 4, score)
        total = (s * ds).sum()
        for t in range(3):
            own = s[t][ids[t].long()]
            total = total + 1.5 * (dw[t] * (own / own.sum() if renorm else own)).sum()
        return total.item()

    h = 2.0 ** -18  # error h^2 / 6 of a third derivative of order one, and 1e-15 / h
    for t in range(3):
        for e in range(9):
            if l[t, e] == -INF:
                assert got[t, e] == 0
                continue
            a, b = l.clone(), l.clone()
            a[t, e] += h
            b[t, e] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - got[t, e].item()) < 1e-8


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_gradient_by_pairs_is_the_formula(score, renorm):
    """The sums over pairs of experts against the formula, in 64 bits, and what they keep where the formula loses it."""
    g = torch.Generator().manual_seed(8)
    l, ds = torch.randn(5, 9, generator=g), torch.randn(5, 9, generator=g)
    dw, ids = torch.randn(5, 4, generator=g), torch.rand(5, 9, generator=g).argsort(1)[:, :4].to(torch.int32)
    for d in (None, ds):
        a, b = (f(l, ids, dw, score, renorm, 1.5, d)[0] for f in (ref.backward, ref.backward_sure))
        assert (a - b).abs().max() < 1e-13
    # two experts 50 apart, the surer one chosen: s (1 - s) d, 1 - s = 1 / (1 + e^50)
    l = torch.tensor([[50.0, 0.0]])
    got, bound = ref.backward_sure(l, torch.tensor([[0]]), torch.tensor([[3.0]]), "softmax", False, 1.0)
    want = 3 / (1 + math.exp(50.0)) * (1 / (1 + math.exp(-50.0)))
    assert abs(got[0, 0].item() / want - 1) < 1e-14 and abs(got[0, 1].item() / want + 1) < 1e-14
    assert (bound < 2e-5 * want).all()


def test_keys_convert_nothing_out_of_range(tmp_path):
    """The 32-bit keys' conversion to whole numbers, built with a check of its range: experts that are left out, rows of
    them, infinite choices (whose distance to the largest is NaN), choices far below the largest."""
    src, exe = tmp_path / "keys.cpp", tmp_path / "keys"
    src.write_text("""
#include <math.h>
#include <stdio.h>
#include "select_keys.h"
int main() {
  const float inf = INFINITY, rows[][2] = {{-inf, 0.f}, {-inf, -inf}, {-inf, inf}, {inf, inf}, {0.f, inf}, {-3e38f, 3e38f},
                                           {-40.f, 0.f}, {1.f, 1.f}, {0.75f, 1.f}, {-1e-40f, 0.f}};
  for (const auto& r : rows) {
    volatile float c = r[0], high = r[1];
    printf("%u ", moe::choice_key(c, fmaf(c - high, 0x1p19f, 0x1p24f - 1.f), 5));
  }
}
""")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-I", pkg_build.CSRC, "-fsanitize=float-cast-overflow",
                        "-fno-sanitize-recover=all", str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-500:]
    most = (1 << 24) - 1
    want = [0, 0, 0, 1, 1, 1, 1, most, most - (1 << 17), most]
    assert [int(x) for x in r.stdout.split()] == [x << 8 | 250 for x in want]


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_check_of_the_gradients_finds_mistakes(score, renorm):
    """What the layer's test asks of a training pass, asked of right results and of each planted mistake."""
    g = torch.Generator().manual_seed(3)
    T, k, E, H = 12, 3, 8, 32
    l, ds = torch.randn(T, E, generator=g), torch.randn(T, E, generator=g)
    ids = ref.select(l, k, score)[0]
    y, dout = torch.randn(T * k, H, generator=g), torch.randn(T, H, generator=g).bfloat16()
    pos = torch.randperm(T * k, generator=g).view(T, k)
    ids[2, 1], pos[2, 1] = -1, -1
    rows = torch.where(pos[..., None] >= 0, y[pos.clamp(min=0)], 0.0)
    dw = (rows.double() * dout.double()[:, None]).sum(2).float()
    back = lambda d, r=renorm, sc=2.5: ref.backward(l, ids, d, score, r, sc, ds)[0].float()  # noqa: E731
    def holds(dw, dl):
        a, b, share = ref.gradient_chain(y, dout, pos, dw, l, ids, dl, ds, score, renorm, 2.5)
        return a <= 1 and b <= 1 and share < 1e-3

    assert holds(dw, back(dw))
    wrong = [(dw, torch.zeros(T, E)), (dw, back(0 * dw)), (dw, back(dw.roll(1, 1))), (dw.roll(1, 1), back(dw.roll(1, 1))),
             (dw.roll(1, 0), back(dw.roll(1, 0))), (dw, back(dw, sc=1.0)), (dw, back(dw, r=not renorm)), (dw, back(dw).roll(1, 1)),
             (0 * dw, back(0 * dw)), (dw, back(dw * (1 + 2.0 ** -9)))]
    for i, w in enumerate(wrong):
        assert not holds(*w), i
