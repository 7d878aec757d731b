"""4-bit integer weights on the host: the plain form by hand, and every refusal before anything is enqueued."""
import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import w4_ref as ref

OK, INVAL, UNSUP = 0, 1, 2
GB = 1 << 30
A, B, C, D, F, G = (i * (GB << 8) for i in range(1, 7))
MIS = A + 4
Q = dict(x=A, dt=1, tr=0, B=1, R=64, C=256, g=64, codes=B, sdt=1, s=C, z=D, st=None)
DQ = dict(codes=A, sdt=1, s=B, z=None, R=4, K=256, g=128, dt=1, out=C, st=None)
P = dict(a=A, a_rows=64, idx=None, div=1, w=B, sdt=1, s=C, z=None, g=128, M=64, K=256, N=64, E=4, off=D, odt=1, out=F,
         st=None)


def call(fn, defaults, **kw):
    assert not set(kw) - set(defaults)
    return getattr(moe.load_library(), fn)(*{**defaults, **kw}.values())


def test_quantise_refusals():
    f = lambda **kw: call("moe_w4_quantize", Q, **kw)  # noqa: E731
    assert f(R=0, x=None, codes=None, s=None) == OK and f(B=0, x=None) == OK
    for bad in (dict(x=None), dict(codes=None), dict(s=None), dict(x=MIS), dict(codes=MIS), dict(s=MIS), dict(z=MIS),
                dict(dt=2), dict(sdt=2), dict(tr=2), dict(B=-1), dict(R=-1), dict(C=0), dict(codes=A), dict(s=A),
                dict(z=A), dict(s=B), dict(z=B), dict(z=C)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(g=16), dict(g=0), dict(g=-64), dict(g=256), dict(C=96), dict(tr=1, R=96), dict(tr=1, C=12),
                dict(R=1 << 31), dict(B=1 << 31), dict(R=(1 << 31) - 1, C=1 << 20)):
        assert f(**bad) == UNSUP, bad


@pytest.mark.parametrize("trans,Bn,R,C,want", [
    (0, 1, (1 << 24) - 1, 2048, INVAL), (0, 1, 1 << 24, 2048, UNSUP), (0, 1, 1, 1 << 30, INVAL),
    (0, 1, 1, (1 << 30) + 128, UNSUP), (1, (1 << 23) - 1, 128, 8, INVAL), (1, 1 << 23, 128, 8, UNSUP),
    (1, 1, 1 << 30, 8, INVAL), (1, 1, (1 << 30) + 128, 8, UNSUP)])
def test_quantise_limits(trans, Bn, R, C, want):
    assert moe.load_library().moe_w4_quantize(None, 1, trans, Bn, R, C, 128, A, 1, B, None, None) == want


def test_dequantise_refusals():
    f = lambda **kw: call("moe_w4_dequantize", DQ, **kw)  # noqa: E731
    assert f(R=0, codes=None, s=None, out=None) == OK
    for bad in (dict(codes=None), dict(s=None), dict(out=None), dict(codes=MIS), dict(s=MIS), dict(out=MIS), dict(z=MIS),
                dict(R=-1), dict(K=0), dict(dt=3), dict(sdt=-1), dict(out=A), dict(out=B), dict(z=D, out=D)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(K=192), dict(g=48), dict(R=1 << 24, K=2048), dict(R=1 << 40, K=1 << 20)):
        assert f(**bad) == UNSUP, bad
    assert f(R=(1 << 24) - 1, K=2048, out=None) == INVAL


def test_product_refusals():
    f = lambda **kw: call("moe_w4_grouped_gemm", P, **kw)  # noqa: E731
    assert f(M=0, a=None, w=None, s=None, off=None, out=None) == OK
    for bad in (dict(a=None), dict(w=None), dict(s=None), dict(off=None), dict(out=None), dict(a=MIS), dict(w=MIS),
                dict(s=MIS), dict(z=MIS), dict(out=MIS), dict(off=MIS), dict(idx=MIS), dict(M=-1), dict(K=0), dict(N=0),
                dict(E=0), dict(sdt=2), dict(odt=3), dict(a_rows=63), dict(a_rows=0, idx=G), dict(idx=G, div=0),
                dict(out=A), dict(out=B), dict(out=C), dict(out=D), dict(z=G, out=G), dict(idx=G + 64, out=G)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(E=257), dict(K=192), dict(g=96), dict(N=60), dict(M=1 << 29, a_rows=1 << 29), dict(a_rows=1 << 31),
                dict(K=(1 << 20) + 128), dict(N=(1 << 20) + 8), dict(M=1 << 26, a_rows=1 << 26, N=512)):
        assert f(**bad) == UNSUP, bad


def test_binding_refusals():
    bf, u8 = torch.bfloat16, torch.uint8
    x, c, s = torch.zeros(6, 128, dtype=bf), torch.zeros(6, 64, dtype=u8), torch.zeros(6, 2, dtype=bf)
    w, ws, out = torch.zeros(2, 8, 64, dtype=u8), torch.zeros(2, 8, 2, dtype=bf), torch.zeros(6, 8, dtype=bf)
    off = torch.tensor([0, 2, 6], dtype=torch.int32)
    bad = [
        lambda: moe.moe_w4_quantize(x, c, s),  # host tensors
        lambda: moe.moe_w4_quantize(x, c[:, :32], s),
        lambda: moe.moe_w4_quantize(x, c.int(), s),
        lambda: moe.moe_w4_quantize(x, c, s[:5]),
        lambda: moe.moe_w4_quantize(x, c, torch.zeros(6, 3, dtype=bf)),
        lambda: moe.moe_w4_quantize(x, c, s[:, :0]),
        lambda: moe.moe_w4_quantize(x, c, s, zeros=torch.zeros(6, 2)),
        lambda: moe.moe_w4_quantize(x, c, s, zeros=torch.zeros(6, 4, dtype=u8)),
        lambda: moe.moe_w4_quantize(x, c, s, trans=True),
        lambda: moe.moe_w4_quantize(x[0], c[0], s[0]),
        lambda: moe.moe_w4_dequantize(c, s, x[:, :64]),
        lambda: moe.moe_w4_dequantize(c, s, x),
        lambda: moe.moe_w4_grouped_gemm(x, w, ws, off, out),
        lambda: moe.moe_w4_grouped_gemm(x.float(), w, ws, off, out),
        lambda: moe.moe_w4_grouped_gemm(x[:, :64], w, ws, off, out),
        lambda: moe.moe_w4_grouped_gemm(x, w, ws[:, :4], off, out),
        lambda: moe.moe_w4_grouped_gemm(x, w, ws, off[:2], out),
        lambda: moe.moe_w4_grouped_gemm(x, w, ws, off, out[:, :4]),
        lambda: moe.moe_w4_grouped_gemm(x, w, ws, off, out, zeros=torch.zeros(2, 8, 1, dtype=u8)),
        lambda: moe.moe_w4_grouped_gemm(x, w, ws, off, out, row_index=torch.zeros(5, dtype=torch.int32)),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: moe.moe_w4_quantize(x.half(), c, s), lambda: moe.moe_w4_quantize(x, c, s.half()),
              lambda: moe.moe_w4_dequantize(c, s, x.half()), lambda: moe.moe_w4_grouped_gemm(x, w, ws, off, out.half())):
        with pytest.raises(TypeError):
            f()


def test_plain_form():
    """By hand: ties to even, clamping, zeros, values that are no numbers, zero points."""
    # 7 * (1/7) and 15 * (1/15) are 1 in fp32
    x = torch.zeros(5, 32)
    x[0, :6] = torch.tensor([7.0, -7.0, 0.5, 1.5, -2.5, 3.4])
    x[2, 3], x[3, 4] = float("inf"), float("nan")
    x[4, :3] = torch.tensor([1e-45, -1e-45, 0.0])
    q, s, _ = ref.quantise(x, 32, False, torch.float32)
    assert s[0, 0] == 1 and q[0, :6].tolist() == [15, 1, 8, 10, 6, 11]
    assert s[1, 0] == 0 and q[1:].unique().tolist() == [8] and s[2:4].isnan().all() and s[4, 0] == 0
    x[0, :4] = torch.tensor([10.0, -5.0, 0.5, 2.5])
    q, s, z = ref.quantise(x[:2], 32, True, torch.float32)
    assert s[0, 0] == 1 and z.tolist() == [[5], [0]] and q[0, :5].tolist() == [15, 0, 5, 7, 3]
    assert ref.weights64(ref.pack(q), s, z)[0, :5].tolist() == [10.0, -5.0, 0.0, 2.0, -2.0]
    assert ref.unpack(ref.pack(q)).equal(q)
