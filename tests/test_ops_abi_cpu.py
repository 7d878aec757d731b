"""Refusals of the operators around the layer, on the host: every invalid or
unsupported call returns before anything is enqueued (fake aligned addresses)."""
import ctypes

import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref as ref

OK, INVAL, UNSUP = 0, 1, 2
GB = 1 << 30
A, B, C, D, F, G = (i * (GB << 8) for i in range(1, 7))
MIS = A + 4


def call(fn, defaults, **kw):
    a = dict(defaults)
    assert not set(kw) - set(a)
    a.update(kw)
    return getattr(moe.load_library(), fn)(*a.values())


GEMM = dict(a=A, dt=1, a_rows=64, idx=None, div=1, w=B, tr=0, M=64, K=128, N=64, E=4, off=C, odt=1, out=D,
            st=None)
WGRAD = dict(a=A, dt=1, a_rows=64, idx=None, div=1, d=B, M=64, K=128, N=64, E=4, off=C, odt=0, acc=0, dw=D,
             st=None)
MX = dict(a=A, asc=B, a_rows=64, idx=None, div=1, w=C, wsc=D, M=64, K=128, N=64, E=4, off=F, odt=1, out=G,
          st=None)


def test_grouped_gemm_refusals():
    f = lambda **kw: call("moe_grouped_gemm", GEMM, **kw)  # noqa: E731
    assert f(M=0, a=None, w=None, off=None, out=None) == OK
    for bad in (dict(a=None), dict(w=None), dict(off=None), dict(out=None), dict(a=MIS), dict(w=MIS),
                dict(out=MIS), dict(off=MIS), dict(idx=MIS), dict(M=-1), dict(K=0), dict(N=0), dict(E=0),
                dict(dt=2), dict(odt=3), dict(tr=2), dict(a_rows=63), dict(a_rows=0, idx=F), dict(idx=F, div=0),
                dict(out=A), dict(out=A + 64 * 128 * 2 - 16), dict(out=B), dict(out=C), dict(out=F, idx=F + 64)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(E=257), dict(K=100), dict(N=60), dict(M=1 << 29, a_rows=1 << 29), dict(a_rows=1 << 31),
                dict(K=(1 << 20) + 8), dict(N=(1 << 20) + 8), dict(M=1 << 26, a_rows=1 << 26, N=512)):
        assert f(**bad) == UNSUP, bad


def test_grouped_wgrad_refusals():
    f = lambda **kw: call("moe_grouped_wgrad", WGRAD, **kw)  # noqa: E731
    for bad in (dict(a=None), dict(d=None), dict(off=None), dict(dw=None), dict(M=0, dw=None), dict(M=0, off=None),
                dict(acc=2), dict(dw=MIS), dict(d=MIS), dict(a_rows=63), dict(idx=F, div=-1), dict(dw=A),
                dict(dw=B), dict(dw=C - 16), dict(dt=7), dict(odt=2)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(acc=1, odt=1), dict(E=300), dict(K=4), dict(N=12), dict(M=1 << 30, a_rows=1 << 30)):
        assert f(**bad) == UNSUP, bad


def test_swiglu_refusals():
    f = lambda **kw: call("moe_swiglu", dict(a=A, dt=1, M=8, I=64, h=B, st=None), **kw)  # noqa: E731
    assert f(M=0, a=None, h=None) == OK
    for bad in (dict(a=None), dict(h=None), dict(a=MIS), dict(h=MIS), dict(M=-1), dict(I=0), dict(dt=2), dict(h=A)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(I=12), dict(M=1 << 31), dict(M=(1 << 31) - 1, I=1 << 20)):
        assert f(**bad) == UNSUP, bad
    g = lambda **kw: call("moe_swiglu_backward",  # noqa: E731
                          dict(a=A, dh=B, dt=1, M=8, I=64, da=C, h=D, st=None), **kw)
    assert g(M=0, a=None, dh=None, da=None, h=None) == OK
    for bad in (dict(a=None), dict(dh=None), dict(da=None), dict(h=MIS), dict(da=B), dict(da=A + 16), dict(h=A),
                dict(h=C), dict(h=B + 16), dict(da=D)):
        assert g(**bad) == INVAL, bad


def test_finalize_backward_refusals():
    f = lambda **kw: call("moe_finalize_backward",  # noqa: E731
                          dict(dout=A, dt=1, y=B, pp=C, w=D, T=4, k=2, H=128, ydt=1, dy=F, dw=G, st=None), **kw)
    assert f(T=0, dout=None, y=None, pp=None, w=None, dy=None, dw=None) == OK
    for bad in (dict(dout=None), dict(pp=None), dict(w=None), dict(y=None), dict(dy=None, dw=None), dict(dy=MIS),
                dict(dw=MIS), dict(y=MIS), dict(dt=2), dict(ydt=2), dict(T=-1), dict(k=0), dict(H=0), dict(dy=A),
                dict(dy=B), dict(dw=D), dict(dw=F)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(k=9), dict(H=96), dict(T=1 << 24)):
        assert f(**bad) == UNSUP, bad


def test_finalize_backward_widest_row():
    # a lane's column index runs 8192 past H: 2^31 - 64 would wrap
    args = dict(dout=A, dt=1, y=B, pp=C, w=D, T=1, k=1, H=(1 << 30) + 64, ydt=1, dy=F, dw=G, st=None)
    assert call("moe_finalize_backward", args) == UNSUP
    assert call("moe_finalize_backward", dict(args, H=(1 << 31) - 64)) == UNSUP


def test_mxfp4_refusals():
    lib = moe.load_library()
    assert [lib.moe_mxfp4_scale_stride(K) for K in (32, 128, 160, 5120, 48, 0, -32)] == [4, 4, 8, 160, 0, 0, 0]
    f = lambda **kw: call("moe_mxfp4_quantize",  # noqa: E731
                          dict(x=A, dt=1, tr=0, B=1, R=64, C=64, codes=B, sc=C, st=None), **kw)
    assert f(R=0, x=None, codes=None, sc=None) == OK
    for bad in (dict(x=None), dict(codes=None), dict(sc=None), dict(x=MIS), dict(codes=MIS), dict(sc=MIS), dict(dt=2),
                dict(tr=2), dict(B=-1), dict(R=-1), dict(C=0), dict(codes=A), dict(sc=A), dict(sc=B)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(C=48), dict(tr=1, R=48), dict(tr=1, C=12), dict(R=1 << 31), dict(R=(1 << 31) - 1, C=1 << 20)):
        assert f(**bad) == UNSUP, bad
    g = lambda **kw: call("moe_mxfp4_dequantize",  # noqa: E731
                          dict(codes=A, sc=B, R=4, K=64, dt=1, out=C, st=None), **kw)
    assert g(R=0, codes=None, sc=None, out=None) == OK
    for bad in (dict(codes=None), dict(sc=None), dict(out=None), dict(R=-1), dict(K=0), dict(dt=3), dict(out=A),
                dict(out=B)):
        assert g(**bad) == INVAL, bad
    assert g(K=40) == UNSUP and g(R=1 << 40, K=1 << 20) == UNSUP


def test_mxfp4_grouped_gemm_refusals():
    f = lambda **kw: call("moe_mxfp4_grouped_gemm", MX, **kw)  # noqa: E731
    assert f(M=0, a=None, asc=None, w=None, wsc=None, off=None, out=None) == OK
    for bad in (dict(a=None), dict(asc=None), dict(w=None), dict(wsc=None), dict(off=None), dict(out=None),
                dict(a=MIS), dict(asc=MIS), dict(wsc=MIS), dict(odt=2), dict(a_rows=63), dict(idx=C, div=0),
                dict(out=A), dict(out=B), dict(out=C), dict(out=D), dict(out=F)):
        assert f(**bad) == INVAL, bad
    for bad in (dict(K=48), dict(N=4), dict(E=257), dict(M=1 << 29, a_rows=1 << 29),
                dict(a_rows=1 << 30)):
        assert f(**bad) == UNSUP, bad


def test_binding_refusals():
    bf, f32 = torch.bfloat16, torch.float32
    a, w, out = torch.zeros(6, 16, dtype=bf), torch.zeros(2, 16, 8, dtype=bf), torch.zeros(6, 8, dtype=bf)
    off = torch.tensor([0, 2, 6], dtype=torch.int32)
    bad = [
        lambda: moe.moe_grouped_gemm(a, w, off, out),  # host tensors
        lambda: moe.moe_grouped_gemm(a, w, off, out[:, :4]),
        lambda: moe.moe_grouped_gemm(a, w, off, out, w_trans=True),
        lambda: moe.moe_grouped_gemm(a, w.float(), off, out),
        lambda: moe.moe_grouped_gemm(a, w, off[:2], out),
        lambda: moe.moe_grouped_gemm(a, w, off.long(), out),
        lambda: moe.moe_grouped_gemm(a, w, off, out, row_index=torch.zeros(5, dtype=torch.int32)),
        lambda: moe.moe_grouped_gemm(a, w, off, out, row_index=torch.zeros(6, dtype=torch.int32), row_div=0),
        lambda: moe.moe_grouped_wgrad(a, out, off, w[:, :8]),
        lambda: moe.moe_grouped_wgrad(a, out.float(), off, w),
        lambda: moe.moe_swiglu(a, a),
        lambda: moe.moe_swiglu(a, torch.zeros(6, 8, dtype=f32)),
        lambda: moe.moe_swiglu_backward(a, out, out),
        lambda: moe.moe_finalize_backward(a, None, off, torch.zeros(6, 1), None, torch.zeros(6, 1)),
        lambda: moe.moe_finalize_backward(a, torch.zeros(6, 16), torch.zeros(6, dtype=torch.int32), torch.zeros(6, 1),
                                          torch.zeros(5, 16), None),
        lambda: moe.moe_mxfp4_quantize(torch.zeros(2, 48, dtype=bf), torch.zeros(2, 24, dtype=torch.uint8),
                                       torch.zeros(2, 4, dtype=torch.uint8)),
        lambda: moe.moe_mxfp4_quantize(torch.zeros(2, 64, dtype=bf), torch.zeros(2, 32, dtype=torch.uint8),
                                       torch.zeros(2, 2, dtype=torch.uint8)),
        lambda: moe.moe_mxfp4_dequantize(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8),
                                         torch.zeros(2, 32, dtype=bf)),
        lambda: moe.moe_mxfp4_grouped_gemm(torch.zeros(6, 16, dtype=torch.uint8), torch.zeros(6, 4, dtype=torch.uint8),
                                           torch.zeros(2, 8, 16, dtype=torch.uint8),
                                           torch.zeros(2, 8, 1, dtype=torch.uint8), off, out),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
        del f
    with pytest.raises(TypeError):
        moe.moe_swiglu(torch.zeros(2, 16, dtype=torch.float16), torch.zeros(2, 8, dtype=torch.float16))


def test_plain_mxfp4_form():
    """The plain encoder against hand-made blocks: ties to even, saturation, zeros, NaN, subnormals."""
    x = torch.zeros(5, 32)
    x[0, :8] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -5.0])
    x[1, 0] = 7.9
    x[3, 1], x[3, 2] = float("nan"), 3.0
    x[4, 0] = 2.0 ** -127
    code, scale = ref.mx_encode(x)
    assert scale[:, 0].tolist() == [127, 127, 0, 255, 0]
    assert code[0, :8].tolist() == [6, 0, 2, 2, 4, 4, 6, 14]
    assert code[1, 0] == 7 and not code[2].any() and not code[3].any() and code[4, 0] == 2
    v = ref.mx_decode64(ref.mx_pack(code), scale)
    assert v[0, :8].tolist() == [4, 0, 1, 1, 2, 2, 4, -4] and v[1, 0] == 6
    assert v[3].isnan().all() and v[4, 0] == 2.0 ** -127
