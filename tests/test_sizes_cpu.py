"""Sizes that an int32 parameter of the C ABI cannot hold: ctypes would pass them on modulo 2^32, past the
library's own checks, so the bindings refuse them (meta tensors: shapes without memory)."""
import pytest
import torch

import sparse_moe_layer_gemm_amd as moe

BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
WRAP = 1 << 32  # + a valid size: that size, modulo 2^32


def t(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="meta")


def off(E):
    return t(E + 1, dtype=I32)


def gemm(K=64, N=64, E=2, trans=False, **kw):
    moe.moe_grouped_gemm(t(4, K), t(E, N, K) if trans else t(E, K, N), off(E), t(4, N), w_trans=trans, **kw)


def wgrad(K=64, N=64, E=2, **kw):
    moe.moe_grouped_wgrad(t(4, K), t(4, N), off(E), t(E, K, N), **kw)


def mx(K=64, N=64, E=2, **kw):
    S = (K // 32 + 3) // 4 * 4
    moe.moe_mxfp4_grouped_gemm(t(4, K // 2, dtype=U8), t(4, S, dtype=U8), t(E, N, K // 2, dtype=U8),
                               t(E, N, S, dtype=U8), off(E), t(4, N), **kw)


def fin(k=2, H=64):
    moe.moe_finalize_backward(t(1, H), t(k, H, dtype=F32), t(k, dtype=I32), t(1, k, dtype=F32), t(k, H),
                              t(1, k, dtype=F32))


def quant(R, C, trans):
    K, rows = (R, C) if trans else (C, R)
    moe.moe_mxfp4_quantize(t(R, C), t(rows, K // 2, dtype=U8), t(rows, (K // 32 + 3) // 4 * 4, dtype=U8), trans=trans)


def dequant(K):
    moe.moe_mxfp4_dequantize(t(1, K // 2, dtype=U8), t(1, (K // 32 + 3) // 4 * 4, dtype=U8), t(1, K))


def index(n=4):
    return t(n, dtype=I32)


WIDE = [
    lambda n: gemm(K=n + 64), lambda n: gemm(N=n + 64), lambda n: gemm(E=n + 2), lambda n: gemm(N=n + 64, trans=True),
    lambda n: gemm(row_index=index(), row_div=n + 2),
    lambda n: wgrad(K=n + 64), lambda n: wgrad(N=n + 64), lambda n: wgrad(E=n + 2),
    lambda n: wgrad(row_index=index(), row_div=n + 2),
    lambda n: moe.moe_swiglu(t(1, 2 * (n + 8)), t(1, n + 8)),
    lambda n: moe.moe_swiglu_backward(t(1, 2 * (n + 8)), t(1, n + 8), t(1, 2 * (n + 8))),
    lambda n: fin(k=n + 2), lambda n: fin(H=n + 64),
    lambda n: quant(1, n + 64, False), lambda n: quant(64, n + 64, True),
    lambda n: dequant(n + 64),
    lambda n: moe.moe_mxfp4_scale_stride(n + 64),
    lambda n: mx(K=n + 64), lambda n: mx(N=n + 64), lambda n: mx(E=n + 2), lambda n: mx(row_index=index(), row_div=n + 2),
]


@pytest.mark.parametrize("n", [1 << 31, WRAP])
@pytest.mark.parametrize("call", range(len(WIDE)))
def test_operators_refuse_sizes_past_31_bits(call, n):
    with pytest.raises(ValueError, match="below 2\\^31"):
        WIDE[call](n)


def test_ordinary_sizes_pass_the_size_checks():
    for f in (gemm, wgrad, mx, fin, lambda: quant(4, 64, False), lambda: quant(64, 8, True), lambda: dequant(64)):
        with pytest.raises(ValueError, match="device tensors"):  # the next check: meta tensors have no memory
            f()
    with pytest.raises(ValueError, match="row_div must be positive"):
        gemm(row_index=index(), row_div=-WRAP + 2)
    with pytest.raises(ValueError, match="below 2\\^31"):
        moe.moe_mxfp4_scale_stride(-WRAP + 64)
    assert moe.moe_mxfp4_scale_stride((1 << 31) - 32) == 1 << 26
    assert [moe.moe_mxfp4_scale_stride(K) for K in (0, -32, 33)] == [0, 0, 0]


# ---- the layer's own steps (stream 0: nothing is enqueued)
def experts(H=64, I=64, E=2, k=2, rows16=False):
    w = moe.ExpertWeights(moe.MOE_BF16, t(2, 64, 128), t(2, 64, 64))
    a = (t(1, H), I, E, k, off(2), t(2, dtype=I32), w)
    ws = t(1, dtype=U8)
    if rows16:
        moe.moe_experts_rows16(*a, t(2, 64, dtype=torch.int16), t(2, 1, dtype=U8), ws, stream=0)
    else:
        moe.moe_experts(*a, t(2, 64, dtype=F32), ws, stream=0)


def forward(fn, H=64, E=2, I=64, k=2):
    w = moe.ExpertWeights(moe.MOE_BF16, t(2, 64, 128), t(2, 64, 64))
    a = (t(1, H), t(1, E, dtype=F32), None, w, I, k)
    ws = t(1, dtype=U8)
    if fn == "norm":
        moe.moe_forward_norm(*a, t(1, 64), t(64), t(64), 1e-6, t(1, 64), t(1, 64), ws, stream=0)
    elif fn == "noalloc":
        moe.moe_forward_noalloc(*a, t(1, 64), stream=0)
    else:
        moe.moe_forward(*a, t(1, 64), ws, stream=0)


def finalize(fn, k=2, H=64):
    y, w, o = t(2, H, dtype=F32), t(1, k, dtype=F32), t(1, 64)
    g = (t(1, 64), t(64), t(64), 1e-6, t(1, 64), t(1, 64))
    pp, sc = t(2, dtype=I32), t(2, 1, dtype=U8)
    {"plain": lambda: moe.moe_finalize(y, pp, w, o, stream=0),
     "rows16": lambda: moe.moe_finalize_rows16(y, sc, pp, w, o, stream=0),
     "norm": lambda: moe.moe_finalize_norm(y, pp, w, *g, stream=0),
     "norm rows16": lambda: moe.moe_finalize_norm_rows16(y, sc, pp, w, *g, stream=0)}[fn]()


def route(H=64, E=8, k=2):
    moe.moe_route(t(1, H), t(1, E, dtype=F32), None, k, moe.MOE_BF16, None, None, t(1, 2, dtype=I32),
                  t(1, 2, dtype=F32), None, stream=0)


def permute(k=2, E=8):
    moe.moe_permute(t(1, k, dtype=I32), E, t(8, dtype=I32), off(8), t(2, dtype=I32), t(2, dtype=I32), t(1, dtype=U8),
                    stream=0)


def weights():
    return moe.ExpertWeights(moe.MOE_BF16, t(2, 64, 128), t(2, 64, 64))


LAYER = [
    lambda n: route(H=n + 64), lambda n: route(E=n + 8), lambda n: route(k=n + 2), lambda n: route(k=2 - n - 2),
    lambda n: permute(k=n + 2), lambda n: permute(E=n + 8),
    *[lambda n, a=a, r=r: experts(**{a: n + 64 if a in "HI" else n + 2}, rows16=r) for a in "HIEk" for r in (False, True)],
    *[lambda n, a=a, f=f: finalize(f, **{a: n + 64 if a == "H" else n + 2}) for a in "kH"
      for f in ("plain", "rows16", "norm", "norm rows16")],
    *[lambda n, a=a, f=f: forward(f, **{a: n + 64 if a in "HI" else n + 2}) for a in "HIEk"
      for f in ("plain", "norm", "noalloc")],
    lambda n: moe.moe_route_workspace_size(1, n + 64, 8), lambda n: moe.moe_route_workspace_size(1, 64, n + 8),
    lambda n: moe.moe_permute_workspace_size(1, n + 2, 8), lambda n: moe.moe_permute_workspace_size(1, 2, n + 8),
    lambda n: moe.moe_experts_workspace_size(1, n + 64, 64, 8, 2, weights()),
    lambda n: moe.moe_experts_workspace_size(1, 64, n + 64, 8, 2, weights()),
    lambda n: moe.moe_forward_workspace_size(1, 64, 64, n + 8, 2, weights()),
    lambda n: moe.moe_forward_workspace_size(1, 64, 64, 8, n + 2, weights()),
]


@pytest.mark.parametrize("call", range(len(LAYER)))
def test_layer_refuses_sizes_past_31_bits(call):
    with pytest.raises(ValueError, match="below 2\\^31"):
        LAYER[call](WRAP)


def test_ordinary_layer_sizes_reach_the_library():
    """Addresses of meta tensors are null: the library's own check is the next one."""
    for f in (route, permute, experts, lambda: experts(rows16=True), lambda: finalize("plain"), lambda: finalize("rows16"),
              lambda: finalize("norm"), lambda: finalize("norm rows16"), lambda: forward("plain"),
              lambda: forward("norm"), lambda: forward("noalloc")):
        with pytest.raises(moe.MoEError):
            f()
    assert moe.moe_route_workspace_size(64, 5120, 256) == moe.load_library().moe_route_workspace_size(64, 5120, 256)
