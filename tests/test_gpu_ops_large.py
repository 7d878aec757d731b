"""The kernels that large calls of the operators take, against plain 64-bit forms: the finalize gradient from 512
tokens on, elementwise calls above 128 MB (they load and store past the caches), and arrays of more than 2^31 elements."""
import random

import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref as ref
from tests.test_gpu_ops import BF, F32, NAN, awkward, close, gen, normal, quantised

pytestmark = pytest.mark.gpu
STREAMED = 128 << 20  # bytes above which an elementwise call streams


# ------------------------------------------------------------------ SwiGLU
def swiglu64(a, dh):
    """(h, da's two halves, and the magnitudes that their errors scale with), in 64 bits."""
    I = dh.shape[1]
    G, U, D = a[:, :I].double(), a[:, I:].double(), dh.double()
    s = torch.sigmoid(G)
    h, dg, du = G * s * U, D * U * s * (1 + G * (1 - s)), D * G * s
    return G, (h, h.abs()), (dg, (D * U * s).abs() * (1 + G.abs())), (du, du.abs())


def swiglu_close(got, want, G, dtype):
    """As for the small calls: s is off by (|g| + 8) 2^-22 (the exponent's argument, exp2, the sum and the reciprocal),
    1 - s absolutely, times |g|; then one rounding to dtype. Values below 2^-120 may be flushed."""
    v, mag = want
    rel = (G.abs() + 8) * 2.0 ** -22 * mag
    close(got, v, rel + ref.HALF[dtype] * (v.abs() + rel) + 2.0 ** -120)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,I", [(15991, 1416), (2796229, 8)])
def test_swiglu_streamed(M, I, dtype):
    g = gen(M)
    size = 2 if dtype == BF else 4
    assert 3 * M * I * size > STREAMED
    a, dh = normal(g, M, 2 * I, dtype=dtype, scale=3.0), normal(g, M, I, dtype=dtype)
    h, hbig = ref.guarded(torch.zeros_like(dh), 16, 7.0)
    h2, h2big = ref.guarded(torch.zeros_like(dh), 16, 7.0)
    da, dbig = ref.guarded(torch.zeros_like(a), 16, 7.0)
    moe.moe_swiglu(a, h)
    moe.moe_swiglu_backward(a, dh, da, h=h2)
    assert torch.equal(h, h2)
    assert all(ref.guards_intact(b, 16, 7.0) for b in (hbig, h2big, dbig))
    G, hw, gw, uw = swiglu64(a, dh)
    swiglu_close(h, hw, G, dtype)
    swiglu_close(da[:, :I], gw, G, dtype)
    swiglu_close(da[:, I:], uw, G, dtype)
    a2, dh2, da3 = a.clone(), dh.clone(), torch.empty_like(a)
    moe.moe_swiglu_backward(a2, dh2, a2, h=dh2)  # in place
    moe.moe_swiglu_backward(a, dh, da3)          # without h
    assert torch.equal(a2, da) and torch.equal(dh2, h) and torch.equal(da3, da)


def test_swiglu_past_31_bits():
    M, I = 1000003, 1080  # a has 2.16e9 elements
    g = gen(4)
    a, dh = torch.empty(M, 2 * I, dtype=BF, device="cuda"), torch.empty(M, I, dtype=BF, device="cuda")
    edge = (1 << 31) // (2 * I)
    rows = torch.tensor([0, 1, edge - 1, edge, edge + 1, M - 2, M - 1], device="cuda")
    a.fill_(1.0), dh.fill_(1.0)
    a[rows], dh[rows] = normal(g, len(rows), 2 * I), normal(g, len(rows), I)
    h, da = torch.full_like(dh, NAN), torch.full_like(a, NAN)
    moe.moe_swiglu(a, h)
    moe.moe_swiglu_backward(a, dh, da)
    G, hw, gw, uw = swiglu64(a[rows], dh[rows])
    swiglu_close(h[rows], hw, G, BF)
    swiglu_close(da[rows][:, :I], gw, G, BF)
    swiglu_close(da[rows][:, I:], uw, G, BF)
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[rows] = False
    one = int(rest.nonzero()[0, 0])
    G, hw, gw, uw = swiglu64(a[one:one + 1], dh[one:one + 1])
    for got, want in ((h[one:one + 1], hw), (da[one:one + 1, :I], gw), (da[one:one + 1, I:], uw)):
        swiglu_close(got, want, G, BF)
    assert bool((h[rest] == h[one, 0]).all()) and bool((da[rest] == da[one]).all())


# ------------------------------------------------------------------ finalize gradient
def positions(rng, P, gone):
    pos = list(range(P))
    rng.shuffle(pos)
    for p in range(gone, P, 5) if gone else ():
        pos[p] = rng.choice([-1, -7, P, 2 ** 31 - 1])
    return torch.tensor(pos, dtype=torch.int32, device="cuda")


def finalize_backward64(dout, y, pos, w):
    """dy (7 where no pair points), dw and the sum of |terms| of dw."""
    (T, k), (P, H) = w.shape, y.shape
    token = torch.arange(P, device="cuda") // k
    ok = (pos >= 0) & (pos < P)
    r, t = pos[ok].long(), token[ok]
    dy = torch.full((P, H), 7.0, dtype=torch.float64, device="cuda")
    dy[r] = w.flatten()[ok].double()[:, None] * dout[t].double()
    terms = dout[t].double() * y[r].double()
    dw, mag = (torch.zeros(P, dtype=torch.float64, device="cuda") for _ in range(2))
    dw[ok], mag[ok] = terms.sum(1), terms.abs().sum(1)
    return dy, dw, mag


@pytest.mark.parametrize("dout_dtype,dy_dtype", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,k,H,gone", [(511, 3, 576, 4), (512, 1, 576, 4), (512, 8, 64, 0), (513, 3, 576, 4),
                                        (513, 8, 5120, 4), (700, 2, 8256, 3), (2051, 8, 1408, 4)])
def test_finalize_backward_many_tokens(T, k, H, gone, dout_dtype, dy_dtype):
    """512 tokens and more take all slots in one workgroup; the last size moves more than 128 MB."""
    g, P = gen(T + k), T * k
    pos = positions(random.Random(T), P, gone)
    dout, y, w = normal(g, T, H, dtype=dout_dtype), normal(g, P, H, dtype=F32), torch.rand(T, k, generator=g, device="cuda")
    dy, big = ref.guarded(torch.full((P, H), 7.0, device="cuda", dtype=dy_dtype), 16, 7.0)
    dw, dwbig = ref.guarded(torch.full((T, k), NAN, device="cuda"), 16, 7.0)
    moe.moe_finalize_backward(dout, y, pos, w, dy, dw)
    want_dy, want_dw, mag = finalize_backward64(dout, y, pos, w)
    # one product in fp32 (half a step of fp32), then the rounding to dy_dtype
    close(dy, want_dy, want_dy.abs() * (ref.HALF[dy_dtype] + ref.HALF[F32] * 1.01))
    close(dw.flatten(), want_dw, ref.sum_bound(want_dw, mag, H, F32))
    assert ref.guards_intact(big, 16, 7.0) and ref.guards_intact(dwbig, 16, 7.0)
    only_dy, only_dw = torch.full_like(dy, 7.0), torch.empty_like(dw)
    moe.moe_finalize_backward(dout, None, pos, w, only_dy, None)
    moe.moe_finalize_backward(dout, y, pos, w, None, only_dw)
    assert torch.equal(only_dy, dy) and torch.equal(only_dw, dw)


@pytest.mark.parametrize("dy_dtype", [BF, F32])
def test_finalize_backward_past_31_bits(dy_dtype):
    T, k, H = 60000, 8, 4480  # y and dy have 2.15e9 elements
    g, P = gen(6), T * k
    pos = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    dout, w = normal(g, T, H), torch.rand(T, k, generator=g, device="cuda")
    y = torch.randint(-3, 4, (P, H), generator=g, device="cuda", dtype=torch.int8).to(F32)
    dy, dw = torch.full((P, H), NAN, device="cuda", dtype=dy_dtype), torch.full((T, k), NAN, device="cuda")
    moe.moe_finalize_backward(dout, y, pos, w, dy, dw)
    for lo in range(0, P, 40000):
        r, t = pos[lo:lo + 40000].long(), torch.arange(lo, min(lo + 40000, P), device="cuda") // k
        rows = dout[t].double()
        want = w.flatten()[lo:lo + 40000].double()[:, None] * rows
        close(dy[r], want, want.abs() * (ref.HALF[dy_dtype] + ref.HALF[F32] * 1.01))
        rows *= y[r]
        close(dw.flatten()[lo:lo + 40000], rows.sum(1), ref.sum_bound(rows.sum(1), rows.abs().sum(1), H, F32))


# ------------------------------------------------------------------ MXFP4
def check_rows(x, codes, scales):
    """Codes and scales of rows x against the plain encoder, some rows at a time."""
    nb = x.shape[-1] // 32
    for lo in range(0, x.shape[0], 2000):
        code, scale = ref.mx_encode(x[lo:lo + 2000])
        assert torch.equal(codes[lo:lo + 2000], ref.mx_pack(code)), lo
        assert torch.equal(scales[lo:lo + 2000, :nb], scale), lo
    assert bool((scales[:, nb:] == 127).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,K", [(13127, 5120), (699123, 96)])
def test_mxfp4_rows_streamed(rows, K, dtype):
    assert rows * K * (2 if dtype == BF else 4) > STREAMED
    x = awkward(gen(rows), rows, K, dtype)
    codes, scales = quantised(x)
    check_rows(x, codes, scales)
    out, big = ref.guarded(torch.zeros(rows, K, dtype=dtype, device="cuda"), 16, 7.0)
    moe.moe_mxfp4_dequantize(codes, scales, out)
    for lo in range(0, rows, 20000):
        want = ref.mx_decode64(codes[lo:lo + 20000], scales[lo:lo + 20000])
        assert torch.equal(out[lo:lo + 20000].double().nan_to_num(nan=1e300), want.nan_to_num(nan=1e300)), lo
    assert ref.guards_intact(big, 16, 7.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_mxfp4_transposed_streamed(dtype):
    g, (B, K, C) = gen(5), (3, 5152, 4360)
    assert B * K * C * (2 if dtype == BF else 4) > STREAMED
    x = torch.stack([awkward(g, C, K, dtype).t().contiguous() for _ in range(B)])
    codes, scales = quantised(x, trans=True)
    for b in range(B):
        check_rows(x[b].t().contiguous(), codes[b], scales[b])


@pytest.mark.parametrize("trans", [False, True])
def test_mxfp4_past_31_bits(trans):
    g = gen(7)
    B, R, C = (300, 5120, 1400) if trans else (1, 420007, 5120)  # 2.15e9 elements
    x = torch.empty(B, R, C, dtype=BF, device="cuda")
    assert x.numel() > 1 << 31
    x.normal_(generator=g)
    codes, scales = quantised(x, trans=trans)
    K = R if trans else C
    back = torch.full((*codes.shape[:-1], K), NAN, dtype=BF, device="cuda")
    moe.moe_mxfp4_dequantize(codes, scales, back)
    flat = lambda t: t.view(-1, t.shape[-1])  # noqa: E731
    codes, scales, back = flat(codes), flat(scales), flat(back)
    edge = (1 << 31) // K  # the row that crosses 2^31 elements
    n = codes.shape[0]
    picked = torch.tensor([0, 1, n // 2, edge - 1, edge, edge + 1, n - 2, n - 1], device="cuda")
    rows = torch.stack([x[p // C, :, p % C] if trans else x[0, p] for p in picked.tolist()])
    check_rows(rows, codes[picked], scales[picked])
    assert torch.equal(back[picked].double(), ref.mx_decode64(codes[picked], scales[picked]))
    assert not back.isnan().any()
