"""Calls of the operators that their documentation allows and ordinary programs seldom make: experts that start behind
row 0, operands at the ends of 32-bit buffers and past 4 GiB, a stream given by the caller, infinities in SwiGLU."""
import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref as ref
from tests.test_gpu_ops import BF, F32, NAN, close, gen, normal, quantised, wide_index

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ experts that start behind row 0
@pytest.mark.parametrize("kind", ["bf16 nn", "bf16 nt", "fp32", "mxfp4"])
@pytest.mark.parametrize("first,counts,N", [(5, [7, 0, 28], 72), (300, [900, 0, 1, 2100] * 3, 2824)])
def test_rows_ahead_of_the_first_expert(first, counts, N, kind):
    """offsets[0] > 0: those rows are neither read nor written (few rows: streaming; many: tiles)."""
    g, E, K, used = gen(first), len(counts), 96, sum(counts)
    M = first + used + 9
    dt = F32 if kind == "fp32" else BF
    a, w = normal(g, M, K, dtype=dt), normal(g, E, N, K, dtype=dt, scale=K ** -0.5)
    off = ref.offsets_of(counts) + first
    out = torch.full((M, N), 7.0, device="cuda")
    if kind == "mxfp4":
        (ca, sa), (cw, sw) = quantised(a), quantised(w)
        sa[:first], sa[first + used:] = 255, 255
        moe.moe_mxfp4_grouped_gemm(ca, sa, cw, sw, off, out)
        x, w64 = ref.mx_decode64(ca, sa), ref.mx_decode64(cw, sw)
    else:
        a[:first], a[first + used:] = NAN, NAN
        if kind == "bf16 nt":
            moe.moe_grouped_gemm(a, w, off, out, w_trans=True)
        else:
            moe.moe_grouped_gemm(a, w.transpose(1, 2).contiguous(), off, out)
        x, w64 = a.double(), w
    want, mag = ref.product64(x[first:first + used], w64, counts, True)
    close(out[first:first + used], want, ref.sum_bound(want, mag, K, F32))
    assert bool((out[:first] == 7.0).all()) and bool((out[first + used:] == 7.0).all())
    if kind != "mxfp4":
        d = normal(g, M, N, dtype=dt)
        d[:first], d[first + used:] = NAN, NAN
        dw = torch.full((E, K, N), NAN, device="cuda")
        moe.moe_grouped_wgrad(a, d, off, dw)
        want, mag = ref.wgrad64(a[first:first + used].double(), d[first:first + used], counts)
        close(dw, want, ref.sum_bound(want, mag, max(counts), F32))


# ------------------------------------------------------------------ the ends of 32 bits
@pytest.mark.parametrize("rows,K", [(1048320, 8192), (0x3FFC0000, 32)])
def test_mxfp4_rows_at_the_end_of_a_buffer(rows, K):
    """Codes of 0xFFF00000 bytes, the most that are addressed in 32 bits; and as many bytes of scales, the most there may be."""
    assert rows * (K // 2) == 0xFFF00000 or rows * moe.moe_mxfp4_scale_stride(K) == 0xFFF00000
    g, per, N = gen(K), 700, 16392
    idx = wide_index(per, rows)
    picked = idx.long().unique()
    ca = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
    sa = torch.full((rows, moe.moe_mxfp4_scale_stride(K)), 255, dtype=torch.uint8, device="cuda")
    ca[picked], sa[picked] = quantised(normal(g, picked.numel(), K))
    cw, sw = quantised(normal(g, 2, N, K, scale=K ** -0.5))
    off, out = ref.offsets_of([0, per]), torch.full((per, N), NAN, device="cuda")
    moe.moe_mxfp4_grouped_gemm(ca, sa, cw, sw, off, out, row_index=idx)
    x = ref.mx_decode64(ca[idx.long()], sa[idx.long()])
    want, mag = ref.product64(x, ref.mx_decode64(cw, sw), [0, per], True)
    close(out, want, ref.sum_bound(want, mag, K, F32))


@pytest.mark.parametrize("w_trans", [False, True])
@pytest.mark.parametrize("counts", [[3, 200], [5, 900]])
def test_weights_past_4_gib(counts, w_trans):
    """The last two of 40 experts, in w and in dw (few rows for 40: streaming; more: tiles)."""
    g, E, K, N, M = gen(21), 40, 8192, 8192, sum(counts)
    w = torch.full((E, K, N), NAN, dtype=BF, device="cuda")
    w[-2:] = normal(g, 2, K, N, scale=K ** -0.5)
    loads = [0] * (E - 2) + counts
    off, a, out = ref.offsets_of(loads), normal(g, M, K), torch.full((M, N), NAN, device="cuda")
    moe.moe_grouped_gemm(a, w, off, out, w_trans=w_trans)
    want, mag = ref.product64(a.double(), w[-2:], counts, w_trans)
    close(out, want, ref.sum_bound(want, mag, K, F32))
    del w
    d = normal(g, M, N)
    for t in (F32, BF):
        dw = torch.full((E, K, N), NAN, dtype=t, device="cuda")
        moe.moe_grouped_wgrad(a, d, off, dw)
        want, mag = ref.wgrad64(a.double(), d, counts)
        close(dw[-2:], want, ref.sum_bound(want, mag, max(counts), t))
        assert not dw[:-2].any()
        del dw


@pytest.mark.parametrize("counts", [[3, 200], [5, 1900]])
def test_mxfp4_weights_past_4_gib(counts):
    g, E, K, N, M = gen(22), 72, 8192, 16384, sum(counts)
    cw = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    sw = torch.full((E, N, moe.moe_mxfp4_scale_stride(K)), 255, dtype=torch.uint8, device="cuda")
    assert cw.numel() > 1 << 32
    cw[-2:], sw[-2:] = quantised(normal(g, 2, N, K, scale=K ** -0.5))
    ca, sa = quantised(normal(g, M, K))
    out = torch.full((M, N), NAN, device="cuda")
    moe.moe_mxfp4_grouped_gemm(ca, sa, cw, sw, ref.offsets_of([0] * (E - 2) + counts), out)
    want, mag = ref.product64(ref.mx_decode64(ca, sa), ref.mx_decode64(cw[-2:], sw[-2:]), counts, True)
    close(out, want, ref.sum_bound(want, mag, K, F32))


# ------------------------------------------------------------------ streams
@pytest.mark.parametrize("raw", [False, True])
def test_stream_given_by_the_caller(raw):
    """Inputs that are written late on a side stream, and every call told to run there (as an object or as an address)."""
    g, st = gen(23), torch.cuda.Stream()
    K, N, counts = 64, 72, [30, 0, 47]
    M, off = sum(counts), ref.offsets_of(counts)
    src = dict(a=normal(g, M, K), w=normal(g, 3, K, N), d=normal(g, M, N), gu=normal(g, M, 2 * K), dh=normal(g, M, K),
               dout=normal(g, M, K), y=normal(g, M, K, dtype=F32), pos=torch.randperm(M, generator=g, device="cuda").to(torch.int32),
               tw=torch.rand(M, 1, generator=g, device="cuda"), wt=normal(g, 3, N, K))

    def calls(s, stream):
        e = lambda *sh, t=BF: torch.empty(*sh, dtype=t, device="cuda")  # noqa: E731
        o = dict(out=e(M, N), dw=e(3, K, N, t=F32), h=e(M, K), da=e(M, 2 * K), dy=e(M, K), dtw=e(M, 1, t=F32),
                 ca=e(M, K // 2, t=torch.uint8), sa=e(M, 4, t=torch.uint8), cw=e(3, N, K // 2, t=torch.uint8),
                 sw=e(3, N, 4, t=torch.uint8), back=e(M, K), mx=e(M, N))
        yield o
        moe.moe_grouped_gemm(s["a"], s["w"], off, o["out"], stream=stream)
        moe.moe_grouped_wgrad(s["a"], s["d"], off, o["dw"], stream=stream)
        moe.moe_swiglu(s["gu"], o["h"], stream=stream)
        moe.moe_swiglu_backward(s["gu"], s["dh"], o["da"], stream=stream)
        moe.moe_finalize_backward(s["dout"], s["y"], s["pos"], s["tw"], o["dy"], o["dtw"], stream=stream)
        moe.moe_mxfp4_quantize(s["a"], o["ca"], o["sa"], stream=stream)
        moe.moe_mxfp4_quantize(s["wt"], o["cw"], o["sw"], stream=stream)
        moe.moe_mxfp4_dequantize(o["ca"], o["sa"], o["back"], stream=stream)
        moe.moe_mxfp4_grouped_gemm(o["ca"], o["sa"], o["cw"], o["sw"], off, o["mx"], stream=stream)
        yield o

    *_, want = calls(src, None)
    late = {n: torch.zeros_like(t) for n, t in src.items()}
    late["pos"].copy_(src["pos"])  # indices are right from the start
    steps = calls(late, st.cuda_stream if raw else st)
    next(steps)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        for n, t in src.items():
            late[n].copy_(t)
    got = next(steps)  # enqueued while the side stream still waits
    st.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n


# ------------------------------------------------------------------ SwiGLU at the ends of its range
@pytest.mark.parametrize("dtype", [BF, F32])
def test_swiglu_infinities_and_nan(dtype):
    """As the formula in 64 bits: NaN where it is NaN, infinite where it is infinite, and neighbours untouched."""
    I = 64
    g = gen(24)
    a, dh = normal(g, 3, 2 * I, dtype=dtype), normal(g, 3, I, dtype=dtype)
    a[0, :6] = torch.tensor([float("inf"), float("-inf"), NAN, 3e38, -3e38, 0.0], device="cuda").to(dtype)
    a[0, I:I + 6], dh[0, :6] = 0.5, 0.5
    a[1, I:I + 3] = torch.tensor([float("inf"), float("-inf"), NAN], device="cuda").to(dtype)
    dh[2, :3] = torch.tensor([float("inf"), float("-inf"), NAN], device="cuda").to(dtype)
    h, da = torch.empty_like(dh), torch.empty_like(a)
    moe.moe_swiglu(a, h)
    moe.moe_swiglu_backward(a, dh, da)
    G, U, D = a[:, :I].double(), a[:, I:].double(), dh.double()
    s = torch.sigmoid(G)
    for got, want in ((h, G * s * U), (da[:, :I], D * U * s * (1 + G * (1 - s))), (da[:, I:], D * G * s)):
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.isinf(), want.isinf())
        assert torch.equal(got.double()[want.isinf()], want[want.isinf()])
    big = a[0, 3].double().item()  # the largest gates: s is 1 or 0
    assert h[0, 3:6].tolist() == [big / 2, 0.0, 0.0]
    assert da[0, 3:6].tolist() == [0.25, 0.0, 0.125] and da[0, I + 3:I + 6].tolist() == [big / 2, 0.0, 0.0]
