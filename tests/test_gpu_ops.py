"""The operators around the layer on the GPU against plain 64-bit forms: grouped
products and weight gradients, SwiGLU, the finalize gradient, MXFP4; a training
pass and a serving pass through them; streams and graphs."""
import random

import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def ragged(rng, E, total):
    """Loads of E experts that add up to total: some empty, some of one row, the rest uneven."""
    cuts = sorted(rng.randint(0, total) for _ in range(E - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def index_for(rng, M, rows, div, bad):
    idx = [rng.randrange(rows * div) for _ in range(M)]
    if bad:  # rows of zeros: negative indices and ones past the tokens
        for i in range(0, M, 7):
            idx[i] = rng.choice([-1, -5, rows * div, rows * div + 3, 2 ** 31 - 1, -2 ** 31])
    return torch.tensor(idx, dtype=torch.int32, device="cuda")


def close(got, want, bound):
    err = (got.double() - want).abs()
    worst = (err - bound).max().item() if err.numel() else 0.0
    assert not err.isnan().any() and worst <= 0, f"off by {err.max().item():.3g}, {worst:.3g} over the bound"


# (loads, K, N): empty experts, single rows, tile edges of 16 / 32 / 64 / 128 / 256, depths that end inside a step
SHAPES = [
    ([1], 8, 8),
    ([0, 1, 0], 72, 40),
    ([3, 0, 16, 1, 17], 64, 64),
    ([5, 33, 0, 31], 264, 136),
    ([64, 65, 2], 136, 520),
    ([127, 0, 129, 1], 200, 264),
    ([256, 257, 255], 96, 256),
    ([300, 0, 0, 7, 600], 544, 328),
    ([0, 0], 64, 64),
    ([1] * 9, 1544, 200),
    ([2, 1, 4] * 21, 320, 512),
    ([700], 1032, 776),
    # many tiles or long experts: the tiled kernels
    ([2000, 0, 1, 700, 255, 2500], 544, 328),
    ([4000], 1032, 776),
    ([65, 129, 257] * 22, 200, 520),
    ([0, 40, 96, 3, 200, 33, 64] * 10, 136, 520),
    ([300, 31, 600], 64, 16392),
    # one long expert among short ones: the streaming kernels
    ([300] + [0, 1] * 40, 320, 200),
    # as many experts as there may be
    ([0, 1, 2, 3] * 64, 96, 72),
    ([40, 0, 17, 90] * 64, 64, 72),
]


@pytest.mark.parametrize("w_trans", [False, True])
@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_grouped_gemm(case, w_trans, dtype, out_dtype):
    counts, K, N = SHAPES[case]
    rng, g = random.Random(case), gen(case)
    E, used, spare = len(counts), sum(counts), 5
    M = used + spare  # rows behind the last expert: NaN in, left as they were
    gather = case % 3 != 1
    div = 1 + case % 4
    rows = 23 if gather else M
    a, abig = ref.guarded(normal(g, rows, K, dtype=dtype), 16, NAN)
    w, wbig = ref.guarded(normal(g, E, *((N, K) if w_trans else (K, N)), dtype=dtype, scale=K ** -0.5), 16, NAN)
    idx = index_for(rng, M, rows, div, case % 2 == 0) if gather else None
    if not gather:
        a[used:] = NAN
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = NAN
    out, obig = ref.guarded(torch.full((M, N), 7.0, device="cuda", dtype=out_dtype), 16, 7.0)
    off = ref.offsets_of(counts)
    moe.moe_grouped_gemm(a, w, off, out, row_index=idx, row_div=div, w_trans=w_trans)
    x = ref.gather64(a, used, idx[:used] if gather else None, div)
    want, mag = ref.product64(x, w, counts, w_trans)
    close(out[:used], want, ref.sum_bound(want, mag, K, out_dtype))
    assert bool((out[used:] == 7.0).all()) and ref.guards_intact(obig, 16, 7.0)
    again = torch.full_like(out, 7.0)
    moe.moe_grouped_gemm(a, w, off, again, row_index=idx, row_div=div, w_trans=w_trans)
    assert torch.equal(again, out)


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("dtype,out_dtype,acc", [(BF, BF, False), (BF, F32, False), (BF, F32, True), (F32, F32, True),
                                                 (F32, BF, False)])
def test_grouped_wgrad(case, dtype, out_dtype, acc):
    counts, K, N = SHAPES[case]
    rng, g = random.Random(100 + case), gen(100 + case)
    E, used, spare = len(counts), sum(counts), 3
    M = used + spare
    gather, div = case % 3 != 2, 1 + case % 3
    rows = 31 if gather else M
    a, _ = ref.guarded(normal(g, rows, K, dtype=dtype), 16, NAN)
    d, _ = ref.guarded(normal(g, M, N, dtype=dtype), 16, NAN)
    d[used:] = NAN
    if not gather:
        a[used:] = NAN
    idx = index_for(rng, M, rows, div, case % 2 == 1) if gather else None
    start = normal(g, E, K, N, dtype=F32) if acc else torch.full((E, K, N), NAN, device="cuda")
    dw, big = ref.guarded(start.to(out_dtype), 16, 7.0)
    off = ref.offsets_of(counts)
    moe.moe_grouped_wgrad(a, d, off, dw, row_index=idx, row_div=div, accumulate=acc)
    x = ref.gather64(a, used, idx[:used] if gather else None, div)
    want, mag = ref.wgrad64(x, d[:used], counts)
    if acc:
        want, mag = want + start.double(), mag + start.double().abs()
    close(dw, want, ref.sum_bound(want, mag, max(counts) + 1, out_dtype))
    assert ref.guards_intact(big, 16, 7.0)


@pytest.mark.parametrize("rows", [2047, 2048, 2049, 5000])
def test_grouped_wgrad_long_expert(rows):
    """One expert with many rows among short ones, gathered: sums over thousands of rows."""
    rng, g = random.Random(rows), gen(rows)
    counts, K, N = [3, rows, 0, 40], 72, 136
    M = sum(counts)
    a, d = normal(g, 97, K), normal(g, M, N)
    idx = index_for(rng, M, 97, 2, True)
    dw = torch.empty(4, K, N, device="cuda")
    moe.moe_grouped_wgrad(a, d, ref.offsets_of(counts), dw, row_index=idx, row_div=2)
    want, mag = ref.wgrad64(ref.gather64(a, M, idx, 2), d, counts)
    close(dw, want, ref.sum_bound(want, mag, rows, F32))


SKEWED = {
    "falling": [1200 // (e + 1) for e in range(256)],
    "rising": [1200 // (256 - e) for e in range(256)],
    "one": [0] * 131 + [2000] + [0] * 124,
    "ends": [700] + [0] * 254 + [900],
    "one in eight": [300 if e % 8 == 7 else 0 for e in range(96)],
    "even": [64] * 256,
    "empty": [0] * 200,
    "few": [5, 0, 4000],
}


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("load", SKEWED)
def test_grouped_wgrad_skewed_loads(load, acc):
    """More tiles than workgroups, shared out by uneven costs: every tile is written once."""
    g, counts = gen(11), SKEWED[load]
    K, N, M = 264, 520, sum(counts)
    if len(counts) < 64:
        K, N = 2056, 2568
    a, d = normal(g, M, K), normal(g, M, N)
    start = normal(g, len(counts), K, N, dtype=F32) if acc else torch.full((len(counts), K, N), NAN, device="cuda")
    dw, big = ref.guarded(start, 16, 7.0)
    moe.moe_grouped_wgrad(a, d, ref.offsets_of(counts), dw, accumulate=acc)
    want, mag = ref.wgrad64(a.double(), d, counts)
    if acc:
        want, mag = want + start.double(), mag + start.double().abs()
    close(dw, want, ref.sum_bound(want, mag, max(counts) + 1, F32))
    assert ref.guards_intact(big, 16, 7.0)


@pytest.mark.parametrize("load", ["rising", "one in eight", "few"])
def test_grouped_wgrad_skewed_gathered_bf16(load):
    """The same with gathered rows (an index twice and bad ones) and bf16 results, rows behind the last expert."""
    rng, g, counts = random.Random(3), gen(12), SKEWED[load]
    K, N, used = (264, 520, sum(counts)) if len(counts) > 64 else (2056, 2568, sum(counts))
    a, d = normal(g, 501, K), normal(g, used + 9, N)
    d[used:] = NAN
    idx = index_for(rng, used + 9, 501, 3, True)
    dw, big = ref.guarded(torch.full((len(counts), K, N), NAN, device="cuda", dtype=BF), 16, 7.0)
    moe.moe_grouped_wgrad(a, d, ref.offsets_of(counts), dw, row_index=idx, row_div=3)
    want, mag = ref.wgrad64(ref.gather64(a, used, idx[:used], 3), d[:used], counts)
    close(dw, want, ref.sum_bound(want, mag, max(counts) + 1, BF))
    assert ref.guards_intact(big, 16, 7.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_grouped_wgrad_empty_experts_keep_dw(dtype):
    """accumulate: an expert without rows keeps dw bit for bit (-0 and NaN payloads too)."""
    g, counts, K, N = gen(5), [0, 70, 0, 3, 0], 72, 136
    M = sum(counts)
    a, d = normal(g, M, K, dtype=dtype), normal(g, M, N, dtype=dtype)
    dw = torch.full((5, K, N), -0.0, device="cuda")
    dw[:, 3] = torch.tensor([0x7FA12345], dtype=torch.int32, device="cuda").view(F32)
    start = dw.clone()
    moe.moe_grouped_wgrad(a, d, ref.offsets_of(counts), dw, accumulate=True)
    for e, c in enumerate(counts):
        assert torch.equal(dw[e].view(torch.int32), start[e].view(torch.int32)) == (c == 0), e


def test_grouped_no_rows():
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    a, w = torch.empty(0, 64, device="cuda", dtype=BF), torch.full((3, 64, 64), NAN, device="cuda", dtype=BF)
    moe.moe_grouped_gemm(a, w, off, torch.empty(0, 64, device="cuda", dtype=BF))
    moe.moe_grouped_wgrad(a, torch.empty(0, 64, device="cuda", dtype=BF), off, w)
    assert not w.any()


@pytest.mark.parametrize("layout", ["nn", "nt", "mx"])
@pytest.mark.parametrize("per", [2, 300, 3000])
def test_bad_rows_stay_where_they_are(layout, per):
    """An infinity or a NaN in one row reaches that row's products only; bounds outside [0, M] are clamped."""
    g, E, K, N = gen(3), 3, 256, 264
    M = E * per
    a, w = normal(g, M, K), normal(g, E, N, K)
    a[1, 5], a[per, 0], a[M - 1, K - 1] = NAN, float("inf"), float("-inf")
    off = torch.tensor([-4, per, 2 * per, M + 999], dtype=torch.int32, device="cuda")
    out = torch.empty(M, N, device="cuda")
    if layout == "mx":
        ca, sa = quantised(a)
        cw, sw = quantised(w.view(E * N, K))
        moe.moe_mxfp4_grouped_gemm(ca, sa, cw.view(E, N, -1), sw.view(E, N, -1), off, out)
    elif layout == "nt":
        moe.moe_grouped_gemm(a, w, off, out, w_trans=True)
    else:
        moe.moe_grouped_gemm(a, w.transpose(1, 2).contiguous(), off, out)
    fine = torch.isfinite(out).all(1)
    assert sorted((~fine).nonzero().flatten().tolist()) == sorted({1, per, M - 1})
    assert not torch.isfinite(out[[1, per, M - 1]]).any()


def wide_index(M, rows):
    """Rows spread over the whole of a long array, its last one among them."""
    idx = (torch.arange(M, dtype=torch.int64, device="cuda") * 7919 * 131) % rows
    idx[-1] = rows - 1
    return idx.to(torch.int32)


@pytest.mark.parametrize("per,N", [(3, 72), (700, 16392)])
@pytest.mark.parametrize("mx", [False, True])
def test_rows_past_32_bits(mx, per, N):
    """Gathered from arrays of more than 4 GiB, by the streaming and the tiled kernels."""
    g, K = gen(8), 8192
    rows = (1 << 20) + 4000 if mx else (1 << 18) + 4000
    idx = wide_index(per, rows)
    picked = idx.long().unique()
    off, out = ref.offsets_of([0, per]), torch.empty(per, N, device="cuda")
    w = normal(g, 2, N, K, scale=K ** -0.5)
    if mx:
        a = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
        sa = torch.full((rows, moe.moe_mxfp4_scale_stride(K)), 255, dtype=torch.uint8, device="cuda")
        a[picked], sa[picked] = quantised(normal(g, picked.numel(), K))
        cw, sw = quantised(w)
        moe.moe_mxfp4_grouped_gemm(a, sa, cw, sw, off, out, row_index=idx)
        x, w64 = ref.mx_decode64(a[idx.long()], sa[idx.long()]), ref.mx_decode64(cw, sw)
    else:
        a = torch.empty(rows, K, dtype=BF, device="cuda")
        a[picked] = normal(g, picked.numel(), K)
        moe.moe_grouped_gemm(a, w, off, out, row_index=idx, w_trans=True)
        x, w64 = a[idx.long()].double(), w
    want, mag = ref.product64(x, w64, [0, per], True)
    close(out, want, ref.sum_bound(want, mag, K, F32))


def test_results_past_32_bits():
    """Rows of out, and of d, past the first 4 GiB."""
    g, K, N, M = gen(9), 8, 1024, (1 << 20) + 4321
    counts = [M - 700, 0, 700]
    off, a, w = ref.offsets_of(counts), normal(g, M, K), normal(g, 3, K, N)
    out = torch.empty(M, N, device="cuda")
    moe.moe_grouped_gemm(a, w, off, out)
    for lo in (0, M - 1400, M - 700):
        e = 0 if lo < M - 700 else 2
        want = a[lo:lo + 700].double() @ w[e].double()
        close(out[lo:lo + 700], want, ref.sum_bound(want, a[lo:lo + 700].double().abs() @ w[e].double().abs(), K, F32))
    d = torch.zeros(2 * M, N, dtype=BF, device="cuda")
    d[-700:] = normal(g, 700, N)
    a2 = torch.zeros(2 * M, K, dtype=BF, device="cuda")
    a2[-700:] = normal(g, 700, K)
    dw = torch.empty(3, K, N, device="cuda")
    moe.moe_grouped_wgrad(a2, d, ref.offsets_of([2 * M - 700, 0, 700]), dw)
    want, mag = ref.wgrad64(a2[-700:].double(), d[-700:], [700])
    close(dw[2:], want, ref.sum_bound(want, mag, 700, F32))
    assert not dw[:2].any()


def test_two_row_indices_of_one_row():
    """The same source row under many sorted rows, on both sides of an expert's border."""
    g, K, N = gen(10), 64, 72
    counts = [37, 91]
    idx = torch.full((128,), 5, dtype=torch.int32, device="cuda")
    a, w, d = normal(g, 9, K), normal(g, 2, K, N), normal(g, 128, N)
    out, dw = torch.empty(128, N, device="cuda"), torch.empty(2, K, N, device="cuda")
    off = ref.offsets_of(counts)
    moe.moe_grouped_gemm(a, w, off, out, row_index=idx)
    moe.moe_grouped_wgrad(a, d, off, dw, row_index=idx)
    x = ref.gather64(a, 128, idx)
    want, mag = ref.product64(x, w, counts, False)
    close(out, want, ref.sum_bound(want, mag, K, F32))
    want, mag = ref.wgrad64(x, d, counts)
    close(dw, want, ref.sum_bound(want, mag, 91, F32))


# ------------------------------------------------------------------ SwiGLU
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,I", [(1, 8), (3, 40), (129, 264), (1000, 1416)])
def test_swiglu_and_gradient(M, I, dtype):
    g = gen(M)
    a = normal(g, M, 2 * I, dtype=dtype, scale=3.0)
    a[0, :4] = torch.tensor([0.0, -88.0, 60.0, -120.0], device="cuda").to(dtype)
    dh = normal(g, M, I, dtype=dtype)
    G, U, D = a[:, :I].double(), a[:, I:].double(), dh.double()
    s = torch.sigmoid(G)
    h64, dg64, du64 = G * s * U, D * U * s * (1 + G * (1 - s)), D * G * s
    h, h2, da = torch.empty_like(dh), torch.empty_like(dh), torch.empty_like(a)
    moe.moe_swiglu(a, h)
    moe.moe_swiglu_backward(a, dh, da, h=h2)
    assert torch.equal(h, h2)
    # s: the exponent's argument g log2(e) is rounded (|g| 2^-23 in the power), then exp2, the sum and the reciprocal
    # take a few steps each; 1 - s loses 2^-22 absolutely, times |g|; last the rounding to dtype. Values below the
    # smallest normal number may be flushed.
    rel = (G.abs() + 8) * 2.0 ** -22
    tiny = 2.0 ** -120
    for got, want, mag in ((h, h64, h64.abs()), (da[:, I:], du64, du64.abs()),
                           (da[:, :I], dg64, (D * U * s).abs() * (1 + G.abs()))):
        close(got, want, rel * mag + ref.HALF[dtype] * (want.abs() + rel * mag) + tiny)
    # in place, and without h
    a2, dh2 = a.clone(), dh.clone()
    moe.moe_swiglu_backward(a2, dh2, a2, h=dh2)
    assert torch.equal(a2, da) and torch.equal(dh2, h)
    da3 = torch.empty_like(a)
    moe.moe_swiglu_backward(a, dh, da3)
    assert torch.equal(da3, da)


# ------------------------------------------------------------------ finalize gradient
@pytest.mark.parametrize("dout_dtype,dy_dtype", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,k,H", [(1, 1, 64), (5, 8, 576), (33, 3, 5120), (7, 2, 16448)])
def test_finalize_backward(T, k, H, dout_dtype, dy_dtype):
    g, rng, P = gen(T), random.Random(T), T * k
    pos = list(range(P))
    rng.shuffle(pos)
    gone = [p for p in range(P) if p % 5 == 4]
    for p in gone:
        pos[p] = rng.choice([-1, -7, P, 2 ** 31 - 1])
    pos_t = torch.tensor(pos, dtype=torch.int32, device="cuda")
    dout, y, w = normal(g, T, H, dtype=dout_dtype), normal(g, P, H, dtype=F32), torch.rand(T, k, generator=g, device="cuda")
    dy, big = ref.guarded(torch.full((P, H), 7.0, device="cuda", dtype=dy_dtype), 16, 7.0)
    dw = torch.full((T, k), NAN, device="cuda")
    moe.moe_finalize_backward(dout, y, pos_t, w, dy, dw)
    want_dy, want_dw, mag = torch.full((P, H), 7.0, dtype=torch.float64, device="cuda"), torch.zeros(P, dtype=torch.float64, device="cuda"), torch.zeros(P, dtype=torch.float64, device="cuda")
    for p in range(P):
        if 0 <= pos[p] < P:
            r, d = pos[p], dout[p // k].double()
            want_dy[r] = w.flatten()[p].double() * d
            want_dw[p], mag[p] = (d * y[r].double()).sum(), (d * y[r].double()).abs().sum()
    # one product in fp32 (half a step of fp32), then the rounding to dy_dtype
    close(dy, want_dy, want_dy.abs() * (ref.HALF[dy_dtype] + ref.HALF[F32] * 1.01))
    close(dw.flatten(), want_dw, ref.sum_bound(want_dw, mag, H, F32))
    assert ref.guards_intact(big, 16, 7.0)
    only_dy, only_dw = torch.full_like(dy, 7.0), torch.empty_like(dw)
    moe.moe_finalize_backward(dout, None, pos_t, w, only_dy, None)
    moe.moe_finalize_backward(dout, y, pos_t, w, None, only_dw)
    assert torch.equal(only_dy, dy) and torch.equal(only_dw, dw)


# ------------------------------------------------------------------ MXFP4
def quantised(x, trans=False):
    rows = (*x.shape[:-2], x.shape[-1]) if trans else x.shape[:-1]
    K = x.shape[-2] if trans else x.shape[-1]
    codes = torch.full((*rows, K // 2), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((*rows, moe.moe_mxfp4_scale_stride(K)), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_mxfp4_quantize(x, codes, scales, trans=trans)
    return codes, scales


def awkward(g, rows, K, dtype):
    """Values that try the encoder: wide scales, every midpoint and its neighbours, zeros, infinities, subnormals."""
    x = normal(g, rows, K, dtype=F32)
    x *= torch.exp2(torch.randint(-140, 120, (rows, 1), generator=g, device="cuda").float())
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0], device="cuda")
    near = torch.cat((mids, -mids, mids * (1 + 2 ** -7), mids * (1 - 2 ** -7)))[:31]
    x[0, :31], x[0, 31] = near, 4.0
    if rows > 4:
        x[1] = 0.0
        x[2, 3], x[3, 0], x[4, K - 1] = NAN, float("inf"), -0.0
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,K", [(1, 32), (7, 96), (130, 160), (64, 5120)])
def test_mxfp4_rows(rows, K, dtype):
    x = awkward(gen(rows), rows, K, dtype)
    codes, scales = quantised(x)
    code, scale = ref.mx_encode(x)
    assert torch.equal(codes, ref.mx_pack(code))
    assert torch.equal(scales[:, : K // 32], scale) and bool((scales[:, K // 32:] == 127).all())
    for t in (BF, F32):
        out, big = ref.guarded(torch.zeros(rows, K, dtype=t, device="cuda"), 16, 7.0)
        moe.moe_mxfp4_dequantize(codes, scales, out)
        want = ref.mx_decode64(codes, scales)
        assert torch.equal(out.double().nan_to_num(nan=1e300), want.nan_to_num(nan=1e300)) and ref.guards_intact(big, 16, 7.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,K,C", [(1, 32, 8), (3, 96, 72), (2, 288, 136), (2, 1024, 264)])
def test_mxfp4_transposed(B, K, C, dtype):
    g = gen(K)
    x = torch.stack([awkward(g, C, K, dtype).t().contiguous() for _ in range(B)])
    codes, scales = quantised(x, trans=True)
    want = quantised(x.transpose(1, 2).contiguous())
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


def test_mxfp4_every_code_and_scale():
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 16, 16).expand(256, 16, 16).reshape(256, 256).contiguous()
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1).expand(256, 16).contiguous()
    out = torch.empty(256, 512, device="cuda")
    moe.moe_mxfp4_dequantize(codes, scales, out)
    want = ref.mx_decode64(codes, scales).float()  # above the fp32 range: infinity
    assert torch.equal(out.nan_to_num(nan=3e38, posinf=2e38, neginf=-2e38), want.nan_to_num(nan=3e38, posinf=2e38, neginf=-2e38))


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_mxfp4_grouped_gemm(case, out_dtype):
    counts, K, N = SHAPES[case]
    K = (K + 31) // 32 * 32
    rng, g = random.Random(case), gen(50 + case)
    E, used, spare = len(counts), sum(counts), 5
    M, gather, div = used + spare, case % 3 != 1, 1 + case % 4
    rows = 23 if gather else M
    ca, sa = quantised(normal(g, rows, K) * torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g, device="cuda")))
    cw, sw = quantised(normal(g, E * N, K, scale=K ** -0.5))
    # padding bytes hold no scale: any value may stand there
    sa[:, K // 32:], sw[:, K // 32:] = 255, 255
    (ca, _), (sa, _) = ref.guarded(ca, 16, 0x77), ref.guarded(sa, 16, 255)
    (cw, _), (sw, _) = ref.guarded(cw.view(E, N, -1), 16, 0x77), ref.guarded(sw.view(E, N, -1), 16, 255)
    idx = index_for(rng, M, rows, div, case % 2 == 0) if gather else None
    if not gather:
        sa[used:] = 255
    for e, c in enumerate(counts):
        if c == 0:
            sw[e] = 255
    out, big = ref.guarded(torch.full((M, N), 7.0, device="cuda", dtype=out_dtype), 16, 7.0)
    off = ref.offsets_of(counts)
    moe.moe_mxfp4_grouped_gemm(ca, sa, cw, sw, off, out, row_index=idx, row_div=div)
    a64, w64 = ref.mx_decode64(ca, sa), ref.mx_decode64(cw, sw)
    x = ref.gather64(a64, used, idx[:used] if gather else None, div)
    want, mag = ref.product64(x, w64, counts, True)
    close(out[:used], want, ref.sum_bound(want, mag, K, out_dtype))
    assert bool((out[used:] == 7.0).all()) and ref.guards_intact(big, 16, 7.0)


@pytest.mark.parametrize("K", [8192, 12800, 13312])
@pytest.mark.parametrize("counts", [[3, 0, 2], [40, 60]])
def test_mxfp4_long_depth(K, counts):
    """Depths whose scales fill the streaming kernels' LDS, and one past that."""
    g, E, N, M = gen(K), len(counts), 72, sum(counts)
    ca, sa = quantised(normal(g, M, K))
    cw, sw = quantised(normal(g, E, N, K, scale=K ** -0.5))
    out = torch.empty(M, N, device="cuda")
    moe.moe_mxfp4_grouped_gemm(ca, sa, cw, sw, ref.offsets_of(counts), out)
    want, mag = ref.product64(ref.mx_decode64(ca, sa), ref.mx_decode64(cw, sw), counts, True)
    close(out, want, ref.sum_bound(want, mag, K, F32))


# ------------------------------------------------------------------ together
def layer(seed, T, k, E, H, I, dtype):
    g = gen(seed)
    x, wgu, wd = (normal(g, *s, dtype=dtype, scale=c) for s, c in
                  (((T, H), 1.0), ((E, H, 2 * I), H ** -0.5), ((E, I, H), I ** -0.5)))
    ids = (torch.randn(T, E, generator=g, device="cuda")).topk(k, dim=1).indices.to(torch.int32).contiguous()
    w = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
    dout = normal(g, T, H, dtype=dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, off, sp, pp = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32), torch.empty(T * k, **i32)
    moe.moe_permute(ids, E, counts, off, sp, pp)
    return dict(x=x, wgu=wgu, wd=wd, ids=ids, w=w, dout=dout, off=off, sp=sp, pp=pp, T=T, k=k, E=E, H=H, I=I, dtype=dtype)


def buffers(L):
    P, H, I, dt = L["T"] * L["k"], L["H"], L["I"], L["dtype"]
    e = lambda *s, t=dt: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    return dict(a=e(P, 2 * I), h=e(P, I), y=e(P, H, t=F32), out=e(L["T"], H), dy=e(P, H), dw=e(L["T"], L["k"], t=F32),
                dh=e(P, I), da=e(P, 2 * I), h2=e(P, I), dxs=e(P, H, t=F32), dx=e(L["T"], H), dx32=e(L["T"], H, t=F32),
                dwd=e(L["E"], I, H, t=F32), dwgu=e(L["E"], H, 2 * I, t=F32), ones=torch.ones(L["T"], L["k"], device="cuda"))


def train_pass(L, b):
    """Forward and backward of the expert block, every step a call of the library."""
    k, off, sp, pp = L["k"], L["off"], L["sp"], L["pp"]
    moe.moe_grouped_gemm(L["x"], L["wgu"], off, b["a"], row_index=sp, row_div=k)
    moe.moe_swiglu(b["a"], b["h"])
    moe.moe_grouped_gemm(b["h"], L["wd"], off, b["y"])
    moe.moe_finalize(b["y"], pp, L["w"], b["out"])
    moe.moe_finalize_backward(L["dout"], b["y"], pp, L["w"], b["dy"], b["dw"])
    moe.moe_grouped_gemm(b["dy"], L["wd"], off, b["dh"], w_trans=True)
    moe.moe_swiglu_backward(b["a"], b["dh"], b["da"], h=b["h2"])
    moe.moe_grouped_wgrad(b["h2"], b["dy"], off, b["dwd"])
    moe.moe_grouped_wgrad(L["x"], b["da"], off, b["dwgu"], row_index=sp, row_div=k)
    moe.moe_grouped_gemm(b["da"], L["wgu"], off, b["dxs"], w_trans=True)
    moe.moe_finalize(b["dxs"], pp, b["ones"], b["dx"], out_f32=b["dx32"])


def block64(L, x, wgu, wd, w):
    """The expert block in fp64, token by slot."""
    out = torch.zeros(L["T"], L["H"], dtype=torch.float64)
    for e in range(L["E"]):
        t, j = (L["ids"].cpu() == e).nonzero(as_tuple=True)
        a = x[t] @ wgu[e]
        h = torch.nn.functional.silu(a[:, :L["I"]]) * a[:, L["I"]:]
        out = out.index_add(0, t, w[t, j].unsqueeze(1) * (h @ wd[e]))
    return out


@pytest.mark.parametrize("dtype,tol", [(F32, 2e-5), (BF, 2e-2)])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 64, 64), (37, 3, 5, 128, 64), (200, 2, 3, 192, 128)])
def test_training_pass(T, k, E, H, I, dtype, tol):
    """Gradients of the whole expert block against fp64 and against differences of the fp64 block.
    In fp32 every stage is a sum of at most 256 terms (2-norm error well below 256 * 2^-24 = 1.5e-5). In bf16 five
    results are rounded on the longest way (a, h, dy, dh, da), each by at most 2^-8 of its value: 5 * 2^-8 = 2e-2."""
    L = layer(T, T, k, E, H, I, dtype)
    b = buffers(L)
    train_pass(L, b)
    leaves = [L[n].double().cpu().requires_grad_() for n in ("x", "wgu", "wd", "w")]
    out = block64(L, *leaves)
    dout = L["dout"].double().cpu()
    grads = torch.autograd.grad(out, leaves, dout)
    for name, want in zip(("out", "dx32", "dwgu", "dwd", "dw"), (out, *grads)):
        got = b[name].double().cpu()
        rel = ((got - want).norm() / want.norm()).item()
        assert rel <= tol + (2.0 ** -8 if name == "out" else 0), (name, rel)
    # differences along a random direction
    gcpu = torch.Generator().manual_seed(T)
    dirs = [torch.randn(t.shape, generator=gcpu, dtype=torch.float64) * t.detach().std() for t in leaves]
    eps = 1e-5
    with torch.no_grad():
        up, down = (block64(L, *(t + s * eps * v for t, v in zip(leaves, dirs))) for s in (1, -1))
        slope = ((up - down) * dout).sum() / (2 * eps)
        got = sum((b[n].double().cpu() * v).sum() for n, v in zip(("dx32", "dwgu", "dwd", "dw"), dirs))
        size = sum((b[n].double().cpu().norm() * v.norm()) for n, v in zip(("dx32", "dwgu", "dwd", "dw"), dirs))
    assert abs(got - slope) <= tol * size


def test_grouped_products_match_the_layer():
    """The composed forward pass gives what moe_experts and moe_finalize give, to the rounding of a and h."""
    L = layer(5, 64, 4, 8, 256, 128, BF)
    b = buffers(L)
    train_pass(L, b)
    wt = moe.ExpertWeights(moe.MOE_BF16, L["wgu"], L["wd"])
    ws = moe.workspace(moe.moe_experts_workspace_size(64, 256, 128, 8, 4, wt))
    y = torch.empty_like(b["y"])
    moe.moe_experts(L["x"], 128, 8, 4, L["off"], L["sp"], wt, y, ws)
    assert ((b["y"] - y).norm() / y.norm()).item() <= 3 * 2.0 ** -8


def test_serving_pass_mxfp4():
    """Expert block with MXFP4 weights and activations against fp64 on the same codes, stage by stage."""
    T, k, E, H, I = 45, 4, 8, 320, 160
    L = layer(9, T, k, E, H, I, BF)
    b = buffers(L)
    cgu, sgu = quantised(L["wgu"], trans=True)
    cd, sd = quantised(L["wd"], trans=True)
    cx, sx = quantised(L["x"])
    moe.moe_mxfp4_grouped_gemm(cx, sx, cgu, sgu, L["off"], b["a"], row_index=L["sp"], row_div=k)
    moe.moe_swiglu(b["a"], b["h"])
    ch, sh = quantised(b["h"])
    moe.moe_mxfp4_grouped_gemm(ch, sh, cd, sd, L["off"], b["y"])
    moe.moe_finalize(b["y"], L["pp"], L["w"], b["out"])
    counts = (L["off"][1:] - L["off"][:-1]).tolist()
    x = ref.gather64(ref.mx_decode64(cx, sx), T * k, L["sp"], k)
    want, mag = ref.product64(x, ref.mx_decode64(cgu, sgu), counts, True)
    close(b["a"], want, ref.sum_bound(want, mag, H, BF))
    code, scale = ref.mx_encode(b["h"])
    assert torch.equal(ch, ref.mx_pack(code)) and torch.equal(sh[:, : I // 32], scale)
    want, mag = ref.product64(ref.mx_decode64(ch, sh), ref.mx_decode64(cd, sd), counts, True)
    close(b["y"], want, ref.sum_bound(want, mag, I, F32))
    rows = b["y"].double()[L["pp"].long()].view(T, k, H)
    terms = L["w"].double().unsqueeze(-1) * rows
    close(b["out"], terms.sum(1), ref.sum_bound(terms.sum(1), terms.abs().sum(1), k + 1, BF))


@pytest.mark.parametrize("T,k,E,H,I", [(70, 3, 6, 128, 96), (1500, 4, 40, 320, 264)])
def test_streams_and_graph(T, k, E, H, I):
    """Two passes side by side on two streams, and both captured and replayed among eager work."""
    Ls = [layer(s, T, k, E, H, I, BF) for s in (1, 2)]
    want = []
    for L in Ls:
        b = buffers(L)
        train_pass(L, b)
        want.append(b)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [buffers(L) for L in Ls]
    for st, L, b in zip(streams, Ls, got):
        with torch.cuda.stream(st):
            train_pass(L, b)
    torch.cuda.synchronize()
    graphs, cap = [], [buffers(L) for L in Ls]
    for L, b in zip(Ls, cap):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            train_pass(L, b)
        graphs.append(gr)
    for _ in range(3):
        for b in cap:
            for t in ("a", "y", "dx", "dwd", "dwgu", "dw"):
                b[t].zero_()
        for gr in graphs:
            gr.replay()
        train_pass(Ls[0], got[0])  # eager work between
        torch.cuda.synchronize()
        for b, v in list(zip(cap, want)) + list(zip(got, want)):
            for n in ("a", "h", "y", "out", "dy", "dw", "dh", "da", "dx", "dwd", "dwgu"):
                assert torch.equal(b[n], v[n]), n
