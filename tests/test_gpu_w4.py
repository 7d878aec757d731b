"""4-bit integer weights with group scales on the GPU against plain 64-bit forms: quantisation, dequantisation, grouped
products."""
import random

import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref, w4_ref as ref
from tests.test_gpu_ops import BF, F32, NAN, close, gen, index_for, normal

pytestmark = pytest.mark.gpu
INF, U8 = float("inf"), torch.uint8


def buffers(rows, K, group, zeros, sdtype):
    codes, cb = ops_ref.guarded(torch.zeros(*rows, K // 2, dtype=U8, device="cuda"), 16, 0xA5)
    s, sb = ops_ref.guarded(torch.zeros(*rows, K // group, dtype=sdtype, device="cuda"), 16, 3.0)
    z, zb = ops_ref.guarded(torch.zeros(*rows, K // group, dtype=U8, device="cuda"), 16, 0xA5)
    return codes, s, z if zeros else None, (cb, sb, zb)


def check_quantise(x, group, zeros, sdtype, trans=False):
    rows_of = x.transpose(-2, -1).contiguous() if trans else x
    rows, K = rows_of.shape[:-1], rows_of.shape[-1]
    codes, s, z, bigs = buffers(rows, K, group, zeros, sdtype)
    moe.moe_w4_quantize(x, codes, s, zeros=z, trans=trans)
    wq, ws, wz = ref.quantise(rows_of, group, zeros, sdtype)
    assert torch.equal(s.nan_to_num(nan=-1.0), ws.nan_to_num(nan=-1.0))
    assert torch.equal(ref.unpack(codes), wq)
    assert z is None or torch.equal(z, wz)
    for big, v in zip(bigs, (0xA5, 3.0, 0xA5)):
        assert ops_ref.guards_intact(big, 16, v)
    return codes, s, z


def special(x, group):
    """Groups of zeros, an infinity, NaN, tiny and huge values, one sign, one value."""
    v = x.view(-1, group)
    ops = [lambda r: r.zero_(), lambda r: r[3:4].fill_(INF), lambda r: r[-1:].fill_(NAN), lambda r: r.mul_(1e-42),
           lambda r: r.mul_(1e-38), lambda r: r.abs_(), lambda r: r.abs_().neg_(), lambda r: r.mul_(5e37),
           lambda r: r.fill_(2.5), lambda r: r[1:].zero_(), lambda r: r[0:1].fill_(-INF), lambda r: r.mul_(1e-30),
           lambda r: r.copy_(torch.arange(group, device="cuda") / 2 - 7)]
    for i, f in enumerate(ops):
        if 2 * i + 1 < v.shape[0]:
            f(v[2 * i + 1])
    return x


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sdtype", [BF, F32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantise(dtype, sdtype, zeros, group):
    g = gen(group)
    for shape in ((1, group), (7, 3 * group), (130, 5 * group), (3, 5, 2 * group)):
        x = special(normal(g, *shape, dtype=dtype), group)
        codes, s, z = check_quantise(x, group, zeros, sdtype)
        for t in (BF, F32):
            out, big = ops_ref.guarded(torch.full(shape, 7.0, dtype=t, device="cuda"), 16, 7.0)
            moe.moe_w4_dequantize(codes, s, out, zeros=z)
            want = ref.weights64(codes, s, z)
            ok = ~want.isnan()
            assert torch.equal(out.isnan(), ~ok) and ops_ref.guards_intact(big, 16, 7.0)
            # rounded to fp32 and to out's type (subnormal results: to multiples of 2^-149, 2^-133 in bf16)
            bound = (2.0 ** -24 + ops_ref.HALF[t]) * want.abs() * 1.01 + (2.0 ** -134 if t is BF else 2.0 ** -150)
            assert bool(((out.double() - want).abs() <= bound)[ok].all())
    for shape in ((8, group), (264, 3 * group), (2, 40, 2 * group), (3, 136, 384)):  # [.., C, K]
        x = special(normal(g, *shape, dtype=dtype), group).transpose(-2, -1).contiguous()
        check_quantise(x, group, zeros, sdtype, trans=True)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("sdtype", [F32, BF])
def test_quantise_every_tie(zeros, sdtype):
    """Quotients at, just below and just above every half, in fp32, for scales of all kinds of mantissas."""
    g, group = gen(3), 32
    top = torch.exp2(torch.rand(400000, 1, generator=g, device="cuda") * 120 - 60)
    s = (top * torch.tensor(1 / 15 if zeros else 1 / 7, dtype=F32, device="cuda")).to(sdtype).float()
    ok = (s.view(torch.int32) & 31) == 0  # scales whose multiples by halves are fp32 numbers
    top, s = top[ok][:4096, None], s[ok][:4096, None]
    half = torch.arange(-6, 6, device="cuda") + 0.5 + (7 if zeros else 0)
    mid = s * half  # exact: 19 by 5 bits
    x = torch.cat((mid, torch.nextafter(mid[:, :9], torch.zeros_like(mid[:, :9])),
                   torch.nextafter(mid[:, 3:], 1e30 * torch.sign(mid[:, 3:])), top, 0 * s), 1)
    assert x.shape == (4096, group)
    assert torch.equal(check_quantise(x.contiguous(), group, zeros, sdtype)[1].float(), s)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("power", [0, -100, -126, 100])
def test_quantise_every_bf16(zeros, power):
    """All mantissas of bf16 values under all mantissas of bf16 scales, over the exponents of quotients 1/32 .. 16."""
    m = torch.arange(128, 256, device="cuda").double()
    values = torch.cat([m * 2.0 ** e for e in range(-9, 1)])
    values = torch.cat((values, -values, torch.zeros(10 * 127 * 3 - 2560, dtype=torch.float64, device="cuda")))
    top = m * (1.0 if zeros else 0.5)
    top = torch.cat((top, top * 2))
    x = torch.zeros(len(top), 30, 128, dtype=torch.float64, device="cuda")
    x[:, :, :127] = values.view(30, 127).clamp(min=-m.max() * (0.0 if zeros else 1.0))
    x = torch.minimum(torch.maximum(x, -top[:, None, None]), top[:, None, None])
    x[:, :, 127] = top[:, None]
    x = (x * 2.0 ** (power - 7)).to(BF).view(len(top), 30 * 128)
    check_quantise(x, 128, zeros, BF)


def weights(g, E, N, K, group, zeros, sdtype):
    """Codes of every value, scales and zero points (bytes of all sizes among them), between guards."""
    codes, _ = ops_ref.guarded(torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda").to(U8), 16, 0xFF)
    s, _ = ops_ref.guarded((torch.randn(E, N, K // group, generator=g, device="cuda") * K ** -0.5 / 4).to(sdtype), 16, NAN)
    z = None
    if zeros:
        z = torch.randint(0, 16, (E, N, K // group), generator=g, device="cuda")
        z = torch.where(torch.rand(z.shape, generator=g, device="cuda") < 0.02, 255 - z, z).to(U8)
        z, _ = ops_ref.guarded(z, 16, 0xFF)
    return codes, s, z


def check_product(a, counts, codes, s, z, out_dtype, idx=None, div=1, spare=5, first=0):
    E, N = codes.shape[:2]
    K, used = a.shape[1], sum(counts)
    M = first + used + spare
    out, big = ops_ref.guarded(torch.full((M, N), 7.0, device="cuda", dtype=out_dtype), 16, 7.0)
    off = ops_ref.offsets_of(counts) + first
    moe.moe_w4_grouped_gemm(a, codes, s, off, out, zeros=z, row_index=idx, row_div=div)
    x = ops_ref.gather64(a, M, idx, div)[first:first + used]
    lo = 0
    for e, c in enumerate(counts):
        if c:
            w, spread = ref.weights64(codes[e], s[e], None if z is None else z[e]), ref.spread64(
                codes[e], s[e], None if z is None else z[e])
            want = x[lo:lo + c] @ w.t().contiguous()
            mag = x[lo:lo + c].abs() @ spread.t().contiguous()
            # K products exact, each added in fp32 within its group; a group's result takes four more roundings
            close(out[first + lo:first + lo + c], want, ops_ref.sum_bound(want, mag, K + 8, out_dtype))
        lo += c
    assert bool((out[:first] == 7.0).all()) and bool((out[first + used:] == 7.0).all())
    assert ops_ref.guards_intact(big, 16, 7.0)
    again = torch.full_like(out, 7.0)
    moe.moe_w4_grouped_gemm(a, codes, s, off, again, zeros=z, row_index=idx, row_div=div)
    assert torch.equal(again, out)


# (loads, K in groups of 128, N): empty experts, single rows, tile edges, depths that end inside a stage
SHAPES = [
    ([1], 1, 8), ([0, 1, 0], 3, 40), ([2], 41, 72), ([3, 0, 16, 1, 17], 2, 64), ([5, 33, 0, 31], 7, 136),
    ([64, 65, 2], 4, 520), ([127, 0, 129, 1], 5, 264), ([0, 0], 2, 64), ([1] * 9, 13, 200), ([2, 1, 4] * 21, 8, 512),
    ([700], 9, 776), ([4] * 5 + [9, 8, 7], 6, 72), ([300] + [0, 1] * 40, 3, 200), ([0, 1, 2, 3] * 64, 1, 72),
    ([2000, 0, 1, 700, 255, 2500], 5, 328), ([65, 129, 257] * 22, 2, 520), ([4000], 9, 776),
    ([0, 40, 96, 3, 200, 33, 64] * 10, 2, 520), ([300, 31, 600], 1, 16392),
    ([0, 1, 2500, 700, 130, 2930], 4, 776), ([40] * 30 + [64, 17, 130, 0], 11, 904), ([3, 0, 20], 120, 72),
    ([1000, 900, 1100, 1024, 960, 1088], 2, 1032),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros,sdtype,out_dtype", [(False, BF, BF), (True, BF, F32), (False, F32, F32), (True, F32, BF)])
def test_product(case, group, zeros, sdtype, out_dtype):
    counts, n128, N = SHAPES[case]
    K = n128 * 128 if group == 128 else n128 * 128 - 32 * (case % 4) if group == 32 else n128 * 128 - 64 * (case % 2)
    K = max(K, group)
    rng, g = random.Random(case), gen(case)
    E, used = len(counts), sum(counts)
    gather, div = case % 3 != 1, 1 + case % 4
    rows = 23 if gather else used + 5
    a, _ = ops_ref.guarded(normal(g, rows, K), 16, NAN)
    idx = index_for(rng, used + 5, rows, div, case % 2 == 0) if gather else None
    if not gather:
        a[used:] = NAN
    codes, s, z = weights(g, E, N, K, group, zeros, sdtype)
    for e, c in enumerate(counts):
        if c == 0:
            s[e] = NAN
    check_product(a, counts, codes, s, z, out_dtype, idx, div)


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("counts,N", [([1, 2, 0, 5], 264), ([70, 300, 0, 600], 264), ([70, 300, 0, 600], 3080),
                                      ([700, 3000, 0, 2600], 776)])
def test_product_exact_on_small_numbers(group, zeros, counts, N):
    """Whole-number rows and power-of-two scales: fp32 sums are exact, so are the results."""
    g, K = gen(5), 640
    M = sum(counts)
    a = torch.randint(-8, 9, (M, K), generator=g, device="cuda").to(BF)
    codes, s, z = weights(g, 4, N, K, group, zeros, F32)
    s = torch.exp2(torch.randint(-2, 3, s.shape, generator=g, device="cuda").float())
    out = torch.empty(M, N, device="cuda")
    moe.moe_w4_grouped_gemm(a, codes, s, ops_ref.offsets_of(counts), out, zeros=z)
    lo = 0
    for e, c in enumerate(counts):
        w = ref.weights64(codes[e], s[e], None if z is None else z[e])
        assert torch.equal(out[lo:lo + c].double(), a[lo:lo + c].double() @ w.t().contiguous())
        lo += c


@pytest.mark.parametrize("per,N", [(1, 136), (3, 136), (20, 136), (300, 136), (300, 3080), (2500, 800)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_bad_rows_and_scales_stay_where_they_are(per, N, group):
    """An infinity or a NaN in a row reaches that row alone, a NaN scale its column alone; a depth that ends in a stage."""
    g, E, K = gen(3), 3, 384
    M = E * per
    a = normal(g, M, K)
    codes, s, z = weights(g, E, N, K, group, True, BF)
    off = ops_ref.offsets_of([per] * E)
    clean, out = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    moe.moe_w4_grouped_gemm(a, codes, s, off, clean, zeros=z)
    a[0, 5], a[M - 1, K - 1] = INF, NAN
    s[1, 77, -1] = NAN
    moe.moe_w4_grouped_gemm(a, codes, s, off, out, zeros=z)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[0], bad[M - 1] = True, True
    bad[per:2 * per, 77] = True
    assert torch.equal(out[~bad], clean[~bad]) and not out[bad].isfinite().any()
    # bounds outside [0, M] count as 0 or M
    wild = off.clone()
    wild[0], wild[-1] = -9, M + 100
    again = torch.empty_like(out)
    moe.moe_w4_grouped_gemm(a, codes, s, wild, again, zeros=z)
    assert torch.equal(again[~bad], clean[~bad])


@pytest.mark.parametrize("counts", [[7, 0, 28], [900, 0, 1, 400]])
@pytest.mark.parametrize("N", [200, 2056, 3080])
def test_rows_ahead_of_the_first_expert(counts, N):
    g, first, K = gen(6), 37, 256
    a = normal(g, first + sum(counts) + 9, K)
    a[:first], a[first + sum(counts):] = NAN, NAN
    codes, s, z = weights(g, len(counts), N, K, 64, True, BF)
    check_product(a, counts, codes, s, z, BF, spare=9, first=first)


def test_no_rows():
    codes, s, _ = weights(gen(1), 3, 64, 64, 64, False, BF)
    out = torch.empty(0, 64, device="cuda", dtype=BF)
    moe.moe_w4_grouped_gemm(torch.empty(0, 64, device="cuda", dtype=BF), codes, s,
                            torch.zeros(4, dtype=torch.int32, device="cuda"), out)
    e = lambda *sh, t: torch.empty(*sh, dtype=t, device="cuda")  # noqa: E731
    moe.moe_w4_quantize(e(0, 64, t=BF), e(0, 32, t=U8), e(0, 1, t=BF))
    moe.moe_w4_dequantize(e(0, 32, t=U8), e(0, 1, t=BF), e(0, 64, t=BF))


@pytest.mark.parametrize("counts", [[3, 20], [5, 900], [5, 2400], [5, 17995]])
def test_weights_past_4_gib(counts):
    """The last two of 72 experts of 8192 x 16384."""
    g, E, K, N = gen(22), 72, 8192, 16384
    codes = torch.zeros(E, N, K // 2, dtype=U8, device="cuda")
    s = torch.full((E, N, K // 128), NAN, device="cuda")
    assert codes.numel() > 1 << 32
    codes[-2:], s[-2:], _ = weights(g, 2, N, K, 128, False, F32)
    a = normal(g, sum(counts), K)
    off = ops_ref.offsets_of([0] * (E - 2) + counts)
    out = torch.full((sum(counts), N), NAN, device="cuda")
    moe.moe_w4_grouped_gemm(a, codes, s, off, out)
    lo = 0
    for e, c in ((E - 2, counts[0]), (E - 1, counts[1])):
        want = a[lo:lo + c].double() @ ref.weights64(codes[e], s[e]).t().contiguous()
        mag = a[lo:lo + c].double().abs() @ ref.spread64(codes[e], s[e]).t().contiguous()
        close(out[lo:lo + c], want, ops_ref.sum_bound(want, mag, K + 8, F32))
        lo += c


@pytest.mark.parametrize("M,N", [(3, 1 << 20), (1 << 22, 8), (70000, 16384)])
def test_widest_and_tallest(M, N):
    """2^20 columns; 2^22 rows; grids of more than 2^16 workgroups."""
    g, K = gen(M), 64
    codes, s, z = weights(g, 2, N, K, 32, True, BF)
    a = normal(g, M, K)
    out = torch.empty(M, N, device="cuda", dtype=BF)
    moe.moe_w4_grouped_gemm(a, codes, s, ops_ref.offsets_of([M // 3, M - M // 3]), out, zeros=z)
    for e, (lo, hi) in enumerate(((0, M // 3), (M // 3, M))):
        rows = torch.arange(lo, hi, device="cuda")
        rows = rows if M < 100 else torch.cat((rows[:70], rows[-70:]))
        want = a[rows].double() @ ref.weights64(codes[e], s[e], z[e]).t().contiguous()
        mag = a[rows].double().abs() @ ref.spread64(codes[e], s[e], z[e]).t().contiguous()
        close(out[rows], want, ops_ref.sum_bound(want, mag, K + 8, BF))


def test_quantise_past_32_bits():
    """More than 2^31 values, by rows and transposed: the last ones."""
    x = torch.zeros(1100, 1024, 2048, dtype=BF, device="cuda")
    x[-1] = normal(gen(9), 1024, 2048)
    for trans, rows, K in ((False, 1024, 2048), (True, 2048, 1024)):
        codes = torch.empty(1100, rows, K // 2, dtype=U8, device="cuda")
        s = torch.empty(1100, rows, K // 64, dtype=BF, device="cuda")
        moe.moe_w4_quantize(x, codes, s, trans=trans)
        wq, ws, _ = ref.quantise(x[-1].t().contiguous() if trans else x[-1], 64, False, BF)
        assert torch.equal(ref.unpack(codes[-1]), wq) and torch.equal(s[-1], ws)
        assert bool((codes[:-1] == 0x88).all()) and not s[:-1].any()
    out = torch.empty(1100, 2048, 1024, dtype=BF, device="cuda")
    moe.moe_w4_dequantize(codes, s, out)
    assert torch.equal(out[-1].double(), ref.weights64(codes[-1], s[-1]).to(BF).double()) and not out[:-1].any()


def test_streams_and_graphs():
    g = gen(13)
    K, N, counts = 512, 264, [3, 0, 1, 9]
    M, off = sum(counts), ops_ref.offsets_of(counts)
    codes, s, z = weights(g, 4, N, K, 128, True, BF)
    xs = [normal(g, M, K) for _ in range(3)]
    want = []
    for x in xs:
        want.append(torch.empty(M, N, device="cuda"))
        moe.moe_w4_grouped_gemm(x, codes, s, off, want[-1], zeros=z)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [torch.empty(M, N, device="cuda") for _ in xs]
    for x, o, st in zip(xs, got, streams):
        moe.moe_w4_grouped_gemm(x, codes, s, off, o, zeros=z, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, o = xs[0].clone(), torch.empty(M, N, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_w4_grouped_gemm(x, codes, s, off, o, zeros=z)
    for i in (0, 1, 2, 1):
        x.copy_(xs[i])
        graph.replay()
        eager = torch.empty_like(o)
        moe.moe_w4_grouped_gemm(xs[2], codes, s, off, eager, zeros=z)
        torch.cuda.synchronize()
        assert torch.equal(o, want[i]) and torch.equal(eager, want[2])


@pytest.mark.parametrize("per,N", [(1, 136), (20, 136), (300, 136), (2500, 800)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("sdtype", [F32, BF])
def test_largest_scales(per, N, group, sdtype):
    """Scales just below 2^120 with zero points of 255, at which s z is just inside fp32: rows of zeros, and rows whose
    sums over a group vanish, have finite results, the former zeros."""
    g, E, K = gen(group), 2, 384
    M = E * per
    a = normal(g, M, K // 2) * 2.0 ** -20
    a = torch.stack((a, -a), 2).flatten(1).to(BF)
    a[::3] = 0
    codes, s, z = weights(g, E, N, K, group, True, sdtype)
    s.copy_(torch.sign(s.float()) * 2.0 ** 120 * (1 - 2.0 ** -8))
    z[..., ::2] = 255
    check_product(a, [per] * E, codes, s, z, F32, spare=0)
    out = torch.empty(M, N, device="cuda")
    moe.moe_w4_grouped_gemm(a, codes, s, ops_ref.offsets_of([per] * E), out, zeros=z)
    assert out.isfinite().all() and not out[::3].any() and out[1::3].any() == (M > 1)


@pytest.mark.parametrize("K", [7168, 9728, 9760, 11392, 11424, 14336, 16256, 16288, 18944, 18976])
@pytest.mark.parametrize("counts,N", [([1], 136), ([0, 3, 4], 72), ([5, 9], 72), ([16, 0, 1], 264), ([64], 520), ([1] * 9, 4096)])
@pytest.mark.parametrize("sdtype", [F32, BF])
def test_scales_of_long_rows(K, counts, N, sdtype):
    """Depths whose scales and zero points fill LDS beside the streaming form's stages. The last that fit, and the next:
    fp32 scales 9728 with 16 rows to a tile, 11392 with 8; bf16 ones 16256 and 18944."""
    g = gen(K)
    a = normal(g, sum(counts), K)
    codes, s, z = weights(g, len(counts), N, K, 32, True, sdtype)
    check_product(a, counts, codes, s, z, BF, spare=0)
