"""Grouped MXFP4 products whose rows have whole 16-byte groups of scales (their tiles load 32 bytes of scales a row),
and depths around the one whose scales no longer fit beside the streaming kernels' rings."""
import random

import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref as ref
from tests.test_gpu_ops import BF, F32, NAN, close, gen, index_for, normal, quantised

pytestmark = pytest.mark.gpu

# last tiles of at most 64, 128, 192 and 256 rows; 143 row by column tiles at least, so that the tiles run
COUNTS, N = [1, 64, 65, 128, 0, 129, 192, 193, 256, 257, 300, 700], 2824


# 480 and 992 end in a byte of padding; a chunk of scales is 1024 deep: half of one, one, one and a half, two, two
# and a half, five
@pytest.mark.parametrize("K", [480, 512, 992, 1024, 1536, 2048, 2560, 5120])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_whole_groups_of_scales(K, gather, out_dtype):
    S = moe.moe_mxfp4_scale_stride(K)
    assert S % 16 == 0
    rng, g, E, used = random.Random(K), gen(K), len(COUNTS), sum(COUNTS)
    M, div = used + 5, 3
    rows = 401 if gather else M
    x = normal(g, rows, K) * torch.exp2(torch.randint(-6, 7, (rows, K // 32), generator=g, device="cuda")).repeat_interleave(32, 1)
    w = normal(g, E * N, K, scale=K ** -0.5) * torch.exp2(torch.randint(-3, 4, (E * N, K // 32), generator=g, device="cuda")).repeat_interleave(32, 1)
    (ca, sa), (cw, sw) = quantised(x), quantised(w)
    sa[:, K // 32:], sw[:, K // 32:] = 255, 255  # padding holds no scale
    (ca, _), (sa, _) = ref.guarded(ca, 16, 0x77), ref.guarded(sa, 16, 255)
    (cw, _), (sw, _) = ref.guarded(cw.view(E, N, -1), 16, 0x77), ref.guarded(sw.view(E, N, -1), 16, 255)
    idx = index_for(rng, M, rows, div, True) if gather else None
    if not gather:
        sa[used:] = 255
    sw[COUNTS.index(0)] = 255
    off = ref.offsets_of(COUNTS)
    out, big = ref.guarded(torch.full((M, N), 7.0, device="cuda", dtype=out_dtype), 16, 7.0)
    moe.moe_mxfp4_grouped_gemm(ca, sa, cw, sw, off, out, row_index=idx, row_div=div)
    a64, w64 = ref.mx_decode64(ca, sa), ref.mx_decode64(cw, sw)
    want, mag = ref.product64(ref.gather64(a64, used, idx[:used] if gather else None, div), w64, COUNTS, True)
    close(out[:used], want, ref.sum_bound(want, mag, K, out_dtype))
    assert bool((out[used:] == 7.0).all()) and ref.guards_intact(big, 16, 7.0)
    # a NaN block in one row and in one column stays there
    row, col = 400, 1000
    if not gather:
        sa[row, K // 32 - 1] = 255
    sw[5, col, 0] = 255
    again = torch.full_like(out, 7.0)
    moe.moe_mxfp4_grouped_gemm(ca, sa, cw, sw, off, again, row_index=idx, row_div=div)
    bad = torch.zeros_like(out, dtype=torch.bool)
    lo = sum(COUNTS[:5])
    bad[lo:lo + COUNTS[5], col] = True
    if not gather:
        bad[row] = True
    assert torch.equal(again.isnan(), bad) and torch.equal(again[~bad], out[~bad])


@pytest.mark.parametrize("K", [13312, 13344, 13440, 13824, 16384])
@pytest.mark.parametrize("counts", [[3, 0, 2], [40, 60], [0, 300, 1]])
def test_depths_around_the_streaming_limit(K, counts):
    """13312 is the last depth whose 96 rows of scales take at most 40 KB of LDS; from 13344 on the tiles take few rows
    too, with dwords of scales (13344, 13440) and with whole groups (13824, 16384)."""
    g, E, n, M = gen(K), len(counts), 72, sum(counts)
    ca, sa = quantised(normal(g, M, K))
    cw, sw = quantised(normal(g, E, n, K, scale=K ** -0.5))
    out = torch.full((M, n), NAN, device="cuda")
    moe.moe_mxfp4_grouped_gemm(ca, sa, cw, sw, ref.offsets_of(counts), out)
    want, mag = ref.product64(ref.mx_decode64(ca, sa), ref.mx_decode64(cw, sw), counts, True)
    close(out, want, ref.sum_bound(want, mag, K, F32))
