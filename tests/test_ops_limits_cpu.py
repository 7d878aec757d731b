"""Row limits of the grouped products, on the host. A null or misaligned output is refused after the sizes, so
INVALID_ARGUMENT says that the sizes were taken, and no accepted call is ever enqueued."""
import pytest

import sparse_moe_layer_gemm_amd as moe

INVAL, UNSUP = 1, 2
A, B, C = (i << 48 for i in range(1, 4))


def gemm(M, K, N, E, dt=1):
    return moe.load_library().moe_grouped_gemm(A, dt, M, None, 1, B, 0, M, K, N, E, C, dt, None, None)


def wgrad(M, K, N, E, dt=1):
    return moe.load_library().moe_grouped_wgrad(A, dt, M, None, 1, B, M, K, N, E, C, 0, 0, None, None)


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("M,K,N,E", [(1 << 28, 8, 8, 256), (3_500_000, 1536, 5120, 64), ((1 << 29) - 1, 8, 64, 1),
                                     (1 << 20, 5120, 1 << 14, 1)])
def test_weight_gradient_takes_any_rows(M, K, N, E, dt):
    """Its grid goes by dw's tiles: rows only lengthen the sums."""
    assert wgrad(M, K, N, E, dt) == INVAL
    assert wgrad(1 << 29, K, N, E, dt) == UNSUP


@pytest.mark.parametrize("M,N,E,want", [
    # (M / 16 + min(E, M)) * ceil(N / 64) against 2^24 - 64
    ((1 << 28) - 66 * 16, 64, 1, INVAL), ((1 << 28) - 65 * 16, 64, 1, UNSUP),
    ((1 << 28) - 321 * 16, 64, 256, INVAL), ((1 << 28) - 320 * 16, 64, 256, UNSUP), (1, 1 << 20, 256, INVAL)])
def test_product_row_limit(M, N, E, want):
    assert gemm(M, 8, N, E) == want


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("M,I,want", [((1 << 31) - 1, 8, INVAL), (1 << 31, 8, UNSUP), (1, 1 << 30, INVAL),
                                      (1, (1 << 30) + 8, UNSUP), ((1 << 27) - 8, 256, INVAL), ((1 << 27) - 1, 256, UNSUP),
                                      ((1 << 24) - 1, 2048, INVAL), (1 << 24, 2048, UNSUP)])
def test_swiglu_limits(M, I, want, bwd):
    """M * I up to 2^35 - 2^11."""
    f = moe.load_library()
    assert (f.moe_swiglu_backward(None, B, 1, M, I, C, None, None) if bwd else f.moe_swiglu(None, 1, M, I, B, None)) == want


@pytest.mark.parametrize("trans,Bn,R,C,want", [
    (0, 1, (1 << 24) - 1, 2048, INVAL), (0, 1, 1 << 24, 2048, UNSUP), (0, 4, 1 << 22, 2048, UNSUP),
    (0, 1, 1, 1 << 30, INVAL), (0, 1, 1, (1 << 30) + 32, UNSUP),
    # B * ceil(K / 256) * ceil(C / 128) below 2^23
    (1, (1 << 23) - 1, 32, 8, INVAL), (1, 1 << 23, 32, 8, UNSUP), (1, 1 << 10, 256 * 128, 128 * 64, UNSUP),
    (1, (1 << 10) - 1, 256 * 128, 128 * 64, INVAL), (1, 1, 1 << 30, 8, INVAL), (1, 1, (1 << 30) + 32, 8, UNSUP)])
def test_quantise_limits(trans, Bn, R, C, want):
    assert moe.load_library().moe_mxfp4_quantize(None, 1, trans, Bn, R, C, A, B, None) == want


@pytest.mark.parametrize("R,K,want", [((1 << 24) - 1, 2048, INVAL), (1 << 24, 2048, UNSUP), (1, (1 << 31) - 32, INVAL)])
def test_dequantise_limits(R, K, want):
    assert moe.load_library().moe_mxfp4_dequantize(None, B, R, K, 1, C, None) == want
