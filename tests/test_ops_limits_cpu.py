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
