"""Weight gradients over more rows than a product's grid could hold."""
import pytest
import torch

import sparse_moe_layer_gemm_amd as moe
from tests import ops_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wgrad_of_2_28_rows(dtype):
    """256 experts, uneven, 2^28 + 5 rows in all; values -1, 0 and 1, so that every sum is a whole number below 2^24 and
    exact in fp32."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    E, K, N, M = 256, 8, 8, (1 << 28) + 5
    counts = [1 << 20] * E
    counts[3], counts[4], counts[255] = 0, (1 << 21) + 1, (1 << 20) + 4
    assert sum(counts) == M
    a, d = (torch.randint(-1, 2, (M, n), generator=g, device="cuda", dtype=torch.int8).to(dtype) for n in (K, N))
    dw = torch.full((E, K, N), float("nan"), device="cuda")
    moe.moe_grouped_wgrad(a, d, ref.offsets_of(counts), dw)
    lo = 0
    for e, c in enumerate(counts):
        want = (a[lo:lo + c, :, None].double() * d[lo:lo + c, None, :].double()).sum(0)
        assert torch.equal(dw[e].double(), want), e
        lo += c
