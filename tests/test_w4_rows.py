"""The product's rows do not depend on one another: a row computed alone, or
among others of the same kernel form, is the same to the bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K,N", [(2000, 555), (130, 4096), (8192, 64)])
@pytest.mark.parametrize("few,many", [(1, 2), (3, 8), (9, 16), (17, 32)])
def test_a_row_alone_and_among_others(libgemm, kind, K, N, few, many):
    from accelerator_gb300 import lowbit
    W = lowbit.w4_quantize(torch.randn(K, N, device="cuda"), 64)
    X = torch.randn(many, K, device="cuda").to(kind)
    all_rows = lowbit.gemm_w4(X, W, dtype=torch.float32)
    assert torch.equal(lowbit.gemm_w4(X[:few].contiguous(), W, dtype=torch.float32), all_rows[:few])
    assert torch.equal(lowbit.gemm_w4(X[-few:].contiguous(), W, dtype=torch.float32), all_rows[-few:])
    assert libgemm.debug_status() == libgemm.OK
