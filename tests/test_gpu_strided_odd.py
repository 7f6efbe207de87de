"""gemm_strided with an MN-major A of an odd number of columns: the last value of
its last row sits alone in a 32-bit word."""
import pytest
import torch

import dense_gemm_swizzled_amd as sg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(1, 8, 1), (33, 64, 3), (129, 136, 70), (2049, 2048, 128),
                                   (4097, 4096, 192)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_odd_columns(M, N, K, dtype):
    gen = torch.Generator().manual_seed(M)
    lda = -(-M // 8) * 8
    A = torch.zeros(K, lda)
    A[:, :M] = torch.randn(K, M, generator=gen)
    B = torch.randn(K, N, generator=gen)
    A, B = A.to(dtype).cuda(), B.to(dtype).cuda()
    D = sg.gemm_strided(A[:, :M], B, a_major="mn", b_major="mn", out_dtype=torch.float32)
    a, b = A[:, :M].double().t().contiguous(), B.double()
    want = a @ b
    # exact products, at most K roundings of 2^-23 (truncation) of the sum's terms
    bound = (K + 2) * 2.0 ** -23 * (a.abs() @ b.abs())
    assert bool(((D.double() - want).abs() <= bound).all())
