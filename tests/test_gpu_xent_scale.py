"""The scale of the cross entropy's gradient terms at the ends of its range: up to
64 tokens, more, and beyond 8192, which find the largest weight each in their own
way."""
import math

import pytest
import torch

import dense_gemm_swizzled_amd as sg

import _xent_ref as ref
from test_gpu_xent import close

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("M", [40, 300, 9000])
@pytest.mark.parametrize("w,alpha", [
    (2.0 ** -116, 2.0 ** 30), (2.0 ** -120, 2.0 ** 30), (2.0 ** -130, 2.0 ** 40),
    (2.0 ** -126, 1.0), (2.0 ** -102, 1.0), (2.0 ** -60, 2.0 ** -40), (2.0 ** 60, 2.0 ** 30)])
@pytest.mark.parametrize("only", ["loss", "lse"])
def test_weights_and_factors_far_from_one(M, w, alpha, only):
    """Small weights, whose reciprocal fp32 does not hold, under a large factor of
    the logits (and the other way round)."""
    A, B, t = ref.inputs(M, 300, 64, BF, 3, alpha=alpha, known=0.0)
    _, lse = sg.gemm_xent(A, B, t, alpha=alpha)
    gen = torch.Generator().manual_seed(M)
    d = (torch.randn(M, generator=gen) * w).cuda()
    dlse = None
    if only == "lse":
        d, dlse = torch.zeros_like(d), d
    dA, dB = sg.gemm_xent_backward(d, A, B, t, lse, alpha=alpha, dlse=dlse)
    wA, wB, bA, bB = ref.backward(d, A, B, t, alpha, dlse)
    close(dA, wA, bA, "dA")
    close(dB, wB, bB, "dB")


@pytest.mark.parametrize("M", [40, 300, 9000])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", ["dloss", "dlse"])
def test_a_weight_that_is_no_number(M, dtype, bad, where):
    """One token's weight is infinite or NaN: its own row of dA is no number, and
    the other rows are what they are without it."""
    A, B, t = ref.inputs(M, 900, 64, dtype, 3, ignored=0.0)
    _, lse = sg.gemm_xent(A, B, t)
    d = torch.full((M,), 1e-4, device="cuda")
    z = torch.full((M,), 1e-5, device="cuda")
    want, _, bound, _ = ref.backward(d, A, B, t, 1.0, z)
    (d if where == "dloss" else z)[3] = bad
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[3] = False
    dA, _ = sg.gemm_xent_backward(d, A, B, t, lse, dlse=z, need=(True, False))
    close(dA[keep], want[keep], bound[keep], "dA")
    assert not bool(torch.isfinite(dA[3]).any())
