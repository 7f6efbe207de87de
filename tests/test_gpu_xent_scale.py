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
