"""The cross entropy's gradients on paths that only many tokens or several runs of
words take: beyond 8192 tokens a launch of its own looks for the largest weight;
up to 64 tokens the scale and the second copy of A are made in the first run only
and dA is summed over the runs (tests/plans/xent_plans.cpp has their plans)."""
import math

import pytest
import torch

import dense_gemm_swizzled_amd as sg

import _xent_ref as ref
from test_gpu_xent import close

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def check_back(d, A, B, t, dlse=None, need=(True, True)):
    loss, lse = sg.gemm_xent(A, B, t)
    want = ref.forward(A, B, t, 1.0)
    close(loss, want[0], want[2], "loss")
    close(lse, want[1], want[3], "lse")
    wA, wB, bA, bB = ref.backward(d, A, B, t, 1.0, dlse)
    dA, dB = sg.gemm_xent_backward(d, A, B, t, lse, dlse=dlse, need=need)
    assert (dA is not None) == need[0] and (dB is not None) == need[1]
    if need[0]:
        close(dA, wA, bA, "dA")
    if need[1]:
        close(dB, wB, bB, "dB")
    return dA, dB


# 8193: a token alone in the last workgroup.  262144 + 1500: more than 256
# workgroups' worth, which go on to their next tokens.
@pytest.mark.parametrize("M,N,K", [(8193, 70, 72), (9500, 300, 64), (262144 + 1500, 9, 8)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_more_than_8192_tokens(M, N, K, dtype):
    A, B, t = ref.inputs(M, N, K, dtype, M)
    gen = torch.Generator().manual_seed(M)
    d = (torch.randn(M, generator=gen) * 10.0 ** torch.linspace(-4, 0, M)).cuda()
    dlse = (0.1 * torch.randn(M, generator=gen)).cuda()
    check_back(d, A, B, t)
    check_back(d, A, B, t, dlse)
    check_back(torch.zeros(M, device="cuda"), A, B, t, dlse)
    check_back(torch.zeros(M, device="cuda"), A, B, t)


@pytest.mark.parametrize("M", [8193, 262144 + 1500])
@pytest.mark.parametrize("at", ["first", "second", "last"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_the_largest_weight_anywhere(M, at, dtype):
    """One weight is 2^15 times the others: in fp16 the gradient of its token
    overflows unless it sets the scale."""
    N, K = 9, 8
    A, B, t = ref.inputs(M, N, K, dtype, 3, ignored=0.0)
    i = {"first": 0, "second": M // 2 + 300, "last": M - 1}[at]
    d = torch.full((M,), 2.0 ** -10, device="cuda")
    d[i] = 2.0 ** 5
    dA, dB = check_back(d, A, B, t)
    assert float(dA[i].abs().max()) > 1.0
    d[i] = 2.0 ** -10
    dlse = d.clone()
    dlse[i] = -2.0 ** 5
    check_back(d, A, B, t, dlse)


@pytest.mark.parametrize("M", [1, 33, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_few_tokens_in_several_runs(M, dtype):
    """Rows of B a mebibyte apart: seven runs of 1792 words, the last of one word."""
    N, K, ldb = 10753, 136, 1 << 19
    A, B, t = ref.inputs(M, N, K, dtype, M, ignored=0.0)
    t[0] = N - 1
    t[-1] = N - 1 if M == 1 else 1792
    wide = torch.full((N, ldb), math.nan, dtype=dtype, device="cuda")
    wide[:, :K] = B
    view = wide[:, :K]
    assert view.stride(0) == ldb
    gen = torch.Generator().manual_seed(M)
    d = (torch.randn(M, generator=gen) + 2).cuda()
    dlse = (0.1 * torch.randn(M, generator=gen)).cuda()
    both = check_back(d, A, view, t, dlse)
    one = check_back(d, A, view, t, dlse, need=(True, False))
    two = check_back(d, A, view, t, dlse, need=(False, True))
    assert torch.equal(one[0], both[0]) and torch.equal(two[1], both[1])
    check_back(d, A, view, t)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_more_words_than_a_run_may_have(dtype):
    """More than 2^22 words at a time would make the pitch of the logits' gradient
    wrap the 32-bit offsets of dB's tiles."""
    M, N, K = 3, (1 << 22) + 5003, 8
    A, B, t = ref.inputs(M, N, K, dtype, 1, ignored=0.0)
    t[0], t[1], t[2] = 0, N - 1, 1 << 22
    check_back(torch.tensor([1.0, -2.0, 0.5], device="cuda"), A, B, t)


@pytest.mark.parametrize("alpha", [-1.0, 0.5, 0.0])
@pytest.mark.parametrize("M,N,K", [(40, 3001, 72), (4100, 4099, 64)])
def test_scaled_logits_of_few_and_of_many_tokens(alpha, M, N, K):
    """64x64 tiles with the gradient in two parts, and 256x256 tiles."""
    A, B, t = ref.inputs(M, N, K, BF, 5, alpha=alpha)
    loss, lse = sg.gemm_xent(A, B, t.to(torch.int32), alpha=alpha)
    want = ref.forward(A, B, t, alpha)
    close(loss, want[0], want[2], "loss")
    close(lse, want[1], want[3], "lse")
    gen = torch.Generator().manual_seed(1)
    d, dlse = (torch.randn(M, generator=gen).cuda() for _ in range(2))
    dA, dB = sg.gemm_xent_backward(d, A, B, t.to(torch.int32), lse, alpha=alpha, dlse=dlse)
    wA, wB, bA, bB = ref.backward(d, A, B, t, alpha, dlse)
    close(dA, wA, bA, "dA")
    close(dB, wB, bB, "dB")


def pitched(x, pitch, fill):
    wide = torch.full((x.shape[0], pitch), fill, dtype=x.dtype, device="cuda")
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


@pytest.mark.parametrize("M,N,K", [(40, 600, 72), (200, 600, 72), (250, 70000, 64)])
def test_the_widest_pitches(M, N, K):
    """A's rows eight mebibytes apart (a panel of 256 of them just below 2^31 bytes),
    B's too where they are few; gradients whose places need more than 32 bits."""
    A, B, t = ref.inputs(M, N, K, BF, 6)
    a = pitched(A, (1 << 22) - 8, math.nan)
    b = pitched(B, (1 << 22) - 8, math.nan) if N < 1000 else B
    loss, lse = sg.gemm_xent(a, b, t)
    want = ref.forward(A, B, t, 1.0)
    close(loss, want[0], want[2], "loss")
    close(lse, want[1], want[3], "lse")
    d = torch.rand(M, generator=torch.Generator().manual_seed(2)).cuda() / M
    zero_A, zero_B = torch.zeros_like(A), torch.zeros_like(B)
    out = pitched(zero_A, 1 << 24, 7.0) if M > 200 else zero_A, \
        pitched(zero_B, 1 << 22, 7.0) if N < 1000 else zero_B
    dA, dB = sg.gemm_xent_backward(d, a, b, t, lse, out=out)
    wA, wB, bA, bB = ref.backward(d, A, B, t, 1.0)
    close(dA, wA, bA, "dA")
    close(dB, wB, bB, "dB")
    # (what lies between the rows is left as it was)
    base = dA._base if M > 200 else None
    assert base is None or bool((base[:, K:K + 64] == 7).all())
