"""The vocabulary's cross entropy: the kernels that only larger or odder sizes
take, several calls at once, and the losses of a training step together."""
import math

import pytest
import torch

import dense_gemm_swizzled_amd as sg

import _xent_ref as ref
from test_gpu_xent import check, close

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
U = ref.U


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


# Few tokens on 128x128 tiles (the gradient in two parts), then on each tile of
# the gradients' products, split and not, with K and the tokens multiples of 64
# and not.
@pytest.mark.parametrize("M,N,K", [
    (40, 66001, 72), (64, 70016, 64), (1, 66000, 136), (90, 20011, 1032), (64, 9000, 2048),
    (2049, 20000, 1032), (2048, 20032, 1024), (8192, 300, 1032), (8192, 320, 1024),
    (8129, 300, 1160), (3000, 70, 520), (100, 300, 4096), (70, 4099, 4160), (300, 9001, 2304)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_every_kernel(M, N, K, dtype):
    A, B, t = ref.inputs(M, N, K, dtype, M + N + K)
    check(A, B, t)


@pytest.mark.parametrize("M", [1, 33, 64])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_few_tokens_lose_nothing(M, dtype):
    """Up to 64 tokens dA and dB are as near as their own rounding: the gradient
    of the logits is kept to twice as many bits."""
    N, K = 3001, 136
    A, B, t = ref.inputs(M, N, K, dtype, 2 * M, known=0.0, ignored=0.0)
    _, lse = sg.gemm_xent(A, B, t)
    gen = torch.Generator().manual_seed(M)
    dloss = torch.rand(M, generator=gen).cuda() + 0.5
    dA, dB = sg.gemm_xent_backward(dloss, A, B, t, lse)
    half = ref.HALF[dtype]
    ref.HALF[dtype] = half * half       # (two parts: a half step of what is left)
    try:
        wA, wB, bA, bB = ref.backward(dloss, A, B, t, 1.0)
    finally:
        ref.HALF[dtype] = half
    # plus the rounding of the results themselves
    close(dA, wA, bA + half * (wA.abs() + bA), "dA")
    close(dB, wB, bB + half * (wB.abs() + bB), "dB")


@pytest.mark.parametrize("M,N", [(300, 70000), (1000, 5000), (40, 70000)])
def test_no_columns(M, N):
    """K = 0: all logits are zero."""
    A, B = (torch.ones(n, 0, dtype=BF, device="cuda") for n in (M, N))
    t = torch.zeros(M, dtype=torch.int64, device="cuda")
    loss, lse = sg.gemm_xent(A, B, t)
    # log N, the exact sum of N ones, rounded by logf's two steps
    assert bool(((lse.double() - math.log(N)).abs() <= 4 * U * math.log(N)).all())
    assert torch.equal(loss, lse)


@pytest.mark.parametrize("weights", ["one", "mixed", "tiny", "huge", "zero", "dlse only"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_weights_of_any_size(weights, dtype):
    """dloss scales the gradients, whatever its size (fp16 within its range)."""
    M, N, K = 100, 900, 64
    A, B, t = ref.inputs(M, N, K, dtype, 31)
    _, lse = sg.gemm_xent(A, B, t)
    gen = torch.Generator().manual_seed(5)
    d = torch.randn(M, generator=gen).cuda()
    dlse = None
    if weights == "one":
        d = torch.zeros(M, device="cuda")
        d[17] = 3.0
    elif weights == "mixed":
        d = d * 10.0 ** torch.linspace(-6, 2, M).cuda()
    elif weights == "tiny":
        d = d * (1e-4 if dtype is FP else 1e-25)
    elif weights == "huge":
        d = d * (1e2 if dtype is FP else 1e25)
    elif weights == "zero":
        d = torch.zeros(M, device="cuda")
    else:
        d, dlse = torch.zeros(M, device="cuda"), d
    wA, wB, bA, bB = ref.backward(d, A, B, t, 1.0, dlse)
    dA, dB = sg.gemm_xent_backward(d, A, B, t, lse, dlse=dlse)
    close(dA, wA, bA, "dA")
    close(dB, wB, bB, "dB")


@pytest.mark.parametrize("M,N,K", [(50, 300, 64), (150, 9001, 72), (2100, 8200, 192)])
def test_padding_holds_anything(M, N, K):
    """Tokens without a weight have no part in dA, NaN or not; others that are NaN
    have NaN."""
    A, B, t = ref.inputs(M, N, K, BF, 35, ignored=0.0)
    t[::4] = -100
    want, lse0 = sg.gemm_xent(A, B, t)
    d = torch.full((M,), 1.0 / M, device="cuda")
    clean, _ = sg.gemm_xent_backward(d, A, B, t, lse0)
    a = A.clone()
    a[::4] = math.nan
    a[4, :] = math.inf
    loss, lse = sg.gemm_xent(a, B, t)
    assert torch.equal(loss, want)
    dA, none = sg.gemm_xent_backward(d, a, B, t, lse, need=(True, False))
    assert none is None and torch.equal(dA, clean) and bool((dA[::4] == 0).all())
    d[::4] = math.nan                       # (a mean over no tokens)
    dA, _ = sg.gemm_xent_backward(d, a, B, t, lse, need=(True, False))
    assert torch.equal(dA, clean)
    # (the largest weight, which scales the gradients, is not theirs either)
    a[1] = math.nan
    loss, lse = sg.gemm_xent(a, B, t)
    dA, _ = sg.gemm_xent_backward(d, a, B, t, lse, need=(True, False))
    assert bool(torch.isnan(dA[1]).all()) and torch.equal(dA[2:], clean[2:])


@pytest.mark.parametrize("M,N", [(300, 5000), (2049, 20000), (40, 3000)])
def test_padding_of_minus_infinity(M, N):
    """A token without a weight whose logits are all -inf, lse too: its row of dA
    is 0.  One with a weight has NaN."""
    A, B, t = ref.inputs(M, N, 64, BF, M, ignored=0.0)
    B[:, 0] = 1.0
    A[3, 0] = A[4, 0] = -math.inf
    t[3] = -1
    t[4] = 7
    loss, lse = sg.gemm_xent(A, B, t)
    assert bool((lse[3:5] == -math.inf).all()) and float(loss[3]) == 0.0
    d = torch.full((M,), 1.0 / M, device="cuda")
    dA, _ = sg.gemm_xent_backward(d, A, B, t, lse, need=(True, False))
    assert bool((dA[3] == 0).all()) and bool(torch.isnan(dA[4]).all())
    d[4] = 0.0
    dA, _ = sg.gemm_xent_backward(d, A, B, t, lse, need=(True, False))
    assert bool((dA[3:5] == 0).all()) and bool(torch.isfinite(dA).all())


def test_losses_may_be_changed_in_place():
    A, B, t = ref.inputs(50, 300, 64, BF, 32)
    a = A.clone().requires_grad_()
    loss, lse = sg.gemm_xent(a, B, t)
    loss *= 2.0
    (loss.sum() + lse.sum()).backward()
    ones = torch.ones(50, device="cuda")
    _, l0 = sg.gemm_xent(A, B, t)
    assert torch.equal(a.grad, sg.gemm_xent_backward(2 * ones, A, B, t, l0, dlse=ones)[0])


def test_calls_at_the_same_time():
    """Two streams, each with workspaces of its own."""
    cases = [ref.inputs(700, 7001, 136, BF, 33), ref.inputs(60, 9001, 264, FP, 34)]
    one = [torch.full((c[0].shape[0],), 0.01, device="cuda") for c in cases]

    def step(c, d):
        loss, lse = sg.gemm_xent(*c)
        return loss, lse, *sg.gemm_xent_backward(d, *c, lse)

    want = [step(c, d) for c, d in zip(cases, one)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(cases[i], one[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            for a, b in zip(g, want[i]):
                assert torch.equal(a, b)


def test_a_head_of_more_than_2_31_values():
    """Words whose place needs more than 32 bits, dB of as many values."""
    M, N, K = 70, 600011, 4096
    gen = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randn(M, K, generator=gen, device="cuda").to(BF)
    B = torch.empty(N, K, dtype=BF, device="cuda")
    for i in range(0, N, 50000):
        B[i:i + 50000] = (torch.randn(min(50000, N - i), K, generator=gen, device="cuda")
                          * (1.5 / 64)).to(BF)
    assert B.numel() > 2 ** 31
    t = torch.randint(0, N, (M,), generator=gen, device="cuda")
    t[0], t[1], t[2] = 0, N - 1, N
    loss, lse = sg.gemm_xent(A, B, t)
    z = torch.empty(M, N, dtype=torch.float64, device="cuda")
    for i in range(0, N, 50000):
        z[:, i:i + 50000] = A.double() @ B[i:i + 50000].double().t().contiguous()
    want = torch.logsumexp(z, 1)
    ok = ref.has_target(t, N)
    nll = torch.where(ok, want - z.gather(1, torch.where(ok, t, 0)[:, None])[:, 0], 0)
    # dz of _xent_ref with the terms' sum at most |A| |B| by columns
    S = float(A.double().abs().sum(1).max()) * float(B.abs().max())
    tol = (K / 16 + 18) * 4 * U * S + 1e-4
    assert bool(((lse.double() - want).abs() <= tol).all())
    assert bool(((loss.double() - nll).abs() <= 2 * tol).all())
    assert float((lse.double() - want).abs().max()) < 1e-4
    dloss = torch.full((M,), 1.0 / M, device="cuda")
    dA, dB = sg.gemm_xent_backward(dloss, A, B, t, lse)
    g = torch.exp(z - want[:, None]) * (ok / M)[:, None]
    rows = torch.nonzero(ok)[:, 0]
    g[rows, t[ok]] -= 1.0 / M
    pick = torch.cat([torch.tensor([0, 1, N - 2, N - 1], device="cuda"), t[ok],
                      torch.randint(0, N, (500,), generator=gen, device="cuda")])
    half = ref.HALF[BF]
    wB = g[:, pick].t().contiguous() @ A.double()
    aB = g[:, pick].t().abs().contiguous() @ A.double().abs()
    close(dB[pick], wB, half * wB.abs() + (half + 1e-4) * aB, "dB")
    wA = torch.zeros(M, K, dtype=torch.float64, device="cuda")
    aA = torch.zeros_like(wA)
    for i in range(0, N, 50000):
        b = B[i:i + 50000].double()
        wA += g[:, i:i + 50000].contiguous() @ b
        aA += g[:, i:i + 50000].abs().contiguous() @ b.abs()
    # (64-bit sums of N terms err by less than 1e-9 of aA)
    close(dA, wA, half * wA.abs() + (half + 1e-4) * aA, "dA")


def test_the_losses_of_a_training_step():
    """Cross entropy of a mixture's output, a penalty on lse, and the balance of
    the routing: the gradients of the head, of the experts' outputs and of the
    router's logits, against 64 bits with the experts' choice taken as given."""
    T, E, k, H, V = 48, 16, 3, 64, 700
    gen = torch.Generator().manual_seed(41)
    r = torch.randn(T, E, generator=gen).cuda().requires_grad_()
    outs = torch.randn(T, k, H, generator=gen).cuda()
    head = (torch.randn(V, H, generator=gen) * 0.2).to(BF).cuda().requires_grad_()
    t = torch.randint(0, V, (T,), generator=gen).cuda()
    t[5] = -100

    w, ids = sg.moe_route(r, k, score="sigmoid")
    h = (w[:, :, None] * outs).sum(1)
    hb = h.to(BF)
    hb.retain_grad()
    loss, lse = sg.gemm_xent(hb, head, t)
    balance, counts, tokens = sg.moe_balance(r, ids, score="sigmoid")
    total = loss.sum() / T + 1e-3 * (lse ** 2).sum() / T + 0.02 * balance
    total.backward()
    assert int(counts.sum()) == T * k and int(tokens) == T

    # The head and the mixture's output: gemm_xent's own bounds.
    d = torch.full((T,), 1.0 / T, device="cuda")
    dl = (2e-3 / T * lse.detach())
    wA, wB, bA, bB = ref.backward(d, hb.detach(), head.detach(), t, 1.0, dl)
    close(head.grad, wB, bB, "head")
    close(hb.grad, wA, bA, "hidden")
    # The router: the mixture's output gradient (as it came, in bf16) through the
    # weights, and the balance.
    x = r.detach().double().requires_grad_()
    s = torch.sigmoid(x)
    chosen = s.gather(1, ids.long())
    w64 = chosen / chosen.sum(1, keepdim=True)
    share = s / s.sum(1, keepdim=True)
    load = E * counts.double() / counts.sum()
    dh = hb.grad.double()
    value = (w64[:, :, None] * outs.double() * dh[:, None, :]).sum() \
        + 0.02 * (load * share.sum(0) / T).sum()
    value.backward()
    # fp32: dw is a sum of H products (H + 2 units of its terms), the route's
    # gradient another 100 units of dw's terms' size over the weights, the
    # balance's 40 units of its own; added once.
    dw = (outs.double().abs() * dh.abs()[:, None, :]).sum(2).amax(1, keepdim=True)
    bound = (H + 102) * U * dw + 60 * U * 0.02 * load.max() / T
    err = (r.grad.double() - x.grad).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
    assert float(x.grad.abs().max()) > 100 * float(bound.max())
