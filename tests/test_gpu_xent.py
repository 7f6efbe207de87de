"""The vocabulary's cross entropy and its gradients on the GPU, against 64 bits
(_xent_ref.py has the reference and the bounds)."""
import math

import pytest
import torch

import dense_gemm_swizzled_amd as sg

import _xent_ref as ref

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def close(got, want, bound, what):
    err = (got.double() - want).abs()
    assert got.shape == want.shape
    assert bool(torch.isfinite(got.double()).all()), f"{what}: not finite"
    bad = err > bound
    assert not bool(bad.any()), (what, int(bad.sum()), float(err.max()),
                                 float((err / bound.clamp_min(1e-300)).max()))


def check(A, B, t, alpha=1.0, dlse=True, seed=0, **kw):
    loss, lse = sg.gemm_xent(A, B, t, alpha=alpha)
    want = ref.forward(A, B, t, alpha)
    close(loss, want[0], want[2], "loss")
    close(lse, want[1], want[3], "lse")
    M = A.shape[0]
    gen = torch.Generator().manual_seed(seed + 77)
    dloss = (torch.randn(M, generator=gen) / max(M, 1)).cuda()
    dl = (0.1 * torch.randn(M, generator=gen) / max(M, 1)).cuda() if dlse else None
    dA, dB = sg.gemm_xent_backward(dloss, A, B, t, lse, alpha=alpha, dlse=dl, **kw)
    wA, wB, bA, bB = ref.backward(dloss, A, B, t, alpha, dl)
    if dA is not None:
        close(dA, wA, bA, "dA")
    if dB is not None:
        close(dB, wB, bB, "dB")
    return loss, lse, dA, dB


# Every kernel: tiles of 64, 128 and 256, with M, N and K that end inside a
# tile, a fragment, a chunk and a K tile.
SIZES = [
    (1, 1, 8), (1, 7, 8), (2, 64, 64), (3, 65, 72), (4, 1000, 128), (17, 129, 40),
    (64, 513, 256), (65, 257, 200), (63, 4099, 136), (127, 2049, 64), (130, 8190, 320),
    (333, 5003, 72), (500, 4097, 264), (1021, 1023, 104), (1025, 2563, 136), (700, 7001, 64),
    (2048, 3001, 8), (2000, 8200, 192), (4099, 4100, 200), (4096, 4096, 128),
]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_sizes(M, N, K, dtype):
    A, B, t = ref.inputs(M, N, K, dtype, M + N + K)
    check(A, B, t)


@pytest.mark.parametrize("alpha", [0.5, -1.0, 3.0, 0.0])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_scaled_logits(alpha, dtype):
    A, B, t = ref.inputs(70, 1001, 96, dtype, 5, alpha=alpha)
    check(A, B, t, alpha=alpha)


@pytest.mark.parametrize("M,N,K", [(300, 600, 72), (4100, 4099, 136)])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_rows_of_any_pitch(M, N, K, kind):
    A, B, t = ref.inputs(M, N, K, BF, 9)
    wa = torch.full((M, K + 24), math.nan, dtype=BF, device="cuda")
    wb = torch.full((N, K + 8), math.nan, dtype=BF, device="cuda")
    wa[:, 8:K + 8], wb[:, :K] = A, B
    want = check(A, B, t)
    da = torch.full((M, K + 16), 7.0, dtype=BF, device="cuda")
    db = torch.full((N, K + 40), 7.0, dtype=BF, device="cuda")
    got = check(wa[:, 8:K + 8], wb[:, :K], t.to(kind), out=(da[:, 8:K + 8], db[:, 16:K + 16]))
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert bool((da[:, :8] == 7).all() and (da[:, K + 8:] == 7).all())
    assert bool((db[:, :16] == 7).all() and (db[:, K + 16:] == 7).all())


def test_runs_of_words():
    """A gradient of the logits beyond 512 MB goes in runs of words, the last
    ending inside a K tile; dA is summed over the runs."""
    M, N, K = 5000, 100003, 72
    assert sg.gemm_xent_backward_workspace_bytes(M, N, K, K) < 2 * M * N
    A, B, t = ref.inputs(M, N, K, BF, 3)
    check(A, B, t)


def test_runs_of_words_in_fp16_and_one_side_at_a_time():
    M, N, K = 6000, 50001, 64
    A, B, t = ref.inputs(M, N, K, FP, 4)
    _, _, dA, dB = check(A, B, t, dlse=False)
    for need in ((True, False), (False, True), (False, False)):
        _, _, a, b = check(A, B, t, dlse=False, need=need)
        assert (a is not None) == need[0] and (b is not None) == need[1]
        assert a is None or torch.equal(a, dA)
        assert b is None or torch.equal(b, dB)


@pytest.mark.parametrize("M,N,K", [(0, 50, 16), (5, 0, 16), (5, 50, 0), (0, 0, 0), (300, 0, 64)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_empty(M, N, K, dtype):
    A = torch.ones(M, K, dtype=dtype, device="cuda")
    B = torch.ones(N, K, dtype=dtype, device="cuda")
    t = torch.zeros(M, dtype=torch.int64, device="cuda")
    loss, lse = sg.gemm_xent(A, B, t)
    assert loss.shape == lse.shape == (M,)
    if N == 0:
        assert bool((loss == 0).all()) and bool((lse == -math.inf).all())
    elif K == 0:
        assert bool(((lse - math.log(N)).abs() < 1e-6).all()) and torch.equal(loss, lse)
    out = (torch.full((M, K), 7.0, dtype=dtype, device="cuda"),
           torch.full((N, K), 7.0, dtype=dtype, device="cuda"))
    dA, dB = sg.gemm_xent_backward(torch.ones(M, device="cuda"), A, B, t, lse, out=out)
    assert dA is out[0] and dB is out[1]
    assert bool((dA == 0).all()) and bool((dB == 0).all())


@pytest.mark.parametrize("M,N,K", [(40, 300, 64), (700, 7001, 64)])
@pytest.mark.parametrize("bad", [-1, -100, "N", 2 ** 40, -2 ** 40, 2 ** 31])
def test_tokens_without_a_target(M, N, K, bad):
    A, B, t = ref.inputs(M, N, K, BF, 6, ignored=0.0)
    t[::3] = N if bad == "N" else bad
    loss, lse, _, _ = check(A, B, t)
    assert bool((loss[::3] == 0).all())
    t[:] = -100
    _, _, dA, dB = check(A, B, t, dlse=False)
    assert bool((dA == 0).all()) and bool((dB == 0).all())


def test_every_target_column():
    """A target in every column of the first and the last tile."""
    for M, N, K in ((300, 256 + 129, 64), (769, 4096 + 257, 64)):
        A, B, _ = ref.inputs(M, N, K, BF, 8)
        for first in (0, N - M if N > M else 0):
            t = (torch.arange(M, device="cuda") + first) % N
            check(A, B, t)


@pytest.mark.parametrize("dtype,size", [(BF, 300.0), (FP, 60.0)])
def test_large_logits(dtype, size):
    """Logits of thousands: the exponentials of all but a few underflow."""
    A, B, t = ref.inputs(90, 700, 64, dtype, 11, known=0.0)
    check((A.float() * size).to(dtype), B, t)
    z = torch.zeros(90, 64, dtype=dtype, device="cuda")
    check(z, B, t)                                           # all equal
    check((A.float() * size).to(dtype), (B[:1].float() * 0 + 1).to(dtype).expand(700, 64)
          .contiguous(), t)


@pytest.mark.parametrize("M,N,K", [(70, 500, 64), (700, 7001, 64)])
def test_infinities_and_nan(M, N, K):
    A, B, t = ref.inputs(M, N, K, BF, 12, ignored=0.0)
    want, want_lse = sg.gemm_xent(A, B, t)
    a = A.clone()
    a[5] = math.nan
    a[6, 0] = math.inf
    b = B.clone()
    b[:, 0] = 1.0       # row 6: every logit is +inf
    loss, lse = sg.gemm_xent(a, b, t)
    assert bool(torch.isnan(loss[5:7]).all()) and bool(torch.isnan(lse[5:7]).all())
    clean, clean_lse = sg.gemm_xent(A, b, t)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[5:7] = False
    assert torch.equal(loss[keep], clean[keep]) and torch.equal(lse[keep], clean_lse[keep])
    # A word of logit -inf: probability 0, an infinite loss where it is the target.
    b = B.clone()
    b[9] = 0.0
    b[9, 0] = -math.inf
    a = A.clone()
    a[:, 0] = a[:, 0].abs() + 0.1
    t = torch.where(t == 9, 10, t)
    t[0] = 9
    loss, lse = sg.gemm_xent(a, b, t)
    z = a.double() @ b.double().t().contiguous()
    assert float(loss[0]) == math.inf
    assert bool(((lse.double() - torch.logsumexp(z, 1)).abs() < 1e-4).all())
    # All logits -inf.
    b = torch.zeros_like(B)
    b[:, 0] = -math.inf
    t[1] = -1
    loss, lse = sg.gemm_xent(a, b, t)
    assert bool((lse == -math.inf).all())
    assert float(loss[1]) == 0.0 and bool(torch.isnan(loss[0]))


def test_the_same_result_every_time():
    for M, N, K in ((4, 9001, 128), (700, 7001, 64), (4099, 4100, 200)):
        A, B, t = ref.inputs(M, N, K, BF, 13)
        first = check(A, B, t)
        work = torch.full((max(sg.gemm_xent_workspace_bytes(M, N, K),
                               sg.gemm_xent_backward_workspace_bytes(M, N, K, K)) + 64,), 255,
                          dtype=torch.uint8, device="cuda")
        out = torch.empty(2, M, device="cuda").unbind(0)
        loss, lse = sg.gemm_xent(A, B, t, out=out, workspace=work)
        assert loss is out[0] and torch.equal(loss, first[0]) and torch.equal(lse, first[1])
        work.fill_(255)
        gen = torch.Generator().manual_seed(77)
        dloss = (torch.randn(M, generator=gen) / M).cuda()
        dl = (0.1 * torch.randn(M, generator=gen) / M).cuda()
        dA, dB = sg.gemm_xent_backward(dloss, A, B, t, lse, dlse=dl, workspace=work)
        assert torch.equal(dA, first[2]) and torch.equal(dB, first[3])


def test_gradients_against_differences():
    """The loss changes along a direction by what the gradients say."""
    A, B, t = ref.inputs(50, 333, 64, FP, 14)
    gen = torch.Generator().manual_seed(3)
    c = torch.rand(50, generator=gen).cuda()
    z = (0.2 * torch.rand(50, generator=gen)).cuda()
    _, lse = sg.gemm_xent(A, B, t)
    dA, dB = sg.gemm_xent_backward(c, A, B, t, lse, dlse=z)
    vA, vB = (torch.randn(x.shape, generator=gen).cuda() * x.std() for x in (A, B))

    def value(h):   # 64 bits, by the definition
        x = (A.double() + h * vA.double()) @ (B.double() + h * vB.double()).t().contiguous()
        l = torch.logsumexp(x, 1)
        ok = ref.has_target(t, 333)
        nll = torch.where(ok, l - x.gather(1, torch.where(ok, t, 0)[:, None])[:, 0], 0)
        return float((c * nll + z * l).sum())
    h = 1e-5
    slope = (value(h) - value(-h)) / (2 * h)
    got = float((dA.double() * vA).sum() + (dB.double() * vB).sum())
    _, _, bA, bB = ref.backward(c, A, B, t, 1.0, z)
    # The differences err by h^2 of the third derivative: 1e-10 of the terms' size.
    tol = float((bA * vA.abs()).sum() + (bB * vB.abs()).sum()) + 1e-6 * abs(slope) + 1e-6
    assert abs(got - slope) <= tol
    # (The bound means something: it is small beside the terms of the slope.)
    assert tol < 0.05 * float((dA.double() * vA).abs().sum() + (dB.double() * vB).abs().sum())


def test_autograd():
    A, B, t = ref.inputs(90, 700, 64, BF, 15)
    a, b = A.clone().requires_grad_(), B.clone().requires_grad_()
    loss, lse = sg.gemm_xent(a, b, t, alpha=0.5)
    want, want_lse = sg.gemm_xent(A, B, t, alpha=0.5)
    assert torch.equal(loss, want) and torch.equal(lse, want_lse)
    n = 90
    (loss.sum() / n + 1e-2 * (lse * lse).sum() / n).backward()
    one = torch.full((n,), 1.0, device="cuda") / n
    dlse = torch.autograd.grad(1e-2 * (want_lse.requires_grad_() ** 2).sum() / n, want_lse)[0]
    dA, dB = sg.gemm_xent_backward(one, A, B, t, want_lse.detach(), alpha=0.5, dlse=dlse)
    assert torch.equal(a.grad, dA) and torch.equal(b.grad, dB)
    # One side frozen, the loss alone, lse alone.
    loss, _ = sg.gemm_xent(a.detach(), b, t)
    (db,) = torch.autograd.grad(loss.sum(), b)
    _, l0 = sg.gemm_xent(A, B, t)
    ones, none = torch.ones(n, device="cuda"), torch.zeros(n, device="cuda")
    assert torch.equal(db, sg.gemm_xent_backward(ones, A, B, t, l0)[1])
    _, lse = sg.gemm_xent(a, b.detach(), t)
    (da,) = torch.autograd.grad(lse.sum(), a)
    assert torch.equal(da, sg.gemm_xent_backward(none, A, B, t, l0, dlse=ones)[0])
    with torch.no_grad():
        assert not sg.gemm_xent(a, b, t)[0].requires_grad
    out = torch.empty(2, n, device="cuda").unbind(0)
    assert not sg.gemm_xent(a, b, t, out=out)[0].requires_grad
    loss, _ = sg.gemm_xent(a, b, t)
    (da,) = torch.autograd.grad(loss, a, ones, create_graph=True)
    with pytest.raises(RuntimeError):
        da.sum().backward()


def test_changed_operands_are_noticed():
    A, B, t = ref.inputs(9, 70, 64, BF, 16)
    leaf = A.requires_grad_()
    x = leaf * 1.0
    loss, _ = sg.gemm_xent(x, B, t)
    with torch.no_grad():
        x.zero_()
    with pytest.raises(RuntimeError, match="modified"):
        torch.autograd.grad(loss.sum(), leaf)


def test_on_a_side_stream():
    A, B, t = ref.inputs(300, 5003, 136, BF, 17)
    want = sg.gemm_xent(A, B, t)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = sg.gemm_xent(A, B, t)
        grads = sg.gemm_xent_backward(torch.ones(300, device="cuda"), A, B, t, got[1])
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for a, b in zip(grads, sg.gemm_xent_backward(torch.ones(300, device="cuda"), A, B, t,
                                                 want[1])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("M,N,K,dtype", [(40, 3001, 64, BF), (700, 7001, 136, FP)])
def test_in_a_graph(M, N, K, dtype):
    A, B, t = ref.inputs(M, N, K, dtype, 18)
    a, b = A.clone().requires_grad_(), B.clone().requires_grad_()
    one = torch.full((M,), 1.0 / M, device="cuda")

    def step():     # (no graph of the leaves outlives it)
        loss, lse = sg.gemm_xent(a, b, t)
        return (loss.detach(), lse.detach(),
                *torch.autograd.grad((loss, lse), (a, b), (one, 0.01 * one)))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        with torch.no_grad():
            x, y, s = ref.inputs(M, N, K, dtype, 20 + i)
            a.copy_(x), b.copy_(y), t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        now = [x.detach().clone() for x in got]
        for x, y in zip(now, step()):
            assert torch.equal(x, y)
