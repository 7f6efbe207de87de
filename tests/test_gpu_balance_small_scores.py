"""The balance of sigmoid scores that fp32 does not hold: a token whose logits are
all far below zero still has shares of its scores, as long as their sum is not
below 2^-126, and falling ones from there on.  Bounds as in test_gpu_balance.py
(there for logits of up to 88 in size; the largest here, 104, weighs 60 u where
88 is given 4 * 90: each share is made from differences to the row's largest
logit and from 2^(-126 - top log2 e), whose argument is off by 24 u and by top
times the constant's rounding)."""
import math

import pytest
import torch

import dense_gemm_swizzled_amd as sg

from test_gpu_balance import HALF, TINY, U, check, shares

pytestmark = pytest.mark.gpu
F32, BF, FP = torch.float32, torch.bfloat16, torch.float16


def rows(T, E, dtype, seed):
    """Rows around -55 to -108, among them ordinary, masked and dead ones, rows
    whose largest logit stands far above the others, and halves of a row masked."""
    gen = torch.Generator().manual_seed(seed)
    mid = -55 - 53 * torch.rand(T, 1, generator=gen)
    x = mid + torch.randn(T, E, generator=gen)
    kind = torch.randint(0, 12, (T, 1), generator=gen)
    x = torch.where(kind == 0, torch.randn(T, E, generator=gen), x)
    x = torch.where(kind == 1, -math.inf, x)
    x = torch.where((kind == 2) & (torch.arange(E) % 2 == 1), math.nan, x)
    x = torch.where((kind == 3) & (torch.arange(E) == seed % E), x + 30, x)
    x = torch.where(kind == 4, x - 1000, x)
    return x.to(dtype).cuda()


def gradient(x, counts, n, dloss):
    """By automatic differentiation of the definition in 64 bits."""
    E = x.shape[1]
    y = torch.where(torch.isnan(x), -math.inf, x).double().requires_grad_()
    s = torch.sigmoid(y)
    total = s.sum(1, keepdim=True)
    # (at the floor itself the derivative jumps: no row may lie on it)
    near = (torch.log2(total.detach().clamp_min(1e-300)) + 126).abs()
    assert float(near.min()) > 1e-3
    share = s / total.clamp_min(2.0 ** -126)
    coef = dloss * E * counts.double() / (float(counts.sum()) * n)
    (share * coef).sum().backward()
    p = share.detach()
    scale = coef.abs() + (p * coef.abs()).sum(1, keepdim=True)
    return y.grad.nan_to_num(0.0), p, scale


@pytest.mark.parametrize("T,E", [(37, 16), (300, 16), (700, 40), (900, 100), (1000, 200),
                                 (5000, 256), (130, 3), (40, 1)])
@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_scores_that_underflow(T, E, dtype):
    x = rows(T, E, dtype, T + E)
    ids = (torch.arange(T, device="cuda") * 3 % E).to(torch.int32)[:, None].contiguous()
    _, counts, tokens = check(x, ids, "sigmoid")
    n = int(tokens)
    dloss = 100.0 * T
    got = sg.moe_balance_backward(torch.tensor(dloss, device="cuda"), x, counts, tokens,
                                  score="sigmoid")
    want, p, scale = gradient(x, counts, n, dloss)
    rel = shares(x, "sigmoid")[4]
    bound = (rel + (p * rel).sum(1, keepdim=True) + (12 + math.log2(E)) * U) * p * scale
    bound = bound + 2.0 ** -96 * scale
    bound = bound + HALF[dtype] * (want.abs() + bound) + TINY[dtype]
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((err <= bound).all()), (float(err.max()), float((err / bound).max()))
    far = (x.float().nan_to_num(-math.inf).amax(1) < -89) & (p.amax(1) > 1e-3)
    assert T < 100 or int(far.sum()) > 5      # (rows whose scores fp32 does not hold)


@pytest.mark.parametrize("at", [-60.0, -86.5, -87.5, -88.5, -91.0])
def test_an_even_load_of_small_scores(at):
    """Equal logits, however small: every share is 1/E, the loss 1."""
    E = 256
    x = torch.full((640, E), at, device="cuda")
    ids = (torch.arange(640 * 4, device="cuda") % E).to(torch.int32).reshape(640, 4)
    loss, counts, tokens = sg.moe_balance(x, ids, score="sigmoid")
    assert abs(float(loss) - 1) < 1e-5 and int(tokens) == 640


def test_in_a_graph_with_padding():
    """Padding among small scores, replayed among eager work of other data."""
    x = rows(2000, 72, BF, 1)
    ids = (torch.arange(4000, device="cuda") % 72).to(torch.int32).reshape(2000, 2)
    d = torch.ones((), device="cuda")

    def step():
        loss, counts, tokens = sg.moe_balance(x, ids, score="sigmoid")
        return loss, sg.moe_balance_backward(d, x, counts, tokens, score="sigmoid")

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        x.copy_(rows(2000, 72, BF, 30 + i))
        graph.replay()
        torch.cuda.synchronize()
        now = [t.clone() for t in got]
        for a, b in zip(now, step()):
            assert torch.equal(a, b)
