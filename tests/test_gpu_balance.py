"""The routing's balance loss and its gradient on the GPU, against 64 bits.

u = 2^-24.  A score is off by a few u: softmax by u |x - top| log2 e for the
rounded difference and product (at most 3u (1 + |x - top|), which weighs e^-|x -
top|: 4u of the row's sum) and u of 2^x; sigmoid by |x| u of
e^-x (its argument's rounding is half a step of |x| log2 e, 2^a changes by ln 2 a
unit of a: |x| u), then 4u (2^x, a sum, a reciprocal of one step, a product).  A
row's sum of E adds log2 E u.  So a share is off by at most rel = (4 * (2 +
spread) + log2 E + 4) u of itself, where spread is the largest |x - top| (|x| for
sigmoid, up to 88 where scores underflow), and 2^-126 where a result
underflows."""
import math

import pytest
import torch

import dense_gemm_swizzled_amd as sg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}
F32, BF, FP = torch.float32, torch.bfloat16, torch.float16


def inputs(T, E, k, dtype, seed, dead=0.1, masked=0.05, size=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = size * (torch.randn(T, E, generator=gen) + 0.5 * torch.randn(1, E, generator=gen))
    if masked:
        x[torch.rand(T, E, generator=gen) < masked] = -math.inf
    if dead:
        x[torch.rand(T, generator=gen) < dead] = -math.inf
    x = x.to(dtype).cuda()
    ids = sg.moe_route(x, k)[1]
    return x, ids


def shares(x, score):
    """(live tokens, scores, shares, each share's relative error), float64."""
    x = x.double()
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=3.4028234663852886e38)
    on = x > -math.inf
    live = on.any(1)
    if score == "softmax":
        top = torch.where(live, x.amax(1), 0)[:, None]
        s = torch.where(on, torch.exp(x - top), 0)
        spread = torch.where(on, top - x, 0).clamp(max=104.0)
    else:
        s = torch.where(on, torch.sigmoid(x), 0)
        spread = torch.where(on, x.abs(), 0).clamp(max=88.0)
    total = s.sum(1, keepdim=True).clamp_min(2.0 ** -126)
    rel = (4 * (2 + spread) + math.log2(x.shape[1]) + 4 + 12) * U
    return live, s, total, s / total, rel


def reference(x, ids, score):
    E = x.shape[1]
    live, _, _, p, rel = shares(x, score)
    flat = ids.reshape(-1).long()
    counts = torch.bincount(flat[(flat >= 0) & (flat < E)], minlength=E)
    n, c = int(live.sum()), int(counts.sum())
    if n == 0 or c == 0:
        return 0.0, counts, n, 0.0
    load = E * counts.double() / c
    loss = float((load * p.sum(0)).sum() / n)
    # A lane adds a token at a time: T / (256 * 64) of them and at least 4, then
    # 64 lanes' and 256 workgroups' sums.
    depth = x.shape[0] / (256 * 64) + 4 + 8 + 16 + 64 + 4
    bound = float((load * (p * rel).sum(0)).sum() / n) + (depth + 2) * U * loss + 1e-37
    return loss, counts, n, bound


def check(x, ids, score):
    loss, counts, tokens = sg.moe_balance(x, ids, score=score)
    want, want_counts, n, bound = reference(x, ids, score)
    assert loss.shape == tokens.shape == () and loss.dtype is torch.float32
    assert torch.equal(counts.long(), want_counts) and int(tokens) == n
    assert abs(float(loss) - want) <= bound, (float(loss), want, bound)
    return loss, counts, tokens


def check_grad(x, counts, tokens, score, dloss=0.37, **kw):
    d = torch.tensor(dloss, device="cuda")
    got = sg.moe_balance_backward(d, x, counts, tokens, score=score, **kw)
    E = x.shape[1]
    _, s, total, p, rel = shares(x, score)
    c, n = float(counts.sum()), int(tokens)
    coef = torch.zeros(E, dtype=torch.float64, device="cuda")
    if c > 0 and n > 0:
        coef = float(d) * E * counts.double() / (c * n)
    dot = (p * coef).sum(1, keepdim=True)
    rest = 1 - s if score == "sigmoid" else torch.ones_like(s)
    if score == "sigmoid":
        xd = torch.where(torch.isnan(x.double()), -math.inf, x.double())
        rest = torch.sigmoid(-xd)
    want = p * rest * (coef - dot)
    # The share, 1 - s (4u), the coefficients and their mean (4u and E terms).
    size = p * rest * (coef.abs() + (p * coef.abs()).sum(1, keepdim=True))
    bound = (rel + (p * rel).sum(1, keepdim=True) + (12 + math.log2(E)) * U) * size
    bound = bound + HALF[x.dtype] * (want.abs() + bound) + TINY[x.dtype]
    assert got.shape == x.shape and got.dtype is x.dtype
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (float(err.max()), float((err / bound).max()))
    return got


# Every kernel (8, 16 lanes with 1, 2, 4 quads), one workgroup and several, with
# experts and tokens that end inside a quad, a wave's tokens and a chunk.
SIZES = [(1, 1, 1), (1, 8, 2), (3, 7, 7), (37, 64, 4), (64, 32, 8), (65, 33, 3), (256, 256, 8),
         (257, 256, 8), (300, 200, 5), (1000, 97, 2), (4097, 128, 8), (5000, 31, 4),
         (16385, 129, 6), (20011, 65, 32), (33000, 12, 1)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sizes(T, E, k, dtype, score):
    x, ids = inputs(T, E, k, dtype, T + E)
    _, counts, tokens = check(x, ids, score)
    check_grad(x, counts, tokens, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [30.0, 1000.0])
def test_large_logits(score, size):
    x, ids = inputs(400, 40, 4, F32, 3, size=size)
    _, counts, tokens = check(x, ids, score)
    check_grad(x, counts, tokens, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_masks(score, dtype):
    x, ids = inputs(300, 24, 3, dtype, 4, dead=0.0, masked=0.0)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, 3:] = -math.inf
    x[3, :20] = math.nan
    x[4] = math.inf
    x[5, 7] = math.inf
    x[6] = torch.finfo(dtype).min
    x[7] = torch.finfo(dtype).max
    x[8, 1:] = torch.finfo(dtype).min
    ids[10] = -1
    ids[11] = 24
    ids[12] = 2 ** 31 - 1
    ids[13] = -2 ** 31
    ids[14] = 5                       # the same expert three times counts three times
    _, counts, tokens = check(x, ids, score)
    assert int(tokens) == 298 and int(counts.sum()) == 296 * 3
    dx = check_grad(x, counts, tokens, score)
    off = ~(x > -math.inf)
    assert bool((dx[off] == 0).all())


@pytest.mark.parametrize("T", [0, 5, 700])
def test_nothing_to_balance(T):
    x = torch.full((T, 16), -math.inf, device="cuda")
    ids = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    loss, counts, tokens = check(x, ids, "softmax")
    assert float(loss) == 0 and int(tokens) == 0
    assert bool((check_grad(x, counts, tokens, "softmax") == 0).all())
    x, _ = inputs(max(T, 1), 16, 2, F32, 0, dead=0.0)
    ids = torch.full((max(T, 1), 2), -1, dtype=torch.int32, device="cuda")
    loss, counts, tokens = check(x, ids, "sigmoid")
    assert float(loss) == 0 and bool((counts == 0).all())
    assert bool((check_grad(x, counts, tokens, "sigmoid") == 0).all())


def test_even_and_one_sided_loads():
    x = torch.zeros(640, 64, device="cuda")
    ids = (torch.arange(640 * 4, device="cuda") % 64).to(torch.int32).reshape(640, 4)
    loss, counts, _ = check(x, ids, "softmax")
    assert abs(float(loss) - 1) < 1e-5 and bool((counts == 40).all())
    x[:, 5] = 60.0
    loss, _, _ = check(x, torch.full_like(ids, 5), "softmax")
    assert abs(float(loss) - 64) < 1e-3


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_rows_of_any_pitch(dtype, score):
    x, ids = inputs(500, 50, 4, dtype, 6)
    loss, counts, tokens = check(x, ids, score)
    dx = check_grad(x, counts, tokens, score)
    for pad, at in ((14, 0), (13, 7), (3, 1)):
        wide = torch.full((500, 50 + pad), 9.0, dtype=dtype, device="cuda")
        wide[:, at:at + 50] = x
        view = wide[:, at:at + 50]
        for a, b in zip(sg.moe_balance(view, ids, score=score), (loss, counts, tokens)):
            assert torch.equal(a, b)
        out = torch.full((500, 50 + pad), 9.0, dtype=dtype, device="cuda")
        got = check_grad(view, counts, tokens, score, out=out[:, at:at + 50])
        assert torch.equal(got, dx)
        assert bool((out[:, :at] == 9).all()) and bool((out[:, at + 50:] == 9).all())


def test_written_outputs_and_workspace():
    x, ids = inputs(3000, 100, 4, BF, 7)
    want = check(x, ids, "softmax")
    work = torch.full((sg.moe_balance_workspace_bytes(3000, 100),), 255, dtype=torch.uint8,
                      device="cuda")
    out = (torch.empty((), device="cuda"), torch.empty(100, dtype=torch.int32, device="cuda"),
           torch.empty((), dtype=torch.int32, device="cuda"))
    for _ in range(3):
        got = sg.moe_balance(x, ids, out=out, workspace=work)
        assert all(a is b for a, b in zip(got, out))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_autograd_and_several_calls():
    x, ids = inputs(900, 40, 4, F32, 8)
    leaf = x.clone().requires_grad_()
    loss, counts, tokens = sg.moe_balance(leaf, ids, score="sigmoid")
    want = sg.moe_balance(x, ids, score="sigmoid")
    assert all(torch.equal(a, b) for a, b in zip((loss, counts, tokens), want))
    assert loss.requires_grad and not counts.requires_grad and not tokens.requires_grad
    (0.01 * loss).backward()
    d = torch.tensor(0.01, device="cuda")
    assert torch.equal(leaf.grad, sg.moe_balance_backward(d, x, counts, tokens, score="sigmoid"))
    with torch.no_grad():
        assert not sg.moe_balance(leaf, ids)[0].requires_grad
    # The counts of two halves added up: the gradient of the whole.
    a, b = (sg.moe_balance(x[i], ids[i], score="sigmoid") for i in (slice(0, 450),
                                                                   slice(450, 900)))
    c, n = a[1] + b[1], a[2] + b[2]
    assert torch.equal(c, counts) and torch.equal(n, tokens)
    half = sg.moe_balance_backward(d, x[450:], c, n, score="sigmoid")
    assert torch.equal(half, leaf.grad[450:])


def test_gradient_against_differences():
    x, ids = inputs(60, 24, 3, F32, 9, masked=0.0)
    gen = torch.Generator().manual_seed(1)
    v = torch.randn(60, 24, generator=gen).cuda()
    for score in ("softmax", "sigmoid"):
        _, counts, tokens = sg.moe_balance(x, ids, score=score)
        dx = check_grad(x, counts, tokens, score, dloss=1.0)
        live = torch.isfinite(x).all(1)

        def value(h):
            return reference((x.double() + h * v.double())[live], ids[live], score)[0]
        h = 1e-4
        slope = (value(h) - value(-h)) / (2 * h)
        got = float((dx.double()[live] * v.double()[live]).sum())
        terms = float((dx.double()[live] * v.double()[live]).abs().sum())
        # h^2 of the third derivative, and 64-bit sums divided by h
        assert abs(got - slope) <= (1e-6 + h * h) * terms + 1e-10


def test_in_a_graph_and_on_a_side_stream():
    x, ids = inputs(2000, 72, 4, BF, 10)
    leaf = x.clone().requires_grad_()

    def step():     # (no graph of the leaf outlives it)
        loss, counts, tokens = sg.moe_balance(leaf, ids)
        return loss.detach(), counts, tokens, torch.autograd.grad(loss, leaf)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, step()):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        with torch.no_grad():
            y, j = inputs(2000, 72, 4, BF, 20 + i)
            leaf.copy_(y), ids.copy_(j)
        graph.replay()
        torch.cuda.synchronize()
        now = [t.detach().clone() for t in got]
        for a, b in zip(now, step()):
            assert torch.equal(a, b)


def test_more_than_2_31_logits():
    T, E, k = (1 << 23) + 77, 256, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.empty(T, E, dtype=BF, device="cuda")
    step = 1 << 20
    for i in range(0, T, step):
        n = min(step, T - i)
        x[i:i + n] = torch.randn(n, E, generator=gen, device="cuda").to(BF)
    assert x.numel() > 2 ** 31
    x[:, 7] += 1.0
    x[T - 3] = -math.inf
    ids = torch.randint(0, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    ids[T - 3] = -1
    loss, counts, tokens = sg.moe_balance(x, ids)
    flat = ids.reshape(-1).long()
    assert torch.equal(counts.long(), torch.bincount(flat[flat >= 0], minlength=E))
    assert int(tokens) == T - 1
    total = torch.zeros(E, dtype=torch.float64, device="cuda")
    for i in range(0, T, step):
        y = x[i:i + step].double()
        total += torch.softmax(y[y[:, 0] > -math.inf], 1).sum(0)
    load = E * counts.double() / counts.sum()
    want = float((load * total).sum() / (T - 1))
    # A lane adds T / (256 * 16) tokens one after another, half a step of the sum
    # so far each time: at most T / 4096 / 2 steps of the sum; shares by 1e-5.
    assert abs(float(loss) - want) <= (T / 8192 * 2 * U + 1e-5) * want
    d = torch.tensor(float(T), device="cuda")
    dx = sg.moe_balance_backward(d, x, counts, tokens)
    for rows in (slice(0, 50), slice(T - 50, T), slice(T // 2, T // 2 + 50)):
        y = x[rows].double()
        p = torch.where(y > -math.inf, torch.softmax(y, 1), 0).nan_to_num(0.0)
        coef = T * load / (T - 1)
        dot = (p * coef).sum(1, keepdim=True)
        exact = p * (coef - dot)
        size = p * (coef + dot)
        assert bool(((dx[rows].double() - exact).abs()
                     <= HALF[BF] * exact.abs() + 1e-5 * size + 1e-30).all())
    torch.cuda.empty_cache()
