"""Expert routing on the GPU: the choice and its weights, their gradient and
the plan against 64-bit references, and the operators together as a layer."""
import math

import numpy as np
import pytest
import torch

import dense_gemm_swizzled_amd as sg

pytestmark = pytest.mark.gpu

TINY = 2.0 ** -126
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
# Relative error of a weight in fp32, in units of 2^-24, for logits within 20
# of the row's largest: the rounded difference in the exponent (20), expf (4),
# the sum over the experts (10), the division (1): 35; the sum of the chosen
# carries the same error and adds 10; division and scale add 2.  82 in all.
W_TOL = 82 * 2.0 ** -24


def scores64(x, score):
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, np.finfo(np.float32).max))
    live = x > -np.inf
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        if score == "sigmoid":
            return np.where(live, np.where(x < 0, np.exp(np.minimum(x, 0)), 1.0) /
                            (1 + np.exp(-np.abs(x))), 0.0), live
        m = x.max(1, keepdims=True)
        e = np.where(live, np.exp(np.where(live, x - m, -np.inf)), 0.0)
        return e / np.maximum(e.sum(1, keepdims=True), TINY), live


def route_reference(x, k, score="softmax", bias=None, n_groups=1, top_groups=None,
                    group_score="max", renorm=True, scale=1.0):
    """Token by token, in 64 bits."""
    x = x.double().numpy()
    T, E = x.shape
    top_groups = n_groups if top_groups is None else top_groups
    s, live = scores64(x, score)
    choose = n_groups > 1 and top_groups < n_groups
    if bias is None and not (choose and group_score == "top2"):
        key = np.where(live, np.minimum(x, np.finfo(np.float32).max), -np.inf)
    else:
        key = s + (0.0 if bias is None else bias.double().numpy())
    key = np.where(live & (key > -np.inf), key, -np.inf)
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        kt = key[t].copy()
        if choose:
            g = kt.reshape(n_groups, -1)
            top = np.sort(g, 1)[:, ::-1]
            gs = top[:, 0].copy()
            if group_score == "top2" and g.shape[1] > 1:
                gs += np.where(top[:, 1] > -np.inf, top[:, 1], 0)
            order = sorted(range(n_groups), key=lambda i: (-gs[i], i))
            for i in order[top_groups:]:
                g[i] = -np.inf
        order = sorted((e for e in range(E) if kt[e] > -np.inf), key=lambda e: (-kt[e], e))[:k]
        ids[t, :len(order)] = order
        w[t, :len(order)] = s[t, order]
    if renorm:
        w = w / np.maximum(w.sum(1, keepdims=True), TINY)
    return w * scale, ids


def check_route(x, k, **kw):
    rw, rid = route_reference(x, k, **kw)
    kw = dict(kw)
    if kw.get("bias") is not None:
        kw["bias"] = kw["bias"].cuda()
    w, ids = sg.moe_route(x.cuda(), k, **kw)
    assert np.array_equal(ids.cpu().numpy(), rid)
    err = np.abs(w.cpu().double().numpy() - rw)
    # Weights with renorm add up to the scale, unless the scores' sum is below
    # 2^-126 and is divided by that instead: the scores are then denormals,
    # 2^-149 apart, and expf's 2 units and half a unit of the division are
    # 2.5 * 2^-149 / 2^-126 < 2^-21 in the weight.
    scale = kw.get("scale", 1.0)
    floored = kw.get("renorm", True) & (rw.sum(1, keepdims=True) < 0.99 * scale)
    lim = W_TOL * rw + np.where(floored, scale * 2.0 ** -21, 0.0)
    assert bool((err <= lim).all()), (err - lim).max()
    return w, ids


def logits(rng, T, E, dtype, spread=2.0):
    return torch.from_numpy((spread * rng.standard_normal((T, E))).astype(np.float32)
                            .clip(-9, 9)).to(dtype)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 8), (65, 20, 3), (7, 32, 5), (33, 33, 4),
                                   (50, 60, 6), (40, 64, 1), (31, 100, 8), (9, 128, 12),
                                   (5, 129, 32), (70, 160, 6), (41, 256, 8), (3, 256, 32)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route(T, E, k, dtype, score):
    rng = np.random.default_rng(T * E + k)
    x = logits(rng, T, E, dtype)
    check_route(x, k, score=score)
    check_route(x, k, score=score, renorm=False, scale=2.5)
    bias = torch.from_numpy((0.2 * rng.standard_normal(E)).astype(np.float32))
    check_route(x, k, score=score, bias=bias)


@pytest.mark.parametrize("E,n_groups,top_groups,k", [(16, 4, 2, 3), (64, 8, 3, 8), (60, 5, 2, 7),
                                                     (256, 8, 4, 8), (96, 32, 5, 6), (32, 32, 4, 4),
                                                     (128, 2, 1, 4), (24, 3, 3, 5)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_groups(E, n_groups, top_groups, k, group_score, with_bias):
    rng = np.random.default_rng(E + n_groups)
    for score, dtype in (("sigmoid", torch.float32), ("softmax", torch.bfloat16)):
        x = logits(rng, 37, E, dtype)
        x[3] = -math.inf
        x[5, : E // 2] = -math.inf
        bias = torch.from_numpy((0.2 * rng.standard_normal(E)).astype(np.float32))
        check_route(x, k, score=score, bias=bias if with_bias else None, n_groups=n_groups,
                    top_groups=top_groups, group_score=group_score)


@pytest.mark.parametrize("E", [8, 60, 200])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lowest_index(E, with_bias):
    rng = np.random.default_rng(E)
    x = torch.from_numpy(rng.integers(-1, 2, (64, E)).astype(np.float32)).to(torch.bfloat16)
    x[0] = 0.5
    bias = torch.zeros(E) if with_bias else None
    _, ids = check_route(x, 8, score="sigmoid", bias=bias)
    assert ids[0].tolist() == list(range(8))
    groups = 4
    check_route(x, 2, score="softmax", bias=bias, n_groups=groups, top_groups=2,
                group_score="top2")


@pytest.mark.parametrize("E", [12, 64, 250])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_and_extreme_logits(E, score, with_bias):
    rng = np.random.default_rng(E)
    k = 6
    low = float(torch.finfo(torch.bfloat16).min)
    x = logits(rng, 12, E, torch.bfloat16)
    x[0] = -math.inf                        # a padding token
    x[1] = math.nan
    x[2, 4:] = -math.inf                    # fewer experts left than top_k
    x[3, ::2] = math.nan
    x[4, 3] = math.inf
    x[5, 2], x[5, 7] = math.inf, math.inf
    x[6] = low                              # the type's lowest value is no mask
    x[7, 2:] = low
    x[8] = 80.0
    bias = None
    if with_bias:
        bias = torch.from_numpy((0.1 * rng.standard_normal(E)).astype(np.float32))
        bias[1], bias[6] = -math.inf, math.nan
    w, ids = check_route(x, k, score=score, bias=bias)
    assert bool((ids[:2] == -1).all()) and bool((w[:2] == 0).all())
    assert bool(torch.isfinite(w).all())


def test_close_scores_are_ordered_in_64_bits():
    """Keys that fp32 cannot tell apart: a bias of steps of 2^-30 over equal
    scores near one half, in shuffled order."""
    rng = np.random.default_rng(2)
    E = 128
    steps = rng.permutation(E).astype(np.float32)
    bias = torch.from_numpy(steps * np.float32(2.0 ** -30))
    x = torch.zeros(5, E)
    check_route(x, 16, score="sigmoid", bias=bias)


def test_small_sigmoid_scores_keep_their_ratios():
    x = torch.full((2, 16), -70.0)
    x[0, 3], x[0, 9] = -69.0, -69.5
    check_route(x, 4, score="sigmoid")
    x = torch.full((1, 16), -95.0)          # sums below 2^-126
    w, _ = check_route(x, 4, score="sigmoid")
    assert bool((w < 1e-2).all())


def test_route_of_strided_logits_into_buffers():
    rng = np.random.default_rng(4)
    wide = logits(rng, 20, 90, torch.float16).cuda()
    x = wide[2:18, 5:69]
    w = torch.full((18, 4), 9.0, device="cuda")
    ids = torch.full((18, 4), 9, dtype=torch.int32, device="cuda")
    sg.moe_route(x, 4, out=(w[1:17], ids[1:17]))
    rw, rid = route_reference(x.cpu(), 4)
    assert np.array_equal(ids[1:17].cpu().numpy(), rid)
    assert bool((w[[0, 17]] == 9).all()) and bool((ids[[0, 17]] == 9).all())


# -------------------------------------------------------------------- the gradient

def weights64(x, ids, score, renorm, scale):
    s, _ = scores64(x, score)
    w = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), 1), 0.0)
    if renorm:
        w = w / np.maximum(w.sum(1, keepdims=True), TINY)
    return w * scale


def grad_reference(x, ids, g, score, renorm, scale):
    s, live = scores64(x, score)
    in_ = (ids >= 0) & (ids < x.shape[1])
    sel = np.where(in_, np.take_along_axis(s, np.where(in_, ids, 0), 1), 0.0)
    g = np.where(in_, g * scale, 0.0)
    tot = np.maximum(sel.sum(1, keepdims=True), TINY)
    d = (g - (g * sel).sum(1, keepdims=True) / tot) / tot if renorm else g
    full = np.zeros_like(s)
    for t in range(len(s)):
        np.add.at(full[t], np.where(in_[t], ids[t], 0), np.where(in_[t], d[t], 0.0))
    if score == "sigmoid":
        return np.where(live, full * s * (1 - s), 0.0)
    return np.where(live, s * (full - (full * s).sum(1, keepdims=True)), 0.0)


def check_grad(x, ids, g, dtype, **kw):
    dx = sg.moe_route_backward(g.cuda(), x.cuda(), ids.cuda(), **kw)
    ref = grad_reference(x.double().numpy(), ids.numpy(), g.double().numpy(), kw["score"],
                         kw["renorm"], kw["scale"])
    assert dx.dtype == dtype
    err = np.abs(dx.cpu().double().numpy() - ref)
    # Scores and ratios are 82 units of 2^-24 off as in the forward pass; a
    # gradient is a difference of terms of at most max|g| scale (times the
    # score's own size), the mean of g over up to 32 terms adds 32 units and
    # the last steps 8: 122 in all, twice over for the two terms; then the
    # rounding to the logits' type.
    top = np.abs(g.double().numpy()).max(1, keepdims=True) * kw["scale"]
    lim = 2 * 122 * 2.0 ** -24 * top + HALF[dtype] * np.abs(ref) + 2.0 ** -25
    assert bool((err <= lim).all()), (err - lim).max()
    return dx, ref


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 8), (65, 20, 3), (33, 64, 4), (31, 100, 8),
                                   (5, 129, 32), (41, 256, 8)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward(T, E, k, dtype, score, renorm):
    rng = np.random.default_rng(T * E + k)
    x = logits(rng, T, E, dtype, 1.5)
    _, ids = sg.moe_route(x.cuda(), k, score=score)
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    check_grad(x, ids.cpu(), g, dtype, score=score, renorm=renorm, scale=1.0)
    check_grad(x, ids.cpu(), g, dtype, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward_against_differences(score, renorm):
    rng = np.random.default_rng(9)
    T, E, k, h = 6, 24, 5, 1e-5
    x = logits(rng, T, E, torch.float32)
    _, ids = sg.moe_route(x.cuda(), k, score=score)
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    dx, _ = check_grad(x, ids.cpu(), g, torch.float32, score=score, renorm=renorm, scale=1.5)
    x64, i64, g64 = x.double().numpy(), ids.cpu().numpy(), g.double().numpy()
    for e in range(E):
        up, dn = x64.copy(), x64.copy()
        up[:, e] += h
        dn[:, e] -= h
        d = ((weights64(up, i64, score, renorm, 1.5) - weights64(dn, i64, score, renorm, 1.5))
             * g64).sum(1) / (2 * h)
        # the difference quotient's error: h^2 times a third derivative of at
        # most about 10 g, and 1e-16 / h of rounding; then the fp32 bound
        lim = 1e-9 * 10 + 1e-10 + 2 * 122 * 2.0 ** -24 * np.abs(g64).max(1) * 1.5
        assert bool((np.abs(dx[:, e].cpu().double().numpy() - d) <= lim).all())


def test_route_backward_of_masked_and_repeated_ids():
    rng = np.random.default_rng(10)
    x = logits(rng, 8, 40, torch.float32)
    x[0] = -math.inf
    x[1, 10:] = -math.inf
    x[2, 5] = math.nan
    ids = torch.from_numpy(rng.integers(0, 10, (8, 6)).astype(np.int32))
    ids[0] = -1
    ids[1, 3:] = -1
    ids[2] = torch.tensor([1, 1, 2, 2, 2, 3])          # named more than once
    ids[3] = torch.tensor([1, 40, 2, 2 ** 31 - 1, -2 ** 31, 3])   # outside the experts
    g = torch.from_numpy(rng.standard_normal((8, 6)).astype(np.float32))
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            dx, _ = check_grad(x, ids, g, torch.float32, score=score, renorm=renorm, scale=1.0)
            assert bool((dx[0] == 0).all()) and bool((dx[1, 10:] == 0).all())
            assert dx[2, 5] == 0 and bool(torch.isfinite(dx).all())


def test_route_backward_strided():
    rng = np.random.default_rng(12)
    wide = logits(rng, 9, 50, torch.bfloat16).cuda()
    x = wide[1:8, 3:35]
    _, ids = sg.moe_route(x, 3)
    g = torch.from_numpy(rng.standard_normal((7, 3)).astype(np.float32)).cuda()
    buf = torch.full((9, 60), 5.0, dtype=torch.bfloat16, device="cuda")
    sg.moe_route_backward(g, x, ids, out=buf[1:8, 7:39])
    assert torch.equal(buf[1:8, 7:39], sg.moe_route_backward(g, x.contiguous(), ids))
    buf[1:8, 7:39] = 5.0
    assert bool((buf == 5.0).all())


# Every split of a token's experts over lanes, on both sides of each change,
# with a last block that is part full and experts that are not whole quads.
# The sums of a row's scores take 10 roundings in every split (3 in a quad, the
# quads, the lanes), as the bound of check_grad counts.
@pytest.mark.parametrize("T,E,k,split", [
    (16383, 61, 4, "16,1"), (16389, 64, 4, "8,2"), (8191, 128, 8, "32,1"),
    (8197, 125, 8, "16,2"), (32767, 66, 3, "16,2"), (32773, 101, 8, "8,4"),
    (32771, 128, 32, "8,4"), (4095, 256, 8, "64,1"), (4097, 250, 8, "32,2"),
    (16383, 131, 2, "32,2"), (16387, 256, 8, "16,4"), (16385, 139, 19, "16,4"),
    (40001, 32, 6, "8,1")])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_of_many_tokens(T, E, k, split, score):
    rng = np.random.default_rng(T + E)
    dtype = DTYPES[(T + E) % 3]
    x = logits(rng, T, E, dtype, 1.5)
    x[5] = -math.inf
    x[T - 1, 1:] = -math.inf
    x[::7, E - 1] = math.nan
    _, ids = sg.moe_route(x.cuda(), k, score=score)
    ids = ids.cpu()
    ids[3, :2] = E - 2                                # one expert twice
    ids[9, 0], ids[10, 1] = E, -2 ** 31               # outside the experts
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    for renorm in (True, False):
        dx, _ = check_grad(x, ids, g, dtype, score=score, renorm=renorm, scale=1.5)
        assert sg.gemm_last_kernel().endswith(split + ">"), sg.gemm_last_kernel()
        assert bool((dx[5] == 0).all()) and bool(torch.isfinite(dx).all())
    # strided rows that no vector fits, with what lies between them kept
    wide = torch.full((T, E + 3), 7.0, dtype=dtype, device="cuda")
    odd = torch.zeros(T, E + 1, dtype=dtype, device="cuda")
    odd[:, 1:] = x.cuda()
    sg.moe_route_backward(g.cuda(), odd[:, 1:], ids.cuda(), score=score, renorm=False, scale=1.5,
                          out=wide[:, 1:E + 1])
    assert torch.equal(wide[:, 1:E + 1], dx)
    assert bool((wide[:, 0] == 7).all()) and bool((wide[:, E + 1:] == 7).all())


def test_no_tokens():
    x = torch.zeros(0, 8, device="cuda")
    w, ids = sg.moe_route(x, 2)
    assert w.shape == ids.shape == (0, 2)
    assert sg.moe_route_backward(w, x, ids).shape == (0, 8)


def test_routing_on_another_stream():
    rng = np.random.default_rng(14)
    x = logits(rng, 300, 64, torch.float32).cuda()
    want = sg.moe_route(x, 6, score="sigmoid")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w, ids = sg.moe_route(x, 6, score="sigmoid")
        plan = sg.moe_plan(ids, 64)
        dx = sg.moe_route_backward(w, x, ids, score="sigmoid")
    side.synchronize()
    assert torch.equal(w, want[0]) and torch.equal(ids, want[1])
    for a, b in zip(plan, sg.moe_plan(want[1], 64)):
        assert torch.equal(a, b)
    assert torch.equal(dx, sg.moe_route_backward(want[0], x, want[1], score="sigmoid"))


# ------------------------------------------------------------------------ the plan

def plan_reference(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    key = np.where(ok, flat, E)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(E + 1))
    rows = np.where(key[order] < E, order // k, -1)
    slots = np.empty(T * k, np.int64)
    slots[order] = np.arange(T * k)
    return offsets, rows, np.where(ok, slots, -1).reshape(T, k)


def check_plan(ids, E, **kw):
    got = sg.moe_plan(ids.cuda(), E, **kw)
    for a, b in zip(got, plan_reference(ids.numpy().astype(np.int64), E)):
        assert a.dtype == torch.int32
        assert np.array_equal(a.cpu().numpy(), b)
    return got


@pytest.mark.parametrize("T,k,E", [(0, 1, 4), (1, 1, 1), (1, 8, 8), (63, 1, 5), (64, 1, 2),
                                   (65, 1, 256), (100, 3, 60), (512, 8, 128), (4096, 1, 256),
                                   (4097, 1, 256), (1366, 3, 255), (5000, 8, 64), (20000, 8, 256),
                                   (300000, 1, 3), (70000, 8, 17)])
def test_plan(T, k, E):
    rng = np.random.default_rng(T + k + E)
    ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32))
    check_plan(ids, E)
    if T:
        ids = torch.from_numpy(rng.integers(-1, E + 1, (T, k)).astype(np.int32))
        ids[0, 0] = 2 ** 31 - 1
        check_plan(ids, E)


@pytest.mark.parametrize("T", [50, 9000])
def test_plan_of_one_expert_and_of_none(T):
    check_plan(torch.full((T, 4), 7, dtype=torch.int32), 8)
    check_plan(torch.full((T, 4), -1, dtype=torch.int32), 8)


# Both sides of each change of the split: workgroups of 1024 pairs that count
# by themselves (up to 16), chunks of 1024, 2048, 4096 and 8192 pairs with
# counts of their own, partial last chunks, and divisions by every kind of k.
@pytest.mark.parametrize("T,k,E,kind", [
    (1025, 1, 256, "alone"), (341, 3, 2, "alone"), (2048, 8, 256, "alone"),
    (64, 256, 256, "alone"), (65, 255, 9, "counted"), (16385, 1, 1, "counted"),
    (5462, 3, 256, "counted"), (8193, 4, 256, "counted"), (16385, 8, 256, "counted"),
    (29128, 9, 129, "counted"), (90001, 11, 60, "counted"), (262147, 8, 200, "counted")])
@pytest.mark.parametrize("spread", ["all", "one", "sorted"])
def test_plan_splits(T, k, E, kind, spread):
    rng = np.random.default_rng(T + k + E)
    ids = rng.integers(-1, E + 1, (T, k)).astype(np.int32)
    if spread == "one":
        ids[rng.random((T, k)) < 0.97] = E - 1
    if spread == "sorted":
        ids = np.sort(ids.reshape(-1))[::-1].reshape(T, k).copy()
    check_plan(torch.from_numpy(ids), E)
    assert sg.gemm_last_kernel() == "moe_plan_place_kernel<%s>" % kind


def test_plan_of_the_most_pairs():
    k = 7
    T = (2 ** 31 - 1) // k
    P, half = T * k, T * k // 2
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    flat = ids.view(-1)
    flat[:half] = 1                                   # the first half goes behind the second
    flat[P - 5:] = 3                                  # and five pairs name no expert
    offsets, rows, slots = sg.moe_plan(ids, 3)
    n0 = P - 5 - half
    assert offsets.tolist() == [0, n0, P - 5, P - 5]
    i = torch.arange(P, dtype=torch.int32, device="cuda")
    slots = slots.view(-1)
    assert torch.equal(slots[:half], i[:half] + n0) and torch.equal(slots[half:P - 5], i[:n0])
    assert bool((slots[P - 5:] == -1).all()) and bool((rows[P - 5:] == -1).all())
    i //= k
    assert torch.equal(rows[:n0], i[half:P - 5]) and torch.equal(rows[n0:P - 5], i[:half])


@pytest.mark.parametrize("T,E", [(4097, 8), (16385, 256), (65537, 256)])
def test_plan_writes_its_workspace_only(T, E):
    ids = torch.from_numpy(np.random.default_rng(T).integers(0, E, (T, 4)).astype(np.int32))
    n = sg.moe_plan_workspace_bytes(T * 4, E)
    ws = torch.full((n + 132,), 85, dtype=torch.uint8, device="cuda")
    check_plan(ids, E, workspace=ws[68:])             # 4-byte aligned
    assert n > 0 and bool((ws[:68] == 85).all()) and bool((ws[68 + n:] == 85).all())


def test_plan_into_buffers_with_a_workspace():
    rng = np.random.default_rng(6)
    T, k, E = 3000, 4, 40
    ids = torch.from_numpy(rng.integers(0, E, (T, k)).astype(np.int32))
    out = (torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"),
           torch.full((T * k,), -9, dtype=torch.int32, device="cuda"),
           torch.full((T, k), -9, dtype=torch.int32, device="cuda"))
    ws = torch.full((sg.moe_plan_workspace_bytes(T * k, E) + 64,), 85, dtype=torch.uint8,
                    device="cuda")
    n = ws.numel() - 64
    check_plan(ids, E, out=out, workspace=ws)
    assert bool((ws[n:] == 85).all())


# ------------------------------------------------------------- the layer together

def layer(x, wr, bias, q1, s1, q2, s2, k):
    """Router, plan, first product (gate and up), SiLU, second product, sum."""
    weights, ids = sg.moe_route(x.float() @ wr, k, score="sigmoid", bias=bias, n_groups=4,
                                top_groups=2, group_score="top2")
    offsets, rows, slots = sg.moe_plan(ids, wr.shape[1])
    qx, sx = sg.i8_quant(x)
    h = sg.i8_grouped_gemm(qx, sx, q1, s1, offsets, rows=rows, out_dtype=torch.bfloat16)
    gate, up = h.float().chunk(2, 1)
    a = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16)
    qa, sa = sg.i8_quant(a)
    y = sg.i8_grouped_gemm(qa, sa, q2, s2, offsets, out_dtype=torch.bfloat16)
    picked = torch.where((slots >= 0)[:, :, None], y[slots.clamp_min(0).long()].float(), 0.0)
    return (picked * weights[:, :, None]).sum(1), dict(
        weights=weights, ids=ids, offsets=offsets, rows=rows, slots=slots, qx=qx, sx=sx, h=h,
        a=a, qa=qa, sa=sa, y=y)


def layer_inputs(T, H, F, E, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = n(T, H).to(torch.bfloat16)
    wr, bias = n(H, E) / math.sqrt(H), 0.1 * n(E)
    w1, w2 = n(E, 2 * F, H) / math.sqrt(H), n(E, H, F) / math.sqrt(F)
    (q1, s1), (q2, s2) = (sg.i8_quant(w.reshape(-1, w.shape[2])) for w in (w1, w2))
    return (x, wr, bias, q1.view(E, 2 * F, H), s1.view(E, -1), q2.view(E, H, F), s2.view(E, -1))


@pytest.mark.parametrize("T,H,F,E,k", [(1, 64, 32, 8, 2), (37, 128, 96, 16, 4),
                                       (700, 256, 128, 16, 4), (2100, 512, 256, 8, 2)])
def test_layer(T, H, F, E, k):
    args = layer_inputs(T, H, F, E, T)
    out, st = layer(*args, k)
    c = {n: v.cpu() for n, v in st.items()}
    x, wr, bias, q1, s1, q2, s2 = (a.cpu() for a in args)
    off, rows = c["offsets"].tolist(), c["rows"].long()
    assert off[-1] == T * k
    tol = 2.0 ** -8 + 4 * 2.0 ** -24
    want_out = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e] == off[e + 1]:
            continue
        t = rows[r]
        h = (c["qx"][t].double() @ q1[e].double().t()) * c["sx"][t].double()[:, None] \
            * s1[e].double()
        assert bool(((c["h"][r].double() - h).abs() <= tol * h.abs()).all())
        y = (c["qa"][r].double() @ q2[e].double().t()) * c["sa"][r].double()[:, None] \
            * s2[e].double()
        assert bool(((c["y"][r].double() - y).abs() <= tol * y.abs()).all())
    w, y = c["weights"].double(), c["y"].double()
    for j in range(k):
        want_out += w[:, j:j + 1] * y[c["slots"][:, j].long()]
    # fp32 products and a sum of k terms: k + 1 roundings of the terms' size
    size = sum(w[:, j:j + 1] * y[c["slots"][:, j].long()].abs() for j in range(k))
    assert bool(((out.cpu().double() - want_out).abs() <= (k + 1) * 2.0 ** -24 * size).all())


def test_layer_in_a_graph():
    """Captured once, replayed with other tokens (masked ones among them) and
    eager work between the replays: every replay equals the eager layer."""
    T, H, F, E, k = 96, 128, 64, 16, 4
    args = list(layer_inputs(T, H, F, E, 1))
    x = args[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(*args, k)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, st = layer(*args, k)
    for i in range(4):
        fresh = torch.randn(T, H, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16)
        x.copy_(fresh)
        g.replay()
        torch.cuda.synchronize()
        got, ids = out.clone(), st["ids"].clone()
        want, st2 = layer(*args, k)
        assert torch.equal(ids, st2["ids"]) and torch.equal(got, want)


def test_two_graphs_of_large_plans_do_not_share_a_workspace():
    """Each captured call allocated its own counts: replays that overlap on two
    streams both give their own plan."""
    rng = np.random.default_rng(1)
    E = 64
    ids = [torch.from_numpy(rng.integers(0, E, (9000, 4)).astype(np.int32)).cuda()
           for _ in range(2)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    sg.moe_plan(ids[0], E)
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sg.moe_plan(ids[i], E))
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for a, b in zip(outs[i], plan_reference(ids[i].cpu().numpy().astype(np.int64), E)):
                assert np.array_equal(a.cpu().numpy(), b)
            for a in outs[i]:
                a.zero_()
        torch.cuda.synchronize()
