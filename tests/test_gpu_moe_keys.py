"""Experts and groups in the order of their 64-bit keys, where keys made in
32 bits would put them in another."""
import numpy as np
import pytest
import torch

import dense_gemm_swizzled_amd as sg

pytestmark = pytest.mark.gpu


def keys64(x, score, bias):
    x = x.astype(np.float64)
    if score == "sigmoid":
        s = np.where(x < 0, np.exp(np.minimum(x, 0)), 1.0) / (1 + np.exp(-np.abs(x)))
    else:
        e = np.exp(x - x.max(1, keepdims=True))
        s = e / e.sum(1, keepdims=True)
    return s if bias is None else s + bias.astype(np.float64)


def choice64(key, k, n_groups=1, top_groups=1):
    """(ids, sums): the choice by top-2 groups for keys [T][E], and the groups'
    sums [T][n_groups]."""
    T, E = key.shape
    key = key.copy()
    sums = None
    if n_groups > 1:
        g = key.reshape(T, n_groups, E // n_groups)
        top = -np.sort(-g, axis=2)[:, :, :2]
        sums = top[:, :, 0] + (top[:, :, 1] if top.shape[2] > 1 else 0)
        order = np.argsort(-sums, axis=1, kind="stable")
        np.put_along_axis(g, order[:, top_groups:, None], -np.inf, axis=1)
        key = g.reshape(T, E)
    return np.argsort(-key, axis=1, kind="stable")[:, :k], sums


def gpu_ids(x, k, bias, **kw):
    b = None if bias is None else torch.from_numpy(bias).cuda()
    return sg.moe_route(torch.from_numpy(x).cuda(), k, bias=b, **kw)[1].cpu().numpy()


def halves(rng, n, base):
    """(logits, bias): two groups of two sigmoid experts whose keys lie in the
    middle between two fp32 values near `base`, those of group 0 by a little
    above it and those of group 1 below in fp32: each key is off by half a
    step u in favour of group 0, and so is each group's sum (by u).  The exact
    sums favour group 1 by less than 2^-25."""
    u = float(np.spacing(np.float32(base)))
    # Experts 0 and 2: scores that fp32 rounds to 1/2, keys on the middle, from
    # where an odd step rounds up and an even one down.
    q0, q2, q1, q3 = 1, 2, 40, 37
    bias = base + np.array([(q0 + 0.5) * u - 0.5, q1 * u, (q2 + 0.5) * u - 0.5, q3 * u])
    assert np.array_equal(bias.astype(np.float32).astype(np.float64), bias)
    x = np.empty((n, 4))
    x[:, 0], x[:, 2] = -rng.uniform(2e-8, 5e-8, n), rng.uniform(2e-8, 5e-8, n)
    # Experts 1 and 3: small scores (fp32 has them to 2^-31) next to the middle,
    # with equal whole steps in both groups, one more than a multiple of four.
    r1 = 4 * rng.integers(max(1, int(9e-4 / u / 4)), int(6e-3 / u / 4), n)
    r1 += (1 - q0 - q1) % 4
    r3 = r1 + q0 + q1 - q2 - q3
    for e, s in ((1, (r1 + 0.5) * u + 1.2e-9), (3, (r3 + 0.5) * u - 1.2e-9)):
        x[:, e] = np.log(s / (1 - s))
    return x.astype(np.float32), bias.astype(np.float32)


@pytest.mark.parametrize("base", [8, 16, 64, 128, 512, 1024])
@pytest.mark.parametrize("swap", [False, True])
def test_group_sums_whose_rounding_matters(base, swap):
    x, bias = halves(np.random.default_rng(base), 4000, base)
    if swap:
        x, bias = np.ascontiguousarray(x[:, [2, 3, 0, 1]]), bias[[2, 3, 0, 1]]
    want, sums = choice64(keys64(x, "sigmoid", bias), 2, 2, 1)
    # Far beyond what 64 bits leave open (2^-52 of the base a sum), and nearly
    # always against the order of the fp32 sums.
    clear = np.abs(sums[:, 0] - sums[:, 1]) > 2.0 ** -48 * base
    assert clear.mean() > 0.99 and (want[:, 0] // 2 == (0 if swap else 1)).mean() > 0.9
    got = gpu_ids(x, 2, bias, score="sigmoid", n_groups=2, top_groups=1, group_score="top2")
    wrong = (got != want).any(1) & clear
    assert not wrong.any(), (int(wrong.sum()), x[wrong][:3].tolist())


def test_a_group_sum_off_by_its_rounding():
    x = np.array([[-3e-8, -6.795358, 3e-8, -6.958249]], np.float32)
    bias = np.array([63.50004196, 64.00019836, 63.50015640, 64.00025177], np.float32)
    want, _ = choice64(keys64(x, "sigmoid", bias), 2, 2, 1)
    got = gpu_ids(x, 2, bias, score="sigmoid", n_groups=2, top_groups=1, group_score="top2")
    assert np.array_equal(got, want)


def test_group_sums_beyond_the_largest_float():
    """Biases whose sums of two pass fp32's range: large ones, and the type's
    lowest value as a mask, which is finite and no -inf."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 16)).astype(np.float32)
    low = float(np.finfo(np.float32).min)
    # (two of a group's four experts; unequal, so that only the sums are close)
    for groups in ([(3.0e38, 3.1e38), (3.3e38, 3.2e38), (2.9e38, 3.2e38), (0.0, 3.4e38)],
                   [(low, 0.9 * low), (low, 0.8 * low), (0.7 * low, 0.9 * low), (low, low)],
                   [(0.9 * low, 0.8 * low), (0.7 * low, 0.6 * low), (0.75 * low, 0.5 * low),
                    (0.1 * low, 0.95 * low)],
                   [(3.3e38, low), (low, 0.9 * low), (2.0e38, 3.0e38), (3.4e38, 1.0)]):
        bias = np.full(16, low, np.float32)
        for g, pair in enumerate(groups):
            bias[4 * g:4 * g + 2] = pair
        for score in ("sigmoid", "softmax"):
            for top, k in ((1, 1), (1, 2), (2, 1), (2, 2), (2, 3), (3, 4)):
                want, _ = choice64(keys64(x, score, bias), k, 4, top)
                got = gpu_ids(x, k, bias, score=score, n_groups=4, top_groups=top,
                              group_score="top2")
                assert np.array_equal(got, want), (groups, score, top, k)


@pytest.mark.parametrize("E,n_groups", [(16, 4), (64, 8), (256, 8)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_sums_of_scores_that_are_denormal(E, n_groups, with_bias):
    """Sigmoid scores below 2^-126 are 2^-149 apart in fp32, far coarser than
    a relative bound of their error."""
    rng = np.random.default_rng(E)
    x = rng.uniform(-103.9, -88.0, (3000, E)).astype(np.float32)
    x[:1000] = rng.uniform(-103.9, -100.0, (1000, E))
    bias = (2.0 ** -146 * rng.integers(0, 3, E)).astype(np.float32) if with_bias else None
    want, _ = choice64(keys64(x, "sigmoid", bias), 4, n_groups, n_groups // 2)
    got = gpu_ids(x, 4, bias, score="sigmoid", n_groups=n_groups, top_groups=n_groups // 2,
                  group_score="top2")
    wrong = (got != want).any(1)
    assert not wrong.any(), (int(wrong.sum()), x[wrong][:1].tolist())


OFF = [-1e3, -1e4, -1e9, -3e38]


@pytest.mark.parametrize("E,k,n_groups,top_groups", [(16, 4, 1, 1), (64, 6, 8, 3), (128, 8, 1, 1),
                                                     (256, 8, 8, 4)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_experts_switched_off_by_a_bias(E, k, n_groups, top_groups, score):
    rng = np.random.default_rng(E)
    x = (2 * rng.standard_normal((500, E))).astype(np.float32)
    for off in OFF + [1e9]:                           # (or forced to the front)
        bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
        bias[[1, E // 2, E - 1]] = off
        bias[2] = np.float32(0.9) * off
        want, _ = choice64(keys64(x, score, bias), k, n_groups, top_groups)
        got = gpu_ids(x, k, bias, score=score, n_groups=n_groups, top_groups=top_groups,
                      group_score="top2")
        assert np.array_equal(got, want), off


@pytest.mark.parametrize("n_groups,top_groups", [(1, 1), (8, 1), (8, 3)])
def test_experts_forced_by_an_infinite_bias(n_groups, top_groups):
    rng = np.random.default_rng(9)
    x = (2 * rng.standard_normal((300, 64))).astype(np.float32)
    for forced in ([5], [5, 6], [5, 50], [50, 51, 3]):
        bias = (0.1 * rng.standard_normal(64)).astype(np.float32)
        bias[forced] = np.inf
        bias[[9, 60]] = -np.inf
        for k in (1, 4):
            want, _ = choice64(keys64(x, "sigmoid", bias), k, n_groups, top_groups)
            got = gpu_ids(x, k, bias, score="sigmoid", n_groups=n_groups, top_groups=top_groups,
                          group_score="top2")
            assert np.array_equal(got, want), (forced, k)


@pytest.mark.parametrize("n_groups,top_groups", [(1, 1), (8, 4)])
def test_an_expert_switched_off_costs_nothing(n_groups, top_groups):
    """Its bias takes no part in the choice, so no more tokens need 64 bits:
    counted with its size, every token did, and a call took 1.8 times as long."""
    T, E, k = 32768, 256, 8
    x = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).cuda()
    biases = [torch.zeros(E, device="cuda") for _ in range(2)]
    biases[1][5] = -1e9
    out = sg.moe_route(x, k, score="sigmoid", bias=biases[0])

    def once(bias):
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        marks[0].record()
        for _ in range(10):
            sg.moe_route(x, k, score="sigmoid", bias=bias, n_groups=n_groups,
                         top_groups=top_groups, group_score="top2", out=out)
        marks[1].record()
        marks[1].synchronize()
        return marks[0].elapsed_time(marks[1])

    times = np.array([[once(b) for b in biases] for _ in range(12)])[2:]
    plain, off = np.median(times, axis=0)
    assert off < 1.35 * plain, (plain, off)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_infinite_logit_is_the_largest_float(score):
    top = float(np.finfo(np.float32).max)
    x = torch.zeros(4, 12)
    x[0, 3] = float("inf")
    x[1, [2, 7]] = float("inf")
    x[2, 5], x[2, 9] = float("inf"), top
    x[3, 4], x[3, 9] = top, float("inf")
    w, ids = sg.moe_route(x.cuda(), 2, score=score)
    w2, ids2 = sg.moe_route(x.clamp(max=top).cuda(), 2, score=score)
    assert torch.equal(w, w2) and torch.equal(ids, ids2)
    assert ids.tolist() == [[3, 0], [2, 7], [5, 9], [4, 9]]
    if score == "softmax":
        assert w.tolist() == [[1, 0], [0.5, 0.5], [0.5, 0.5], [0.5, 0.5]]
    g = torch.ones(4, 2).cuda()
    assert torch.equal(sg.moe_route_backward(g, x.cuda(), ids, score=score),
                       sg.moe_route_backward(g, x.clamp(max=top).cuda(), ids, score=score))
