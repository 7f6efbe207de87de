"""Routing and 8-bit operators on tensors of more than 2^31 elements, checked
on sampled rows (their first and last among them) against references."""
import numpy as np
import pytest
import torch

import dense_gemm_swizzled_amd as sg

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def sampled(n, count=60):
    rng = np.random.default_rng(n)
    i = np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, count)]))
    return torch.from_numpy(i).cuda()


def codes(gen, *shape):
    return torch.randint(-128, 128, shape, generator=gen, device="cuda", dtype=torch.int8)


def product(a, sa, b, sb):
    s = torch.from_numpy(a.cpu().numpy().astype(np.float64) @ b.cpu().numpy().astype(np.float64).T)
    return s * sa.cpu().double()[:, None] * sb.cpu().double()


# The integer sum is exact; fp32 conversion and two products, then bf16.
TOL = 3 * 2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -10)


@pytest.mark.parametrize("M,N,K", [(33000, 66000, 128),      # 256 x 256 tiles
                                   (60, 36000000, 16)])      # 64 x 64 tiles of few rows
def test_d_of_more_than_2_31_values(M, N, K):
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, b = codes(gen, M, K), codes(gen, N, K)
    sa, sb = (0.5 + torch.rand(n, generator=gen, device="cuda") for n in (M, N))
    d = sg.i8_gemm(a, sa, b, sb)
    assert d.numel() > 2 ** 31
    r, c = sampled(M, 30), sampled(N, 2000)
    got, want = d[r][:, c].cpu().double(), product(a[r], sa[r], b[c], sb[c])
    assert bool(((got - want).abs() <= TOL * want.abs()).all())


def test_grouped_weights_of_more_than_2_31_bytes():
    gen = torch.Generator(device="cuda").manual_seed(2)
    G, N, K, R = 40, 8200, 8192, 320
    b = torch.empty(G, N, K, dtype=torch.int8, device="cuda")
    for g in range(G):
        b[g] = codes(gen, N, K)
    assert b.numel() > 2 ** 31
    for rows in (None, torch.randint(0, R, (R,), generator=gen, device="cuda").int()):
        a, sa = codes(gen, R, K), 0.5 + torch.rand(R, generator=gen, device="cuda")
        sb = 0.5 + torch.rand(G, N, generator=gen, device="cuda")
        off = (torch.arange(G + 1, device="cuda") * (R // G)).int()
        d = sg.i8_grouped_gemm(a, sa, b, sb, off, rows=rows)
        src = torch.arange(R, device="cuda") if rows is None else rows.long()
        for g in (0, 17, G - 1):
            s = src[off[g]:off[g + 1]]
            want = product(a[s], sa[s], b[g], sb[g])
            got = d[off[g]:off[g + 1]].cpu().double()
            assert bool(((got - want).abs() <= TOL * want.abs()).all())


def test_quantised_rows_beyond_2_31_values():
    R, K = 33001, 66000
    x = torch.empty(R, K, dtype=torch.bfloat16, device="cuda").normal_()
    q, s = sg.i8_quant(x)
    r = sampled(R)
    xs = x[r].float().cpu().numpy()                   # (numpy: the GPU's division is not rounded once)
    a = np.abs(xs).max(1)
    assert np.array_equal(s[r].cpu().numpy(), a / np.float32(127))
    assert np.array_equal(q[r].cpu().numpy(), np.rint(xs * (np.float32(127) / a)[:, None]))


def test_logits_beyond_2_31_values():
    T, E, k = 8400000, 256, 4
    x = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_()
    w, ids = sg.moe_route(x, k, score="sigmoid", renorm=False)
    dx = sg.moe_route_backward(torch.ones_like(w), x, ids, score="sigmoid", renorm=False)
    r = sampled(T)
    order = np.argsort(-x[r].float().cpu().numpy(), axis=1, kind="stable")[:, :k]
    assert np.array_equal(ids[r].cpu().numpy(), order)
    s = torch.sigmoid(x[r].double().cpu())
    got = w[r].cpu().double()
    want = s.gather(1, torch.from_numpy(order))
    assert bool(((got - want).abs() <= 6 * 2.0 ** -24 * want).all())
    g = torch.zeros_like(s).scatter_(1, torch.from_numpy(order), 1) * s * (1 - s)
    err = (dx[r].cpu().double() - g).abs()
    assert bool((err <= (2.0 ** -8 + 20 * 2.0 ** -24) * g.abs()).all())
