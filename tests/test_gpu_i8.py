"""8-bit products and their quantiser on the GPU against 64-bit references.

Tolerance of a product: the integer sum is exact, so D differs from the exact
value by its conversion to fp32, two fp32 products (2^-24 relative each) and
the rounding to D's type (half a step: bf16 2^-8, f16 2^-11, fp32 none left),
plus half of f16's smallest step where the result is subnormal.
"""
import math

import numpy as np
import pytest
import torch

import dense_gemm_swizzled_amd as sg

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def codes(rng, *shape, full=True):
    lo = -128 if full else -127
    return torch.from_numpy(rng.integers(lo, 128, shape, dtype=np.int8))


def scales(rng, *shape):
    return torch.from_numpy((0.5 + rng.random(shape)).astype(np.float32) * 2.0 ** -10)


def reference(a, sa, b, sb):
    """64-bit D (the integer sums, below 2^31, are exact in it)."""
    return (a.double() @ b.double().t()) * sa.double()[:, None] * sb.double()[None, :]


def check(d, ref):
    ref = ref.numpy()
    got = d.detach().cpu().double().numpy()
    lim = (3 * 2.0 ** -24 + HALF[d.dtype]) * (1 + 2.0 ** -20) * np.abs(ref)
    if d.dtype == torch.float16:
        lim = lim + 2.0 ** -25
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    bad = ~(np.abs(got - ref) <= lim) & ~np.isnan(ref)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


def run(a, sa, b, sb, **kw):
    return sg.i8_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), **kw)


# Sizes that reach every kernel, with edges in M, N and K.
SIZES = [
    (1, 1, 16, "stream"), (1, 8, 0, "stream"), (1, 257, 1040, "stream"), (3, 40, 48, "stream"),
    (16, 128, 4096, "stream"), (17, 100, 80, "stream"), (32, 264, 528, "stream"),
    (33, 130, 144, "stream"), (64, 513, 2064, "stream"), (65, 72, 272, "mid"),
    (100, 999, 128, "mid"), (300, 264, 208, "mid"), (129, 4097, 144, "mid"),
    (1000, 2050, 400, "mid"), (200, 264, 16, "mid"), (2000, 2304, 16, "pingpong"), (4096, 4096, 128, "pingpong"),
    (4000, 4111, 192, "pingpong"), (8200, 2056, 80, "pingpong"), (4097, 4096, 256, "pingpong"),
    (4096, 4000, 384, "pingpong"), (5100, 4111, 640, "pingpong"), (9000, 5001, 256, "pingpong"),
]


@pytest.mark.parametrize("M,N,K,kind", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_i8_gemm(M, N, K, kind, dtype):
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    a, b = codes(rng, M, K), codes(rng, N, K)
    sa, sb = scales(rng, M), scales(rng, N)
    d = run(a, sa, b, sb, out_dtype=dtype)
    check(d, reference(a, sa, b, sb))
    assert kind in sg.gemm_last_kernel(), sg.gemm_last_kernel()


# One size for every instantiation that the tile choice can pick.
KERNELS = [
    (1, 4096, 1040, "i8_stream_kernel<16,16,dense>"), (7, 4500, 1040, "i8_stream_kernel<16,32,dense>"),
    (16, 33000, 112, "i8_stream_kernel<16,64,dense>"), (20, 200, 528, "i8_stream_kernel<32,16,dense>"),
    (29, 5001, 528, "i8_stream_kernel<32,32,dense>"), (32, 9000, 272, "i8_stream_kernel<32,32,dense>"),
    (50, 2900, 1040, "i8_stream_kernel<64,32,dense>"), (64, 9000, 272, "i8_mid_kernel<64,64,dense>"),
    (333, 4104, 1040, "i8_mid_kernel<64,128,dense>"), (768, 4096, 1040, "i8_mid_kernel<128,128,dense>"),
]


@pytest.mark.parametrize("M,N,K,name", KERNELS)
def test_every_dense_kernel(M, N, K, name):
    rng = np.random.default_rng(M + N + K)
    a, b, sa, sb = codes(rng, M, K), codes(rng, N, K), scales(rng, M), scales(rng, N)
    for dtype in (torch.bfloat16, torch.float32):
        d = run(a, sa, b, sb, out_dtype=dtype)
        assert sg.gemm_last_kernel() == name
        check(d, reference(a, sa, b, sb))


GROUPED_KERNELS = [
    # G, N, K, rows of each group on average
    (3, 200, 528, 4, "i8_stream_kernel<16,16,%s>"), (9, 1000, 1040, 8, "i8_stream_kernel<16,32,%s>"),
    (40, 1000, 80, 5, "i8_stream_kernel<16,64,%s>"), (6, 300, 272, 40, "i8_mid_kernel<64,64,%s>"),
    (5, 2800, 1040, 60, "i8_mid_kernel<64,128,%s>"), (4, 2000, 1040, 300, "i8_mid_kernel<128,128,%s>"),
    (32, 2048, 144, 30, "i8_pingpong_kernel<%s>"), (32, 2048, 256, 30, "i8_pingpong_kernel<%s>"),
    (20, 2100, 384, 500, "i8_pingpong_kernel<%s>"), (3, 4111, 640, 2500, "i8_pingpong_kernel<%s>"),
]


@pytest.mark.parametrize("G,N,K,mean,name", GROUPED_KERNELS)
@pytest.mark.parametrize("gather", [True, False])
def test_every_grouped_kernel(G, N, K, mean, name, gather):
    rng = np.random.default_rng(G + N + K)
    sizes = rng.multinomial(G * mean, rng.dirichlet(np.full(G, 2.0)))
    offsets = [0] + np.cumsum(sizes).tolist()
    R = offsets[-1]
    T = R // 2 + 1 if gather else R
    rows = rng.integers(0, T, R) if gather else np.arange(R)
    a, b, sa, sb = codes(rng, T, K), codes(rng, G, N, K), scales(rng, T), scales(rng, G, N)
    d = sg.i8_grouped_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(),
                           torch.tensor(offsets, dtype=torch.int32).cuda(),
                           rows=torch.from_numpy(rows.astype(np.int32)).cuda() if gather else None)
    assert sg.gemm_last_kernel() == name % ("grouped,rows" if gather else "grouped")
    want = torch.empty(R, N, dtype=torch.float64)
    for g in range(G):
        r = rows[offsets[g]:offsets[g + 1]]
        want[offsets[g]:offsets[g + 1]] = reference(a[r], sa[r], b[g], sb[g])
    check(d, want)


@pytest.mark.parametrize("M", [1, 40, 70, 200])
def test_largest_sum_is_exact(M):
    K = 131056
    a = torch.full((M, K), -128, dtype=torch.int8)
    b = torch.full((8, K), -128, dtype=torch.int8)
    b[1] = 127
    one = torch.ones
    d = run(a, one(M), b, one(8), out_dtype=torch.float32)
    # 2^14 K = 2147221504 and -128 * 127 K: fp32 rounds the sums to 2^7
    want = torch.tensor([2147221504.0] + [-128.0 * 127 * K] + [2147221504.0] * 6).float()
    assert torch.equal(d.cpu(), want.expand(M, 8))


@pytest.mark.parametrize("M,N,K", [(5, 50, 96), (50, 33, 160), (90, 75, 272), (300, 2001, 144),
                                   (4096, 4100, 144), (4200, 4100, 256)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_padded_rows_are_read_and_kept(M, N, K, dtype):
    """Rows of A, B and D inside wider buffers: the padding of A and B (127s)
    is not used, the cells around D keep their value."""
    rng = np.random.default_rng(K)
    wide_a = torch.full((M, K + 32), 127, dtype=torch.int8)
    wide_b = torch.full((N, K + 16), 127, dtype=torch.int8)
    a, b = codes(rng, M, K), codes(rng, N, K)
    wide_a[:, :K], wide_b[:, :K] = a, b
    sa, sb = scales(rng, M), scales(rng, N)
    for off, ldd in ((0, N + (-N) % 8 + 8), (3, N + 5)):
        buf = torch.full((M + 2, ldd), 7.0, dtype=dtype, device="cuda")
        out = buf[1:M + 1, off:off + N]
        sg.i8_gemm(wide_a.cuda()[:, :K], sa.cuda(), wide_b.cuda()[:, :K], sb.cuda(), out=out)
        check(out, reference(a, sa, b, sb))
        buf[1:M + 1, off:off + N] = 7.0
        assert bool((buf == 7.0).all())


def test_nan_scales_make_rows_and_columns_nan():
    rng = np.random.default_rng(3)
    for M in (4, 40, 200):
        a, b, sa, sb = codes(rng, M, 64), codes(rng, 24, 64), scales(rng, M), scales(rng, 24)
        sa[M // 2], sb[5] = math.nan, math.nan
        d = run(a, sa, b, sb, out_dtype=torch.float32).cpu()
        want = torch.zeros(M, 24, dtype=torch.bool)
        want[M // 2], want[:, 5] = True, True
        assert torch.equal(torch.isnan(d), want)


# ---------------------------------------------------------------- the grouped form

def grouped_reference(a, sa, b, sb, offsets, rows):
    R = len(rows)
    out = torch.full((R, b.shape[1]), math.nan, dtype=torch.float64)
    for g in range(b.shape[0]):
        for r in range(offsets[g], offsets[g + 1]):
            t = rows[r]
            if 0 <= t < a.shape[0]:
                out[r] = (b[g].double() @ a[t].double()) * sa[t].double() * sb[g].double()
            else:
                out[r] = 0.0
    return out


GROUPED = [
    # T, G, N, K, rows of each group
    (5, 1, 24, 64, [9]), (9, 3, 40, 48, [0, 7, 0]), (20, 4, 33, 80, [1, 0, 30, 2]),
    (64, 7, 129, 144, [20, 40, 0, 1, 17, 33, 16]), (40, 2, 100, 272, [64, 65]),
    (300, 5, 200, 128, [130, 1, 0, 300, 128]), (33, 256, 16, 32, None),
    (600, 3, 2048, 192, [255, 256, 700]), (2000, 2, 4096, 128, [1500, 2700]),
]


@pytest.mark.parametrize("T,G,N,K,sizes", GROUPED)
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_i8_grouped_gemm(T, G, N, K, sizes, gather, dtype):
    rng = np.random.default_rng(T + N + K)
    if sizes is None:
        sizes = rng.integers(0, 6, G).tolist()
    offsets = [0] + np.cumsum(sizes).tolist()
    R = offsets[-1] + 3                      # three rows behind the last group
    rows = rng.integers(0, T, R).tolist()
    rows[0] = T - 1
    if gather and R > 6:
        rows[2], rows[4] = -1, T             # outside A: zero rows
    if not gather:
        T, rows = R, list(range(R))
    a, b = codes(rng, T, K), codes(rng, G, N, K)
    sa, sb = scales(rng, T), scales(rng, G, N)
    out = torch.full((R, N), -3.0, dtype=dtype, device="cuda")
    sg.i8_grouped_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(),
                       torch.tensor(offsets, dtype=torch.int32).cuda(),
                       rows=torch.tensor(rows, dtype=torch.int32).cuda() if gather else None,
                       out=out)
    n = offsets[-1]
    check(out[:n], grouped_reference(a, sa, b, sb, offsets, rows)[:n])
    assert bool((out[n:] == -3.0).all())


def test_grouped_matches_the_dense_product_bit_for_bit():
    rng = np.random.default_rng(11)
    a, b = codes(rng, 700, 208), codes(rng, 3, 264, 208)
    sa, sb = scales(rng, 700), scales(rng, 3, 264)
    off = [0, 10, 10, 700]
    d = sg.i8_grouped_gemm(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(),
                           torch.tensor(off, dtype=torch.int32).cuda())
    for g in range(3):
        lo, hi = off[g], off[g + 1]
        if hi > lo:
            assert torch.equal(d[lo:hi], run(a[lo:hi], sa[lo:hi], b[g], sb[g]))


@pytest.mark.parametrize("R,N,K,name", [(6, 48, 64, "stream"), (60, 48, 64, "mid"),
                                        (600, 48, 64, "mid"), (9000, 2048, 256, "pingpong")])
def test_bad_offsets_stay_inside_d(R, N, K, name):
    """The device clamps offsets: whatever they are, nothing outside D's rows
    is written."""
    rng = np.random.default_rng(R)
    G = 4
    a, b = codes(rng, R, K).cuda(), codes(rng, G, N, K).cuda()
    sa, sb = scales(rng, R).cuda(), scales(rng, G, N).cuda()
    top = 2 ** 31 - 1
    for off in ([0, R, 0, R, R], [-5, 2, 9 * R, -top, top], [top] * 5, [-top - 1] * 5,
                [R, R // 2, 3, 1, 0], [0, 0, 0, 0, 0]):
        buf = torch.full((R + 2, N), 5.0, device="cuda")
        sg.i8_grouped_gemm(a, sa, b, sb, torch.tensor(off, dtype=torch.int32).cuda(),
                           out=buf[1:R + 1])
        torch.cuda.synchronize()
        assert name in sg.gemm_last_kernel()
        assert bool((buf[0] == 5.0).all()) and bool((buf[-1] == 5.0).all())


@pytest.mark.parametrize("M,N", [(3, 40), (20, 40), (60, 40), (100, 72), (4096, 4100)])
def test_k_of_zero_gives_zeros(M, N):
    a, b = torch.zeros(M, 0, dtype=torch.int8), torch.zeros(N, 0, dtype=torch.int8)
    for dtype in DTYPES:
        out = torch.full((M, N), 3.0, dtype=dtype, device="cuda")
        run(a, torch.ones(M), b, torch.ones(N), out=out)
        assert bool((out == 0).all())
    off = torch.tensor([0, M // 2, M], dtype=torch.int32).cuda()
    out = torch.full((M, N), 3.0, device="cuda")
    sg.i8_grouped_gemm(a.cuda(), torch.ones(M).cuda(), torch.zeros(2, N, 0, dtype=torch.int8).cuda(),
                       torch.ones(2, N).cuda(), off, out=out)
    assert bool((out == 0).all())


def test_quant_of_no_columns_and_no_rows():
    q, s = sg.i8_quant(torch.zeros(3, 0, device="cuda"))
    assert q.shape == (3, 0) and bool((s == 2.0 ** -100 / 127).all())
    q, s = sg.i8_quant(torch.zeros(0, 40, device="cuda"))
    assert q.shape == (0, 48) and s.shape == (0,)


def test_no_rows_and_empty_a():
    off = torch.zeros(3, dtype=torch.int32).cuda()
    b, sb = torch.zeros(2, 8, 16, dtype=torch.int8).cuda(), torch.ones(2, 8).cuda()
    a, sa = torch.zeros(0, 16, dtype=torch.int8).cuda(), torch.ones(0).cuda()
    assert sg.i8_grouped_gemm(a, sa, b, sb, off).shape == (0, 8)
    # every index lies outside an empty A: rows of zeros
    off[1:] = 2
    d = sg.i8_grouped_gemm(a, sa, b, sb, off, rows=torch.zeros(2, dtype=torch.int32).cuda())
    assert bool((d == 0).all())


# -------------------------------------------------------------------- the quantiser

def quant_reference(x):
    """The definition's fp32 steps, each one correctly rounded by numpy."""
    x = x.float().numpy()
    R, K = x.shape
    a = np.abs(x).max(1, initial=0.0) if K else np.zeros(R, np.float32)
    ok = np.isfinite(a)
    a = np.where(ok, np.maximum(a, np.float32(2.0 ** -100)), np.float32(1)).astype(np.float32)
    inv = np.float32(127) / a
    q = np.rint(np.where(ok[:, None], x, 0).astype(np.float32) * inv[:, None])
    q = np.pad(q, ((0, 0), (0, -K % 16))).astype(np.int8)
    return q, np.where(ok, a / np.float32(127), np.float32(np.nan))


@pytest.mark.parametrize("R,K", [(1, 1), (3, 7), (5, 16), (9, 24), (4, 500), (2, 512), (3, 520),
                                 (2, 1032), (7, 5003), (3, 4096), (2, 8192), (2, 10008),
                                 (2, 16384), (3, 16392), (2, 40001), (300, 128),
                                 (17, 130), (33, 250), (2, 32768), (1, 70003)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_i8_quant(R, K, dtype):
    rng = np.random.default_rng(R * K)
    x = torch.from_numpy((rng.standard_normal((R, K)) *
                          np.exp(rng.standard_normal((R, 1)))).astype(np.float32)).to(dtype)
    q, s = sg.i8_quant(x.cuda())
    rq, rs = quant_reference(x)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)
    # a code is at most half a step off, and the fp32 steps add two roundings
    # of a value of at most 127
    back = q.cpu().double()[:, :K] * s.cpu().double()[:, None]
    lim = (0.5 + 127 * 3 * 2.0 ** -24) * s.cpu().double()[:, None]
    assert bool(((back - x.double()).abs() <= lim).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("K", [40, 3000])
def test_quant_of_odd_rows(dtype, K):
    """Zero rows, the largest and smallest values, infinities and NaN."""
    x = torch.zeros(9, K, dtype=torch.float32)
    fin = torch.finfo(dtype)
    x[1, K - 1] = fin.max
    x[2, 0], x[2, 1] = fin.min, fin.max
    x[3] = fin.tiny
    x[4, K // 2] = math.inf
    x[5, K - 1] = -math.inf
    x[6, 3] = math.nan
    x[7, 0], x[7, 1] = math.inf, math.nan
    x[8, :5] = torch.tensor([1.0, -1.0, 0.5, 2.5 / 127, 1.5 / 127])
    x = x.to(dtype)
    q, s = sg.i8_quant(x.cuda())
    rq, rs = quant_reference(x)
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)
    assert bool(torch.isnan(s[4:8]).all()) and bool((q[4:8] == 0).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_quant_of_views_and_into_buffers(dtype):
    rng = np.random.default_rng(5)
    wide = torch.from_numpy(rng.standard_normal((12, 700)).astype(np.float32)).to(dtype)
    for c0, K in ((0, 512), (8, 600), (1, 333), (3, 17)):
        x = wide[1:9, c0:c0 + K]
        Kp = -(-K // 16) * 16
        buf = torch.full((10, Kp + 32), 99, dtype=torch.int8, device="cuda")
        s = torch.full((10,), 4.0, device="cuda")
        sg.i8_quant(wide.cuda()[1:9, c0:c0 + K], out=buf[1:9, 16:16 + Kp], out_scale=s[1:9])
        rq, rs = quant_reference(x)
        assert np.array_equal(buf[1:9, 16:16 + Kp].cpu().numpy(), rq)
        assert np.array_equal(s[1:9].cpu().numpy(), rs)
        buf[1:9, 16:16 + Kp] = 99
        assert bool((buf == 99).all()) and s[0] == 4.0 and s[9] == 4.0


def test_quant_then_product_is_near_the_float_product():
    """Codes are half a step off: |error of a_k| <= s_a / 2 and the same for
    b, so |error of D| <= sum |a| s_b / 2 + |b| s_a / 2 + s_a s_b / 4, up to
    the fp32 steps (2^-16 of it covers 127 * 3 roundings)."""
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.standard_normal((70, 1003)).astype(np.float32)).to(torch.bfloat16)
    w = torch.from_numpy(rng.standard_normal((90, 1003)).astype(np.float32)).to(torch.bfloat16)
    qx, sx = sg.i8_quant(x.cuda())
    qw, sw = sg.i8_quant(w.cuda())
    d = sg.i8_gemm(qx, sx, qw, sw, out_dtype=torch.float32).cpu().double()
    x, w, sx, sw = x.double(), w.double(), sx.cpu().double(), sw.cpu().double()
    ex, ew = sx[:, None] / 2, sw[None, :] / 2
    lim = x.abs().sum(1)[:, None] * ew + w.abs().sum(1)[None, :] * ex + 1003 * ex * ew
    assert bool(((d - x @ w.t()).abs() <= lim * (1 + 2.0 ** -16)).all())


def test_other_stream_and_graph_replays():
    """On a side stream, and captured: each replay gives what eager calls give
    on the same inputs."""
    rng = np.random.default_rng(21)
    M, N, K = 48, 136, 320
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    w = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).cuda()
    qw, sw = sg.i8_quant(w)
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.i8_quant(x, out=q, out_scale=s)
        sg.i8_gemm(q, s, qw, sw, out=d)
    side.synchronize()
    assert bool((d == 0).all())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sg.i8_quant(x, out=q, out_scale=s)
        sg.i8_gemm(q, s, qw, sw, out=d)
    for i in range(4):
        x.copy_(torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)))
        q.zero_(), d.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = d.clone()
        q2, s2 = sg.i8_quant(x)
        assert torch.equal(q, q2) and torch.equal(got, sg.i8_gemm(q2, s2, qw, sw))
