"""The vocabulary's cross entropy and its gradients in 64 bits, with the bounds
of the kernels' errors (u = 2^-24, half a step of fp32 relative to the value).

A logit is alpha times a sum of K exact products, added in fp32 by matrix
instructions that take at least 16 of them at a time: K/16 roundings of the
accumulator and at most 16 inside an instruction, each (truncation included) at
most 2u of the sum of the products' magnitudes S, then two roundings of a
product with alpha: dz = (K/16 + 18) * 2u * |alpha| S.
"""
import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step of the value


def logits(A, B, alpha):
    """z and the bound dz of its error, float64."""
    a, b = A.double(), B.double()
    K = A.shape[1]
    z = alpha * (a @ b.t().contiguous())
    dz = (K / 16 + 18) * 2 * U * abs(alpha) * (a.abs() @ b.abs().t().contiguous())
    return z, dz


def has_target(t, N):
    return (t >= 0) & (t < N)


def forward(A, B, t, alpha):
    """(loss, lse, bound of loss, bound of lse).

    The exponentials of z - max are each off by dz, by u of (z - max) log2 e for
    the difference, u for the product and u of 2^x (z - max in [-104, 0] where it
    counts: at most 4 * 151 u, and only for terms below e^-100; relative to the
    sum the mean of (z - max) e^(z - max) is at most 1/e a term of N, so 4 u
    (1 + log N) covers it), and joined over the tiles (log2 of a tile's maximum
    less the row's, again such a factor for each of two joins): 16 u (1 + log N).
    The sum adds 64 + N/256 + 32 numbers one after another at most."""
    N = B.shape[0]
    z, dz = logits(A, B, alpha)
    lse = torch.logsumexp(z, 1)
    ok = has_target(t, N)
    at = torch.where(ok, t, 0).long()[:, None]
    zt = z.gather(1, at)[:, 0]
    loss = torch.where(ok, lse - zt, 0)
    logn = torch.log(torch.tensor(float(N)))
    d = dz.amax(1) + U * (16 * (1 + logn) + 96 + N / 256)
    d_lse = d + 4 * U * (z.amax(1).abs() + lse.abs())
    # The loss is the maximum less the target's logit plus the sum's logarithm,
    # one rounding each.
    d_loss = d + dz.gather(1, at)[:, 0] + 4 * U * ((z.amax(1) - zt).abs() + logn + loss)
    return loss, lse, d_loss, d_lse


def backward(dloss, A, B, t, alpha, dlse=None):
    """(dA, dB, bound of dA, bound of dB)."""
    N, K = B.shape
    M = A.shape[0]
    half = HALF[A.dtype]
    z, dz = logits(A, B, alpha)
    lse = torch.logsumexp(z, 1)
    ok = has_target(t, N)
    dl = torch.where(ok, dloss.double(), 0)
    whole = dl if dlse is None else dl + dlse.double()
    p = torch.exp(z - lse[:, None])
    g = p * whole[:, None]
    rows = torch.nonzero(ok)[:, 0]
    g[rows, t[ok].long()] -= dl[rows]
    g *= alpha
    # g: the softmax is off by dz of its logit, the forward pass's error of lse
    # and 4 u of the logits' size (lse rounded, times log2 e, the fused
    # difference), the factors by 4 u; then half a step of 16 bits, and for fp16
    # half the smallest number, 2^-25, at a scale that brings the largest
    # |alpha| (|dl| + |whole|) to 2^13 or more.
    d_lse = forward(A, B, t, alpha)[3]
    rel = dz + d_lse[:, None] + 8 * U * (1 + z.abs() + lse.abs()[:, None])
    dg = abs(alpha) * whole.abs()[:, None] * p * rel + 8 * U * abs(alpha) * (
        dl.abs() + whole.abs())[:, None] * (p + (g != 0))
    dg = dg + half * (g.abs() + dg)
    if A.dtype is torch.float16:
        dg = dg + 2.0 ** -38 * abs(alpha) * float((dl.abs() + whole.abs()).max())
    a, b = A.double(), B.double()

    def product(x, dx, y):
        n = x.shape[1]
        d = dx @ y.abs() + (n / 16 + 18) * 2 * U * (x.abs() @ y.abs())
        out = x @ y
        # rounded once to the type (half its smallest number where it is denormal)
        tiny = 2.0 ** -25 if A.dtype is torch.float16 else 2.0 ** -134
        return out, d + half * (out.abs() + d) + tiny

    dA, bA = product(g, dg, b)
    dB, bB = product(g.t().contiguous(), dg.t().contiguous(), a)
    return dA, dB, bA, bB


def inputs(M, N, K, dtype, seed, known=0.7, ignored=0.1, alpha=1.0, device="cuda"):
    """Hidden states, a head and targets; a share of the targets is likely."""
    gen = torch.Generator().manual_seed(seed)
    B = torch.randn(N, K, generator=gen) * (1.5 / max(K, 1) ** 0.5 / (abs(alpha) or 1.0))
    t = torch.randint(0, max(N, 1), (M,), generator=gen)
    A = torch.randn(M, K, generator=gen)
    if N and K:
        w = B[t]
        up = 10 * torch.rand(M, 1, generator=gen) * (torch.rand(M, 1, generator=gen) < known)
        A = A + up * w / (w * w).sum(1, keepdim=True)
    t = torch.where(torch.rand(M, generator=gen) < ignored, -100, t)
    return A.to(dtype).to(device), B.to(dtype).to(device), t.to(device)
