"""The routing gradient where absolute bounds see nothing: saturated sigmoid
experts and the small gradients of experts that were not chosen, against
64-bit references and with bounds relative to the gradient's own size."""
import numpy as np
import pytest
import torch

import dense_gemm_swizzled_amd as sg

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# The smallest step of the type, halved: results below its normal range.
STEP = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def inputs(T, E, k, dtype, lo, hi):
    rng = np.random.default_rng(T + E + k)
    x = torch.from_numpy(rng.uniform(lo, hi, (T, E)).astype(np.float32)).to(dtype)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    g = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    return x, torch.from_numpy(ids), g


def sigmoid_gradient(x, ids, g, renorm, scale):
    """(gradient, its size) of the chosen experts' logits, in 64 bits; 1 - s
    is made from the logit, not from s."""
    x = np.take_along_axis(x.double().numpy(), ids.numpy().astype(np.int64), 1)
    z = np.exp(-np.abs(x))
    s, rest = np.where(x < 0, z, 1) / (1 + z), np.where(x < 0, 1, z) / (1 + z)
    g = g.double().numpy() * scale
    r = s / s.sum(1, keepdims=True) if renorm else s
    mean = (g * r).sum(1, keepdims=True) if renorm else 0.0
    return r * (g - mean) * rest, r * rest * np.abs(g).max(1, keepdims=True)


# T, E, k: one of each split of the experts over lanes.
@pytest.mark.parametrize("T,E,k", [(40, 24, 6), (33, 64, 8), (50, 100, 4), (21, 256, 32),
                                   (16389, 64, 8), (32773, 101, 6), (16387, 256, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renorm", [True, False])
def test_saturated_experts_keep_their_gradient(T, E, k, dtype, renorm):
    x, ids, g = inputs(T, E, k, dtype, -30.0, 30.0)
    x[1::3] = x[1::3].abs()                           # rows with saturated experts only
    dx = sg.moe_route_backward(g.cuda(), x.cuda(), ids.cuda(), score="sigmoid", renorm=renorm,
                               scale=2.5)
    got = np.take_along_axis(dx.cpu().double().numpy(), ids.numpy().astype(np.int64), 1)
    ref, size = sigmoid_gradient(x, ids, g, renorm, 2.5)
    # In units of 2^-24: a score 6 (expf 4, sum, quotient); the sum of up to 32
    # of them 10 more, so a ratio 6 + 16 + 1 = 23; g times the scale 1; the mean
    # 23 + 2 and 10 for its sum; the difference, of two terms of up to max|g|,
    # 35 + 1 and 2; times the ratio (23 of twice max|g|) 46 + 2; times 1 - s
    # (6 and a rounding, of twice max|g|) 14: 100 in all, then the type.
    lim = 100 * 2.0 ** -24 * size + HALF[dtype] * np.abs(ref) + STEP[dtype]
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), (int(bad.sum()), got[bad][:3], ref[bad][:3])
    far = np.take_along_axis(x.double().numpy(), ids.numpy().astype(np.int64), 1) > 17
    if dtype != torch.float16:                        # the bound leaves no room for zeros
        assert (np.abs(ref) > lim)[far].mean() > 0.5


@pytest.mark.parametrize("T,E,k", [(40, 24, 6), (33, 64, 8), (50, 100, 4), (21, 256, 32),
                                   (16389, 64, 8), (16387, 256, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_not_chosen_in_a_softmax(T, E, k, dtype):
    """Without renormalisation their gradient is -s_e sum_j s_j g_j, about 1/E^2
    of the weights' gradient and less."""
    x, ids, g = inputs(T, E, k, dtype, -9.0, 9.0)
    dx = sg.moe_route_backward(g.cuda(), x.cuda(), ids.cuda(), score="softmax", renorm=False)
    x64, i64 = x.double().numpy(), ids.numpy().astype(np.int64)
    e = np.exp(x64 - x64.max(1, keepdims=True))
    s = e / e.sum(1, keepdims=True)
    sj = np.take_along_axis(s, i64, 1)
    ref = -s * (g.double().numpy() * sj).sum(1, keepdims=True)
    size = s * (np.abs(g.double().numpy()) * sj).sum(1, keepdims=True)
    # Units of 2^-24: an exponential 24 (its rounded argument, up to 18, and
    # expf), a score 35 (the sum 10, the quotient 1), the sum of the products
    # 35 + 2 + 10, its quotient by the total 11, the product with the
    # expert's exponential 24 + 1: 83.
    lim = 83 * 2.0 ** -24 * size * (1 + 2.0 ** -16) + HALF[dtype] * np.abs(ref) + STEP[dtype]
    rest = np.ones_like(s, bool)
    np.put_along_axis(rest, i64, False, 1)
    err = np.abs(dx.cpu().double().numpy() - ref)
    assert bool((err <= lim)[rest].all()), (err - lim)[rest].max()
