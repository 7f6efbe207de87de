"""The calls that carry a gradient have no forward-mode one: a tensor with a tangent
is refused instead of losing it (no GPU)."""
import pytest
import torch
import torch.autograd.forward_ad as forward_ad

import dense_gemm_swizzled_amd as sg

NULL, DTYPE = -1, -4


def dual(x):
    return forward_ad.make_dual(x, torch.ones_like(x))


def code(call):
    with pytest.raises(sg.GemmError) as e:
        call()
    return e.value.code, "tangent" in str(e.value)


@pytest.mark.parametrize("leaf", [False, True])
@pytest.mark.parametrize("given", [False, True])
def test_a_tangent_is_refused(leaf, given):
    a, b = (torch.zeros(n, 16, dtype=torch.bfloat16, requires_grad=leaf) for n in (6, 9))
    t = torch.zeros(6, dtype=torch.int64)
    x = torch.zeros(6, 16, requires_grad=leaf)
    ids = torch.zeros(6, 2, dtype=torch.int32)
    f, n = torch.zeros(6), torch.zeros((), dtype=torch.int32)
    xent = {"out": (f, f.clone())} if given else {}
    route = {"out": (torch.zeros(6, 2), ids)} if given else {}
    balance = {"out": (torch.zeros(()), torch.zeros(16, dtype=torch.int32), n)} if given else {}
    with forward_ad.dual_level():
        for grad in (True, False):
            with torch.set_grad_enabled(grad):
                assert code(lambda: sg.gemm_xent(dual(a), b, t, **xent)) == (DTYPE, True)
                assert code(lambda: sg.gemm_xent(a, dual(b), t, **xent)) == (DTYPE, True)
                assert code(lambda: sg.moe_route(dual(x), 2, **route)) == (DTYPE, True)
                assert code(lambda: sg.moe_balance(dual(x), ids, **balance)) == (DTYPE, True)
                # without a tangent nothing changes (here: no GPU)
                assert code(lambda: sg.gemm_xent(a, b, t, **xent)) == (NULL, False)
                assert code(lambda: sg.moe_route(x, 2, **route)) == (NULL, False)
                assert code(lambda: sg.moe_balance(x, ids, **balance)) == (NULL, False)


def test_functional_transforms_do_not_lose_it_either():
    a = torch.zeros(6, 16, dtype=torch.bfloat16)
    t = torch.zeros(6, dtype=torch.int64)
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: sg.gemm_xent(x, a, t)[0], (a,), (a,))
