"""The gradient of moe_route's weights through autograd."""
import math

import pytest
import torch

import dense_gemm_swizzled_amd as sg

pytestmark = pytest.mark.gpu


def logits(T, E, dtype, seed=0):
    return torch.randn(T, E, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kw", [
    dict(score="softmax"), dict(score="sigmoid", scale=2.5), dict(score="softmax", renorm=False),
    dict(score="sigmoid", renorm=False, n_groups=4, top_groups=2, group_score="top2")])
def test_weights_carry_the_gradient_of_the_logits(dtype, kw):
    x = logits(70, 40, dtype)
    x[3] = -math.inf
    bias = 0.1 * torch.randn(40, generator=torch.Generator().manual_seed(1)).cuda()
    want, want_ids = sg.moe_route(x, 5, bias=bias, **kw)
    assert not want.requires_grad
    leaf = x.clone().requires_grad_()
    w, ids = sg.moe_route(leaf, 5, bias=bias, **kw)
    assert torch.equal(w, want) and torch.equal(ids, want_ids)
    assert w.requires_grad and not ids.requires_grad
    g = torch.randn(70, 5, generator=torch.Generator().manual_seed(2)).cuda()
    w.backward(g)
    form = {n: kw[n] for n in ("score", "renorm", "scale") if n in kw}
    assert torch.equal(leaf.grad, sg.moe_route_backward(g, x, want_ids, **form))
    assert bool((leaf.grad[3] == 0).all()) and bool((leaf.grad != 0).any())


def test_a_router_learns_through_it():
    """The gradient of a router's weight matrix equals the one of the weights
    written in torch operations, the choice taken as given."""
    T, H, E, k = 90, 32, 24, 4
    x = logits(T, H, torch.float32, 3)
    wr = (logits(H, E, torch.float32, 4) / math.sqrt(H)).requires_grad_()
    c = logits(T, k, torch.float32, 5)
    w, ids = sg.moe_route(x @ wr, k, score="sigmoid", scale=1.5)
    (w * c).sum().backward()
    ref = wr.detach().double().cpu().requires_grad_()
    s = torch.sigmoid(x.double().cpu() @ ref).gather(1, ids.long().cpu())
    (1.5 * s / s.sum(1, keepdim=True) * c.double().cpu()).sum().backward()
    # Each gradient of a logit is off by up to 100 units of 2^-24 of its terms,
    # 1.5 max|c| / 4; the product over T tokens by another unit for each term
    # and T for the sum, and its operands' logits by H units.
    bound = (100 + T + H) * 2.0 ** -24 * 1.5 * (x.abs().t() @ c.abs().amax(1, keepdim=True)).max()
    assert float((wr.grad.cpu().double() - ref.grad).abs().max()) <= float(bound)
    assert float(ref.grad.abs().max()) > 100 * float(bound)


def test_gradients_of_any_layout_and_logits_of_any_pitch():
    wide = logits(30, 50, torch.bfloat16)
    x = wide[:, 7:39]
    want, ids = sg.moe_route(x, 3)
    leaf = x.detach().requires_grad_()
    w, _ = sg.moe_route(leaf, 3)
    one = torch.ones((), device="cuda").expand(30, 3)
    (dx,) = torch.autograd.grad(w, leaf, one, retain_graph=True)
    assert torch.equal(dx, sg.moe_route_backward(one.contiguous(), x, ids))
    g = logits(3, 30, torch.float32).t()
    (dx,) = torch.autograd.grad(w, leaf, g)
    assert torch.equal(dx, sg.moe_route_backward(g.contiguous(), x, ids))


def test_no_history_where_none_is_wanted():
    leaf = logits(9, 16, torch.float32).requires_grad_()
    with torch.no_grad():
        assert not sg.moe_route(leaf, 2)[0].requires_grad
    with torch.inference_mode():
        sg.moe_route(leaf, 2)
    out = (torch.empty(9, 2, device="cuda"), torch.empty(9, 2, dtype=torch.int32, device="cuda"))
    w, ids = sg.moe_route(leaf, 2, out=out)
    assert w is out[0] and ids is out[1] and not w.requires_grad
    assert sg.moe_route(leaf[:0], 2)[0].shape == (0, 2)
    w, _ = sg.moe_route(leaf, 2)
    (dx,) = torch.autograd.grad(w, leaf, torch.ones_like(w), create_graph=True)
    with pytest.raises(RuntimeError):                 # differentiable once
        dx.sum().backward()


def test_changed_logits_are_noticed():
    leaf = logits(9, 16, torch.float32).requires_grad_()
    x = leaf * 1.0
    w, _ = sg.moe_route(x, 2)
    with torch.no_grad():
        x.zero_()
    with pytest.raises(RuntimeError, match="modified"):
        torch.autograd.grad(w, leaf, torch.ones_like(w))


def test_forward_and_gradient_in_a_graph():
    x = logits(40, 32, torch.float32).requires_grad_()
    g = logits(40, 4, torch.float32, 1)

    def step():
        # (No graph of x outlives the step: a captured one and an eager one of
        # the same leaf would belong to two streams.)
        w, ids = sg.moe_route(x, 4, score="sigmoid")
        return w.detach(), ids, torch.autograd.grad(w, x, g)[0]

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
            x.copy_(logits(40, 32, torch.float32, 10 + i))
        graph.replay()
        torch.cuda.synchronize()
        got_now = [t.detach().clone() for t in got]
        for a, b in zip(got_now, step()):
            assert torch.equal(a, b)
