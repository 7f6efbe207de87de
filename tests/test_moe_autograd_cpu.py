"""moe_route refuses logits that require a gradient as it does others (no GPU)."""
import pytest
import torch

import dense_gemm_swizzled_amd as sg

NULL, SHAPE, DTYPE, GROUPS = -1, -3, -4, -6


@pytest.mark.parametrize("args,kw,code", [
    ((2,), {}, NULL), ((0,), {}, SHAPE), ((17,), {}, SHAPE), ((2,), dict(score="tanh"), DTYPE),
    ((2,), dict(group_score="mean"), GROUPS), ((2,), dict(bias=torch.zeros(15)), SHAPE)])
def test_refusals(args, kw, code):
    x = torch.zeros(6, 16)
    for logits in (x, x.clone().requires_grad_(), x.clone().requires_grad_() * 2):
        with pytest.raises(sg.GemmError) as e:
            sg.moe_route(logits, *args, **kw)
        assert e.value.code == code
