"""Outputs of the cross entropy beside their inputs in one buffer are taken, over
them refused."""
import pytest
import torch

import dense_gemm_swizzled_amd as sg

import _xent_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("M", [40, 300])
def test_side_by_side_in_one_buffer(M):
    N, K = 700, 64
    A, B, t = ref.inputs(M, N, K, BF, 5)
    _, lse = sg.gemm_xent(A, B, t)
    d = torch.rand(M, device="cuda") / M
    want = sg.gemm_xent_backward(d, A, B, t, lse)
    tokens = torch.zeros(M, 2 * K + 8, dtype=BF, device="cuda")
    words = torch.zeros(N, 2 * K, dtype=BF, device="cuda")
    tokens[:, :K], words[:, K:] = A, B
    out = tokens[:, K + 8:], words[:, :K]
    got = sg.gemm_xent_backward(d, tokens[:, :K], words[:, K:], t, lse, out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(tokens[:, :K], A) and torch.equal(words[:, K:], B)
    # one behind the other
    both = torch.cat([A, torch.zeros_like(A)])
    got, _ = sg.gemm_xent_backward(d, both[:M], B, t, lse, out=(both[M:], None),
                                   need=(True, False))
    assert torch.equal(got, want[0])


@pytest.mark.parametrize("M", [40, 300])
def test_over_an_input(M):
    A, B, t = ref.inputs(M, 700, 64, BF, 6)
    loss, lse = sg.gemm_xent(A, B, t)
    before = A.clone(), B.clone()

    def code(call):
        with pytest.raises(sg.GemmError, match="overlaps") as e:
            call()
        return e.value.code

    back = sg.gemm_xent_backward
    for out in ((A, None), (None, B), (A, B), (B[:M], None)):
        assert code(lambda: back(loss, A, B, t, lse, out=out)) == -2
    x = torch.zeros(M, device="cuda")
    assert code(lambda: sg.gemm_xent(A, B, t, out=(x, x))) == -2
    torch.cuda.synchronize()
    assert torch.equal(A, before[0]) and torch.equal(B, before[1])
