"""Refusals of the balance loss's entry points, before any GPU call (no GPU)."""
import pytest
import torch

import dense_gemm_swizzled_amd as sg

NULL, ALIGN, SHAPE, DTYPE = -1, -2, -3, -4
P = 0x10000  # an aligned fake device address (never dereferenced)


def _run(**kw):
    a = dict(T=900, E=40, k=4, x=P, ldl=40, dt=sg.SG_F32, ids=P, score=0, loss=P, counts=P,
             tokens=P, w=P, wb=1 << 30)
    a.update(kw)
    return sg.moe_balance_run(a["T"], a["E"], a["k"], a["x"], a["ldl"], a["dt"], a["ids"],
                              a["score"], a["loss"], a["counts"], a["tokens"], a["w"], a["wb"],
                              None)


def _back(**kw):
    a = dict(T=900, E=40, dloss=P, x=P, ldl=40, dt=sg.SG_BF16, counts=P, tokens=P, score=1, d=P,
             ldd=40)
    a.update(kw)
    return sg.moe_balance_backward_run(a["T"], a["E"], a["dloss"], a["x"], a["ldl"], a["dt"],
                                       a["counts"], a["tokens"], a["score"], a["d"], a["ldd"],
                                       None)


BOTH = [(dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE), (dict(E=0), SHAPE), (dict(E=257, ldl=257),
                                                                            SHAPE),
        (dict(ldl=39), SHAPE), (dict(dt=sg.SG_E4M3), DTYPE), (dict(score=2), DTYPE),
        (dict(x=None), NULL), (dict(x=P + 1), ALIGN), (dict(counts=None), NULL),
        (dict(counts=P + 2), ALIGN), (dict(tokens=None), NULL), (dict(tokens=P + 1), ALIGN)]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(k=0), SHAPE), (dict(k=41), SHAPE), (dict(k=33), SHAPE), (dict(T=1 << 29), SHAPE),
    (dict(ids=None), NULL), (dict(ids=P + 2), ALIGN), (dict(loss=None), NULL),
    (dict(loss=P + 2), ALIGN), (dict(w=None), NULL), (dict(w=P + 4), ALIGN),
    (dict(wb=sg.moe_balance_workspace_bytes(900, 40) - 1), SHAPE)])
def test_moe_balance_run_rejects(kw, code):
    assert _run(**kw) == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("moe_balance_run")


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(ldd=39), SHAPE), (dict(d=None), NULL), (dict(d=P + 1), ALIGN), (dict(dloss=None), NULL),
    (dict(dloss=P + 2), ALIGN)])
def test_moe_balance_backward_run_rejects(kw, code):
    assert _back(**kw) == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("moe_balance_backward_run")


def test_sizes():
    assert _back(T=0, x=None, d=None, dloss=None, counts=None, tokens=None) == 0
    assert sg.moe_balance_workspace_bytes(256, 256) == 0
    for T in (257, 16384, 1 << 20, (1 << 31) - 1):
        assert 0 < sg.moe_balance_workspace_bytes(T, 256) <= 256 * 258 * 8
    for T, E in ((-1, 8), (1 << 31, 8), (5, 0), (5, 257)):
        assert sg.moe_balance_workspace_bytes(T, E) == SHAPE


def test_wrappers_refuse():
    x, ids = torch.zeros(6, 16), torch.zeros(6, 2, dtype=torch.int32)
    c, n, d = torch.zeros(16, dtype=torch.int32), torch.zeros((), dtype=torch.int32), \
        torch.zeros(())

    def code(call):
        with pytest.raises(sg.GemmError) as e:
            call()
        return e.value.code

    for w in (x, x.clone().requires_grad_()):
        assert code(lambda: sg.moe_balance(w, ids)) == NULL               # not on a GPU
        assert code(lambda: sg.moe_balance(w, ids, score="tanh")) == DTYPE
        assert code(lambda: sg.moe_balance(w, ids.long())) == DTYPE
        assert code(lambda: sg.moe_balance(w, ids[:5])) == SHAPE
        assert code(lambda: sg.moe_balance(w, ids[:, 0])) == SHAPE
        assert code(lambda: sg.moe_balance(w.double(), ids)) == DTYPE
    assert code(lambda: sg.moe_balance(x, ids, out=(d, c[:5], n))) == SHAPE
    assert code(lambda: sg.moe_balance(x, ids, out=(d.reshape(1), c, n))) == SHAPE
    back = sg.moe_balance_backward
    assert code(lambda: back(d, x, c, n)) == NULL
    assert code(lambda: back(d.double(), x, c, n)) == DTYPE
    assert code(lambda: back(d.reshape(1), x, c, n)) == SHAPE
    assert code(lambda: back(d, x, c.long(), n)) == DTYPE
    assert code(lambda: back(d, x, c[:3], n)) == SHAPE
    assert code(lambda: back(d, x, c, n, score="x")) == DTYPE
    assert code(lambda: back(d, x, c, n, out=x[:3])) == SHAPE
    assert code(lambda: back(d, x, c, n, out=x.half())) == DTYPE
