"""Refusals of the cross entropy's entry points, before any GPU call (no GPU)."""
import pytest
import torch

import dense_gemm_swizzled_amd as sg

NULL, ALIGN, SHAPE, DTYPE = -1, -2, -3, -4
P = 0x10000  # an aligned fake device address (never dereferenced)
BIG = 1 << 40


def _run(**kw):
    a = dict(M=33, N=50, K=64, alpha=1.0, A=P, lda=64, B=P, ldb=64, dt=sg.SG_BF16, t=P,
             tt=sg.SG_I64, loss=P, lse=P, w=P, wb=BIG)
    a.update(kw)
    return sg.gemm_xent_run(a["M"], a["N"], a["K"], a["alpha"], a["A"], a["lda"], a["B"],
                            a["ldb"], a["dt"], a["t"], a["tt"], a["loss"], a["lse"], a["w"],
                            a["wb"], None)


def _back(**kw):
    a = dict(M=33, N=50, K=64, alpha=1.0, dloss=P, dlse=None, A=P, lda=64, B=P, ldb=64,
             dt=sg.SG_BF16, t=P, tt=sg.SG_I64, lse=P, dA=P, ldda=64, dB=P, lddb=64, w=P, wb=BIG)
    a.update(kw)
    return sg.gemm_xent_backward_run(a["M"], a["N"], a["K"], a["alpha"], a["dloss"], a["dlse"],
                                     a["A"], a["lda"], a["B"], a["ldb"], a["dt"], a["t"],
                                     a["tt"], a["lse"], a["dA"], a["ldda"], a["dB"], a["lddb"],
                                     a["w"], a["wb"], None)


BOTH = [
    (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(K=-8), SHAPE), (dict(K=60), SHAPE),
    (dict(M=1 << 31), SHAPE), (dict(N=1 << 31), SHAPE), (dict(lda=56), SHAPE),
    (dict(ldb=56), SHAPE), (dict(lda=1 << 22), SHAPE), (dict(ldb=1 << 22), SHAPE),
    (dict(lda=68), ALIGN), (dict(ldb=68), ALIGN), (dict(A=P + 8), ALIGN), (dict(B=P + 2), ALIGN),
    (dict(t=P + 4), ALIGN), (dict(tt=sg.SG_I32, t=P + 2), ALIGN), (dict(w=P + 8), ALIGN),
    (dict(lse=P + 2), ALIGN), (dict(A=None), NULL), (dict(B=None), NULL), (dict(t=None), NULL),
    (dict(lse=None), NULL), (dict(w=None), NULL), (dict(wb=0), SHAPE),
    (dict(dt=sg.SG_F32), DTYPE), (dict(dt=sg.SG_E4M3), DTYPE), (dict(tt=sg.SG_F32), DTYPE),
    (dict(tt=0), DTYPE), (dict(M=1 << 22, N=1 << 30), SHAPE),
]


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(loss=None), NULL), (dict(loss=P + 1), ALIGN),
    (dict(wb=33 * 8 + 33 * 4 - 1), SHAPE)])
def test_gemm_xent_run_rejects(kw, code):
    assert _run(**kw) == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("gemm_xent_run")


@pytest.mark.parametrize("kw,code", BOTH + [
    (dict(M=1 << 22), SHAPE), (dict(ldda=56), SHAPE), (dict(lddb=56), SHAPE),
    (dict(ldda=68), ALIGN), (dict(lddb=68), ALIGN), (dict(dA=P + 8), ALIGN),
    (dict(dB=P + 8), ALIGN), (dict(dloss=None), NULL), (dict(dloss=P + 2), ALIGN),
    (dict(dlse=P + 1), ALIGN), (dict(M=1 << 20, lda=1 << 11), SHAPE),
    (dict(wb=sg.gemm_xent_backward_workspace_bytes(33, 50, 64, 64) - 1), SHAPE)])
def test_gemm_xent_backward_run_rejects(kw, code):
    assert _back(**kw) == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("gemm_xent_backward_run")


def test_calls_that_have_nothing_to_do():
    assert _run(M=0, A=None, t=None, loss=None, lse=None, w=None, wb=0) == 0
    assert _back(dA=None, dB=None, w=None, wb=0) == 0
    assert _back(K=0, lda=0, ldb=0, ldda=0, lddb=0, A=None, B=None, w=None, wb=0) == 0
    assert _back(M=0, dB=None, A=None, t=None, dloss=None, lse=None, w=None, wb=0) == 0
    assert _back(N=0, dA=None, B=None, w=None, wb=0) == 0


def test_workspaces():
    # two floats a token and 256-word tile, one more a token
    assert sg.gemm_xent_workspace_bytes(8192, 131072, 4096) == 8192 * (512 * 8 + 4)
    assert sg.gemm_xent_workspace_bytes(0, 5, 8) == 0
    for M, N, K in ((-1, 5, 8), (5, -1, 8), (5, 5, -8), (1 << 31, 5, 8)):
        assert sg.gemm_xent_workspace_bytes(M, N, K) == SHAPE
    for M, N, K, ldb in ((-1, 5, 8, 8), (1 << 22, 5, 8, 8), (5, 5, 8, 0), (5, 5, 8, 1 << 22)):
        assert sg.gemm_xent_backward_workspace_bytes(M, N, K, ldb) == SHAPE
    # The gradient of the logits stays within 512 MB (or 256 words) and every
    # product's operands below 2^31 bytes.
    for M in (1, 63, 8192, 100003, (1 << 22) - 1):
        for N in (1, 300, 131072, (1 << 31) - 1):
            for ldb in (64, 8192, (1 << 22) - 8):
                n = sg.gemm_xent_backward_workspace_bytes(M, N, 64, ldb)
                # (besides: the tokens' terms, the sums of dA with up to 256
                # workgroups of 128 x 128 values or one of M x K)
                assert 0 < n <= max(1 << 29, 512 * M) + 16 * M + 4096 + 256 * M + (1 << 24)


def test_wrappers_refuse():
    a = torch.zeros(6, 16, dtype=torch.bfloat16)
    b = torch.zeros(9, 16, dtype=torch.bfloat16)
    t = torch.zeros(6, dtype=torch.int64)
    f = torch.zeros(6)

    def code(call):
        with pytest.raises(sg.GemmError) as e:
            call()
        return e.value.code

    for w in (a, a.clone().requires_grad_()):
        assert code(lambda: sg.gemm_xent(w, b, t)) == NULL                # not on a GPU
        assert code(lambda: sg.gemm_xent(w, b[:, :8], t)) == SHAPE
        assert code(lambda: sg.gemm_xent(w, b.half(), t)) == DTYPE
        assert code(lambda: sg.gemm_xent(w.float(), b.float(), t)) == DTYPE
        assert code(lambda: sg.gemm_xent(w, b, t[:5])) == SHAPE
        assert code(lambda: sg.gemm_xent(w, b, t.float())) == DTYPE
        assert code(lambda: sg.gemm_xent(w, b, torch.zeros(12, dtype=torch.int64)[::2])) == ALIGN
        assert code(lambda: sg.gemm_xent(w.t(), b, t)) == ALIGN
        assert code(lambda: sg.gemm_xent(w[0], b, t)) == SHAPE
    assert code(lambda: sg.gemm_xent(a, b, t, out=(f[:5], f))) == SHAPE
    back = sg.gemm_xent_backward
    assert code(lambda: back(f, a, b, t, f)) == NULL
    assert code(lambda: back(f.double(), a, b, t, f)) == DTYPE
    assert code(lambda: back(f, a, b, t, f[:5])) == SHAPE
    assert code(lambda: back(f, a, b, t, f, dlse=f[:3])) == SHAPE
    assert code(lambda: back(f, a, b, t, f, out=(b, b))) == SHAPE
    assert code(lambda: back(f, a, b, t, f, out=(a, b.half()))) == DTYPE
    assert code(lambda: back(f.expand(2, 6)[0][:1].expand(6), a, b, t, f)) == ALIGN
