"""Refusals of the expert-routing and 8-bit entry points: the C ABI and the
torch wrappers, all before any GPU call (no GPU)."""
import pytest
import torch

import dense_gemm_swizzled_amd as sg

NULL, ALIGN, SHAPE, DTYPE, MAJOR, GROUPS = -1, -2, -3, -4, -5, -6
P = 0x10000  # an aligned fake device address (never dereferenced)


def _gemm(**kw):
    a = dict(M=33, N=40, K=64, A=P, lda=64, SA=P, B=P, ldb=64, SB=P, D=P, ldd=40,
             d_dtype=sg.SG_BF16)
    a.update(kw)
    return sg.i8_gemm_run(a["M"], a["N"], a["K"], a["A"], a["lda"], a["SA"], a["B"], a["ldb"],
                          a["SB"], a["D"], a["ldd"], a["d_dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), SHAPE), (dict(K=72, lda=80, ldb=80), SHAPE), (dict(K=131072, lda=131072,
                                                                    ldb=131072), SHAPE),
    (dict(lda=48), SHAPE), (dict(ldb=48), SHAPE), (dict(ldd=39), SHAPE),
    (dict(lda=72), ALIGN), (dict(ldb=72), ALIGN), (dict(A=P + 8), ALIGN), (dict(B=P + 1), ALIGN),
    (dict(SA=P + 2), ALIGN), (dict(SB=P + 2), ALIGN), (dict(D=P + 1), ALIGN),
    (dict(A=None), NULL), (dict(B=None), NULL), (dict(SA=None), NULL), (dict(SB=None), NULL),
    (dict(D=None), NULL), (dict(d_dtype=sg.SG_E4M3), DTYPE), (dict(d_dtype=0), DTYPE),
    (dict(lda=1 << 30), SHAPE), (dict(ldb=1 << 30), SHAPE), (dict(M=1 << 31), SHAPE),
    (dict(N=1 << 31, ldd=1 << 31), SHAPE),
])
def test_i8_gemm_run_rejects(kw, code):
    assert _gemm(**kw) == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("i8_gemm_run")


def test_empty_products_do_nothing():
    assert _gemm(M=0, A=None, SA=None, D=None) == 0
    assert _gemm(N=0, B=None, SB=None, D=None) == 0
    assert sg.i8_quant_run(0, 64, None, 64, sg.SG_F32, None, 64, None, None) == 0
    assert sg.moe_route_run(0, 8, 2, None, 8, sg.SG_F32, None, 0, 1, 1, 0, 1, 1.0, None, None,
                            None) == 0
    assert sg.moe_route_backward_run(0, 8, 2, None, None, 8, sg.SG_F32, None, 0, 1, 1.0, None, 8,
                                     None) == 0


def _grouped(**kw):
    a = dict(G=4, R=33, N=40, K=64, offsets=P, A=P, lda=64, a_rows=33, rows=P, SA=P, B=P, SB=P,
             D=P, ldd=40, d_dtype=sg.SG_F32)
    a.update(kw)
    return sg.i8_grouped_gemm_run(a["G"], a["R"], a["N"], a["K"], a["offsets"], a["A"], a["lda"],
                                  a["a_rows"], a["rows"], a["SA"], a["B"], a["SB"], a["D"],
                                  a["ldd"], a["d_dtype"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(G=0), GROUPS), (dict(G=257), GROUPS), (dict(offsets=None), NULL),
    (dict(rows=None, a_rows=32), SHAPE), (dict(a_rows=-1), SHAPE), (dict(R=-1), SHAPE),
    (dict(a_rows=1 << 26), SHAPE),       # gathered rows beyond 32-bit offsets
    (dict(offsets=P + 2), ALIGN), (dict(rows=P + 2), ALIGN), (dict(K=40, lda=48), SHAPE),
    (dict(A=None), NULL), (dict(SA=None), NULL), (dict(B=None), NULL), (dict(SB=None), NULL),
    (dict(lda=1 << 30, rows=None), SHAPE),
])
def test_i8_grouped_gemm_run_rejects(kw, code):
    assert _grouped(**kw) == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("i8_grouped_gemm_run")


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), SHAPE), (dict(K=-1), SHAPE), (dict(ldx=40), SHAPE), (dict(ldq=48), SHAPE),
    (dict(ldq=56), SHAPE), (dict(ldq=72), ALIGN), (dict(Q=P + 8), ALIGN), (dict(X=P + 1), ALIGN),
    (dict(S=P + 2), ALIGN), (dict(X=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL),
    (dict(dt=sg.SG_E4M3), DTYPE),
])
def test_i8_quant_run_rejects(kw, code):
    a = dict(R=3, K=50, X=P, ldx=50, dt=sg.SG_BF16, Q=P, ldq=64, S=P)
    a.update(kw)
    rc = sg.i8_quant_run(a["R"], a["K"], a["X"], a["ldx"], a["dt"], a["Q"], a["ldq"], a["S"],
                         None)
    assert rc == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("i8_quant_run")


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(E=0, k=1), SHAPE), (dict(E=257, ldl=300), SHAPE),
    (dict(k=0), SHAPE), (dict(k=33, E=64), SHAPE), (dict(k=17), SHAPE), (dict(ldl=15), SHAPE),
    (dict(dt=sg.SG_E8M0), DTYPE), (dict(score=2), DTYPE), (dict(groups=3), GROUPS),
    (dict(groups=0), GROUPS), (dict(groups=4, top=5), GROUPS), (dict(groups=4, top=0), GROUPS),
    (dict(groups=4, top=1, k=5), GROUPS), (dict(gs=2), GROUPS), (dict(logits=None), NULL),
    (dict(w=None), NULL), (dict(ids=None), NULL), (dict(logits=P + 1), ALIGN),
    (dict(bias=P + 2), ALIGN), (dict(w=P + 2), ALIGN), (dict(ids=P + 1), ALIGN),
])
def test_moe_route_run_rejects(kw, code):
    a = dict(T=3, E=16, k=2, logits=P, ldl=16, dt=sg.SG_BF16, bias=None, score=0, groups=1, top=1,
             gs=0, w=P, ids=P)
    a.update(kw)
    a["ldl"] = max(a["ldl"], a["E"]) if "ldl" not in kw else a["ldl"]
    rc = sg.moe_route_run(a["T"], a["E"], a["k"], a["logits"], a["ldl"], a["dt"], a["bias"],
                          a["score"], a["groups"], a["top"], a["gs"], 1, 1.0, a["w"], a["ids"],
                          None)
    assert rc == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("moe_route_run")


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(k=17), SHAPE), (dict(ldl=15), SHAPE), (dict(ldd=15), SHAPE),
    (dict(dt=0), DTYPE), (dict(score=-1), DTYPE), (dict(dw=None), NULL), (dict(ids=None), NULL),
    (dict(out=None), NULL), (dict(logits=None), NULL), (dict(dw=P + 1), ALIGN),
    (dict(out=P + 1), ALIGN),
])
def test_moe_route_backward_run_rejects(kw, code):
    a = dict(T=3, E=16, k=2, dw=P, logits=P, ldl=16, dt=sg.SG_F16, ids=P, score=0, out=P, ldd=16)
    a.update(kw)
    rc = sg.moe_route_backward_run(a["T"], a["E"], a["k"], a["dw"], a["logits"], a["ldl"],
                                   a["dt"], a["ids"], a["score"], 1, 1.0, a["out"], a["ldd"],
                                   None)
    assert rc == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("moe_route_backward_run")


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(E=257), SHAPE), (dict(k=0), SHAPE),
    (dict(k=257), SHAPE), (dict(T=1 << 30, k=2), SHAPE), (dict(ids=None), NULL),
    (dict(offsets=None), NULL), (dict(rows=None), NULL), (dict(slots=None), NULL),
    (dict(ids=P + 2), ALIGN), (dict(ws=P + 2), ALIGN), (dict(T=9000, ws=P, wsb=16), SHAPE),
    (dict(T=9000, ws=None, wsb=1 << 20), NULL),
])
def test_moe_plan_run_rejects(kw, code):
    a = dict(T=3, E=16, k=2, ids=P, offsets=P, rows=P, slots=P, ws=None, wsb=0)
    a.update(kw)
    rc = sg.moe_plan_run(a["T"], a["E"], a["k"], a["ids"], a["offsets"], a["rows"], a["slots"],
                         a["ws"], a["wsb"], None)
    assert rc == code, sg.gemm_last_error()
    assert sg.gemm_last_error().startswith("moe_plan_run")


def test_plan_workspace_bytes():
    assert sg.moe_plan_workspace_bytes(0, 8) == 0
    assert sg.moe_plan_workspace_bytes(4096, 256) == 0
    assert sg.moe_plan_workspace_bytes(16384, 256) == 0
    n = sg.moe_plan_workspace_bytes(16385, 8)
    assert n > 0 and n % (8 * 4) == 0
    # never more than 256 workgroups' counts, however many pairs
    assert sg.moe_plan_workspace_bytes((1 << 31) - 1, 256) <= 256 * 256 * 4
    assert sg.moe_plan_workspace_bytes(-1, 8) == SHAPE
    assert sg.moe_plan_workspace_bytes(8, 257) == SHAPE
    assert sg.moe_plan_workspace_bytes(1 << 31, 8) == SHAPE


# ------------------------------------------------------------ torch wrappers

def _code(fn, *a, **kw):
    with pytest.raises(sg.GemmError) as e:
        fn(*a, **kw)
    return e.value.code


def i8(*shape):
    return torch.zeros(*shape, dtype=torch.int8)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_i8_gemm_checks():
    A, B, sa, sb = i8(8, 32), i8(4, 32), torch.ones(8), torch.ones(4)
    assert _code(sg.i8_gemm, A, sa, B, sb) == NULL          # only the device is wrong
    assert _code(sg.i8_gemm, i8(8, 64)[:, :32], sa, B, sb, out=torch.zeros(8, 7)[:, :4]) == NULL
    assert _code(sg.i8_gemm, A, sa, i8(4, 48), sb) == SHAPE
    assert _code(sg.i8_gemm, A, torch.ones(4), B, sb) == SHAPE
    assert _code(sg.i8_gemm, A, torch.ones(8, 1), B, sb) == SHAPE
    assert _code(sg.i8_gemm, A, torch.ones(16)[::2], B, sb) == ALIGN
    assert _code(sg.i8_gemm, A, sa.double(), B, sb) == DTYPE
    assert _code(sg.i8_gemm, A.float(), sa, B, sb) == DTYPE
    assert _code(sg.i8_gemm, A, sa, B.to(torch.uint8), sb) == DTYPE
    assert _code(sg.i8_gemm, i8(32, 8).t(), sa, B, sb) == ALIGN
    assert _code(sg.i8_gemm, i8(1, 32).expand(8, 32), sa, B, sb) == ALIGN
    assert _code(sg.i8_gemm, A, sa, B, sb, out=torch.zeros(4, 8).t()) == ALIGN
    assert _code(sg.i8_gemm, A, sa, B, sb, out=torch.zeros(8, 5)) == SHAPE
    assert _code(sg.i8_gemm, A, sa, B, sb, out=i32(8, 4)) == DTYPE


def test_i8_grouped_gemm_checks():
    A, B = i8(8, 32), i8(3, 4, 32)
    sa, sb, off, rows = torch.ones(8), torch.ones(3, 4), i32(4), i32(20)
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb, off) == NULL
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb, off, rows=rows, out=torch.zeros(20, 4)) == NULL
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb, i32(3)) == SHAPE
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb, off.long()) == DTYPE
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb, off, rows=rows.long()) == DTYPE
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb, off, rows=i32(4, 5)) == SHAPE
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb, off, rows=i32(40)[::2]) == ALIGN
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb[0], off) == SHAPE
    assert _code(sg.i8_grouped_gemm, A, sa, B[:, :, :16], sb, off) == ALIGN
    assert _code(sg.i8_grouped_gemm, i8(8, 48), sa, B, sb, off) == SHAPE
    assert _code(sg.i8_grouped_gemm, A, sa, B, sb, off, rows=rows, out=torch.zeros(8, 4)) == SHAPE


def test_i8_quant_checks():
    X = torch.zeros(4, 20)
    assert _code(sg.i8_quant, X) == NULL
    assert _code(sg.i8_quant, X[:, 1:7], out=i8(4, 16), out_scale=torch.zeros(4)) == NULL
    assert _code(sg.i8_quant, X.t()) == ALIGN
    assert _code(sg.i8_quant, X.double()) == DTYPE
    assert _code(sg.i8_quant, X[0]) == SHAPE
    assert _code(sg.i8_quant, X, out=i8(4, 20)) == SHAPE
    assert _code(sg.i8_quant, X, out_scale=torch.zeros(5)) == SHAPE
    assert _code(sg.i8_quant, X, out=i8(4, 32).to(torch.uint8)) == DTYPE


def test_moe_route_checks():
    x = torch.zeros(6, 16)
    assert _code(sg.moe_route, x, 2) == NULL
    assert _code(sg.moe_route, x[:, 1:9], 2, bias=torch.zeros(8)) == NULL
    assert _code(sg.moe_route, x.t(), 2) == ALIGN
    assert _code(sg.moe_route, x[0], 2) == SHAPE
    assert _code(sg.moe_route, x, 0) == SHAPE
    assert _code(sg.moe_route, x, 17) == SHAPE
    assert _code(sg.moe_route, x.double(), 2) == DTYPE
    assert _code(sg.moe_route, x, 2, score="tanh") == DTYPE
    assert _code(sg.moe_route, x, 2, group_score="mean") == GROUPS
    assert _code(sg.moe_route, x, 2, bias=torch.zeros(15)) == SHAPE
    assert _code(sg.moe_route, x, 2, bias=torch.zeros(16, dtype=torch.bfloat16)) == DTYPE
    assert _code(sg.moe_route, x, 2, out=(torch.zeros(6, 3), i32(6, 2))) == SHAPE
    assert _code(sg.moe_route, x, 2, out=(torch.zeros(6, 2), torch.zeros(6, 2))) == DTYPE


def test_moe_route_backward_checks():
    x, ids, dw = torch.zeros(6, 16), i32(6, 2), torch.zeros(6, 2)
    assert _code(sg.moe_route_backward, dw, x, ids) == NULL
    assert _code(sg.moe_route_backward, dw, x, ids, out=torch.zeros(6, 20)[:, :16]) == NULL
    assert _code(sg.moe_route_backward, dw, x, i32(5, 2)) == SHAPE
    assert _code(sg.moe_route_backward, dw, x, ids.long()) == DTYPE
    assert _code(sg.moe_route_backward, dw[:, :1], x, ids) == ALIGN
    assert _code(sg.moe_route_backward, dw.half(), x, ids) == DTYPE
    assert _code(sg.moe_route_backward, dw, x, ids, out=torch.zeros(6, 16).half()) == DTYPE
    assert _code(sg.moe_route_backward, dw, x, ids, out=torch.zeros(6, 15)) == SHAPE


def test_moe_plan_checks():
    ids = i32(6, 2)
    assert _code(sg.moe_plan, ids, 8) == NULL
    assert _code(sg.moe_plan, ids.long(), 8) == DTYPE
    assert _code(sg.moe_plan, ids[0], 8) == SHAPE
    assert _code(sg.moe_plan, i32(2, 6).t(), 8) == ALIGN
    assert _code(sg.moe_plan, ids, 0) == SHAPE
    assert _code(sg.moe_plan, ids, 257) == SHAPE
    assert _code(sg.moe_plan, ids, 8, out=(i32(8), i32(12), i32(6, 2))) == SHAPE
    assert _code(sg.moe_plan, ids, 8, out=(i32(9), i32(12), i32(6, 3))) == SHAPE
    big = i32(9000, 2)
    assert _code(sg.moe_plan, big, 8, workspace=torch.zeros(8, dtype=torch.uint8)) == SHAPE
    assert _code(sg.moe_plan, big, 8, workspace=torch.zeros(1 << 16)) == DTYPE


# Sizes that a C int or a byte offset does not hold are refused, not wrapped.
@pytest.mark.parametrize("ld", [1 << 31, 1 << 56, 1 << 57, 1 << 62])
def test_pitches_that_overflow(ld):
    assert _gemm(lda=ld) == SHAPE
    assert _gemm(ldb=ld) == SHAPE
    assert _gemm(M=4097, lda=ld) == SHAPE
    assert _grouped(lda=ld) == SHAPE
    assert _grouped(lda=ld, rows=None) == SHAPE


def test_sizes_beyond_32_bits():
    wide, x, ids = (1 << 32) + 8, torch.zeros(6, 16), i32(6, 2)
    assert _code(sg.moe_plan, ids, wide) == SHAPE
    assert _code(sg.moe_plan, i32(0, wide), 8) == SHAPE
    assert _code(sg.moe_route, torch.zeros(0, wide), 2) == SHAPE
    assert _code(sg.moe_route, x, 2, n_groups=wide) == SHAPE
    assert _code(sg.moe_route, x, 2, n_groups=8, top_groups=wide) == SHAPE
    assert _code(sg.moe_route_backward, torch.zeros(0, 2), torch.zeros(0, wide), i32(0, 2)) == SHAPE
    assert _code(sg.moe_route_backward, torch.zeros(0, wide), torch.zeros(0, 16),
                 i32(0, wide)) == SHAPE
    assert _code(sg.i8_grouped_gemm, i8(8, 16), torch.ones(8), i8(wide, 0, 16),
                 torch.zeros(wide, 0), i32(9)) == SHAPE
