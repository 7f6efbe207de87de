"""The cross entropy's calls refuse outputs and workspaces that overlap an input or
each other, before any GPU call (no GPU).  Areas of memory are laid out on fake
addresses, which are never dereferenced."""
import pytest

import dense_gemm_swizzled_amd as sg

ALIGN = -2
M, N, K = 33, 50, 64
ROW = 2 * K                                     # bytes of a packed row
W = sg.gemm_xent_workspace_bytes(M, N, K)
WB = sg.gemm_xent_backward_workspace_bytes(M, N, K, K)
AT = {name: 0x1000000 * (i + 1) for i, name in enumerate(
    ("A", "B", "targets", "loss", "lse", "dloss", "dlse", "dA", "dB", "work"))}


def run(**at):
    a = {**AT, **at}
    return sg.gemm_xent_run(M, N, K, 1.0, a["A"], K, a["B"], K, sg.SG_BF16, a["targets"],
                            sg.SG_I64, a["loss"], a["lse"], a["work"], W, None)


def back(lda=K, ldb=K, ldda=K, lddb=K, **at):
    a = {**AT, **at}
    need = sg.gemm_xent_backward_workspace_bytes(M, N, K, ldb)
    return sg.gemm_xent_backward_run(M, N, K, 1.0, a["dloss"], a["dlse"], a["A"], lda, a["B"],
                                     ldb, sg.SG_BF16, a["targets"], sg.SG_I64, a["lse"], a["dA"],
                                     ldda, a["dB"], lddb, a["work"], need, None)


def refused(rc, call, *names):
    text = sg.gemm_last_error()
    assert rc == ALIGN and text.startswith(call) and "overlaps" in text, (rc, text)
    assert all(n in text for n in names), text


@pytest.mark.parametrize("out", ["loss", "lse", "work"])
@pytest.mark.parametrize("other,last", [
    ("A", M * ROW - 16), ("B", N * ROW - 16), ("targets", 8 * M - 8), ("loss", 4 * M - 4),
    ("lse", 4 * M - 4), ("work", W // 16 * 16 - 16)])
def test_forward(out, other, last):
    if out == other:
        return
    name = {"work": "workspace"}
    names = name.get(out, out), name.get(other, other)
    # (the addresses that are not "other" + 0 keep the alignment of `out`)
    refused(run(**{out: AT[other]}), "gemm_xent_run", *names)
    refused(run(**{out: AT[other] + last // 16 * 16}), "gemm_xent_run", *names)
    refused(run(**{out: AT[other] - 16}), "gemm_xent_run", *names)


@pytest.mark.parametrize("out", ["dA", "dB", "work"])
@pytest.mark.parametrize("other,size", [
    ("A", M * ROW), ("B", N * ROW), ("targets", 8 * M), ("dloss", 4 * M), ("dlse", 4 * M),
    ("lse", 4 * M), ("dA", M * ROW), ("dB", N * ROW), ("work", WB)])
def test_backward(out, other, size):
    if out == other:
        return
    name = {"work": "workspace"}
    names = name.get(out, out), name.get(other, other)
    for at in (0, (size - 1) // 16 * 16, -16):
        refused(back(**{out: AT[other] + at}), "gemm_xent_backward_run", *names)


def test_rows_that_lie_in_each_other():
    """Padded rows: the columns decide where the pitch is the same."""
    wide = 2 * K + 8
    for shift in (0, 8, K - 8, wide - K + 8, wide - 8, wide + 8, 5 * wide + K - 8):
        refused(back(lda=wide, ldda=wide, dA=AT["A"] + 2 * shift), "gemm_xent_backward_run",
                "dA", "A")
        refused(back(ldb=wide, lddb=wide, B=AT["dB"] + 2 * shift), "gemm_xent_backward_run",
                "dB", "B")
    # a vector in the padding is apart, across a row's end it is not
    refused(back(lda=wide, ldda=wide, dA=AT["lse"] - 2 * wide - 2 * wide + 16),
            "gemm_xent_backward_run", "dA", "lse")
    # two pitches: only one behind the other
    refused(back(lda=wide, ldda=wide + 8, dA=AT["A"] + 2 * K), "gemm_xent_backward_run", "dA", "A")




def test_pitches_that_no_memory_has():
    """(A single row has none; a vocabulary of one word, then one token.)"""
    huge = (1 << 62) + 64
    for m, n in ((M, 1), (1, N)):
        need = sg.gemm_xent_backward_workspace_bytes(m, n, K, K)
        rc = sg.gemm_xent_backward_run(
            m, n, K, 1.0, AT["dloss"], None, AT["A"], K, AT["B"], K, sg.SG_BF16, AT["targets"],
            sg.SG_I64, AT["lse"], AT["A"] if m == 1 else None, huge,
            AT["B"] if n == 1 else None, huge, AT["work"], need, None)
        refused(rc, "gemm_xent_backward_run", "dA" if m == 1 else "dB")
