"""The gradient of the vocabulary's matrix from up to 512 tokens on 256x128 tiles
(xent_twin_kernel): tokens, words and hidden sizes that end inside a stage, a tile
and a fragment, alone, with dA's sum beside it, and in several runs of words."""
import math

import pytest
import torch

import dense_gemm_swizzled_amd as sg

import _xent_ref as ref
from test_gpu_xent import check

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def twin():
    return sg.gemm_last_kernel().startswith("xent_twin_kernel")


@pytest.mark.parametrize("M,N,K", [
    (1, 40003, 264), (33, 20001, 520), (40, 66001, 72), (64, 8192, 1024), (65, 30001, 520),
    (257, 20003, 776), (511, 30001, 520), (512, 20032, 1024)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_sizes(M, N, K, dtype):
    A, B, t = ref.inputs(M, N, K, dtype, M + N + K)
    _, _, _, dB = check(A, B, t)
    assert twin()
    _, _, none, alone = check(A, B, t, need=(False, True))
    assert twin() and none is None and torch.equal(alone, dB)
    check(A, B, t, need=(True, False))


def test_up_to_512_tokens():
    A, B, t = ref.inputs(513, 20032, 1024, BF, 1)
    check(A, B, t)
    assert not twin()


@pytest.mark.parametrize("M", [50, 300])
def test_pitches_hold_anything(M):
    N, K = 30001, 520
    A, B, t = ref.inputs(M, N, K, BF, 9)
    wa = torch.full((M, K + 24), math.nan, dtype=BF, device="cuda")
    wb = torch.full((N, K + 8), math.nan, dtype=BF, device="cuda")
    wa[:, 8:K + 8], wb[:, :K] = A, B
    want = check(A, B, t)
    da = torch.full((M, K + 16), 7.0, dtype=BF, device="cuda")
    db = torch.full((N + 2, K + 40), 7.0, dtype=BF, device="cuda")
    got = check(wa[:, 8:K + 8], wb[:, :K], t, out=(da[:, 8:K + 8], db[1:N + 1, 16:K + 16]))
    assert twin()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert bool((da[:, :8] == 7).all() and (da[:, K + 8:] == 7).all())
    assert bool((db[:, :16] == 7).all() and (db[:, K + 16:] == 7).all())
    assert bool((db[0] == 7).all() and (db[N + 1] == 7).all())


def test_runs_of_words():
    """Two runs, the last of other sizes: dA's sum is beside dB's last one."""
    M, N, K = 500, 600001, 264
    assert sg.gemm_xent_backward_workspace_bytes(M, N, K, K) < 2 * M * N + (1 << 27)
    A, B, t = ref.inputs(M, N, K, BF, 3)
    check(A, B, t)
    assert twin()


def test_in_a_graph():
    """Replays among eager work of other data give the eager results."""
    M, N, K = 60, 20011, 520
    A, B, t = ref.inputs(M, N, K, BF, 6)
    d = torch.rand(M, device="cuda") + 0.5
    out = torch.empty_like(A), torch.empty_like(B)

    def step():
        _, lse = sg.gemm_xent(A, B, t)
        sg.gemm_xent_backward(d, A, B, t, lse, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    assert twin()
    for seed in range(3):
        a, b, u = ref.inputs(M, N, K, BF, 20 + seed)
        A.copy_(a), B.copy_(b), t.copy_(u)
        _, lse = sg.gemm_xent(a, b, u)
        dA, dB = sg.gemm_xent_backward(d, a, b, u, lse)
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], dA) and torch.equal(out[1], dB)
