"""Sizes of the 8-bit products beyond one launch (no GPU)."""
import pytest

import dense_gemm_swizzled_amd as sg

SHAPE = -3
P = 0x10000  # an aligned fake device address (never dereferenced)


# More tiles than a launch of 512 threads each can have, whose threads along x
# stay below 2^32: one row of 2^29 columns (16 x 64 tiles), 16 rows of many
# columns with a long K (16 x 32), and 256 x 256 tiles past the limit.
@pytest.mark.parametrize("M,N,K", [(1, 1 << 29, 16), (16, 1 << 28, 4096),
                                   ((1 << 31) - 1, 64, 16), (1 << 24, 1 << 24, 128)])
def test_more_tiles_than_a_launch_has(M, N, K):
    for ldd in (N, N + 8):
        assert sg.i8_gemm_run(M, N, K, P, K, P, P, K, P, P, ldd, sg.SG_BF16, None) == SHAPE
        assert "tiles" in sg.gemm_last_error()


@pytest.mark.parametrize("G,R,N,K", [(1, (1 << 31) - 1, 1, 16), (256, 1, 1 << 29, 16), (256, 2000, 1 << 24, 16)])
@pytest.mark.parametrize("gather", [True, False])
def test_more_grouped_tiles_than_a_launch_has(G, R, N, K, gather):
    a_rows = 100 if gather else R
    rc = sg.i8_grouped_gemm_run(G, R, N, K, P, P, K, a_rows, P if gather else None, P, P, P, P, N,
                                sg.SG_F32, None)
    assert rc == SHAPE and "tiles" in sg.gemm_last_error()
