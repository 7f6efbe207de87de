"""Python binding of libswizzled_gemm.so (MI355X / gfx950 swizzled GEMM).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/swizzled_gemm.h``.  There is
no CPU fallback: if the shared library is missing, every call raises.

Two layers:

* ``gemm_run``, ``gemm_strided_run``, ``grouped_gemm_run``, ``mx_gemm_run``,
  ``mxfp4_gemm_run``, ``mxfp6_gemm_run``, ``mx_scales_blocks_bytes``,
  ``mx_scales_to_blocks``, ``mx_gemm_blocks_run``, ``gemm_layout_run``,
  ``gemm_layout128_run``, ``gemm_last_error``, ``gemm_version``,
  ``gemm_lds_layout``, ``gemm_lds_layout_mxfp6``, ``gemm_lds_layout_cblock``,
  ``gemm_lds_image``, ``i8_gemm_run``, ``i8_grouped_gemm_run``, ``i8_quant_run``,
  ``moe_route_run``, ``moe_route_backward_run``, ``moe_plan_run``,
  ``moe_plan_workspace_bytes``, ``moe_balance_run``, ``moe_balance_backward_run``,
  ``moe_balance_workspace_bytes``, ``gemm_xent_run``, ``gemm_xent_backward_run``,
  ``gemm_xent_workspace_bytes``, ``gemm_xent_backward_workspace_bytes``: the C entry points under the same names, taking
  integer device pointers.
* ``gemm``, ``gemm_strided``, ``grouped_gemm``, ``mx_gemm``, ``mxfp4_gemm``,
  ``mxfp6_gemm``, ``mx_scales_blocks``, ``mx_gemm_blocks``, ``gemm_layout``,
  ``gemm_layout128``, ``i8_gemm``, ``i8_grouped_gemm``, ``i8_quant``,
  ``moe_route``, ``moe_route_backward``, ``moe_plan``, ``moe_balance``,
  ``moe_balance_backward``, ``gemm_xent``, ``gemm_xent_backward``: the same calls on torch CUDA
  tensors (shapes read from the tensors, output allocated by torch, launched
  on torch's current stream).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

__all__ = [
    "SG_OK", "SG_F16", "SG_BF16", "SG_F32", "SG_E4M3", "SG_E8M0", "SG_NONE",
    "SG_K_MAJOR", "SG_MN_MAJOR", "SG_MAX_GROUPS", "GemmError",
    "gemm_run", "gemm_strided_run", "grouped_gemm_run", "mx_gemm_run", "mxfp4_gemm_run",
    "mxfp6_gemm_run", "gemm_layout_run", "gemm_layout128_run", "gemm_last_error",
    "gemm_version", "gemm_lds_layout", "gemm_lds_layout_mxfp6", "gemm_lds_layout_cblock",
    "gemm_lds_image", "gemm_lds_image_tile", "gemm_mfma_scale_probe", "SG_IMG_HALF",
    "SG_IMG_HALF_KEXACT", "SG_IMG_MN256", "SG_IMG_FP6", "SG_IMG_CBLOCK", "gemm_last_kernel", "gemm_clock_trace", "gemm_clock_probe", "gemm_clock_probe_waves",
    "SG_E2M1", "SG_E2M3", "SG_E3M2", "SG_SF_ROWS", "SG_SF_BLOCKS",
    "mx_scales_blocks_bytes", "mx_scales_to_blocks", "mx_gemm_blocks_run", "mx_scales_blocks",
    "mx_gemm_blocks",
    "gemm", "gemm_plan", "gemm_strided", "grouped_gemm", "mx_gemm", "mxfp4_gemm", "mxfp6_gemm",
    "gemm_layout", "gemm_layout_io", "gemm_layout_io_run",
    "gemm_layout128", "SG_LAYOUT_PAD16",
    "i8_gemm_run", "i8_grouped_gemm_run", "i8_quant_run", "moe_route_run",
    "moe_route_backward_run", "moe_plan_run", "moe_plan_workspace_bytes",
    "i8_gemm", "i8_grouped_gemm", "i8_quant", "moe_route", "moe_route_backward", "moe_plan",
    "SG_SCORE_SOFTMAX", "SG_SCORE_SIGMOID", "SG_GROUP_MAX", "SG_GROUP_TOP2", "SG_MAX_TOP_K",
    "SG_MAX_ROUTE_GROUPS",
    "moe_balance_run", "moe_balance_backward_run", "moe_balance_workspace_bytes",
    "moe_balance", "moe_balance_backward",
    "gemm_xent_run", "gemm_xent_backward_run", "gemm_xent_workspace_bytes",
    "gemm_xent_backward_workspace_bytes", "gemm_xent", "gemm_xent_backward", "SG_I32", "SG_I64",
    "library_path", "load",
]

SG_OK = 0
SG_NONE, SG_F16, SG_BF16, SG_F32, SG_E4M3, SG_E8M0 = 0, 1, 2, 3, 4, 5
SG_E2M1, SG_E2M3, SG_E3M2 = 6, 7, 8
SG_I32, SG_I64 = 9, 10
SG_SF_ROWS, SG_SF_BLOCKS = 0, 1
SG_K_MAJOR, SG_MN_MAJOR = 0, 1
SG_MAX_GROUPS = 256
SG_LAYOUT_PAD16 = -1
SG_SCORE_SOFTMAX, SG_SCORE_SIGMOID = 0, 1
SG_GROUP_MAX, SG_GROUP_TOP2 = 0, 1
SG_MAX_TOP_K, SG_MAX_ROUTE_GROUPS = 32, 32
ERRORS = {-1: "SG_ERR_NULL", -2: "SG_ERR_ALIGN", -3: "SG_ERR_SHAPE",
          -4: "SG_ERR_DTYPE", -5: "SG_ERR_MAJOR", -6: "SG_ERR_GROUPS",
          -7: "SG_ERR_HIP"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libswizzled_gemm.so")
_lib = None


class GemmError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERRORS.get(code, code)}: {msg}")
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load the shared library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is missing: build it with __graft_entry__.build() "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.gemm_run.argtypes = [i64, i64, i64, vp, i32, vp, i32, i32, vp, i32, vp, i32, vp]
    f32 = ctypes.c_float
    lib.gemm_strided_run.argtypes = [i64, i64, i64, f32, vp, i64, i32, vp, i64, i32, i32,
                                     f32, vp, i64, i32, vp, i64, i32, vp]
    lib.grouped_gemm_run.argtypes = [i32, ctypes.POINTER(ctypes.c_int64), i64, i64, vp,
                                     i32, vp, i32, i32, vp, i32, vp]
    lib.mx_gemm_run.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, i32, vp]
    lib.mxfp4_gemm_run.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, i32, vp]
    lib.mxfp6_gemm_run.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, i32, vp]
    lib.gemm_layout_run.argtypes = [i32, i64, i64, i64, vp, vp, vp, i32, vp, i32, vp]
    lib.gemm_layout128_run.argtypes = [i32, i64, i64, i64, vp, vp, vp, i32, vp, i32, vp]
    lib.gemm_layout_io_run.argtypes = [i32, i32, i64, i64, i64, vp, vp, vp, i32, vp, i32, vp]
    lib.gemm_lds_layout.argtypes = [i32, i32, ctypes.POINTER(ctypes.c_int32)]
    lib.gemm_lds_layout_mxfp6.argtypes = [i32, i32, ctypes.POINTER(ctypes.c_int32)]
    lib.gemm_lds_layout_cblock.argtypes = [ctypes.POINTER(ctypes.c_int32)]
    lib.gemm_lds_image.argtypes = [vp, i64, i64, i32, i64, i64, i32, vp, vp]
    lib.gemm_lds_image_tile.argtypes = [i32, vp, i64, i64, i64, i64, vp, vp]
    lib.gemm_mfma_scale_probe.argtypes = [i32, vp, vp, vp, vp, vp, vp]
    lib.gemm_clock_trace.argtypes = [vp, i64, ctypes.POINTER(ctypes.c_int)]
    lib.gemm_clock_probe.argtypes = [i64, vp, vp]
    lib.gemm_clock_probe_waves.argtypes = []
    lib.mx_scales_blocks_bytes.argtypes = [i64, i64]
    lib.mx_scales_blocks_bytes.restype = ctypes.c_int64
    lib.mx_scales_to_blocks.argtypes = [vp, i64, i64, vp, vp]
    lib.mx_gemm_blocks_run.argtypes = [i32, i64, i64, i64, vp, vp, vp, vp, vp, i32, vp]
    lib.i8_gemm_run.argtypes = [i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, i64, i32, vp]
    lib.i8_grouped_gemm_run.argtypes = [i32, i64, i64, i64, vp, vp, i64, i64, vp, vp, vp, vp, vp,
                                        i64, i32, vp]
    lib.i8_quant_run.argtypes = [i64, i64, vp, i64, i32, vp, i64, vp, vp]
    lib.moe_route_run.argtypes = [i64, i32, i32, vp, i64, i32, vp, i32, i32, i32, i32, i32, f32,
                                  vp, vp, vp]
    lib.moe_route_backward_run.argtypes = [i64, i32, i32, vp, vp, i64, i32, vp, i32, i32, f32, vp,
                                           i64, vp]
    lib.moe_plan_run.argtypes = [i64, i32, i32, vp, vp, vp, vp, vp, i64, vp]
    lib.moe_plan_workspace_bytes.argtypes = [i64, i32]
    lib.moe_plan_workspace_bytes.restype = ctypes.c_int64
    lib.moe_balance_run.argtypes = [i64, i32, i32, vp, i64, i32, vp, i32, vp, vp, vp, vp, i64, vp]
    lib.moe_balance_backward_run.argtypes = [i64, i32, vp, vp, i64, i32, vp, vp, i32, vp, i64, vp]
    lib.moe_balance_workspace_bytes.argtypes = [i64, i32]
    lib.moe_balance_workspace_bytes.restype = ctypes.c_int64
    lib.gemm_xent_run.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, i32, vp, i32, vp, vp, vp,
                                  i64, vp]
    lib.gemm_xent_backward_run.argtypes = [i64, i64, i64, f32, vp, vp, vp, i64, vp, i64, i32, vp,
                                           i32, vp, vp, i64, vp, i64, vp, i64, vp]
    lib.gemm_xent_workspace_bytes.argtypes = [i64, i64, i64]
    lib.gemm_xent_backward_workspace_bytes.argtypes = [i64, i64, i64, i64]
    for f in (lib.gemm_xent_workspace_bytes, lib.gemm_xent_backward_workspace_bytes):
        f.restype = i64
    for f in (lib.moe_balance_run, lib.moe_balance_backward_run, lib.gemm_xent_run, lib.gemm_xent_backward_run,
              lib.i8_gemm_run, lib.i8_grouped_gemm_run, lib.i8_quant_run, lib.moe_route_run,
              lib.moe_route_backward_run, lib.moe_plan_run, lib.mx_scales_to_blocks, lib.mx_gemm_blocks_run, lib.gemm_run, lib.gemm_strided_run, lib.grouped_gemm_run, lib.mx_gemm_run,
              lib.mxfp4_gemm_run, lib.mxfp6_gemm_run,
              lib.gemm_layout_run, lib.gemm_layout128_run, lib.gemm_layout_io_run,
              lib.gemm_lds_layout, lib.gemm_lds_layout_mxfp6, lib.gemm_lds_layout_cblock,
              lib.gemm_lds_image, lib.gemm_lds_image_tile, lib.gemm_mfma_scale_probe,
              lib.gemm_clock_trace, lib.gemm_clock_probe,
              lib.gemm_clock_probe_waves):
        f.restype = ctypes.c_int
    lib.gemm_last_error.argtypes = []
    lib.gemm_last_error.restype = ctypes.c_char_p
    lib.gemm_version.argtypes = []
    lib.gemm_version.restype = ctypes.c_char_p
    lib.gemm_last_kernel.argtypes = []
    lib.gemm_last_kernel.restype = ctypes.c_char_p
    _lib = lib
    return lib


# ------------------------------------------------------------ raw C entry points

def gemm_run(M, N, K, A, a_major, B, b_major, ab_dtype, C, c_dtype, D, d_dtype,
             stream) -> int:
    return load().gemm_run(M, N, K, A, a_major, B, b_major, ab_dtype, C, c_dtype,
                           D, d_dtype, stream)


def gemm_strided_run(M, N, K, alpha, A, lda, a_major, B, ldb, b_major, ab_dtype, beta, C,
                     ldc, c_dtype, D, ldd, d_dtype, stream) -> int:
    return load().gemm_strided_run(M, N, K, alpha, A, lda, a_major, B, ldb, b_major,
                                   ab_dtype, beta, C, ldc, c_dtype, D, ldd, d_dtype, stream)


def grouped_gemm_run(G, m_offsets, N, K, A, a_major, B, b_major, ab_dtype, D,
                     d_dtype, stream) -> int:
    offs = None
    if m_offsets is not None:
        offs = (ctypes.c_int64 * len(m_offsets))(*[int(x) for x in m_offsets])
    return load().grouped_gemm_run(G, offs, N, K, A, a_major, B, b_major, ab_dtype,
                                   D, d_dtype, stream)


def mx_gemm_run(M, N, K, A, SFA, B, SFB, D, d_dtype, stream) -> int:
    return load().mx_gemm_run(M, N, K, A, SFA, B, SFB, D, d_dtype, stream)


def mxfp4_gemm_run(M, N, K, A, SFA, B, SFB, D, d_dtype, stream) -> int:
    return load().mxfp4_gemm_run(M, N, K, A, SFA, B, SFB, D, d_dtype, stream)


def mxfp6_gemm_run(fmt, M, N, K, A, SFA, B, SFB, D, d_dtype, stream) -> int:
    return load().mxfp6_gemm_run(fmt, M, N, K, A, SFA, B, SFB, D, d_dtype, stream)


def mx_scales_blocks_bytes(rows, K) -> int:
    return load().mx_scales_blocks_bytes(rows, K)


def mx_scales_to_blocks(SF, rows, K, out, stream) -> int:
    return load().mx_scales_to_blocks(SF, rows, K, out, stream)


def mx_gemm_blocks_run(fmt, M, N, K, A, SFA, B, SFB, D, d_dtype, stream) -> int:
    return load().mx_gemm_blocks_run(fmt, M, N, K, A, SFA, B, SFB, D, d_dtype, stream)


def gemm_layout_run(swz_units, M, N, K, A, B, C, c_dtype, D, d_dtype, stream) -> int:
    return load().gemm_layout_run(swz_units, M, N, K, A, B, C, c_dtype, D, d_dtype, stream)


def gemm_layout_io_run(operand_swz, output_swz, M, N, K, A, B, C, c_dtype, D, d_dtype,
                       stream) -> int:
    return load().gemm_layout_io_run(operand_swz, output_swz, M, N, K, A, B, C, c_dtype, D,
                                     d_dtype, stream)


def gemm_layout128_run(layout, M, N, K, A, B, C, c_dtype, D, d_dtype, stream) -> int:
    return load().gemm_layout128_run(layout, M, N, K, A, B, C, c_dtype, D, d_dtype, stream)


def i8_gemm_run(M, N, K, A, lda, SA, B, ldb, SB, D, ldd, d_dtype, stream) -> int:
    return load().i8_gemm_run(M, N, K, A, lda, SA, B, ldb, SB, D, ldd, d_dtype, stream)


def i8_grouped_gemm_run(G, R, N, K, offsets, A, lda, a_rows, rows, SA, B, SB, D, ldd, d_dtype,
                        stream) -> int:
    return load().i8_grouped_gemm_run(G, R, N, K, offsets, A, lda, a_rows, rows, SA, B, SB, D,
                                      ldd, d_dtype, stream)


def i8_quant_run(R, K, X, ldx, x_dtype, Q, ldq, S, stream) -> int:
    return load().i8_quant_run(R, K, X, ldx, x_dtype, Q, ldq, S, stream)


def moe_route_run(T, E, top_k, logits, ldl, dtype, bias, score, n_groups, top_groups,
                  group_score, renorm, scale, weights, ids, stream) -> int:
    return load().moe_route_run(T, E, top_k, logits, ldl, dtype, bias, score, n_groups,
                                top_groups, group_score, renorm, scale, weights, ids, stream)


def moe_route_backward_run(T, E, top_k, dweights, logits, ldl, dtype, ids, score, renorm, scale,
                           dlogits, lddl, stream) -> int:
    return load().moe_route_backward_run(T, E, top_k, dweights, logits, ldl, dtype, ids, score,
                                         renorm, scale, dlogits, lddl, stream)


def moe_plan_run(T, E, top_k, ids, offsets, rows, slots, workspace, workspace_bytes,
                 stream) -> int:
    return load().moe_plan_run(T, E, top_k, ids, offsets, rows, slots, workspace,
                               workspace_bytes, stream)


def moe_plan_workspace_bytes(P, E) -> int:
    return load().moe_plan_workspace_bytes(P, E)


def moe_balance_run(T, E, top_k, logits, ldl, dtype, ids, score, loss, counts, tokens, workspace,
                    workspace_bytes, stream) -> int:
    return load().moe_balance_run(T, E, top_k, logits, ldl, dtype, ids, score, loss, counts,
                                  tokens, workspace, workspace_bytes, stream)


def moe_balance_backward_run(T, E, dloss, logits, ldl, dtype, counts, tokens, score, dlogits,
                             lddl, stream) -> int:
    return load().moe_balance_backward_run(T, E, dloss, logits, ldl, dtype, counts, tokens,
                                           score, dlogits, lddl, stream)


def moe_balance_workspace_bytes(T, E) -> int:
    return load().moe_balance_workspace_bytes(T, E)


def gemm_xent_run(M, N, K, alpha, A, lda, B, ldb, ab_dtype, targets, target_dtype, loss, lse,
                  workspace, workspace_bytes, stream) -> int:
    return load().gemm_xent_run(M, N, K, alpha, A, lda, B, ldb, ab_dtype, targets, target_dtype,
                                loss, lse, workspace, workspace_bytes, stream)


def gemm_xent_backward_run(M, N, K, alpha, dloss, dlse, A, lda, B, ldb, ab_dtype, targets,
                           target_dtype, lse, dA, ldda, dB, lddb, workspace, workspace_bytes,
                           stream) -> int:
    return load().gemm_xent_backward_run(M, N, K, alpha, dloss, dlse, A, lda, B, ldb, ab_dtype,
                                         targets, target_dtype, lse, dA, ldda, dB, lddb,
                                         workspace, workspace_bytes, stream)


def gemm_xent_workspace_bytes(M, N, K) -> int:
    return load().gemm_xent_workspace_bytes(M, N, K)


def gemm_xent_backward_workspace_bytes(M, N, K, ldb) -> int:
    return load().gemm_xent_backward_workspace_bytes(M, N, K, ldb)


def gemm_last_error() -> str:
    return load().gemm_last_error().decode()


def gemm_version() -> str:
    return load().gemm_version().decode()


def gemm_last_kernel() -> str:
    """The kernel instantiation the last launching call on this thread ran."""
    return load().gemm_last_kernel().decode()


def gemm_lds_layout(rows: int, row_bytes: int) -> np.ndarray:
    """[rows][row_bytes/16] LDS byte offsets of the kernels' swizzled tile."""
    out = np.zeros(max(rows, 0) * max(row_bytes // 16, 0) + 1, dtype=np.int32)
    rc = load().gemm_lds_layout(rows, row_bytes,
                                out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
    if rc != SG_OK:
        raise GemmError(rc, gemm_last_error())
    return out[:-1].reshape(rows, row_bytes // 16)


def gemm_lds_layout_mxfp6(rows: int, unshifted: int = 32) -> np.ndarray:
    """[rows][12] LDS byte offsets of bytes [8q, 8q+8) of each 96-byte row of
    the MXFP6 kernel's operand tile."""
    out = np.zeros(max(rows, 0) * 12 + 1, dtype=np.int32)
    rc = load().gemm_lds_layout_mxfp6(rows, unshifted,
                                      out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
    if rc != SG_OK:
        raise GemmError(rc, gemm_last_error())
    return out[:-1].reshape(rows, 12)


def gemm_lds_layout_cblock() -> np.ndarray:
    """[4][128][8] LDS places of a 16-bit C in the 256x256 kernel's epilogue:
    wave, row and 16-byte chunk of the wave's 128 x 64 block -> quarter *
    16384 + byte offset inside that quarter's 16 KiB half slot."""
    out = np.zeros(4 * 128 * 8, dtype=np.int32)
    rc = load().gemm_lds_layout_cblock(out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
    if rc != SG_OK:
        raise GemmError(rc, gemm_last_error())
    return out.reshape(4, 128, 8)


def gemm_lds_image(X, rows_total, K, elem_bytes, row0, k0, tile_rows, out,
                   stream) -> int:
    return load().gemm_lds_image(X, rows_total, K, elem_bytes, row0, k0, tile_rows,
                                 out, stream)


SG_IMG_HALF, SG_IMG_HALF_KEXACT, SG_IMG_MN256, SG_IMG_FP6, SG_IMG_CBLOCK = 1, 2, 3, 4, 5


def gemm_lds_image_tile(kind, X, rows, row_bytes, row0, byte0, out, stream) -> int:
    return load().gemm_lds_image_tile(kind, X, rows, row_bytes, row0, byte0, out, stream)


def gemm_mfma_scale_probe(fmt, a, b, sa, sb, out, stream) -> int:
    return load().gemm_mfma_scale_probe(fmt, a, b, sa, sb, out, stream)


def gemm_clock_trace(buf, slots: int) -> int:
    """Turns the per-workgroup clock trace of later launches from this
    thread on (buf = device pointer of 4*slots uint64) or off (buf None);
    returns the real-time counter's rate in kHz."""
    khz = ctypes.c_int(0)
    _check(load().gemm_clock_trace(buf, int(slots), ctypes.byref(khz)))
    return khz.value


def gemm_clock_probe(iters: int, out, stream) -> int:
    return load().gemm_clock_probe(int(iters), out, stream)


def gemm_clock_probe_waves() -> int:
    return load().gemm_clock_probe_waves()


# ----------------------------------------------------------- torch convenience
#
# The wrappers check what the C ABI cannot see before they hand over any
# pointer: every tensor is 2-D (3-D for grouped B), densely packed (row-major,
# no transposed or expanded views) except where gemm_strided takes row
# strides, of the shape the problem implies, and on one CUDA device.  A
# failed check raises GemmError with the code of the matching C error:
# SG_ERR_SHAPE for shapes, SG_ERR_ALIGN for a layout the call cannot address,
# SG_ERR_DTYPE for element types, SG_ERR_NULL for a tensor that is not on the
# CUDA device of the others.  The device is checked last, so every other
# check also runs on CPU tensors.

def _check(rc: int):
    if rc != SG_OK:
        raise GemmError(rc, gemm_last_error())


def _dt(t) -> int:
    import torch
    m = {torch.float16: SG_F16, torch.bfloat16: SG_BF16, torch.float32: SG_F32}
    if t not in m:
        raise GemmError(-4, f"unsupported dtype {t}")
    return m[t]


def _stream(device) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _need(cond: bool, code: int, msg: str) -> None:
    if not cond:
        raise GemmError(code, msg)


def _dense(name: str, t, dims: int = 2) -> None:
    """t is a packed row-major tensor of `dims` dimensions."""
    _need(t.dim() == dims, -3, f"{name} must be {dims}-D, got shape {tuple(t.shape)}")
    _need(t.is_contiguous(), -2,
          f"{name} must be contiguous (row-major, no transposed or expanded view); "
          f"strides {tuple(t.stride())}")


def _shape(name: str, t, shape) -> None:
    _need(tuple(t.shape) == tuple(shape), -3,
          f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _dtype_is(name: str, t, dtypes) -> None:
    _need(t.dtype in dtypes, -4, f"{name} has dtype {t.dtype}, expected one of {dtypes}")


def _one_device(*named) -> None:
    """Every (name, tensor) pair with a tensor lives on one CUDA device."""
    dev = None
    for name, t in named:
        if t is None:
            continue
        _need(t.device.type == "cuda", -1, f"{name} is on {t.device}, not a CUDA device")
        if dev is None:
            dev = t.device
        _need(t.device == dev, -1, f"{name} is on {t.device}, the others on {dev}")


def _mk(A, B, a_major: str, b_major: str):
    """(M, N, K) of A (a_major) and B (b_major), checking that K agrees."""
    _need(a_major in ("k", "mn") and b_major in ("k", "mn"), -5,
          f"majorness must be 'k' or 'mn', got {a_major!r}, {b_major!r}")
    M, K = A.shape if a_major == "k" else tuple(reversed(A.shape))
    N, Kb = B.shape if b_major == "k" else tuple(reversed(B.shape))
    _need(Kb == K, -3, f"A and B disagree on K ({K} vs {Kb})")
    _need(A.dtype == B.dtype, -4, f"A and B dtypes differ ({A.dtype} vs {B.dtype})")
    return int(M), int(N), int(K)


def _out(out, shape, dtype, device):
    """`out` checked against `shape`, or a new tensor of `dtype`."""
    import torch
    if out is None:
        return torch.empty(tuple(shape), dtype=dtype, device=device)
    _shape("out", out, shape)
    return out


def _gemm_args(A, B, a_major, b_major, C, out, out_dtype):
    """Checks of gemm()/gemm_plan(): returns (M, N, K, out)."""
    import torch
    _dense("A", A)
    _dense("B", B)
    M, N, K = _mk(A, B, a_major, b_major)
    _dtype_is("A", A, (torch.float16, torch.bfloat16))
    if C is not None:
        _dense("C", C)
        _shape("C", C, (M, N))
        _dtype_is("C", C, (torch.float32, torch.bfloat16, torch.float16))
    if out is not None:
        _dense("out", out)
        _shape("out", out, (M, N))
        _dtype_is("out", out, (torch.float32, torch.bfloat16, torch.float16))
    _one_device(("A", A), ("B", B), ("C", C), ("out", out))
    out = _out(out, (M, N), out_dtype or torch.float32, A.device)
    return M, N, K, out


def gemm(A, B, *, a_major: str = "k", b_major: str = "k", C=None,
         out_dtype=None, out=None):
    """D = A*B (+C) on torch CUDA tensors.

    A: [M][K] (a_major "k") or [K][M] ("mn"); B: [N][K] ("k") or [K][N]
    ("mn"); C: optional [M][N]; returns D [M][N] of out_dtype (default
    torch.float32), or writes `out` [M][N].  Every tensor contiguous and on
    one CUDA device."""
    M, N, K, out = _gemm_args(A, B, a_major, b_major, C, out, out_dtype)
    _check(gemm_run(M, N, K, A.data_ptr(), 0 if a_major == "k" else 1, B.data_ptr(),
                    0 if b_major == "k" else 1, _dt(A.dtype),
                    C.data_ptr() if C is not None else None,
                    _dt(C.dtype) if C is not None else SG_NONE, out.data_ptr(),
                    _dt(out.dtype), _stream(A.device)))
    return out


def gemm_plan(A, B, *, a_major: str = "k", b_major: str = "k", C=None, out):
    """gemm() with its argument marshalling done once: returns a callable
    that launches D = A*B (+C) into `out` on the stream current now, for
    launch-bound small problems where the per-call Python work would
    otherwise take longer than the kernel.  The callable holds references to
    A, B, C and out, so their storage stays allocated while it lives; they
    must not be resized or have their storage replaced meanwhile."""
    _need(out is not None, -1, "gemm_plan needs out")
    M, N, K, out = _gemm_args(A, B, a_major, b_major, C, out, None)
    f = load().gemm_run
    args = (M, N, K, A.data_ptr(), 0 if a_major == "k" else 1, B.data_ptr(),
            0 if b_major == "k" else 1, _dt(A.dtype),
            C.data_ptr() if C is not None else None,
            _dt(C.dtype) if C is not None else SG_NONE, out.data_ptr(), _dt(out.dtype),
            _stream(A.device))

    def run() -> None:
        rc = f(*args)
        if rc != SG_OK:
            raise GemmError(rc, gemm_last_error())
    # The launch takes raw pointers: keep the tensors (and so their memory)
    # alive as long as the callable can be called.
    run.tensors = (A, B, C, out)
    return run


def _ld(t, name: str) -> int:
    _need(t.dim() == 2, -3, f"{name} must be 2-D, got shape {tuple(t.shape)}")
    _need(t.stride(1) == 1 and t.stride(0) >= max(t.shape[1], 1), -2,
          f"{name} must have unit column stride and a row stride of at least its width; "
          f"strides {tuple(t.stride())}")
    return t.stride(0)


def gemm_strided(A, B, *, a_major: str = "k", b_major: str = "k", C=None, alpha: float = 1.0,
                 beta: float = 1.0, out_dtype=None, out=None):
    """D = alpha * A*B + beta * C on 2-D torch CUDA tensors whose rows may be
    padded (views with unit column stride): leading dimensions are the row
    strides.  Shapes as in gemm(); `out` may itself be a padded view."""
    import torch
    lda, ldb = _ld(A, "A"), _ld(B, "B")
    M, N, K = _mk(A, B, a_major, b_major)
    _dtype_is("A", A, (torch.float16, torch.bfloat16))
    if C is not None:
        ldc = _ld(C, "C")
        _shape("C", C, (M, N))
        _dtype_is("C", C, (torch.float32, torch.bfloat16, torch.float16))
    if out is not None:
        _shape("out", out, (M, N))
        _dtype_is("out", out, (torch.float32, torch.bfloat16, torch.float16))
        ldd = _ld(out, "out")
    _one_device(("A", A), ("B", B), ("C", C), ("out", out))
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or torch.float32, device=A.device)
        ldd = N
    _check(gemm_strided_run(M, N, K, float(alpha), A.data_ptr(), lda,
                            0 if a_major == "k" else 1, B.data_ptr(), ldb,
                            0 if b_major == "k" else 1, _dt(A.dtype), float(beta),
                            C.data_ptr() if C is not None else None,
                            ldc if C is not None else N,
                            _dt(C.dtype) if C is not None else SG_NONE, out.data_ptr(),
                            ldd, _dt(out.dtype), _stream(A.device)))
    return out


def _layout_args(A, B, C, out, out_dtype):
    """Checks of the layout-ablation wrappers: bf16 K-major A [M][K] and
    B [N][K]."""
    import torch
    _dense("A", A)
    _dense("B", B)
    M, N, K = _mk(A, B, "k", "k")
    _dtype_is("A", A, (torch.bfloat16,))
    if C is not None:
        _dense("C", C)
        _shape("C", C, (M, N))
        _dtype_is("C", C, (torch.float32, torch.bfloat16, torch.float16))
    if out is not None:
        _dense("out", out)
        _shape("out", out, (M, N))
        _dtype_is("out", out, (torch.float32, torch.bfloat16, torch.float16))
    _one_device(("A", A), ("B", B), ("C", C), ("out", out))
    return M, N, K, _out(out, (M, N), out_dtype or torch.float32, A.device)


def gemm_layout(A, B, swz_units: int, *, C=None, out_dtype=None, out=None):
    """gemm() for bf16 K-major A [M][K] and B [N][K] on the 256x256-tile
    kernel with the LDS layout swz_units (16 = the library's XOR swizzle
    over 256-byte lines, 8 = over 128-byte lines, 0 = none)."""
    M, N, K, out = _layout_args(A, B, C, out, out_dtype)
    _check(gemm_layout_run(swz_units, M, N, K, A.data_ptr(), B.data_ptr(),
                           C.data_ptr() if C is not None else None,
                           _dt(C.dtype) if C is not None else SG_NONE, out.data_ptr(),
                           _dt(out.dtype), _stream(A.device)))
    return out


def gemm_layout_io(A, B, operand_swz: int, output_swz: int, *, C=None, out_dtype=None,
                   out=None):
    """gemm() for bf16 K-major A [M][K] and B [N][K] on the library's 256x256
    kernel with the operand layout operand_swz (16 or 0) and the epilogue's
    C/D staging swizzled (output_swz 1) or not (0); D is 16-bit (default
    bf16), C None or 16-bit."""
    import torch
    M, N, K, out = _layout_args(A, B, C, out, out_dtype or torch.bfloat16)
    _check(gemm_layout_io_run(operand_swz, output_swz, M, N, K, A.data_ptr(), B.data_ptr(),
                              C.data_ptr() if C is not None else None,
                              _dt(C.dtype) if C is not None else SG_NONE, out.data_ptr(),
                              _dt(out.dtype), _stream(A.device)))
    return out


def gemm_layout128(A, B, layout: int, *, C=None, out_dtype=None, out=None):
    """gemm_layout() on 128x128 tiles, where layout may also be
    SG_LAYOUT_PAD16 (rows padded by 16 bytes, no swizzle)."""
    M, N, K, out = _layout_args(A, B, C, out, out_dtype)
    _check(gemm_layout128_run(layout, M, N, K, A.data_ptr(), B.data_ptr(),
                              C.data_ptr() if C is not None else None,
                              _dt(C.dtype) if C is not None else SG_NONE, out.data_ptr(),
                              _dt(out.dtype), _stream(A.device)))
    return out


def grouped_gemm(A, B, m_offsets: Sequence[int], *, out_dtype=None, out=None):
    """Per group g: D[off_g:off_{g+1}] = A[off_g:off_{g+1}] * B[g]^T.

    A: [sum M][K]; B: [G][N][K]; m_offsets: G+1 host ints (m_offsets[-1] is
    A's row count)."""
    import torch
    _dense("A", A)
    _dense("B", B, dims=3)
    G, N, K = (int(x) for x in B.shape)
    offs = [int(x) for x in m_offsets]
    _need(len(offs) == G + 1, -6, f"m_offsets has {len(offs)} entries, expected G+1 = {G + 1}")
    _need(A.shape[0] == offs[-1], -3,
          f"A has {A.shape[0]} rows, m_offsets[-1] = {offs[-1]}")
    _need(A.shape[1] == K, -3, f"A and B disagree on K ({A.shape[1]} vs {K})")
    _need(A.dtype == B.dtype, -4, f"A and B dtypes differ ({A.dtype} vs {B.dtype})")
    _dtype_is("A", A, (torch.float16, torch.bfloat16))
    if out is not None:
        _dense("out", out)
        _shape("out", out, (offs[-1], N))
        _dtype_is("out", out, (torch.float32, torch.bfloat16, torch.float16))
    _one_device(("A", A), ("B", B), ("out", out))
    out = _out(out, (offs[-1], N), out_dtype or torch.bfloat16, A.device)
    _check(grouped_gemm_run(G, offs, N, K, A.data_ptr(), 0, B.data_ptr(), 0,
                            _dt(A.dtype), out.data_ptr(), _dt(out.dtype),
                            _stream(A.device)))
    return out


def _mx_args(A, SFA, B, SFB, out, out_dtype, k_per_byte_num: int, k_per_byte_den: int):
    """Checks of the block-scaled wrappers: uint8 A [M][bytes], B [N][bytes]
    with the same row bytes, SFA [M][K/32], SFB [N][K/32] uint8; returns
    (M, N, K, out)."""
    import torch
    for name, t in (("A", A), ("SFA", SFA), ("B", B), ("SFB", SFB)):
        _dense(name, t)
        _dtype_is(name, t, (torch.uint8,))
    M, N = int(A.shape[0]), int(B.shape[0])
    _need(A.shape[1] == B.shape[1], -3,
          f"A and B rows hold different byte counts ({A.shape[1]} vs {B.shape[1]})")
    K = int(A.shape[1]) * k_per_byte_num // k_per_byte_den
    _need(K * k_per_byte_den == int(A.shape[1]) * k_per_byte_num, -3,
          f"A's row of {A.shape[1]} bytes is not a whole number of elements")
    _shape("SFA", SFA, (M, K // 32))
    _shape("SFB", SFB, (N, K // 32))
    if out is not None:
        _dense("out", out)
        _shape("out", out, (M, N))
        _dtype_is("out", out, (torch.float32, torch.bfloat16))
    _one_device(("A", A), ("SFA", SFA), ("B", B), ("SFB", SFB), ("out", out))
    return M, N, K, _out(out, (M, N), out_dtype or torch.bfloat16, A.device)


_MX_FMTS = {"e4m3": (SG_E4M3, 1, 1), "e2m1": (SG_E2M1, 2, 1), "e2m3": (SG_E2M3, 4, 3),
            "e3m2": (SG_E3M2, 4, 3)}


def mx_scales_blocks(SF, *, out=None):
    """e8m0 scales SF [rows][K/32] (uint8) rearranged into the SG_SF_BLOCKS
    layout: a 1-D uint8 tensor of mx_scales_blocks_bytes(rows, K) bytes
    (allocated by torch unless `out` is given)."""
    import torch
    _dense("SF", SF)
    _dtype_is("SF", SF, (torch.uint8,))
    rows, K = int(SF.shape[0]), int(SF.shape[1]) * 32
    n = int(mx_scales_blocks_bytes(rows, K))
    _check(n if n < 0 else 0)
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=SF.device)
    else:
        _dense("out", out, 1)
        _shape("out", out, (n,))
        _dtype_is("out", out, (torch.uint8,))
    _one_device(("SF", SF), ("out", out))
    _check(mx_scales_to_blocks(SF.data_ptr(), rows, K, out.data_ptr(), _stream(SF.device)))
    return out


def mx_gemm_blocks(A, SFA, B, SFB, *, fmt: str = "e4m3", out_dtype=None, out=None):
    """The block-scaled GEMM of mx_gemm / mxfp4_gemm / mxfp6_gemm (fmt
    "e4m3", "e2m1", "e2m3" or "e3m2"; A and B as there) with SFA and SFB in
    the SG_SF_BLOCKS layout (mx_scales_blocks)."""
    import torch
    _need(fmt in _MX_FMTS, -4, f"fmt must be one of {sorted(_MX_FMTS)}, got {fmt!r}")
    code, num, den = _MX_FMTS[fmt]
    for name, t in (("A", A), ("B", B)):
        _dense(name, t)
        _dtype_is(name, t, (torch.uint8,))
    M, N = int(A.shape[0]), int(B.shape[0])
    _need(A.shape[1] == B.shape[1], -3,
          f"A and B rows hold different byte counts ({A.shape[1]} vs {B.shape[1]})")
    K = int(A.shape[1]) * num // den
    _need(K * den == int(A.shape[1]) * num, -3,
          f"A's row of {A.shape[1]} bytes is not a whole number of elements")
    for name, t, rows in (("SFA", SFA, M), ("SFB", SFB, N)):
        _dense(name, t, 1)
        _dtype_is(name, t, (torch.uint8,))
        n = int(mx_scales_blocks_bytes(rows, K))
        _check(n if n < 0 else 0)
        _shape(name, t, (n,))
    if out is not None:
        _dense("out", out)
        _shape("out", out, (M, N))
        _dtype_is("out", out, (torch.float32, torch.bfloat16))
    _one_device(("A", A), ("SFA", SFA), ("B", B), ("SFB", SFB), ("out", out))
    out = _out(out, (M, N), out_dtype or torch.bfloat16, A.device)
    _check(mx_gemm_blocks_run(code, M, N, K, A.data_ptr(), SFA.data_ptr(), B.data_ptr(),
                              SFB.data_ptr(), out.data_ptr(), _dt(out.dtype), _stream(A.device)))
    return out


def mx_gemm(A, SFA, B, SFB, *, out_dtype=None, out=None):
    """Block-scaled e4m3 GEMM: A [M][K], B [N][K] (uint8 e4m3 codes),
    SFA [M][K/32], SFB [N][K/32] (uint8 e8m0 codes)."""
    M, N, K, out = _mx_args(A, SFA, B, SFB, out, out_dtype, 1, 1)
    _check(mx_gemm_run(M, N, K, A.data_ptr(), SFA.data_ptr(), B.data_ptr(),
                       SFB.data_ptr(), out.data_ptr(), _dt(out.dtype),
                       _stream(A.device)))
    return out


def mxfp4_gemm(A, SFA, B, SFB, *, out_dtype=None, out=None):
    """Block-scaled e2m1 GEMM: A [M][K/2], B [N][K/2] (uint8, two e2m1 per
    byte, element 2i in the low nibble), SFA [M][K/32], SFB [N][K/32] (uint8
    e8m0 codes)."""
    M, N, K, out = _mx_args(A, SFA, B, SFB, out, out_dtype, 2, 1)
    _check(mxfp4_gemm_run(M, N, K, A.data_ptr(), SFA.data_ptr(), B.data_ptr(),
                          SFB.data_ptr(), out.data_ptr(), _dt(out.dtype), _stream(A.device)))
    return out


def mxfp6_gemm(A, SFA, B, SFB, *, fmt: str = "e2m3", out_dtype=None, out=None):
    """Block-scaled FP6 GEMM: A [M][3K/4], B [N][3K/4] (uint8, a 6-bit
    stream of e2m3 or e3m2 codes per row, element k at bits [6k, 6k+6)),
    SFA [M][K/32], SFB [N][K/32] (uint8 e8m0 codes)."""
    _need(fmt in ("e2m3", "e3m2"), -4, f"fmt must be 'e2m3' or 'e3m2', got {fmt!r}")
    code = {"e2m3": SG_E2M3, "e3m2": SG_E3M2}[fmt]
    M, N, K, out = _mx_args(A, SFA, B, SFB, out, out_dtype, 4, 3)
    _check(mxfp6_gemm_run(code, M, N, K, A.data_ptr(), SFA.data_ptr(), B.data_ptr(),
                          SFB.data_ptr(), out.data_ptr(), _dt(out.dtype), _stream(A.device)))
    return out


# ---------------------------------------------- 8-bit products, expert routing
#
# Small calls of these take less time on the GPU than a wrapper of the kind
# above takes to check them (13 to 19 us), so the checks build their messages
# only when they fail and the C functions are called directly (6 to 8 us a
# call, 4 of them the launch itself).  The launches go to the tensors' device
# even when another is current.  moe_route's weights carry autograd history
# (its backward pass is moe_route_backward); the 8-bit results carry none, their
# codes are for serving.

_torch = None
_raw_stream = _current_device = None


def _lib_torch():
    """(the loaded library, torch), imported once."""
    global _torch, _raw_stream, _current_device
    if _torch is None:
        import torch
        load()
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _torch = torch
    return _lib, _torch


def _launch(f, device, *args) -> None:
    """Calls the C function f(*args, stream) with `device` current."""
    index = device.index
    if _current_device() == index:
        rc = f(*args, _raw_stream(index))
    else:
        with _torch.cuda.device(index):
            rc = f(*args, _raw_stream(index))
    if rc:
        raise GemmError(rc, gemm_last_error())


def _fail(code: int, msg: str):
    raise GemmError(code, msg)


def _int(name: str, v) -> int:
    """v as an int that a C int holds."""
    v = int(v)
    if not -0x80000000 <= v <= 0x7fffffff:
        _fail(-3, f"{name}={v} is outside 32 bits")
    return v


def _on_one_device(first, *others) -> None:
    """Every tensor (None passes) is on `first`'s CUDA device."""
    device = first.device
    if not first.is_cuda:
        _fail(-1, f"a tensor is on {device}, not a CUDA device")
    for t in others:
        if t is not None and t.device != device:
            _fail(-1, f"tensors are on {t.device} and {device}")


def _no_tangent(**tensors) -> None:
    """No tensor carries a forward-mode gradient, which the kernels would drop."""
    forward_ad = _torch.autograd.forward_ad
    if getattr(forward_ad, "_current_level", 0) < 0:
        return
    for name, t in tensors.items():
        if forward_ad.unpack_dual(t).tangent is not None:
            _fail(-4, f"{name} has a forward-mode tangent; only reverse mode is supported")


def _vector(name: str, t, n: int, dtype) -> None:
    """t is a packed vector of n elements of dtype."""
    if t.shape != (n,):
        _fail(-3, f"{name} has shape {tuple(t.shape)}, expected ({n},)")
    if t.dtype is not dtype:
        _fail(-4, f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        _fail(-2, f"{name} must be contiguous; strides {t.stride()}")


def _packed(name: str, t, shape, dtype) -> None:
    """t is a packed row-major tensor of `shape` and dtype."""
    if not t.is_contiguous():
        _fail(-2, f"{name} must be contiguous (row-major); strides {t.stride()}")
    if t.shape != shape:
        _fail(-3, f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        _fail(-4, f"{name} has dtype {t.dtype}, expected {dtype}")


def _pitch(name: str, t) -> int:
    """The row stride of a 2-D tensor with unit column stride: at least its
    width, which stands in where no second row tells the stride."""
    if t.dim() != 2:
        _fail(-3, f"{name} must be 2-D, got shape {tuple(t.shape)}")
    rows, cols = t.shape
    s0, s1 = t.stride()
    if cols > 1 and s1 != 1:
        _fail(-2, f"{name} must have unit column stride; strides {t.stride()}")
    if rows <= 1 or cols == 0:
        return cols
    if s0 < cols:
        _fail(-2, f"{name} must have a row stride of at least its width; strides {t.stride()}")
    return s0


def _code_pitch(name: str, t) -> int:
    """_pitch of int8 codes; a single row's is its width rounded up to 16."""
    if t.dtype is not _torch.int8:
        _fail(-4, f"{name} has dtype {t.dtype}, expected torch.int8")
    ld = _pitch(name, t)
    return ld if t.shape[0] > 1 else -(-ld // 16) * 16


def _float_code(name: str, dtype) -> int:
    """The SG_* code of a float type."""
    T = _torch
    if dtype is T.bfloat16:
        return SG_BF16
    if dtype is T.float32:
        return SG_F32
    if dtype is T.float16:
        return SG_F16
    _fail(-4, f"{name} has dtype {dtype}, expected float32, bfloat16 or float16")


def _out_pitch(out, R: int, N: int) -> int:
    if out.shape != (R, N):
        _fail(-3, f"out has shape {tuple(out.shape)}, expected ({R}, {N})")
    _float_code("out", out.dtype)
    return _pitch("out", out)


def i8_quant(X, *, out=None, out_scale=None):
    """X [R][K] (float32, bfloat16 or float16, unit column stride) as 8-bit
    codes with one scale per row: (codes int8 [R][Kp], scales float32 [R]), Kp
    = K rounded up to 16, the columns behind K zero.  X is about codes *
    scales[:, None]; scale = max|x| / 127.  A row with an infinity or a NaN has
    the scale NaN.  out: int8 [R][Kp] whose row stride is a multiple of 16."""
    lib, T = _lib_torch()
    ldx = _pitch("X", X)
    R, K = X.shape
    dt = _float_code("X", X.dtype)
    ldq = Kp = -(-K // 16) * 16
    if out is not None:
        if out.shape != (R, Kp):
            _fail(-3, f"out has shape {tuple(out.shape)}, expected ({R}, {Kp})")
        ldq = _code_pitch("out", out)
    if out_scale is not None:
        _vector("out_scale", out_scale, R, T.float32)
    _on_one_device(X, out, out_scale)
    dev = X.device
    if out is None:
        out = T.empty(R, Kp, dtype=T.int8, device=dev)
    if out_scale is None:
        out_scale = T.empty(R, dtype=T.float32, device=dev)
    _launch(lib.i8_quant_run, dev, R, K, X.data_ptr(), ldx, dt, out.data_ptr(), ldq,
            out_scale.data_ptr())
    return out, out_scale


def i8_gemm(A, SA, B, SB, *, out_dtype=None, out=None):
    """D[m][n] = SA[m] * SB[n] * sum_k A[m][k] * B[n][k] for int8 A [M][K] and
    B [N][K] and float32 scales SA [M], SB [N]; returns D [M][N] of out_dtype
    (default torch.bfloat16), or writes `out`.  K is a multiple of 16 (i8_quant
    pads); rows of A, B and out may be padded."""
    lib, T = _lib_torch()
    lda, ldb = _code_pitch("A", A), _code_pitch("B", B)
    M, K = A.shape
    N, Kb = B.shape
    if Kb != K:
        _fail(-3, f"A and B disagree on K ({K} vs {Kb})")
    _vector("SA", SA, M, T.float32)
    _vector("SB", SB, N, T.float32)
    ldd = N if out is None else _out_pitch(out, M, N)
    _on_one_device(A, SA, B, SB, out)
    dev = A.device
    if out is None:
        out = T.empty(M, N, dtype=out_dtype or T.bfloat16, device=dev)
    _launch(lib.i8_gemm_run, dev, M, N, K, A.data_ptr(), lda, SA.data_ptr(), B.data_ptr(), ldb,
            SB.data_ptr(), out.data_ptr(), ldd, _float_code("out", out.dtype))
    return out


def i8_grouped_gemm(A, SA, B, SB, offsets, *, rows=None, out_dtype=None, out=None):
    """i8_gemm for G experts whose row ranges are on the device: row r of D,
    offsets[g] <= r < offsets[g+1], is A's row rows[r] (or r) times B[g].

    A int8 [T][K], SA [T]; B int8 [G][N][K], SB [G][N]; offsets int32 [G+1] and
    rows int32 [R] as moe_plan returns them (without rows, R = T).  Returns D
    [R][N] of out_dtype (default torch.bfloat16), or writes `out`.  Rows at and
    behind offsets[G] are not written: a new D holds anything there."""
    lib, T = _lib_torch()
    lda = _code_pitch("A", A)
    R, K = A.shape
    if B.dim() != 3:
        _fail(-3, f"B must be [G][N][K], got shape {tuple(B.shape)}")
    G, N, Kb = B.shape
    _int("G", G)
    _packed("B", B, B.shape, T.int8)
    if Kb != K:
        _fail(-3, f"A and B disagree on K ({K} vs {Kb})")
    _vector("SA", SA, R, T.float32)
    _packed("SB", SB, (G, N), T.float32)
    _vector("offsets", offsets, G + 1, T.int32)
    a_rows = R
    if rows is not None:
        R = rows.numel()
        _vector("rows", rows, R, T.int32)
    ldd = N if out is None else _out_pitch(out, R, N)
    _on_one_device(A, SA, B, SB, offsets, rows, out)
    dev = A.device
    if out is None:
        out = T.empty(R, N, dtype=out_dtype or T.bfloat16, device=dev)
    _launch(lib.i8_grouped_gemm_run, dev, G, R, N, K, offsets.data_ptr(), A.data_ptr(), lda,
            a_rows, None if rows is None else rows.data_ptr(), SA.data_ptr(), B.data_ptr(),
            SB.data_ptr(), out.data_ptr(), ldd, _float_code("out", out.dtype))
    return out


_SCORES = {"softmax": SG_SCORE_SOFTMAX, "sigmoid": SG_SCORE_SIGMOID}
_GROUP_SCORES = {"max": SG_GROUP_MAX, "top2": SG_GROUP_TOP2}


def _score_code(score) -> int:
    code = _SCORES.get(score)
    if code is None:
        _fail(-4, f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return code


_route_function = None


def _routed(logits, top_k, score, renorm, scale, rest):
    """moe_route with moe_route_backward as the gradient of the logits."""
    global _route_function
    if _route_function is None:

        class MoeRoute(_torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, top_k, form, rest):  # (gradients are off in here)
                weights, ids = moe_route(logits, top_k, **form, **rest)
                ctx.save_for_backward(logits, ids)
                ctx.form = form
                ctx.mark_non_differentiable(ids)
                return weights, ids

            @staticmethod
            @_torch.autograd.function.once_differentiable
            def backward(ctx, dweights, _):
                logits, ids = ctx.saved_tensors
                return (moe_route_backward(dweights.contiguous(), logits, ids, **ctx.form),
                        None, None, None)

        _route_function = MoeRoute
    return _route_function.apply(logits, top_k, {"score": score, "renorm": renorm, "scale": scale},
                                 rest)


def moe_route(logits, top_k: int, *, score: str = "softmax", bias=None, n_groups: int = 1,
              top_groups: Optional[int] = None, group_score: str = "max", renorm: bool = True,
              scale: float = 1.0, out=None):
    """The top_k experts of each token and their weights, from router logits
    [T][E]: (weights float32 [T][top_k], ids int32 [T][top_k]).

    Experts are chosen by score + bias (bias float32 [E]; softmax or sigmoid
    scores), within the top_groups best of n_groups equal groups; among equal
    ones the lowest index.  Weights are the scores of the chosen ones (without
    the bias), divided by their sum (renorm), times scale.  Logits of -inf or
    NaN are masked (+inf is the largest float); a token with no expert left has
    ids -1 and weights 0.

    Where the logits require a gradient, the weights carry it (the choice held
    fixed; bias gets none; a forward-mode tangent is refused).  out: (weights, ids) to write, which carry no
    history: their gradient is a call of moe_route_backward."""
    lib, T = _lib_torch()
    _no_tangent(logits=logits)
    if out is None and logits.requires_grad and T.is_grad_enabled():
        return _routed(logits, top_k, score, renorm, scale, {
            "bias": bias, "n_groups": n_groups, "top_groups": top_groups,
            "group_score": group_score})
    ldl = _pitch("logits", logits)
    n, E = logits.shape
    dt, code = _float_code("logits", logits.dtype), _score_code(score)
    _int("E", E)
    top_k, n_groups = int(top_k), _int("n_groups", n_groups)
    top_groups = n_groups if top_groups is None else _int("top_groups", top_groups)
    groups = _GROUP_SCORES.get(group_score)
    if groups is None:
        _fail(-6, f"group_score must be one of {sorted(_GROUP_SCORES)}, got {group_score!r}")
    if not 1 <= top_k <= min(E, SG_MAX_TOP_K):
        _fail(-3, f"top_k={top_k} outside 1..min({E}, {SG_MAX_TOP_K})")
    if bias is not None:
        _vector("bias", bias, E, T.float32)
    if out is None:
        _on_one_device(logits, bias)
        weights = T.empty(n, top_k, dtype=T.float32, device=logits.device)
        ids = T.empty_like(weights, dtype=T.int32)
    else:
        weights, ids = out
        _packed("weights", weights, (n, top_k), T.float32)
        _packed("ids", ids, (n, top_k), T.int32)
        _on_one_device(logits, bias, weights, ids)
    _launch(lib.moe_route_run, logits.device, n, E, top_k, logits.data_ptr(), ldl, dt,
            None if bias is None else bias.data_ptr(), code, n_groups, top_groups, groups,
            1 if renorm else 0, float(scale), weights.data_ptr(), ids.data_ptr())
    return weights, ids


def moe_route_backward(dweights, logits, ids, *, score: str = "softmax", renorm: bool = True,
                       scale: float = 1.0, out=None):
    """The gradient of the logits [T][E] (their type) from dweights float32
    [T][top_k], the gradient of moe_route's weights, and its ids."""
    lib, T = _lib_torch()
    ldl = _pitch("logits", logits)
    n, E = logits.shape
    dt, code = _float_code("logits", logits.dtype), _score_code(score)
    if ids.dim() != 2:
        _fail(-3, f"ids must be 2-D, got shape {tuple(ids.shape)}")
    _int("E", E)
    top_k = _int("top_k", ids.shape[1])
    _packed("ids", ids, (n, top_k), T.int32)
    _packed("dweights", dweights, (n, top_k), T.float32)
    lddl = E
    if out is not None:
        if out.shape != (n, E):
            _fail(-3, f"out has shape {tuple(out.shape)}, expected ({n}, {E})")
        if out.dtype is not logits.dtype:
            _fail(-4, f"out has dtype {out.dtype}, expected {logits.dtype}")
        lddl = _pitch("out", out)
    _on_one_device(logits, dweights, ids, out)
    dev = logits.device
    if out is None:
        out = T.empty(n, E, dtype=logits.dtype, device=dev)
    _launch(lib.moe_route_backward_run, dev, n, E, top_k, dweights.data_ptr(),
            logits.data_ptr(), ldl, dt, ids.data_ptr(), code, 1 if renorm else 0, float(scale),
            out.data_ptr(), lddl)
    return out


def moe_plan(ids, n_experts: int, *, out=None, workspace=None):
    """The (token, expert) pairs of ids int32 [T][top_k] sorted by expert,
    stably: (offsets int32 [E+1], rows int32 [T*top_k], slots int32 [T][top_k]).
    Expert e's sorted rows are offsets[e]:offsets[e+1], rows[r] is the token of
    sorted row r (-1 behind offsets[E]) and slots[t][j] the sorted row of pair
    (t, j), -1 where its id is outside [0, E).

    out: (offsets, rows, slots) to write.  workspace: a uint8 tensor of at
    least moe_plan_workspace_bytes(T * top_k, E) bytes; by default one is
    allocated for the call."""
    lib, T = _lib_torch()
    if ids.dim() != 2:
        _fail(-3, f"ids must be 2-D, got shape {tuple(ids.shape)}")
    n, top_k = ids.shape
    _packed("ids", ids, (n, top_k), T.int32)
    _int("top_k", top_k)
    P, n_experts = n * top_k, _int("n_experts", n_experts)
    need = lib.moe_plan_workspace_bytes(P, n_experts)
    if need < 0:
        _fail(need, gemm_last_error())
    dev = ids.device
    if workspace is not None:
        size = workspace.numel()
        _vector("workspace", workspace, size, T.uint8)
        if size < need:
            _fail(-3, f"workspace has {size} bytes, {need} are needed")
    if out is not None:
        offsets, rows, slots = out
        _vector("offsets", offsets, n_experts + 1, T.int32)
        _vector("rows", rows, P, T.int32)
        _packed("slots", slots, (n, top_k), T.int32)
        _on_one_device(ids, offsets, rows, slots, workspace)
    else:
        _on_one_device(ids, workspace)
        offsets = T.empty(n_experts + 1, dtype=T.int32, device=dev)
        rows = T.empty(P, dtype=T.int32, device=dev)
        slots = T.empty_like(ids)
    if workspace is None and need:
        workspace = T.empty(need, dtype=T.uint8, device=dev)
    _launch(lib.moe_plan_run, dev, n, n_experts, top_k, ids.data_ptr(), offsets.data_ptr(),
            rows.data_ptr(), slots.data_ptr(), workspace.data_ptr() if need else None, need)
    return offsets, rows, slots


# ------------------------------------------------- the routing's balance loss

_balance_function = None


def _balanced(logits, ids, score, workspace):
    """moe_balance with moe_balance_backward as the gradient of the logits."""
    global _balance_function
    if _balance_function is None:

        class MoeBalance(_torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, ids, score, workspace):  # (gradients are off in here)
                loss, counts, tokens = moe_balance(logits, ids, score=score, workspace=workspace)
                ctx.save_for_backward(logits, counts, tokens)
                ctx.score = score
                ctx.mark_non_differentiable(counts, tokens)
                return loss, counts, tokens

            @staticmethod
            @_torch.autograd.function.once_differentiable
            def backward(ctx, dloss, *_):
                logits, counts, tokens = ctx.saved_tensors
                return (moe_balance_backward(dloss, logits, counts, tokens, score=ctx.score),
                        None, None, None)

        _balance_function = MoeBalance
    return _balance_function.apply(logits, ids, score, workspace)


def moe_balance(logits, ids, *, score: str = "softmax", out=None, workspace=None):
    """How evenly a router spreads its tokens over the experts, from its logits
    [T][E] and moe_route's ids int32 [T][top_k]: (loss float32 [], counts int32
    [E], tokens int32 []).

    loss = sum over the experts of E * their share of the pairs * the mean over
    the tokens of their share of the token's scores (softmax or sigmoid): 1 for
    an even load, E at most.  counts are the pairs of each expert, tokens those
    that have an expert left; ids outside [0, E) and masked logits (-inf, NaN)
    do not count.

    Where the logits require a gradient, the loss carries it (the counts held
    fixed; a forward-mode tangent is refused).  out: (loss, counts, tokens) to write, which carry no history: their
    gradient is a call of moe_balance_backward.  workspace: a uint8 tensor of at
    least moe_balance_workspace_bytes(T, E) bytes; by default one is allocated
    for the call.  (A captured step with its backward: as for gemm_xent.)"""
    lib, T = _lib_torch()
    _no_tangent(logits=logits)
    if out is None and logits.requires_grad and T.is_grad_enabled():
        return _balanced(logits, ids, score, workspace)
    ldl = _pitch("logits", logits)
    n, E = logits.shape
    dt, code = _float_code("logits", logits.dtype), _score_code(score)
    if ids.dim() != 2:
        _fail(-3, f"ids must be 2-D, got shape {tuple(ids.shape)}")
    _int("E", E)
    top_k = _int("top_k", ids.shape[1])
    _packed("ids", ids, (n, top_k), T.int32)
    if out is None:
        _on_one_device(logits, ids, workspace)
    else:
        loss, counts, tokens = out
        _packed("loss", loss, (), T.float32)
        _vector("counts", counts, E, T.int32)
        _packed("tokens", tokens, (), T.int32)
        _on_one_device(logits, ids, loss, counts, tokens, workspace)
    dev = logits.device
    need = lib.moe_balance_workspace_bytes(n, E)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, dev)
    if out is None:
        loss = logits.new_empty((), dtype=T.float32)
        counts, tokens = ids.new_empty(E), ids.new_empty(())
    _launch(lib.moe_balance_run, dev, n, E, top_k, logits.data_ptr(), ldl, dt, ids.data_ptr(),
            code, loss.data_ptr(), counts.data_ptr(), tokens.data_ptr(),
            workspace.data_ptr() if need else None, need)
    return loss, counts, tokens


def moe_balance_backward(dloss, logits, counts, tokens, *, score: str = "softmax", out=None):
    """The gradient of the logits [T][E] (their type) from dloss float32 [], the
    gradient of moe_balance's loss, and its counts and tokens."""
    lib, T = _lib_torch()
    ldl = _pitch("logits", logits)
    n, E = logits.shape
    dt, code = _float_code("logits", logits.dtype), _score_code(score)
    _int("E", E)
    _packed("dloss", dloss, (), T.float32)
    _vector("counts", counts, E, T.int32)
    _packed("tokens", tokens, (), T.int32)
    lddl = E
    if out is not None:
        if out.shape != (n, E):
            _fail(-3, f"out has shape {tuple(out.shape)}, expected ({n}, {E})")
        if out.dtype is not logits.dtype:
            _fail(-4, f"out has dtype {out.dtype}, expected {logits.dtype}")
        lddl = _pitch("out", out)
    _on_one_device(logits, dloss, counts, tokens, out)
    dev = logits.device
    if out is None:
        out = T.empty(n, E, dtype=logits.dtype, device=dev)
    _launch(lib.moe_balance_backward_run, dev, n, E, dloss.data_ptr(), logits.data_ptr(), ldl, dt,
            counts.data_ptr(), tokens.data_ptr(), code, out.data_ptr(), lddl)
    return out


# ---------------------------------------------- cross entropy over a vocabulary

def _xent_args(A, B, targets):
    """(M, N, K, lda, ldb, the SG_* codes of A's and the targets' types)."""
    T = _torch
    lda, ldb = _pitch("A", A), _pitch("B", B)
    M, K = A.shape
    N, Kb = B.shape
    if Kb != K:
        _fail(-3, f"A and B disagree on K ({K} vs {Kb})")
    if A.dtype is not B.dtype:
        _fail(-4, f"A and B dtypes differ ({A.dtype} vs {B.dtype})")
    dt = _float_code("A", A.dtype)
    if dt == SG_F32:
        _fail(-4, "A has dtype torch.float32, expected float16 or bfloat16")
    wide = targets.dtype is T.int64
    _vector("targets", targets, M, T.int64 if wide else T.int32)
    return M, N, K, lda, ldb, dt, SG_I64 if wide else SG_I32


def _workspace(given, need: int, device):
    """`given` checked against `need` bytes, or a new workspace of them."""
    if need < 0:
        _fail(need, gemm_last_error())
    if given is None:
        return _torch.empty(need, dtype=_torch.uint8, device=device)
    _vector("workspace", given, given.numel(), _torch.uint8)
    if given.numel() < need:
        _fail(-3, f"workspace has {given.numel()} bytes, {need} are needed")
    return given


_xent_function = None


def _xent(A, B, targets, alpha, workspace):
    """gemm_xent with gemm_xent_backward as the gradient of A and B."""
    global _xent_function
    if _xent_function is None:

        class GemmXent(_torch.autograd.Function):
            @staticmethod
            def forward(ctx, A, B, targets, alpha, workspace):  # (gradients are off in here)
                loss, lse = gemm_xent(A, B, targets, alpha=alpha, workspace=workspace)
                ctx.save_for_backward(A, B, targets, lse)
                ctx.alpha = alpha
                ctx.set_materialize_grads(False)
                return loss, lse

            @staticmethod
            @_torch.autograd.function.once_differentiable
            def backward(ctx, dloss, dlse):
                if dloss is None and dlse is None:
                    return None, None, None, None, None
                A, B, targets, lse = ctx.saved_tensors
                dloss = _torch.zeros_like(lse) if dloss is None else dloss.contiguous()
                dA, dB = gemm_xent_backward(
                    dloss, A, B, targets, lse, alpha=ctx.alpha,
                    dlse=None if dlse is None else dlse.contiguous(),
                    need=ctx.needs_input_grad[:2])
                return dA, dB, None, None, None

        _xent_function = GemmXent
    return _xent_function.apply(A, B, targets, alpha, workspace)


def gemm_xent(A, B, targets, *, alpha: float = 1.0, out=None, workspace=None):
    """Softmax cross entropy of M tokens over a vocabulary of N words, logits
    alpha * A @ B.T, which are not kept: (loss float32 [M], lse float32 [M]).

    A [M][K] (tokens) and B [N][K] (a word a row), both float16 or bfloat16,
    rows padded or not; targets int32 or int64 [M].  lse is the logarithm of the
    softmax's divisor, loss = lse - the target's logit, or 0 for a token whose
    target lies outside [0, N).

    Where A or B requires a gradient, loss and lse carry it (reverse mode: a
    forward-mode tangent is refused).  out: (loss, lse) to write, which overlap
    nothing and carry no history: their gradient is a call of gemm_xent_backward.  workspace: a uint8 tensor of at least
    gemm_xent_workspace_bytes(M, N, K) bytes; by default one is allocated for
    the call.

    To capture a step with its backward into a graph, let no autograd graph of A
    or B from outside the capture live: torch would accumulate their gradients on
    the stream of that one."""
    lib, T = _lib_torch()
    alpha = float(alpha)
    _no_tangent(A=A, B=B)
    if out is None and (A.requires_grad or B.requires_grad) and T.is_grad_enabled():
        return _xent(A, B, targets, alpha, workspace)
    M, N, K, lda, ldb, dt, tt = _xent_args(A, B, targets)
    if out is not None:
        loss, lse = out
        _vector("loss", loss, M, T.float32)
        _vector("lse", lse, M, T.float32)
        _on_one_device(A, B, targets, loss, lse, workspace)
    else:
        _on_one_device(A, B, targets, workspace)
    dev = A.device
    workspace = _workspace(workspace, lib.gemm_xent_workspace_bytes(M, N, K), dev)
    if out is None:
        loss = T.empty(M, dtype=T.float32, device=dev)
        lse = T.empty_like(loss)
    _launch(lib.gemm_xent_run, dev, M, N, K, alpha, A.data_ptr(), lda, B.data_ptr(), ldb, dt,
            targets.data_ptr(), tt, loss.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
            workspace.numel())
    return loss, lse


def gemm_xent_backward(dloss, A, B, targets, lse, *, alpha: float = 1.0, dlse=None,
                       need=(True, True), out=None, workspace=None):
    """The gradients (dA [M][K], dB [N][K]), of A's and B's type, from dloss
    float32 [M], the gradient of gemm_xent's loss, and dlse float32 [M], that of
    its lse (None: zero).  lse is gemm_xent's.  The gradient of the logits is
    rounded to A's type on the way, up to 64 tokens to twice as many bits.  M is
    below 2^22, and with dB the rows of A span less than 2^31 bytes.

    need: which of the two are computed; the other is None.  out: (dA, dB) to
    write (None: a new tensor), rows padded or not, that overlap no input and not
    each other.  workspace: a uint8 tensor of
    at least gemm_xent_backward_workspace_bytes(M, N, K, B.stride(0)) bytes."""
    lib, T = _lib_torch()
    M, N, K, lda, ldb, dt, tt = _xent_args(A, B, targets)
    for name, t in (("dloss", dloss), ("lse", lse), ("dlse", dlse)):
        if t is not None or name != "dlse":
            _vector(name, t, M, T.float32)
    out = out or (None, None)
    pitch = []
    for name, t, like, wanted in (("dA", out[0], A, need[0]), ("dB", out[1], B, need[1])):
        if t is None or not wanted:
            pitch.append(K)
            continue
        if t.shape != like.shape:
            _fail(-3, f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape)}")
        if t.dtype is not like.dtype:
            _fail(-4, f"{name} has dtype {t.dtype}, expected {like.dtype}")
        pitch.append(_pitch(name, t))
    _on_one_device(A, B, targets, dloss, dlse, lse, workspace, *out)
    dev = A.device
    size = lib.gemm_xent_backward_workspace_bytes(M, N, K, ldb)
    workspace = _workspace(workspace, size, dev)
    dA, dB = (None if not wanted else T.empty_like(like, memory_format=T.contiguous_format)
              if t is None else t
              for t, like, wanted in ((out[0], A, need[0]), (out[1], B, need[1])))
    _launch(lib.gemm_xent_backward_run, dev, M, N, K, float(alpha), dloss.data_ptr(),
            None if dlse is None else dlse.data_ptr(), A.data_ptr(), lda, B.data_ptr(), ldb, dt,
            targets.data_ptr(), tt, lse.data_ptr(), None if dA is None else dA.data_ptr(),
            pitch[0], None if dB is None else dB.data_ptr(), pitch[1], workspace.data_ptr(),
            workspace.numel())
    return dA, dB
