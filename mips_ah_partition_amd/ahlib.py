"""Thin Python binding of the C ABI in include/ah.h (libah.so, built in-tree).

Argument marshalling only: every function takes torch CUDA (ROCm) tensors,
checks dtype/shape/contiguity, passes raw device pointers and the current
stream to the library and raises ``AHError`` on a non-zero status.  All work
runs in the library's HIP kernels; there is no fallback path: if libah.so is
missing or cannot be loaded, the import of this module's functions fails
loudly.
"""
from __future__ import annotations

import ctypes as C
import functools
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libah.so")

AH_OK, AH_ERR_NULL, AH_ERR_SHAPE, AH_ERR_UNSUPPORTED, AH_ERR_WORKSPACE, AH_ERR_HIP = 0, -1, -2, -3, -4, -5
AH_F32, AH_BF16 = 0, 1
AH_CODES_TILED = -1
AH_MAX_WIDTH = 1 << 20  # n and k of the grouped products

# every symbol include/ah.h declares
EXPORTS = (
    "ah_status_string", "ah_version",
    "ah_partition_workspace_bytes", "ah_partition_score",
    "ah_build_lut",
    "ah_scan_workspace_bytes", "ah_scan_topk", "ah_scan_topk_noalloc",
    "ah_residual_leaf_bias", "ah_scan_topk_residual",
    "ah_sq8_quantize", "ah_sq8_workspace_bytes", "ah_sq8_scan_topk",
    "ah_rslm_rotate", "ah_rslm_encode", "ah_rslm_scan_topk",
    "ah_assign_workspace_bytes", "ah_assign_leaves",
    "ah_kmeans_workspace_bytes", "ah_kmeans_update",
    "ah_encode", "ah_encode_sweep", "ah_pq_update_workspace_bytes", "ah_pq_update",
    "ah_tiled_codes_bytes", "ah_tile_codes",
    "ah_reorder_exact",
    "ah_i8_quantize_rows", "ah_i8_matmul", "ah_i8_linear_workspace_bytes", "ah_i8_linear",
    "ah_group_rows_workspace_bytes", "ah_group_rows", "ah_grouped_matmul",
    "ah_grouped_dx_workspace_bytes", "ah_grouped_matmul_dx", "ah_grouped_matmul_dw",
    "ah_distill_workspace_bytes", "ah_distill_topk",
    "ah_grouped_gated", "ah_grouped_gated_grad",
    "ah_f8_quantize", "ah_f8_matmul", "ah_f8_linear_workspace_bytes", "ah_f8_linear",
    "ah_dropout",
)
# every symbol include/ah_instrument.h declares (measurement hooks)
INSTRUMENT_EXPORTS = ("ah_scan_topk_timed", "ah_scan_workspace_counters", "ah_hbm_read_probe")

_lib = None


class AHError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


def lib() -> C.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
        L.ah_status_string.restype = C.c_char_p
        L.ah_status_string.argtypes = [C.c_int]
        L.ah_version.restype = C.c_int
        L.ah_partition_workspace_bytes.restype = sz
        L.ah_partition_workspace_bytes.argtypes = [i64, i32]
        L.ah_partition_score.restype = C.c_int
        L.ah_partition_score.argtypes = [vp, i64, i32, vp, i32, i32, vp, vp, vp, sz, vp]
        L.ah_build_lut.restype = C.c_int
        L.ah_build_lut.argtypes = [vp, i64, i32, vp, i32, i32, vp, vp, vp, vp, vp]
        L.ah_scan_workspace_bytes.restype = sz
        L.ah_scan_workspace_bytes.argtypes = [i64, i32, i64, i32, i32, i32]
        L.ah_scan_topk.restype = C.c_int
        L.ah_scan_topk.argtypes = [vp, i64, i32, vp, i32, i64, vp, vp, i32, vp, i32, i32, vp, vp, vp, sz, vp]
        L.ah_scan_topk_timed.restype = C.c_int
        L.ah_scan_topk_timed.argtypes = [vp, i64, i32, vp, i32, i64, vp, vp, i32, vp, i32, i32, vp, vp, vp, sz, vp,
                                         vp, vp]
        L.ah_scan_topk_residual.restype = C.c_int
        L.ah_scan_topk_residual.argtypes = [vp, i64, i32, vp, i32, i64, vp, vp, i32, vp, i32, vp, i32, i32, vp, vp,
                                            vp, sz, vp]
        L.ah_residual_leaf_bias.restype = C.c_int
        L.ah_residual_leaf_bias.argtypes = [vp, vp, i64, i32, i32, vp, vp]
        L.ah_rslm_rotate.restype = C.c_int
        L.ah_rslm_rotate.argtypes = [vp, i64, i32, vp, vp, vp, vp]
        L.ah_rslm_encode.restype = C.c_int
        L.ah_rslm_encode.argtypes = [vp, i64, i32, vp, vp, vp, vp]
        L.ah_rslm_scan_topk.restype = C.c_int
        L.ah_rslm_scan_topk.argtypes = [vp, vp, i64, vp, vp, i64, i32, vp, i32, vp, vp, vp, sz, vp]
        L.ah_kmeans_workspace_bytes.restype = sz
        L.ah_kmeans_workspace_bytes.argtypes = [i32, i32]
        L.ah_kmeans_update.restype = C.c_int
        L.ah_kmeans_update.argtypes = [vp, i64, i32, vp, i32, vp, vp, vp, sz, vp]
        L.ah_encode_sweep.restype = C.c_int
        L.ah_encode_sweep.argtypes = [vp, i32, i64, i32, vp, i32, i32, C.c_double, i32, vp, i32, vp]
        L.ah_pq_update_workspace_bytes.restype = sz
        L.ah_pq_update_workspace_bytes.argtypes = [i64, i32, i32]
        L.ah_pq_update.restype = C.c_int
        L.ah_pq_update.argtypes = [vp, i64, i32, vp, i32, i32, i32, C.c_double, vp, vp, sz, vp]
        L.ah_sq8_quantize.restype = C.c_int
        L.ah_sq8_quantize.argtypes = [vp, i64, i32, C.c_double, vp, vp, vp]
        L.ah_sq8_workspace_bytes.restype = sz
        L.ah_sq8_workspace_bytes.argtypes = [i64, i64, i32, i32]
        L.ah_sq8_scan_topk.restype = C.c_int
        L.ah_sq8_scan_topk.argtypes = [vp, vp, i64, vp, vp, i64, i32, i32, vp, vp, vp, sz, vp]
        L.ah_assign_workspace_bytes.restype = sz
        L.ah_assign_workspace_bytes.argtypes = [i64, i32]
        L.ah_assign_leaves.restype = C.c_int
        L.ah_assign_leaves.argtypes = [vp, i64, i32, vp, i32, vp, vp, vp, sz, vp]
        L.ah_encode.restype = C.c_int
        L.ah_encode.argtypes = [vp, i32, i64, i32, vp, i32, i32, C.c_double, i32, vp, i32, vp]
        L.ah_tiled_codes_bytes.restype = sz
        L.ah_tiled_codes_bytes.argtypes = [i64, i32]
        L.ah_tile_codes.restype = C.c_int
        L.ah_tile_codes.argtypes = [vp, i32, i64, i32, vp, sz, vp]
        L.ah_reorder_exact.restype = C.c_int
        L.ah_reorder_exact.argtypes = [vp, i64, i32, vp, i32, i64, vp, i32, i32, vp, vp, vp]
        f32 = C.c_float
        L.ah_i8_quantize_rows.restype = C.c_int
        L.ah_i8_quantize_rows.argtypes = [vp, i32, i64, i32, i64, vp, vp, vp]
        L.ah_i8_matmul.restype = C.c_int
        L.ah_i8_matmul.argtypes = [vp, vp, i64, vp, vp, i64, i32, vp, vp, i32, vp]
        L.ah_i8_linear_workspace_bytes.restype = sz
        L.ah_i8_linear_workspace_bytes.argtypes = [i64, i32]
        L.ah_i8_linear.restype = C.c_int
        L.ah_i8_linear.argtypes = [vp, i32, i64, i32, i64, vp, vp, i64, vp, vp, i32, vp, sz, vp]
        L.ah_group_rows_workspace_bytes.restype = sz
        L.ah_group_rows_workspace_bytes.argtypes = [i64, i32]
        L.ah_group_rows.restype = C.c_int
        L.ah_group_rows.argtypes = [vp, i64, i32, vp, vp, vp, sz, vp]
        L.ah_grouped_matmul.restype = C.c_int
        L.ah_grouped_matmul.argtypes = [vp, i64, vp, i32, i32, i32, vp, vp, i64, i32, vp, i32, vp]
        L.ah_grouped_dx_workspace_bytes.restype = sz
        L.ah_grouped_dx_workspace_bytes.argtypes = [i64, i32, i32]
        L.ah_grouped_matmul_dx.restype = C.c_int
        L.ah_grouped_matmul_dx.argtypes = [vp, i64, vp, i32, i32, i32, vp, vp, i64, i32, vp, i32, vp, sz, vp]
        L.ah_grouped_matmul_dw.restype = C.c_int
        L.ah_grouped_matmul_dw.argtypes = [vp, i64, vp, i64, i32, i32, i32, vp, vp, i64, i32, vp, i32, vp]
        L.ah_distill_workspace_bytes.restype = sz
        L.ah_distill_workspace_bytes.argtypes = [i64, i64, i32]
        L.ah_distill_topk.restype = C.c_int
        L.ah_distill_topk.argtypes = [vp, i32, i64, i64, i64, vp, vp, i32, f32, vp, vp, vp, i64, vp, sz, vp]
        u64, f64 = C.c_uint64, C.c_double
        L.ah_grouped_gated.restype = C.c_int
        L.ah_grouped_gated.argtypes = [vp, i64, vp, i32, i32, i32, vp, vp, i64, i32, i32, f64, u64, vp, vp, vp, i32, vp]
        L.ah_grouped_gated_grad.restype = C.c_int
        L.ah_grouped_gated_grad.argtypes = [vp, i64, vp, i32, i32, i32, vp, vp, i64, vp, i32, f64, u64, vp, vp, vp, vp]
        L.ah_f8_quantize.restype = C.c_int
        L.ah_f8_quantize.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, vp, vp, vp]
        L.ah_f8_matmul.restype = C.c_int
        L.ah_f8_matmul.argtypes = [vp, vp, i32, i64, vp, vp, i32, i64, i64, vp, vp, i32, vp]
        L.ah_f8_linear_workspace_bytes.restype = sz
        L.ah_f8_linear_workspace_bytes.argtypes = [i64, i64]
        L.ah_f8_linear.restype = C.c_int
        L.ah_f8_linear.argtypes = [vp, i32, i64, i64, i64, i32, vp, vp, i32, i64, vp, vp, i32, vp, sz, vp]
        L.ah_dropout.restype = C.c_int
        L.ah_dropout.argtypes = [vp, i32, i64, i64, i64, f64, u64, vp, vp, i64, vp, i64, vp]
        L.ah_scan_topk_noalloc.restype = C.c_int
        L.ah_scan_topk_noalloc.argtypes = [vp, i64, i32, vp, i32, i64, vp, vp, i32, vp, i32, i32, vp, vp, vp]
        L.ah_scan_workspace_counters.restype = C.c_int
        L.ah_scan_workspace_counters.argtypes = [i64, i32, i64, i32, i32, i32, C.POINTER(sz), C.POINTER(sz)]
        L.ah_hbm_read_probe.restype = C.c_int
        L.ah_hbm_read_probe.argtypes = [vp, sz, i32, vp, vp]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ah_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != AH_OK:
        raise AHError(status, where)


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _dev(t, dtype, name, ndim=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    return t


# ----------------------------------------------------------------------------- step 1
def ah_partition_workspace_bytes(nq: int, L: int) -> int:
    return int(lib().ah_partition_workspace_bytes(nq, L))


def ah_partition_score(q, centroids, nl, leaves_out=None, leaf_scores_out=None, workspace=None, stream=None):
    """Best nl leaves per query (and their fp32 scores)."""
    q = _dev(q, torch.float32, "q", 2)
    centroids = _dev(centroids, torch.float32, "centroids", 2)
    nq, d = q.shape
    L = centroids.shape[0]
    if centroids.shape[1] != d:
        raise ValueError("centroids dimension differs from queries")
    if leaves_out is None:
        leaves_out = torch.empty((nq, nl), dtype=torch.int32, device=q.device)
    if leaf_scores_out is None:
        leaf_scores_out = torch.empty((nq, nl), dtype=torch.float32, device=q.device)
    _dev(leaves_out, torch.int32, "leaves_out")
    _dev(leaf_scores_out, torch.float32, "leaf_scores_out")
    need = ah_partition_workspace_bytes(nq, L)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    _check(lib().ah_partition_score(_ptr(q), nq, d, _ptr(centroids), L, nl, _ptr(leaves_out),
                                    _ptr(leaf_scores_out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "ah_partition_score")
    return leaves_out, leaf_scores_out


# ----------------------------------------------------------------------------- step 2
def ah_build_lut(q, codebooks, lut_i8_out=None, scale_out=None, bias_out=None, lut_f32_out=None,
                 want_f32=False, stream=None):
    """int8 tables (and optionally the fp32 ones) for a query batch.
    codebooks: float32 [B, 16, dpb]."""
    q = _dev(q, torch.float32, "q", 2)
    codebooks = _dev(codebooks, torch.float32, "codebooks", 3)
    nq, d = q.shape
    B, _, dpb = codebooks.shape
    dev = q.device
    if lut_i8_out is None:
        lut_i8_out = torch.empty((nq, B, 16), dtype=torch.int8, device=dev)
    if scale_out is None:
        scale_out = torch.empty(nq, dtype=torch.float32, device=dev)
    if bias_out is None:
        bias_out = torch.empty(nq, dtype=torch.float32, device=dev)
    if lut_f32_out is None and want_f32:
        lut_f32_out = torch.empty((nq, B, 16), dtype=torch.float32, device=dev)
    _dev(lut_i8_out, torch.int8, "lut_i8_out")
    _dev(scale_out, torch.float32, "scale_out")
    _dev(bias_out, torch.float32, "bias_out")
    _dev(lut_f32_out, torch.float32, "lut_f32_out")
    _check(lib().ah_build_lut(_ptr(q), nq, d, _ptr(codebooks), B, dpb, _ptr(lut_f32_out), _ptr(lut_i8_out),
                              _ptr(scale_out), _ptr(bias_out), _stream(stream)), "ah_build_lut")
    return lut_i8_out, scale_out, bias_out, lut_f32_out


# ----------------------------------------------------------------------------- steps 3+4
def ah_scan_workspace_bytes(nq: int, B: int, n: int, L: int, nl: int, R: int) -> int:
    return int(lib().ah_scan_workspace_bytes(nq, B, n, L, nl, R))


def ah_sq8_quantize(x, pct=99.9, codes_out=None, scale_out=None, stream=None):
    """Per-row int8 codes and float32 steps (robust percentile scale)."""
    x = _dev(x, torch.float32, "x", 2)
    n, d = x.shape
    if codes_out is None:
        codes_out = torch.empty((n, d), dtype=torch.int8, device=x.device)
    if scale_out is None:
        scale_out = torch.empty(n, dtype=torch.float32, device=x.device)
    _dev(codes_out, torch.int8, "codes_out", 2)
    _dev(scale_out, torch.float32, "scale_out", 1)
    _check(lib().ah_sq8_quantize(_ptr(x), n, d, float(pct), _ptr(codes_out), _ptr(scale_out), _stream(stream)),
           "ah_sq8_quantize")
    return codes_out, scale_out


def ah_sq8_workspace_bytes(nq: int, n: int, d: int, R: int) -> int:
    return int(lib().ah_sq8_workspace_bytes(nq, n, int(d), int(R)))


def ah_sq8_scan_topk(q8, q_scale, d8, d_scale, R, ids_out=None, scores_out=None, workspace=None, stream=None):
    """Top-R documents per query by ((float)(q8 . d8) * q_scale) * d_scale, ties to the lower id."""
    q8 = _dev(q8, torch.int8, "q8", 2)
    d8 = _dev(d8, torch.int8, "d8", 2)
    q_scale = _dev(q_scale, torch.float32, "q_scale", 1)
    d_scale = _dev(d_scale, torch.float32, "d_scale", 1)
    nq, d = q8.shape
    n = d8.shape[0]
    if ids_out is None:
        ids_out = torch.empty((nq, R), dtype=torch.int32, device=q8.device)
    if scores_out is None:
        scores_out = torch.empty((nq, R), dtype=torch.float32, device=q8.device)
    need = ah_sq8_workspace_bytes(nq, n, d, R)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q8.device)
    _check(lib().ah_sq8_scan_topk(_ptr(q8), _ptr(q_scale), nq, _ptr(d8), _ptr(d_scale), n, d, int(R), _ptr(ids_out),
                                  _ptr(scores_out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "ah_sq8_scan_topk")
    return ids_out, scores_out


def ah_rslm_rotate(x, signs, perm, y_out=None, stream=None):
    """Block Hadamard rotation of rows (sign flips, permutation, blocks of up to 128)."""
    x = _dev(x, torch.float32, "x", 2)
    n, d = x.shape
    signs = _dev(signs, torch.float32, "signs", 1)
    perm = _dev(perm, torch.int32, "perm", 1)
    if signs.numel() != d or perm.numel() != d:
        raise ValueError("signs and perm need d entries")
    if y_out is None:
        y_out = torch.empty_like(x)
    _dev(y_out, torch.float32, "y_out", 2)
    _check(lib().ah_rslm_rotate(_ptr(x), n, d, _ptr(signs), _ptr(perm), _ptr(y_out), _stream(stream)),
           "ah_rslm_rotate")
    return y_out


def ah_rslm_encode(y, levels, codes_out=None, step_out=None, stream=None):
    """4-bit nearest-level codes of rotated rows and the norm-restoring row steps;
    levels: 16 ascending floats (host)."""
    y = _dev(y, torch.float32, "y", 2)
    n, d = y.shape
    lv = np.ascontiguousarray(levels, dtype=np.float32)
    if lv.shape != (16,):
        raise ValueError("16 levels")
    if codes_out is None:
        codes_out = torch.empty((n, (d + 1) // 2), dtype=torch.uint8, device=y.device)
    if step_out is None:
        step_out = torch.empty(n, dtype=torch.float32, device=y.device)
    _dev(codes_out, torch.uint8, "codes_out", 2)
    _dev(step_out, torch.float32, "step_out", 1)
    _check(lib().ah_rslm_encode(_ptr(y), n, d, lv.ctypes.data_as(C.c_void_p), _ptr(codes_out), _ptr(step_out),
                                _stream(stream)), "ah_rslm_encode")
    return codes_out, step_out


def ah_rslm_scan_topk(q8, q_scale, codes, step, d, levels_i8, R, ids_out=None, scores_out=None, workspace=None,
                      stream=None):
    """Top-R documents per query over 4-bit codes standing for the int8 values levels_i8 (16, host)."""
    q8 = _dev(q8, torch.int8, "q8", 2)
    q_scale = _dev(q_scale, torch.float32, "q_scale", 1)
    codes = _dev(codes, torch.uint8, "codes", 2)
    step = _dev(step, torch.float32, "step", 1)
    nq = q8.shape[0]
    n = codes.shape[0]
    lv = np.ascontiguousarray(levels_i8, dtype=np.int8)
    if lv.shape != (16,) or q8.shape[1] != d or codes.shape[1] != (d + 1) // 2:
        raise ValueError("shapes")
    if ids_out is None:
        ids_out = torch.empty((nq, R), dtype=torch.int32, device=q8.device)
    if scores_out is None:
        scores_out = torch.empty((nq, R), dtype=torch.float32, device=q8.device)
    need = ah_sq8_workspace_bytes(nq, n, d, R)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q8.device)
    _check(lib().ah_rslm_scan_topk(_ptr(q8), _ptr(q_scale), nq, _ptr(codes), _ptr(step), n, d,
                                   lv.ctypes.data_as(C.c_void_p), int(R), _ptr(ids_out), _ptr(scores_out),
                                   _ptr(workspace), workspace.numel(), _stream(stream)), "ah_rslm_scan_topk")
    return ids_out, scores_out


def ah_kmeans_update(x, leaf_of_row, centroids, counts_out=None, workspace=None, stream=None):
    """In place: each leaf's centroid becomes the mean of its rows (empty leaves keep theirs).
    Returns (centroids, counts int32 [L])."""
    x = _dev(x, torch.float32, "x", 2)
    leaf_of_row = _dev(leaf_of_row, torch.int32, "leaf_of_row", 1)
    centroids = _dev(centroids, torch.float32, "centroids", 2)
    n, d = x.shape
    L = centroids.shape[0]
    if centroids.shape[1] != d or leaf_of_row.numel() != n:
        raise ValueError("shapes")
    if counts_out is None:
        counts_out = torch.empty(L, dtype=torch.int32, device=x.device)
    need = int(lib().ah_kmeans_workspace_bytes(L, d))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib().ah_kmeans_update(_ptr(x), n, d, _ptr(leaf_of_row), L, _ptr(centroids), _ptr(counts_out),
                                  _ptr(workspace), workspace.numel(), _stream(stream)), "ah_kmeans_update")
    return centroids, counts_out


def ah_kmeans_workspace_bytes(L: int, d: int) -> int:
    return int(lib().ah_kmeans_workspace_bytes(L, d))


def ah_encode_sweep(rows, codebooks, eta, codes_inout, sweeps=1, stream=None):
    """Coupled-encoding sweeps started from the codes in codes_inout (updated in place)."""
    codebooks = _dev(codebooks, torch.float32, "codebooks", 3)
    B, _, dpb = codebooks.shape
    if rows.dtype == torch.bfloat16:
        dt = AH_BF16
    else:
        rows = _dev(rows, torch.float32, "rows", 2)
        dt = AH_F32
    n, d = rows.shape
    _dev(codes_inout, torch.uint8, "codes_inout", 2)
    _check(lib().ah_encode_sweep(_ptr(rows), dt, n, d, _ptr(codebooks), B, dpb, float(eta), int(sweeps),
                                 _ptr(codes_inout), codes_inout.shape[1], _stream(stream)), "ah_encode_sweep")
    return codes_inout


def ah_pq_update(x, codes, codebooks, eta, workspace=None, stream=None):
    """Block-by-block closed-form center update at fixed codes (codebooks updated in place)."""
    x = _dev(x, torch.float32, "x", 2)
    codes = _dev(codes, torch.uint8, "codes", 2)
    codebooks = _dev(codebooks, torch.float32, "codebooks", 3)
    n, d = x.shape
    B, _, dpb = codebooks.shape
    need = int(lib().ah_pq_update_workspace_bytes(n, B, dpb))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib().ah_pq_update(_ptr(x), n, d, _ptr(codes), codes.shape[1], B, dpb, float(eta), _ptr(codebooks),
                              _ptr(workspace), workspace.numel(), _stream(stream)), "ah_pq_update")
    return codebooks


def ah_pq_update_workspace_bytes(n: int, B: int, dpb: int) -> int:
    return int(lib().ah_pq_update_workspace_bytes(n, B, dpb))


def ah_assign_workspace_bytes(n: int, L: int) -> int:
    return int(lib().ah_assign_workspace_bytes(n, L))


def ah_assign_leaves(x, centroids, leaf_out=None, score_out=None, workspace=None, want_scores=False, stream=None):
    """Nearest centroid of every row (lowest id on ties); returns (leaves int32 [n], scores or None)."""
    x = _dev(x, torch.float32, "x", 2)
    centroids = _dev(centroids, torch.float32, "centroids", 2)
    n, d = x.shape
    L = centroids.shape[0]
    if centroids.shape[1] != d:
        raise ValueError("centroids dimension differs from rows")
    if leaf_out is None:
        leaf_out = torch.empty(n, dtype=torch.int32, device=x.device)
    if score_out is None and want_scores:
        score_out = torch.empty(n, dtype=torch.float32, device=x.device)
    _dev(leaf_out, torch.int32, "leaf_out")
    _dev(score_out, torch.float32, "score_out")
    need = ah_assign_workspace_bytes(n, L)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib().ah_assign_leaves(_ptr(x), n, d, _ptr(centroids), L, _ptr(leaf_out), _ptr(score_out), _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "ah_assign_leaves")
    return leaf_out, score_out


def ah_encode(rows, codebooks, eta, sweeps=2, codes_out=None, stride=None, stream=None):
    """Anisotropic coupled codes of rows (float32 or bfloat16 [n, d]) for
    codebooks float32 [B, 16, dpb]; returns uint8 [n, stride]."""
    if rows.dtype == torch.float32:
        dt = AH_F32
    elif rows.dtype == torch.bfloat16:
        dt = AH_BF16
    else:
        raise TypeError("rows must be float32 or bfloat16")
    _dev(rows, rows.dtype, "rows", 2)
    codebooks = _dev(codebooks, torch.float32, "codebooks", 3)
    n, d = rows.shape
    B, _, dpb = codebooks.shape
    stride = (B + 1) // 2 if stride is None else int(stride)
    if codes_out is None:
        codes_out = torch.empty((n, stride), dtype=torch.uint8, device=rows.device)
    _dev(codes_out, torch.uint8, "codes_out", 2)
    _check(lib().ah_encode(_ptr(rows), dt, n, d, _ptr(codebooks), B, dpb, float(eta), int(sweeps), _ptr(codes_out),
                           codes_out.shape[1], _stream(stream)), "ah_encode")
    return codes_out


class TiledCodes:
    """Codes in the tiled layout of ah_tile_codes: ``data`` (uint8, device) holds
    ceil(n / 64) tiles; ``n`` rows of ``blocks`` 4-bit codes."""

    def __init__(self, data, n, blocks):
        self.data, self.n, self.blocks = data, int(n), int(blocks)


def ah_tiled_codes_bytes(n: int, B: int) -> int:
    return int(lib().ah_tiled_codes_bytes(n, B))


def ah_tile_codes(codes, B=None, stream=None) -> TiledCodes:
    """Row-major codes uint8 [n, stride] -> TiledCodes (B defaults to 2 * stride)."""
    codes = _dev(codes, torch.uint8, "codes", 2)
    n, stride = codes.shape
    B = 2 * stride if B is None else int(B)
    need = ah_tiled_codes_bytes(n, B)
    out = torch.empty(max(need, 16), dtype=torch.uint8, device=codes.device)
    _check(lib().ah_tile_codes(_ptr(codes), stride, n, B, _ptr(out), out.numel(), _stream(stream)), "ah_tile_codes")
    return TiledCodes(out, n, B)


def ah_scan_topk(lut_i8, codes, R, ids=None, leaf_offsets=None, leaves=None, cand_ids_out=None,
                 cand_scores_out=None, workspace=None, stream=None, main_events=None, leaf_bias=None,
                 bias_bound=0):
    """Top-R rows per query by exact int32 sum of table entries.
    codes: uint8 [n, stride] row-major, or TiledCodes; leaves: int32 [nq, nl] or
    None (scan all rows).  With leaf_bias (int32 [nq, nl], residual variant) the
    call is ah_scan_topk_residual: the j-th leaf's rows add its clipped bias."""
    lut_i8 = _dev(lut_i8, torch.int8, "lut_i8", 3)
    _dev(ids, torch.int32, "ids")
    _dev(leaf_offsets, torch.int64, "leaf_offsets")
    _dev(leaves, torch.int32, "leaves")
    nq, B, _ = lut_i8.shape
    if isinstance(codes, TiledCodes):
        if codes.blocks != B:
            raise ValueError("tiled codes were made for another number of blocks")
        n, stride = codes.n, AH_CODES_TILED
        codes = _dev(codes.data, torch.uint8, "codes", 1)
    else:
        codes = _dev(codes, torch.uint8, "codes", 2)
        n, stride = codes.shape
    L = 0 if leaf_offsets is None else leaf_offsets.numel() - 1
    nl = 0 if leaves is None else leaves.shape[1]
    dev = lut_i8.device
    if cand_ids_out is None:
        cand_ids_out = torch.empty((nq, R), dtype=torch.int32, device=dev)
    if cand_scores_out is None:
        cand_scores_out = torch.empty((nq, R), dtype=torch.int32, device=dev)
    _dev(cand_ids_out, torch.int32, "cand_ids_out")
    _dev(cand_scores_out, torch.int32, "cand_scores_out")
    Lw, nlw = (L, nl) if leaves is not None else (0, 0)
    need = ah_scan_workspace_bytes(nq, B, n, Lw, nlw, R)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    if leaf_bias is not None:
        _dev(leaf_bias, torch.int32, "leaf_bias", 2)
        if main_events is not None:
            raise ValueError("main_events are not supported with leaf_bias")
        _check(lib().ah_scan_topk_residual(_ptr(lut_i8), nq, B, _ptr(codes), stride, n, _ptr(ids), _ptr(leaf_offsets),
                                           L, _ptr(leaves), nl, _ptr(leaf_bias), int(bias_bound), R,
                                           _ptr(cand_ids_out), _ptr(cand_scores_out), _ptr(workspace),
                                           workspace.numel(), _stream(stream)), "ah_scan_topk_residual")
        return cand_ids_out, cand_scores_out
    args = (_ptr(lut_i8), nq, B, _ptr(codes), stride, n, _ptr(ids), _ptr(leaf_offsets), L, _ptr(leaves), nl, R,
            _ptr(cand_ids_out), _ptr(cand_scores_out), _ptr(workspace), workspace.numel(), _stream(stream))
    if main_events is None:
        _check(lib().ah_scan_topk(*args), "ah_scan_topk")
    else:  # (start, stop) raw hipEvent_t handles bracketing the main scan kernel
        _check(lib().ah_scan_topk_timed(*args, C.c_void_p(main_events[0]), C.c_void_p(main_events[1])),
               "ah_scan_topk_timed")
    return cand_ids_out, cand_scores_out


AH_SCAN_SCRATCH_BYTES = 128 << 20


def ah_scan_topk_noalloc(lut_i8, codes, R, ids=None, leaf_offsets=None, leaves=None, cand_ids_out=None,
                         cand_scores_out=None, stream=None):
    """ah_scan_topk on the library's static per-GPU scratch (no workspace);
    the outputs are allocated here only when not given."""
    lut_i8 = _dev(lut_i8, torch.int8, "lut_i8", 3)
    _dev(ids, torch.int32, "ids")
    _dev(leaf_offsets, torch.int64, "leaf_offsets")
    _dev(leaves, torch.int32, "leaves")
    nq, B, _ = lut_i8.shape
    if isinstance(codes, TiledCodes):
        if codes.blocks != B:
            raise ValueError("tiled codes were made for another number of blocks")
        n, stride = codes.n, AH_CODES_TILED
        codes = _dev(codes.data, torch.uint8, "codes", 1)
    else:
        codes = _dev(codes, torch.uint8, "codes", 2)
        n, stride = codes.shape
    L = 0 if leaf_offsets is None else leaf_offsets.numel() - 1
    nl = 0 if leaves is None else leaves.shape[1]
    if cand_ids_out is None:
        cand_ids_out = torch.empty((nq, R), dtype=torch.int32, device=lut_i8.device)
    if cand_scores_out is None:
        cand_scores_out = torch.empty((nq, R), dtype=torch.int32, device=lut_i8.device)
    _dev(cand_ids_out, torch.int32, "cand_ids_out")
    _dev(cand_scores_out, torch.int32, "cand_scores_out")
    _check(lib().ah_scan_topk_noalloc(_ptr(lut_i8), nq, B, _ptr(codes), stride, n, _ptr(ids), _ptr(leaf_offsets), L,
                                      _ptr(leaves), nl, int(R), _ptr(cand_ids_out), _ptr(cand_scores_out),
                                      _stream(stream)), "ah_scan_topk_noalloc")
    return cand_ids_out, cand_scores_out


def ah_residual_leaf_bias(leaf_scores, step, bias_bound, bias_out=None, stream=None):
    """Residual variant's leaf term in table units: int32 [nq, nl] =
    clip(rint((s[q, j] - s[q, 0]) / step[q]), -bias_bound, bias_bound), 0 when step is 0."""
    leaf_scores = _dev(leaf_scores, torch.float32, "leaf_scores", 2)
    step = _dev(step, torch.float32, "step", 1)
    nq, nl = leaf_scores.shape
    if bias_out is None:
        bias_out = torch.empty((nq, nl), dtype=torch.int32, device=leaf_scores.device)
    _dev(bias_out, torch.int32, "bias_out", 2)
    _check(lib().ah_residual_leaf_bias(_ptr(leaf_scores), _ptr(step), nq, nl, int(bias_bound), _ptr(bias_out),
                                       _stream(stream)), "ah_residual_leaf_bias")
    return bias_out


# ----------------------------------------------------------------------------- step 5
def ah_reorder_exact(q, base, cand_ids, k, ids_out=None, scores_out=None, stream=None):
    """Exact rescoring of candidates; base is float32 [n, d] or bfloat16 [n, d]."""
    q = _dev(q, torch.float32, "q", 2)
    cand_ids = _dev(cand_ids, torch.int32, "cand_ids", 2)
    if base.dtype == torch.float32:
        dt = AH_F32
    elif base.dtype == torch.bfloat16:
        dt = AH_BF16
    else:
        raise TypeError("base must be float32 or bfloat16")
    _dev(base, base.dtype, "base", 2)
    nq, d = q.shape
    n = base.shape[0]
    R = cand_ids.shape[1]
    dev = q.device
    if ids_out is None:
        ids_out = torch.empty((nq, k), dtype=torch.int32, device=dev)
    if scores_out is None:
        scores_out = torch.empty((nq, k), dtype=torch.float32, device=dev)
    _dev(ids_out, torch.int32, "ids_out")
    _dev(scores_out, torch.float32, "scores_out")
    _check(lib().ah_reorder_exact(_ptr(q), nq, d, _ptr(base), dt, n, _ptr(cand_ids), R, k, _ptr(ids_out),
                                  _ptr(scores_out), _stream(stream)), "ah_reorder_exact")
    return ids_out, scores_out


# ----------------------------------------------------------------------------- learned query side
_FLOATS = {torch.float32: AH_F32, torch.bfloat16: AH_BF16}


def _at(t):
    """Address for a pointer argument (the argument types are declared, so a plain int will do)."""
    return None if t is None else t.data_ptr()


def _on(stream, t):
    """The raw stream of a call: the one given, or the current one of t's device."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream.cuda_stream


def _is(t, dtype, name, ndim):
    """_dev in one test; what fails it is named by _dev."""
    if not (type(t) is torch.Tensor and t.is_cuda and t.dtype is dtype and t.dim() == ndim and t.is_contiguous()):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a device tensor")
        _dev(t, dtype, name, ndim)
    return t


def _float_code(dtype, name):
    code = _FLOATS.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {dtype}")
    return code


def _rows(t, dtype, name):
    """A 2-D device tensor whose rows may lie further apart than they are long; returns (tensor, stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dims")
    n, d = t.shape
    stride = t.stride(0) if n > 1 else max(t.stride(0), d)
    if (d > 1 and t.stride(1) != 1) or stride < d:
        raise ValueError(f"{name} must have contiguous, non-overlapping rows")
    return t, stride


def _empty(shape, dtype, device, stream):
    """Device memory that belongs to the stream the call runs on (so that it is not
    handed to other work before the call has finished)."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _out(t, shape, dtype, name, device, stream):
    if t is None:
        return _empty(shape, dtype, device, stream)
    _dev(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _work(t, need, name, device, stream):
    if t is None:
        return _empty(need, torch.uint8, device, stream) if need else None
    _dev(t, torch.uint8, name)
    return t


def _nbytes(t):
    return 0 if t is None else t.numel()


def ah_i8_quantize_rows(x, codes_out=None, scale_out=None, stream=None):
    """Int8 codes and float32 steps (max |x| / 127) of the rows of x (float32 or bfloat16 [n, d])."""
    x, xs = _rows(x, None, "x")
    dt = _float_code(x.dtype, "x")
    n, d = x.shape
    codes_out = _out(codes_out, (n, d), torch.int8, "codes_out", x.device, stream)
    scale_out = _out(scale_out, (n,), torch.float32, "scale_out", x.device, stream)
    _check(lib().ah_i8_quantize_rows(_at(x), dt, n, d, xs, _at(codes_out), _at(scale_out), _on(stream, x)),
           "ah_i8_quantize_rows")
    return codes_out, scale_out


def _channels(w8, w_scale, bias, k):
    _is(w8, torch.int8, "w8", 2)
    _is(w_scale, torch.float32, "w_scale", 1)
    if bias is not None:
        _is(bias, torch.float32, "bias", 1)
    n = w8.shape[0]
    if w8.shape[1] != k:
        raise ValueError("w8 and x differ in their width")
    if w_scale.numel() != n or (bias is not None and bias.numel() != n):
        raise ValueError("w_scale and bias need one entry for each row of w8")
    return n


def ah_i8_matmul(x8, x_scale, w8, w_scale, bias=None, out_dtype=torch.float32, out=None, stream=None):
    """((float)(x8 . w8) * x_scale) * w_scale (+ bias) for every row of x8 [m, k] and of w8 [n, k]."""
    _is(x8, torch.int8, "x8", 2)
    _is(x_scale, torch.float32, "x_scale", 1)
    m, k = x8.shape
    if x_scale.numel() != m:
        raise ValueError("x_scale needs one entry for each row of x8")
    n = _channels(w8, w_scale, bias, k)
    dt = _float_code(out_dtype if out is None else out.dtype, "out")
    out = _out(out, (m, n), out_dtype if out is None else out.dtype, "out", x8.device, stream)
    _check(lib().ah_i8_matmul(_at(x8), _at(x_scale), m, _at(w8), _at(w_scale), n, k, _at(bias), _at(out), dt,
                              _on(stream, x8)), "ah_i8_matmul")
    return out


def ah_i8_linear_workspace_bytes(m: int, k: int) -> int:
    return int(lib().ah_i8_linear_workspace_bytes(m, k))


def ah_i8_linear(x, w8, w_scale, bias=None, out_dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """A linear layer in int8: the rows of x (float32 or bfloat16 [m, k]) quantised, times w8 [n, k]."""
    x, xs = _rows(x, None, "x")
    dt = _float_code(x.dtype, "x")
    m, k = x.shape
    n = _channels(w8, w_scale, bias, k)
    odt = _float_code(out_dtype if out is None else out.dtype, "out")
    out = _out(out, (m, n), out_dtype if out is None else out.dtype, "out", x.device, stream)
    workspace = _work(workspace, ah_i8_linear_workspace_bytes(m, k), "workspace", x.device, stream)
    _check(lib().ah_i8_linear(_at(x), dt, m, k, xs, _at(w8), _at(w_scale), n, _at(bias), _at(out), odt,
                              _at(workspace), _nbytes(workspace), _on(stream, x)), "ah_i8_linear")
    return out


def ah_group_rows_workspace_bytes(n: int, L: int) -> int:
    return int(lib().ah_group_rows_workspace_bytes(n, L))


def ah_group_rows(leaves, L, offsets_out=None, order_out=None, workspace=None, stream=None):
    """Slots in leaf order: (offsets int64 [L + 1], order int32 [slots]) for leaves int32 of any
    shape (slots in memory order; a leaf outside [0, L) means none, such slots come last)."""
    _dev(leaves, torch.int32, "leaves")
    n, L = leaves.numel(), int(L)
    offsets_out = _out(offsets_out, (L + 1,), torch.int64, "offsets_out", leaves.device, stream)
    order_out = _out(order_out, (n,), torch.int32, "order_out", leaves.device, stream)
    workspace = _work(workspace, ah_group_rows_workspace_bytes(n, L), "workspace", leaves.device, stream)
    _check(lib().ah_group_rows(_at(leaves), n, L, _at(offsets_out), _at(order_out), _at(workspace),
                               _nbytes(workspace), _on(stream, leaves)), "ah_group_rows")
    return offsets_out, order_out


def _groups(offsets, order, fan, slots, L):
    _is(offsets, torch.int64, "offsets", 1)
    if order is not None:
        _is(order, torch.int32, "order", 1)
    if offsets.numel() != L + 1:
        raise ValueError("offsets needs one entry more than there are leaves")
    if order is not None and order.numel() != slots:
        raise ValueError("order needs one entry for each slot")
    if order is None and fan != 1:
        raise ValueError("rows without an order cannot be shared (fan > 1)")


def ah_grouped_matmul(x, w, offsets, order=None, fan=1, out_dtype=torch.bfloat16, out=None, stream=None):
    """out[s] = W_leaf(s) x[s // fan] for every slot s: x bfloat16 [m, k], w bfloat16 [L, n, k],
    offsets and order as from ah_group_rows; returns [m * fan, n]."""
    x, xs = _rows(x, torch.bfloat16, "x")
    _is(w, torch.bfloat16, "w", 3)
    m, k = x.shape
    L, n, kw = w.shape
    if kw != k:
        raise ValueError("w and x differ in their width")
    slots = m * fan
    _groups(offsets, order, fan, slots, L)
    dtype = out_dtype if out is None else out.dtype
    odt = _float_code(dtype, "out")
    out = _out(out, (slots, n), dtype, "out", x.device, stream)
    _check(lib().ah_grouped_matmul(_at(x), xs, _at(w), L, n, k, _at(offsets), _at(order), slots, fan, _at(out),
                                   odt, _on(stream, x)), "ah_grouped_matmul")
    return out


def ah_grouped_dx_workspace_bytes(slots: int, k: int, fan: int) -> int:
    return int(lib().ah_grouped_dx_workspace_bytes(slots, k, fan))


def ah_grouped_matmul_dx(dy, w, offsets, order=None, fan=1, out_dtype=torch.bfloat16, dx_out=None, workspace=None,
                         stream=None):
    """Gradient of ah_grouped_matmul with respect to x: dy bfloat16 [m * fan, n] -> [m, k]."""
    dy, dys = _rows(dy, torch.bfloat16, "dy")
    _is(w, torch.bfloat16, "w", 3)
    slots, n = dy.shape
    L, nw, k = w.shape
    if nw != n or fan < 1 or slots % fan:
        raise ValueError("dy needs fan rows of the width of w's output for each query")
    _groups(offsets, order, fan, slots, L)
    dtype = out_dtype if dx_out is None else dx_out.dtype
    odt = _float_code(dtype, "dx_out")
    dx_out = _out(dx_out, (slots // fan, k), dtype, "dx_out", dy.device, stream)
    workspace = _work(workspace, ah_grouped_dx_workspace_bytes(slots, k, fan), "workspace", dy.device, stream)
    _check(lib().ah_grouped_matmul_dx(_at(dy), dys, _at(w), L, n, k, _at(offsets), _at(order), slots, fan,
                                      _at(dx_out), odt, _at(workspace), _nbytes(workspace), _on(stream, dy)),
           "ah_grouped_matmul_dx")
    return dx_out


def ah_grouped_matmul_dw(dy, x, offsets, order=None, fan=1, out_dtype=torch.float32, dw_out=None, stream=None):
    """Gradient of ah_grouped_matmul with respect to w: dy bfloat16 [m * fan, n], x bfloat16 [m, k] -> [L, n, k]."""
    dy, dys = _rows(dy, torch.bfloat16, "dy")
    x, xs = _rows(x, torch.bfloat16, "x")
    slots, n = dy.shape
    m, k = x.shape
    if slots != m * fan:
        raise ValueError("dy needs fan rows for each row of x")
    L = offsets.numel() - 1
    _groups(offsets, order, fan, slots, L)
    dtype = out_dtype if dw_out is None else dw_out.dtype
    odt = _float_code(dtype, "dw_out")
    dw_out = _out(dw_out, (L, n, k), dtype, "dw_out", dy.device, stream)
    _check(lib().ah_grouped_matmul_dw(_at(dy), dys, _at(x), xs, L, n, k, _at(offsets), _at(order), slots, fan,
                                      _at(dw_out), odt, _on(stream, dy)), "ah_grouped_matmul_dw")
    return dw_out


def ah_distill_workspace_bytes(n: int, V: int, k: int) -> int:
    return int(lib().ah_distill_workspace_bytes(n, V, k))


def ah_distill_topk(logits, ids, scores, tau=1.0, row_weight=None, want_grad=True, loss_out=None, grad_out=None,
                    workspace=None, stream=None):
    """Loss (float32 [n]) of a student's logits (float32 or bfloat16 [n, V]) against a teacher's best
    (ids int32, scores float32 [n, k]) and, with want_grad, its gradient times row_weight (else None)."""
    logits, zs = _rows(logits, None, "logits")
    dt = _float_code(logits.dtype, "logits")
    n, V = logits.shape
    _is(ids, torch.int32, "ids", 2)
    _is(scores, torch.float32, "scores", 2)
    if ids.shape != scores.shape or ids.shape[0] != n:
        raise ValueError("ids and scores need one row for each row of logits and the same width")
    if row_weight is not None and _is(row_weight, torch.float32, "row_weight", 1).numel() != n:
        raise ValueError("row_weight needs one entry for each row")
    loss_out = _out(loss_out, (n,), torch.float32, "loss_out", logits.device, stream)
    gs = V
    if grad_out is not None:
        grad_out, gs = _rows(grad_out, logits.dtype, "grad_out")
        if tuple(grad_out.shape) != (n, V):
            raise ValueError("grad_out must have the shape of logits")
    elif want_grad:
        grad_out = _empty((n, V), logits.dtype, logits.device, stream)
    workspace = _work(workspace, ah_distill_workspace_bytes(n, V, ids.shape[1]), "workspace", logits.device, stream)
    _check(lib().ah_distill_topk(_at(logits), dt, n, V, zs, _at(ids), _at(scores), ids.shape[1], float(tau),
                                 _at(row_weight), _at(loss_out), _at(grad_out), gs, _at(workspace),
                                 _nbytes(workspace), _on(stream, logits)), "ah_distill_topk")
    return loss_out, grad_out


# ----------------------------------------------------------------------------- gated blocks, 8-bit floats, dropout
_ACTS = {"silu": 0, "gelu": 1, "relu": 2}
_F8 = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}


def _call(name, where, *args):
    """One library call with `where`'s device current, whatever device is."""
    dev = where.get_device()
    if dev == torch._C._cuda_getDevice():
        status = getattr(lib(), name)(*args)
    else:
        with torch.cuda.device(dev):
            status = getattr(lib(), name)(*args)
    _check(status, name)


def _together(where, *tensors):
    dev = where.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors must be on one device")


def _act_code(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    return code


def _count(step):
    if step is not None and _is(step, torch.int64, "step", step.dim() if isinstance(step, torch.Tensor) else 1).numel() != 1:
        raise ValueError("step must be one int64")
    return step


def _leaf_starts(offsets, order, fan, slots, L):
    if offsets is not None:
        _groups(offsets, order, fan, slots, L)
    elif L != 1 or order is not None or fan != 1:
        raise ValueError("rows without offsets belong to one leaf, without an order or a fan")


def ah_grouped_gated(x, w, offsets=None, order=None, fan=1, act="silu", drop=0.0, seed=0, step=None, want_pre=False,
                     out_dtype=torch.bfloat16, out=None, pre_out=None, stream=None):
    """h[s] = act(gate) * up of slot s's leaf, with dropout: x bfloat16 [m, k], w bfloat16 [L, 2n, k] (gate rows, then
    up rows), offsets and order as from ah_group_rows (none: one leaf has every row).  Returns (h [m * fan, n],
    the projections bfloat16 [m * fan, 2n] for the backward pass with want_pre, else None)."""
    x, xs = _rows(x, torch.bfloat16, "x")
    _is(w, torch.bfloat16, "w", 3)
    m, k = x.shape
    L, n2, kw = w.shape
    if kw != k or n2 % 2:
        raise ValueError("w needs two rows of x's width for each output column")
    slots, n = m * fan, n2 // 2
    _leaf_starts(offsets, order, fan, slots, L)
    _count(step)
    _together(x, w, offsets, order, step, out, pre_out)
    dtype = out_dtype if out is None else out.dtype
    odt = _float_code(dtype, "out")
    out = _out(out, (slots, n), dtype, "out", x.device, stream)
    if pre_out is not None or want_pre:
        pre_out = _out(pre_out, (slots, n2), torch.bfloat16, "pre_out", x.device, stream)
    _call("ah_grouped_gated", x, _at(x), xs, _at(w), L, n, k, _at(offsets), _at(order), slots, fan, _act_code(act),
          float(drop), int(seed) & (2 ** 64 - 1), _at(step), _at(pre_out), _at(out), odt, _on(stream, x))
    return out, pre_out


def ah_grouped_gated_grad(dy, w, pre, offsets=None, order=None, act="silu", drop=0.0, seed=0, step=None,
                          want_hidden=True, dpre_out=None, hidden_out=None, stream=None):
    """From the gradient of a gated block's output to its projections': dy bfloat16 [slots, d], w bfloat16 [L, d, n] (the
    output layer), pre bfloat16 [slots, 2n] and the dropout's arguments as in the forward call.  Returns (dpre bfloat16
    [slots, 2n], h bfloat16 [slots, n] computed again from pre for the output layer's gradient, or None)."""
    dy, dys = _rows(dy, torch.bfloat16, "dy")
    _is(w, torch.bfloat16, "w", 3)
    _is(pre, torch.bfloat16, "pre", 2)
    slots, d = dy.shape
    L, dw, n = w.shape
    if dw != d or tuple(pre.shape) != (slots, 2 * n):
        raise ValueError("w and pre must have the widths of dy and of the block")
    _leaf_starts(offsets, order, 1, slots, L)
    _count(step)
    _together(dy, w, pre, offsets, order, step, dpre_out, hidden_out)
    dpre_out = _out(dpre_out, (slots, 2 * n), torch.bfloat16, "dpre_out", dy.device, stream)
    if hidden_out is not None or want_hidden:
        hidden_out = _out(hidden_out, (slots, n), torch.bfloat16, "hidden_out", dy.device, stream)
    _call("ah_grouped_gated_grad", dy, _at(dy), dys, _at(w), L, d, n, _at(offsets), _at(order), slots, _at(pre),
          _act_code(act), float(drop), int(seed) & (2 ** 64 - 1), _at(step), _at(dpre_out), _at(hidden_out),
          _on(stream, dy))
    return dpre_out, hidden_out


def _f8_code(dtype, name):
    code = _F8.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float8_e4m3fn or float8_e5m2, got {dtype}")
    return code


def _f8_shapes(n, d):
    """Shapes of the codes and of the scales of n rows of d."""
    kb = (d + 127) // 128
    return (n, kb * 128), (kb, (n + 15) // 16 * 16)


def ah_f8_quantize(x, dtype=torch.float8_e4m3fn, want_rows=True, want_columns=False, codes_out=None, scale_out=None,
                   codes_t_out=None, scale_t_out=None, stream=None):
    """8-bit codes of x (float32 or bfloat16 [n, d]) with a scale 2^(byte - 127) for each block of 128: (codes [n, d to a
    multiple of 128], scales uint8 [blocks, n to a multiple of 16]) along the rows and, with want_columns, the
    same of x transposed; None, None for what is not wanted."""
    x, xs = _rows(x, None, "x")
    dt, code = _float_code(x.dtype, "x"), _f8_code(dtype, "dtype")
    n, d = x.shape
    _together(x, codes_out, scale_out, codes_t_out, scale_t_out)
    if want_rows or codes_out is not None:
        cs, ss = _f8_shapes(n, d)
        codes_out = _out(codes_out, cs, dtype, "codes_out", x.device, stream)
        scale_out = _out(scale_out, ss, torch.uint8, "scale_out", x.device, stream)
    if want_columns or codes_t_out is not None:
        cs, ss = _f8_shapes(d, n)
        codes_t_out = _out(codes_t_out, cs, dtype, "codes_t_out", x.device, stream)
        scale_t_out = _out(scale_t_out, ss, torch.uint8, "scale_t_out", x.device, stream)
    _call("ah_f8_quantize", x, _at(x), dt, n, d, xs, code, _at(codes_out), _at(scale_out), _at(codes_t_out),
          _at(scale_t_out), _on(stream, x))
    return codes_out, scale_out, codes_t_out, scale_t_out


def _f8_operand(codes, scale, name):
    if not isinstance(codes, torch.Tensor):
        raise TypeError(f"{name} must be a device tensor")
    code = _f8_code(codes.dtype, name)
    _is(codes, codes.dtype, name, 2)
    _is(scale, torch.uint8, "the scale of codes", 2)
    n, kp = codes.shape
    if kp & 127 or scale.shape != (kp >> 7, (n + 15) & -16):
        raise ValueError(f"{name} and its scale must have the shapes that ah_f8_quantize gives")
    return code, n, kp


def _f8_bias(bias, n):
    if bias is not None and _is(bias, torch.float32, "bias", 1).numel() != n:
        raise ValueError("bias needs one entry for each output column")


def ah_f8_matmul(x8, x_scale, w8, w_scale, bias=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """What the rows of x8 and of w8 stand for, multiplied: out [m, n] (+ bias).  Codes and scales as ah_f8_quantize
    makes them."""
    xc, m, k = _f8_operand(x8, x_scale, "x8")
    wc, n, kw = _f8_operand(w8, w_scale, "w8")
    if kw != k:
        raise ValueError("w8 and x8 differ in their width")
    _f8_bias(bias, n)
    _together(x8, x_scale, w8, w_scale, bias, out)
    dtype = out_dtype if out is None else out.dtype
    odt = _float_code(dtype, "out")
    out = _out(out, (m, n), dtype, "out", x8.device, stream)
    if k == 0:  # a sum over nothing
        with torch.cuda.stream(stream):
            return out.zero_() if bias is None else out.copy_(bias.expand(m, n))
    _call("ah_f8_matmul", x8, _at(x8), _at(x_scale), xc, m, _at(w8), _at(w_scale), wc, n, k, _at(bias), _at(out), odt,
          _on(stream, x8))
    return out


@functools.lru_cache(maxsize=256)
def ah_f8_linear_workspace_bytes(m: int, k: int) -> int:
    return int(lib().ah_f8_linear_workspace_bytes(m, k))


def ah_f8_linear(x, w8, w_scale, bias=None, x_type=torch.float8_e4m3fn, out_dtype=torch.bfloat16, out=None,
                 workspace=None, stream=None):
    """A linear layer in 8-bit floats: the rows of x (float32 or bfloat16 [m, k]) quantised to x_type, times w8
    (ah_f8_quantize of weights [n, k])."""
    x, xs = _rows(x, None, "x")
    dt, xc = _float_code(x.dtype, "x"), _f8_code(x_type, "x_type")
    m, k = x.shape
    wc, n, kw = _f8_operand(w8, w_scale, "w8")
    if kw != (k + 127) // 128 * 128:
        raise ValueError("w8 and x differ in their width")
    _f8_bias(bias, n)
    _together(x, w8, w_scale, bias, out, workspace)
    dtype = out_dtype if out is None else out.dtype
    odt = _float_code(dtype, "out")
    out = _out(out, (m, n), dtype, "out", x.device, stream)
    workspace = _work(workspace, ah_f8_linear_workspace_bytes(m, k), "workspace", x.device, stream)
    _call("ah_f8_linear", x, _at(x), dt, m, k, xs, xc, _at(w8), _at(w_scale), wc, n, _at(bias), _at(out), odt,
          _at(workspace), _nbytes(workspace), _on(stream, x))
    return out


def ah_dropout(x, p, seed, step=None, residual=None, out=None, stream=None):
    """x with each element dropped with probability p and the others multiplied by 1 / (1 - p) (+ residual): float32 or
    bfloat16 [rows, n]; p in [0, 1), taken as min(rint(65536 p), 65535) / 65536.  The mask is a function of seed, step
    (int64 on the device, none: 0), row and column; the gradient is the same call on the output's gradient."""
    x, xs = _rows(x, None, "x")
    dt = _float_code(x.dtype, "x")
    rows, n = x.shape
    rs = os_ = n
    if residual is not None:
        residual, rs = _rows(residual, x.dtype, "residual")
        if residual.shape != x.shape:
            raise ValueError("residual must have the shape of x")
    if out is None:
        out = _empty((rows, n), x.dtype, x.device, stream)
    else:
        out, os_ = _rows(out, x.dtype, "out")
        if out.shape != x.shape:
            raise ValueError("out must have the shape of x")
    _count(step)
    _together(x, step, residual, out)
    _call("ah_dropout", x, _at(x), dt, rows, n, xs, float(p), int(seed) & (2 ** 64 - 1), _at(step), _at(residual), rs,
          _at(out), os_, _on(stream, x))
    return out


# ----------------------------------------------------------------------------- measurement hooks
def ah_scan_workspace_counters(nq: int, B: int, n: int, L: int, nl: int, R: int):
    """(appended_offset, control_offset): byte offsets of the scan's counters in its workspace."""
    a, c = C.c_size_t(), C.c_size_t()
    _check(lib().ah_scan_workspace_counters(nq, B, n, L, nl, R, C.byref(a), C.byref(c)), "ah_scan_workspace_counters")
    return a.value, c.value


def scan_counters(workspace, nq: int, B: int, n: int, L: int, nl: int, R: int):
    """(appended rows per query int64 [nq], overflowed queries) as the last scan
    call on `workspace` left them (synchronises the device)."""
    a, c = ah_scan_workspace_counters(nq, B, n, L, nl, R)
    torch.cuda.synchronize()
    appended = workspace[a:a + 4 * nq].view(torch.int32).cpu().numpy().astype(np.int64) & 0xFFFFFFFF
    ctrl = workspace[c:c + 64].view(torch.int32).cpu().numpy()
    return appended, int(ctrl[1])


def ah_hbm_read_probe(data, blocks_per_cu=8, sink=None, stream=None):
    """Plain-stream read of every byte of the device tensor `data` (16-byte loads)."""
    if not data.is_cuda or not data.is_contiguous():
        raise ValueError("data must be a contiguous device tensor")
    nbytes = data.numel() * data.element_size()
    if sink is None:
        sink = torch.zeros(4, dtype=torch.int32, device=data.device)
    _check(lib().ah_hbm_read_probe(_ptr(data), nbytes, int(blocks_per_cu), _ptr(sink), _stream(stream)),
           "ah_hbm_read_probe")
    return sink

