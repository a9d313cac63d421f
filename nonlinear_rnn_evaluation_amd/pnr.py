"""ctypes binding of libpnr (include/pnr.h): argument marshalling only.

Every step of the evaluation runs in the HIP library; this module turns torch tensors
into device pointers and the C structs, passes torch's current stream, and allocates
the output and workspace tensors (PyTorch is used only for device memory and streams).
If ``libpnr.so`` has not been built, loading raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
from typing import NamedTuple, Optional, Union

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpnr.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "pnr.h")

CELL_GRU, CELL_GRU_DIAG, CELL_LSTM_DIAG = 0, 1, 2
JAC_FULL, JAC_DIAG, JAC_ZERO = 0, 1, 2
F64, F32, BF16 = 0, 1, 2
OK, NOT_CONVERGED, NONFINITE = 0, 1, 2
E_INVALID, E_UNSUPPORTED, E_WORKSPACE, E_HIP = -1, -2, -3, -4
DECAY_HEAD, DECAY_TOKEN = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU = 0, 1, 2
STATIC_SCRATCH_BYTES = 64 << 20   # PNR_STATIC_SCRATCH_BYTES of include/pnr.h

_DT = {torch.float64: F64, torch.float32: F32, torch.bfloat16: BF16}


class PnrCell(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("D", ctypes.c_int32), ("D_in", ctypes.c_int32),
                ("T", ctypes.c_int32), ("B", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("state_dtype", ctypes.c_int32), ("jac_every", ctypes.c_int32),
                ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class PnrParams(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("U", ctypes.c_void_p), ("b_x", ctypes.c_void_p),
                ("b_h", ctypes.c_void_p)]


class PnrProfile(ctypes.Structure):
    _fields_ = [("total_ms", ctypes.c_double), ("proj_ms", ctypes.c_double), ("newton_ms", ctypes.c_double),
                ("out_ms", ctypes.c_double), ("passes", ctypes.c_int32), ("resid_only", ctypes.c_int32)]


class PnrLinattn(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("H_kv", ctypes.c_int32),
                ("D_k", ctypes.c_int32), ("D_v", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("decay", ctypes.c_int32), ("scale", ctypes.c_double), ("q_stride", ctypes.c_int64 * 3),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3), ("lens", ctypes.c_void_p),
                ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class PnrNorm(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int32), ("L", ctypes.c_int32), ("C", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("eps", ctypes.c_double),
                ("lens", ctypes.c_void_p), ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class PnrSelscan(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("E", ctypes.c_int32), ("N", ctypes.c_int32),
                ("G", ctypes.c_int32), ("dtype", ctypes.c_int32), ("softplus", ctypes.c_int32),
                ("u_stride", ctypes.c_int64 * 2), ("dt_stride", ctypes.c_int64 * 2), ("z_stride", ctypes.c_int64 * 2),
                ("B_stride", ctypes.c_int64 * 3), ("C_stride", ctypes.c_int64 * 3), ("lens", ctypes.c_void_p),
                ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class PnrCheckpoint(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("E", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("x_stride", ctypes.c_int64 * 2), ("stream", ctypes.c_void_p)]


class PnrConv(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("E", ctypes.c_int32), ("W", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("act", ctypes.c_int32), ("x_stride", ctypes.c_int64 * 2),
                ("lens", ctypes.c_void_p), ("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libpnr.so from the package directory (raises if it is not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libpnr.so not found at {LIB_PATH}; build it with "
                           "`python -m nonlinear_rnn_evaluation_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER
    lib.pnr_workspace_bytes.argtypes = [P(PnrCell), ctypes.c_int]
    lib.pnr_workspace_bytes.restype = ctypes.c_size_t
    lib.pnr_eval.argtypes = [P(PnrCell), P(PnrParams), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                             ctypes.c_int, ctypes.c_double, ctypes.c_int]
    lib.pnr_eval.restype = ctypes.c_int
    lib.pnr_workspace_bytes_damped.argtypes = [P(PnrCell), ctypes.c_int]
    lib.pnr_workspace_bytes_damped.restype = ctypes.c_size_t
    lib.pnr_eval_damped.argtypes = [P(PnrCell), P(PnrParams), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double]
    lib.pnr_eval_damped.restype = ctypes.c_int
    lib.pnr_workspace_bytes_chunked.argtypes = [P(PnrCell), ctypes.c_int, ctypes.c_double, ctypes.c_int]
    lib.pnr_workspace_bytes_chunked.restype = ctypes.c_size_t
    lib.pnr_eval_chunked.argtypes = [P(PnrCell), P(PnrParams), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double, ctypes.c_int]
    lib.pnr_eval_chunked.restype = ctypes.c_int
    lib.pnr_workspace_bytes_backward.argtypes = [P(PnrCell)]
    lib.pnr_workspace_bytes_backward.restype = ctypes.c_size_t
    lib.pnr_backward.argtypes = [P(PnrCell), P(PnrParams)] + [ctypes.c_void_p] * 10
    lib.pnr_backward.restype = ctypes.c_int
    lib.pnr_workspace_bytes_lowrank.argtypes = [P(PnrCell), ctypes.c_int]
    lib.pnr_workspace_bytes_lowrank.restype = ctypes.c_size_t
    lib.pnr_eval_lowrank.argtypes = [P(PnrCell), P(PnrParams), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int, ctypes.c_double, ctypes.c_int]
    lib.pnr_eval_lowrank.restype = ctypes.c_int
    lib.pnr_eval_bounded.argtypes = [P(PnrCell), P(PnrParams), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int, ctypes.c_double, ctypes.c_int]
    lib.pnr_eval_bounded.restype = ctypes.c_int
    lib.pnr_eval_static.argtypes = [P(PnrCell), P(PnrParams), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_int, ctypes.c_double, ctypes.c_int]
    lib.pnr_eval_static.restype = ctypes.c_int
    lib.pnr_backward_approx.argtypes = [P(PnrCell), P(PnrParams)] + [ctypes.c_void_p] * 10 + [ctypes.c_int]
    lib.pnr_backward_approx.restype = ctypes.c_int
    lib.pnr_eval_adaptive.argtypes = [P(PnrCell), P(PnrParams), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double]
    lib.pnr_eval_adaptive.restype = ctypes.c_int
    lib.pnr_workspace_bytes_backward_chunked.argtypes = [P(PnrCell), ctypes.c_int]
    lib.pnr_workspace_bytes_backward_chunked.restype = ctypes.c_size_t
    lib.pnr_backward_chunked.argtypes = [P(PnrCell), P(PnrParams)] + [ctypes.c_void_p] * 10 + [ctypes.c_int]
    lib.pnr_backward_chunked.restype = ctypes.c_int
    lib.pnr_iters_used.argtypes = []
    lib.pnr_iters_used.restype = ctypes.c_int
    lib.pnr_last_residual.argtypes = []
    lib.pnr_last_residual.restype = ctypes.c_double
    lib.pnr_last_residual_history.argtypes = [P(ctypes.c_double), ctypes.c_int]
    lib.pnr_last_residual_history.restype = ctypes.c_int
    lib.pnr_last_error.argtypes = []
    lib.pnr_last_error.restype = ctypes.c_char_p
    lib.pnr_scan_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    lib.pnr_scan_workspace_bytes.restype = ctypes.c_size_t
    lib.pnr_scan.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                             ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    lib.pnr_scan.restype = ctypes.c_int
    lib.pnr_profile_enable.argtypes = [ctypes.c_int]
    lib.pnr_profile_enable.restype = ctypes.c_int
    lib.pnr_last_profile.argtypes = [P(PnrProfile)]
    lib.pnr_last_profile.restype = ctypes.c_int
    vp = ctypes.c_void_p
    for name, args, res in (
            ("pnr_linattn_workspace_bytes", [P(PnrLinattn)], ctypes.c_size_t),
            ("pnr_linattn_forward", [P(PnrLinattn)] + [vp] * 7, ctypes.c_int),
            ("pnr_linattn_step", [P(PnrLinattn)] + [vp] * 6 + [ctypes.c_int, vp, vp], ctypes.c_int),
            ("pnr_linattn_workspace_bytes_backward", [P(PnrLinattn)], ctypes.c_size_t),
            ("pnr_linattn_backward", [P(PnrLinattn)] + [vp] * 12, ctypes.c_int),
            ("pnr_groupnorm_workspace_bytes", [P(PnrNorm)], ctypes.c_size_t),
            ("pnr_groupnorm", [P(PnrNorm)] + [vp] * 7, ctypes.c_int),
            ("pnr_groupnorm_workspace_bytes_backward", [P(PnrNorm)], ctypes.c_size_t),
            ("pnr_groupnorm_backward", [P(PnrNorm)] + [vp] * 11, ctypes.c_int),
            ("pnr_selscan_workspace_bytes", [P(PnrSelscan)], ctypes.c_size_t),
            ("pnr_selscan_forward", [P(PnrSelscan)] + [vp] * 11, ctypes.c_int),
            ("pnr_selscan_step", [P(PnrSelscan)] + [vp] * 10 + [ctypes.c_int, vp, vp], ctypes.c_int),
            ("pnr_selscan_workspace_bytes_backward", [P(PnrSelscan)], ctypes.c_size_t),
            ("pnr_selscan_backward", [P(PnrSelscan)] + [vp] * 20, ctypes.c_int),
            ("pnr_checkpoint_pack", [P(PnrCheckpoint)] + [vp] * 3, ctypes.c_int),
            ("pnr_checkpoint_unpack", [P(PnrCheckpoint)] + [vp] * 3, ctypes.c_int),
            ("pnr_conv_forward", [P(PnrConv)] + [vp] * 7, ctypes.c_int),
            ("pnr_conv_step", [P(PnrConv)] + [vp] * 5 + [ctypes.c_int, vp, vp], ctypes.c_int),
            ("pnr_conv_workspace_bytes_backward", [P(PnrConv)], ctypes.c_size_t),
            ("pnr_conv_backward", [P(PnrConv)] + [vp] * 11, ctypes.c_int)):
        f = getattr(lib, name)
        f.argtypes, f.restype = args, res
    _lib = lib
    return lib


def header_functions() -> list:
    """Names of the functions declared in include/pnr.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"\b(pnr_[a-z_]+)\s*\(", text)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libpnr takes device tensors")
    if not t.is_contiguous():
        raise ValueError("libpnr takes contiguous tensors")
    return t.data_ptr()


def _check(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple) -> Optional[torch.Tensor]:
    """The library reads raw memory, so a tensor of another dtype or shape would be
    reinterpreted, not converted: refuse it."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return t


def _arg(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple) -> Optional[int]:
    return _ptr(_check(t, name, dtype, shape))


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def make_cell(kind: int, D: int, D_in: int, T: int, B: int, x_dtype: int, state_dtype: int,
              jac_every: int = 1, stream: Optional[int] = None, workspace: Optional[int] = None,
              workspace_bytes: int = 0) -> PnrCell:
    return PnrCell(kind, D, D_in, T, B, x_dtype, state_dtype, jac_every, stream, workspace, workspace_bytes)


# ---- the C entry points under their own names ------------------------------------------
def pnr_workspace_bytes(cell: PnrCell, jac_mode: int) -> int:
    return load().pnr_workspace_bytes(ctypes.byref(cell), jac_mode)


def pnr_eval(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h_out: int, max_iters: int,
             tol: float, jac_mode: int) -> int:
    return load().pnr_eval(ctypes.byref(cell), ctypes.byref(params), x, h0, h_out, max_iters, tol, jac_mode)


def pnr_workspace_bytes_lowrank(cell: PnrCell, rank: int) -> int:
    return load().pnr_workspace_bytes_lowrank(ctypes.byref(cell), rank)


def pnr_eval_lowrank(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h_out: int, max_iters: int,
                     tol: float, rank: int) -> int:
    return load().pnr_eval_lowrank(ctypes.byref(cell), ctypes.byref(params), x, h0, h_out, max_iters, tol, rank)


def pnr_eval_bounded(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h_out: int, max_iters: int,
                     tol: float, jac_mode: int) -> int:
    return load().pnr_eval_bounded(ctypes.byref(cell), ctypes.byref(params), x, h0, h_out, max_iters, tol, jac_mode)


def pnr_eval_static(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h_out: int, max_iters: int,
                    tol: float, jac_mode: int) -> int:
    return load().pnr_eval_static(ctypes.byref(cell), ctypes.byref(params), x, h0, h_out, max_iters, tol, jac_mode)


def pnr_eval_adaptive(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h_out: int, max_iters: int,
                      tol: float, jac_mode: int, refresh_ratio: float) -> int:
    return load().pnr_eval_adaptive(ctypes.byref(cell), ctypes.byref(params), x, h0, h_out, max_iters, tol,
                                    jac_mode, refresh_ratio)


def pnr_workspace_bytes_damped(cell: PnrCell, jac_mode: int) -> int:
    return load().pnr_workspace_bytes_damped(ctypes.byref(cell), jac_mode)


def pnr_eval_damped(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h_out: int, max_iters: int,
                    tol: float, jac_mode: int, damping: float) -> int:
    return load().pnr_eval_damped(ctypes.byref(cell), ctypes.byref(params), x, h0, h_out, max_iters, tol, jac_mode,
                                  damping)


def pnr_workspace_bytes_chunked(cell: PnrCell, jac_mode: int, damping: float, chunk_len: int) -> int:
    return load().pnr_workspace_bytes_chunked(ctypes.byref(cell), jac_mode, damping, chunk_len)


def pnr_eval_chunked(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h_out: int, max_iters: int,
                     tol: float, jac_mode: int, damping: float, chunk_len: int) -> int:
    return load().pnr_eval_chunked(ctypes.byref(cell), ctypes.byref(params), x, h0, h_out, max_iters, tol, jac_mode,
                                   damping, chunk_len)


def pnr_workspace_bytes_backward(cell: PnrCell) -> int:
    return load().pnr_workspace_bytes_backward(ctypes.byref(cell))


def pnr_backward(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h: int, grad_h: int,
                 grad_x: Optional[int], grad_W: Optional[int], grad_U: Optional[int], grad_b_x: Optional[int],
                 grad_b_h: Optional[int], grad_h0: Optional[int]) -> int:
    return load().pnr_backward(ctypes.byref(cell), ctypes.byref(params), x, h0, h, grad_h, grad_x, grad_W, grad_U,
                               grad_b_x, grad_b_h, grad_h0)


def pnr_backward_approx(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h: int, grad_h: int,
                        grad_x: Optional[int], grad_W: Optional[int], grad_U: Optional[int],
                        grad_b_x: Optional[int], grad_b_h: Optional[int], grad_h0: Optional[int],
                        jac_mode: int) -> int:
    return load().pnr_backward_approx(ctypes.byref(cell), ctypes.byref(params), x, h0, h, grad_h, grad_x, grad_W,
                                      grad_U, grad_b_x, grad_b_h, grad_h0, jac_mode)


def pnr_workspace_bytes_backward_chunked(cell: PnrCell, chunk_len: int) -> int:
    return load().pnr_workspace_bytes_backward_chunked(ctypes.byref(cell), chunk_len)


def pnr_backward_chunked(cell: PnrCell, params: PnrParams, x: int, h0: Optional[int], h: int, grad_h: int,
                         grad_x: Optional[int], grad_W: Optional[int], grad_U: Optional[int],
                         grad_b_x: Optional[int], grad_b_h: Optional[int], grad_h0: Optional[int],
                         chunk_len: int) -> int:
    return load().pnr_backward_chunked(ctypes.byref(cell), ctypes.byref(params), x, h0, h, grad_h, grad_x, grad_W,
                                       grad_U, grad_b_x, grad_b_h, grad_h0, chunk_len)


def pnr_iters_used() -> int:
    return load().pnr_iters_used()


def pnr_last_residual() -> float:
    return load().pnr_last_residual()


def pnr_last_residual_history() -> list:
    lib = load()
    n = lib.pnr_last_residual_history(None, 0)
    buf = (ctypes.c_double * max(n, 1))()
    lib.pnr_last_residual_history(buf, n)
    return list(buf[:n])


def pnr_last_error() -> str:
    return load().pnr_last_error().decode()


def pnr_scan_workspace_bytes(kind: int, R: int, T: int, tile_len: int = 0) -> int:
    return load().pnr_scan_workspace_bytes(kind, R, T, tile_len)


def pnr_scan(kind: int, R: int, T: int, A: int, b: int, d: int, tile_len: int, workspace: int,
             workspace_bytes: int, stream: Optional[int]) -> int:
    return load().pnr_scan(kind, R, T, A, b, d, tile_len, workspace, workspace_bytes, stream)


def pnr_profile_enable(on: bool) -> int:
    return load().pnr_profile_enable(1 if on else 0)


def pnr_last_profile() -> Optional[dict]:
    p = PnrProfile()
    if load().pnr_last_profile(ctypes.byref(p)) != 0:
        return None
    return {name: getattr(p, name) for name, _ in PnrProfile._fields_}


def pnr_linattn_workspace_bytes(desc: PnrLinattn) -> int:
    return load().pnr_linattn_workspace_bytes(ctypes.byref(desc))


def pnr_linattn_forward(desc: PnrLinattn, q: int, k: int, v: int, log_decay: int, state_in: Optional[int],
                        o: Optional[int], state_out: Optional[int]) -> int:
    return load().pnr_linattn_forward(ctypes.byref(desc), q, k, v, log_decay, state_in, o, state_out)


def pnr_linattn_step(desc: PnrLinattn, q: int, k: int, v: int, log_decay: int, state_in: int,
                     slots: Optional[int], n_slots: int, o: int, state_out: int) -> int:
    return load().pnr_linattn_step(ctypes.byref(desc), q, k, v, log_decay, state_in, slots, n_slots, o, state_out)


def pnr_linattn_workspace_bytes_backward(desc: PnrLinattn) -> int:
    return load().pnr_linattn_workspace_bytes_backward(ctypes.byref(desc))


def pnr_linattn_backward(desc: PnrLinattn, q: int, k: int, v: int, log_decay: int, state_in: Optional[int],
                         grad_o: int, grad_state_out: Optional[int], grad_q: Optional[int], grad_k: Optional[int],
                         grad_v: Optional[int], grad_log_decay: Optional[int], grad_state_in: Optional[int]) -> int:
    return load().pnr_linattn_backward(ctypes.byref(desc), q, k, v, log_decay, state_in, grad_o, grad_state_out,
                                       grad_q, grad_k, grad_v, grad_log_decay, grad_state_in)


def pnr_groupnorm_workspace_bytes(desc: PnrNorm) -> int:
    return load().pnr_groupnorm_workspace_bytes(ctypes.byref(desc))


def pnr_groupnorm(desc: PnrNorm, x: int, weight: Optional[int], bias: Optional[int], gate: Optional[int], y: int,
                  mean: Optional[int], rstd: Optional[int]) -> int:
    return load().pnr_groupnorm(ctypes.byref(desc), x, weight, bias, gate, y, mean, rstd)


def pnr_groupnorm_workspace_bytes_backward(desc: PnrNorm) -> int:
    return load().pnr_groupnorm_workspace_bytes_backward(ctypes.byref(desc))


def pnr_groupnorm_backward(desc: PnrNorm, x: int, weight: Optional[int], bias: Optional[int], gate: Optional[int],
                           grad_y: int, mean: int, rstd: int, grad_x: Optional[int], grad_weight: Optional[int],
                           grad_bias: Optional[int], grad_gate: Optional[int]) -> int:
    return load().pnr_groupnorm_backward(ctypes.byref(desc), x, weight, bias, gate, grad_y, mean, rstd, grad_x,
                                         grad_weight, grad_bias, grad_gate)


def pnr_selscan_workspace_bytes(desc: PnrSelscan) -> int:
    return load().pnr_selscan_workspace_bytes(ctypes.byref(desc))


def pnr_selscan_forward(desc: PnrSelscan, u: int, dt: int, A: int, B: int, C: int, D: Optional[int], z: Optional[int],
                        dt_bias: Optional[int], state_in: Optional[int], y: int, state_out: Optional[int]) -> int:
    return load().pnr_selscan_forward(ctypes.byref(desc), u, dt, A, B, C, D, z, dt_bias, state_in, y, state_out)


def pnr_selscan_step(desc: PnrSelscan, u: int, dt: int, A: int, B: int, C: int, D: Optional[int], z: Optional[int],
                     dt_bias: Optional[int], state_in: int, slots: Optional[int], n_slots: int, y: int,
                     state_out: int) -> int:
    return load().pnr_selscan_step(ctypes.byref(desc), u, dt, A, B, C, D, z, dt_bias, state_in, slots, n_slots, y,
                                   state_out)


def pnr_selscan_workspace_bytes_backward(desc: PnrSelscan) -> int:
    return load().pnr_selscan_workspace_bytes_backward(ctypes.byref(desc))


def pnr_selscan_backward(desc: PnrSelscan, u: int, dt: int, A: int, B: int, C: int, D: Optional[int],
                         z: Optional[int], dt_bias: Optional[int], state_in: Optional[int], grad_y: int,
                         grad_state_out: Optional[int], *grads: Optional[int]) -> int:
    """grads: u, dt, A, B, C, D, z, dt_bias, state_in."""
    return load().pnr_selscan_backward(ctypes.byref(desc), u, dt, A, B, C, D, z, dt_bias, state_in, grad_y,
                                       grad_state_out, *grads)


def pnr_checkpoint_pack(desc: PnrCheckpoint, x: int, codes: int, exponents: int) -> int:
    return load().pnr_checkpoint_pack(ctypes.byref(desc), x, codes, exponents)


def pnr_checkpoint_unpack(desc: PnrCheckpoint, codes: int, exponents: int, x: int) -> int:
    return load().pnr_checkpoint_unpack(ctypes.byref(desc), codes, exponents, x)


def pnr_conv_forward(desc: PnrConv, x: int, exponents: Optional[int], weight: int, bias: Optional[int],
                     state_in: Optional[int], y: int, state_out: Optional[int]) -> int:
    return load().pnr_conv_forward(ctypes.byref(desc), x, exponents, weight, bias, state_in, y, state_out)


def pnr_conv_step(desc: PnrConv, x: int, weight: int, bias: Optional[int], state_in: Optional[int],
                  slots: Optional[int], n_slots: int, y: int, state_out: Optional[int]) -> int:
    return load().pnr_conv_step(ctypes.byref(desc), x, weight, bias, state_in, slots, n_slots, y, state_out)


def pnr_conv_workspace_bytes_backward(desc: PnrConv) -> int:
    return load().pnr_conv_workspace_bytes_backward(ctypes.byref(desc))


def pnr_conv_backward(desc: PnrConv, x: int, exponents: Optional[int], weight: int, bias: Optional[int],
                      state_in: Optional[int], grad_y: int, grad_state_out: Optional[int], grad_x: Optional[int],
                      grad_weight: Optional[int], grad_bias: Optional[int], grad_state_in: Optional[int]) -> int:
    return load().pnr_conv_backward(ctypes.byref(desc), x, exponents, weight, bias, state_in, grad_y, grad_state_out,
                                    grad_x, grad_weight, grad_bias, grad_state_in)


# ---- torch-level conveniences (allocation + marshalling) ---------------------------------
class PnrError(RuntimeError):
    pass


def evaluate(kind: int, W: torch.Tensor, U: torch.Tensor, x: torch.Tensor, *, b_x=None, b_h=None,
             h0=None, max_iters: int = 64, tol: float = 1e-5, jac_mode: int = JAC_FULL,
             jac_every: int = 1, h_out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, damping: Optional[float] = None,
             chunk_len: Optional[int] = None, refresh_ratio: Optional[float] = None,
             static_scratch: bool = False, bounded: bool = False, jac_rank: Optional[int] = None) -> dict:
    """Run pnr_eval (or pnr_eval_damped when `damping` is given, pnr_eval_chunked when
    `chunk_len` is given, pnr_eval_adaptive when `refresh_ratio` is given, pnr_eval_static
    -- no workspace; the library's static device scratch -- when `static_scratch`,
    pnr_eval_bounded when `bounded`, pnr_eval_lowrank when `jac_rank` is given -- the
    jac_mode argument is then FULL) on device tensors; returns dict(h=[B,T,S], status,
    iters, residual, history)."""
    if refresh_ratio is not None and (damping is not None or chunk_len is not None):
        raise ValueError("refresh_ratio combines with neither damping nor chunk_len")
    if static_scratch and (refresh_ratio is not None or damping is not None or chunk_len is not None
                           or workspace is not None):
        raise ValueError("static_scratch is pnr_eval's variant: no damping, chunking, refresh ratio or workspace")
    if jac_rank is not None and (refresh_ratio is not None or damping is not None or chunk_len is not None
                                 or static_scratch or bounded):
        raise ValueError("jac_rank is pnr_eval's variant: no damping, chunking, refresh ratio, bounds or static scratch")
    if bounded and (refresh_ratio is not None or damping is not None or chunk_len is not None or static_scratch):
        raise ValueError("bounded is pnr_eval's variant: no damping, chunking, refresh ratio or static scratch")
    B, T, D_in = x.shape
    D = U.shape[1]
    S = 2 * D if kind == CELL_LSTM_DIAG else D
    if x.dtype not in _DT or U.dtype not in _DT:
        raise TypeError(f"unsupported dtypes x {x.dtype}, U {U.dtype}")
    xdt, sdt = _DT[x.dtype], _DT[U.dtype]
    G = 4 if kind == CELL_LSTM_DIAG else 3
    sd = U.dtype
    args = dict(W=_check(W, "W", x.dtype, (G * D, D_in)),
                U=_check(U, "U", sd, (G * D, D) if kind == CELL_GRU else (G, D)),
                b_x=_check(b_x, "b_x", sd, (G * D,)), b_h=_check(b_h, "b_h", sd, (G * D,)),
                h0=_check(h0, "h0", sd, (B, S)), x=x)
    if h_out is not None:
        _check(h_out, "h_out", sd, (B, T, S))
    ptrs = {k: _ptr(v) for k, v in args.items()}
    cell = make_cell(kind, D, D_in, T, B, xdt, sdt, jac_every, _stream())
    if static_scratch:
        need = 0
    elif jac_rank is not None:
        need = pnr_workspace_bytes_lowrank(cell, jac_rank)
    elif chunk_len is not None:
        need = pnr_workspace_bytes_chunked(cell, jac_mode, damping or 0.0, chunk_len)
    elif damping is None:
        need = pnr_workspace_bytes(cell, jac_mode)
    else:
        need = pnr_workspace_bytes_damped(cell, jac_mode)
    if need == 0 and not static_scratch:
        raise PnrError(pnr_last_error())
    if not static_scratch:
        if workspace is None or workspace.numel() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        cell.workspace = workspace.data_ptr()
        cell.workspace_bytes = workspace.numel()
    if h_out is None:
        h_out = torch.empty(B, T, S, dtype=U.dtype, device=x.device)
    out = _arg(h_out, "h_out", sd, (B, T, S))
    params = PnrParams(ptrs["W"], ptrs["U"], ptrs["b_x"], ptrs["b_h"])
    if jac_rank is not None:
        rc = pnr_eval_lowrank(cell, params, ptrs["x"], ptrs["h0"], out, max_iters, tol, jac_rank)
    elif bounded:
        rc = pnr_eval_bounded(cell, params, ptrs["x"], ptrs["h0"], out, max_iters, tol, jac_mode)
    elif static_scratch:
        rc = pnr_eval_static(cell, params, ptrs["x"], ptrs["h0"], out, max_iters, tol, jac_mode)
    elif chunk_len is not None:
        rc = pnr_eval_chunked(cell, params, ptrs["x"], ptrs["h0"], out, max_iters, tol, jac_mode,
                              damping or 0.0, chunk_len)
    elif refresh_ratio is not None:
        rc = pnr_eval_adaptive(cell, params, ptrs["x"], ptrs["h0"], out, max_iters, tol, jac_mode, refresh_ratio)
    elif damping is None:
        rc = pnr_eval(cell, params, ptrs["x"], ptrs["h0"], out, max_iters, tol, jac_mode)
    else:
        rc = pnr_eval_damped(cell, params, ptrs["x"], ptrs["h0"], out, max_iters, tol, jac_mode, damping)
    if rc < 0:
        raise PnrError(f"pnr_eval returned {rc}: {pnr_last_error()}")
    return {"h": h_out, "status": rc, "iters": pnr_iters_used(), "residual": pnr_last_residual(),
            "history": pnr_last_residual_history(), "workspace": workspace}


def backward(kind: int, W: torch.Tensor, U: torch.Tensor, x: torch.Tensor, h: torch.Tensor, grad_h: torch.Tensor,
             *, b_x=None, b_h=None, h0=None, want=("x", "W", "U", "b_x", "b_h", "h0"),
             workspace: Optional[torch.Tensor] = None, chunk_len: int = 0,
             jac_mode: Optional[int] = None) -> dict:
    """Run pnr_backward on device tensors: gradients of L through the recurrence whose
    states are h, given grad_h = dL/dh.  Returns {name: fp32 tensor} for the names in
    `want` (the others are not computed), plus "workspace" and the adjoint solve's
    "status", "iters", "residual" and "history" (dense GRU: refinement iterations;
    diagonal cells: one scan, iters 0).  chunk_len > 0 runs pnr_backward_chunked: the
    sequence is processed in chunks of that many steps, last chunk first, with a
    workspace sized for one chunk.  jac_mode runs pnr_backward_approx: JAC_FULL exact,
    JAC_DIAG the diagonal approximation in the adjoint recursion."""
    if jac_mode is not None and chunk_len:
        raise ValueError("jac_mode applies to the unchunked backward pass")
    B, T, D_in = x.shape
    G, D = (U.shape[0] // U.shape[1], U.shape[1]) if kind == CELL_GRU else (U.shape[0], U.shape[1])
    S = 2 * D if kind == CELL_LSTM_DIAG else D
    if x.dtype not in _DT or U.dtype not in _DT:
        raise TypeError(f"unsupported dtypes x {x.dtype}, U {U.dtype}")
    sd = U.dtype
    args = dict(h=_check(h, "h", sd, (B, T, S)), grad_h=_check(grad_h, "grad_h", sd, (B, T, S)),
                W=_check(W, "W", x.dtype, (G * D, D_in)), b_x=_check(b_x, "b_x", sd, (G * D,)),
                b_h=_check(b_h, "b_h", sd, (G * D,)), h0=_check(h0, "h0", sd, (B, S)), U=U, x=x)
    ptrs = {k: _ptr(v) for k, v in args.items()}
    cell = make_cell(kind, D, D_in, T, B, _DT[x.dtype], _DT[U.dtype], 1, _stream())
    if chunk_len < 0:
        raise ValueError(f"chunk_len must be >= 0 (got {chunk_len})")
    need = pnr_workspace_bytes_backward_chunked(cell, chunk_len) if chunk_len else pnr_workspace_bytes_backward(cell)
    if need == 0:
        raise PnrError(pnr_last_error())
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    cell.workspace = workspace.data_ptr()
    cell.workspace_bytes = workspace.numel()
    f32 = dict(dtype=torch.float32, device=x.device)
    shapes = {"x": (B, T, D_in), "W": (G * D, D_in), "U": tuple(U.shape), "b_x": (G * D,), "b_h": (G * D,),
              "h0": (B, S)}
    out = {k: torch.empty(shapes[k], **f32) for k in want}
    params = PnrParams(ptrs["W"], ptrs["U"], ptrs["b_x"], ptrs["b_h"])
    grads = [_ptr(out.get(k)) for k in ("x", "W", "U", "b_x", "b_h", "h0")]
    if chunk_len:
        rc = pnr_backward_chunked(cell, params, ptrs["x"], ptrs["h0"], ptrs["h"], ptrs["grad_h"], *grads, chunk_len)
    elif jac_mode is not None:
        rc = pnr_backward_approx(cell, params, ptrs["x"], ptrs["h0"], ptrs["h"], ptrs["grad_h"], *grads, jac_mode)
    else:
        rc = pnr_backward(cell, params, ptrs["x"], ptrs["h0"], ptrs["h"], ptrs["grad_h"], *grads)
    if rc < 0:
        raise PnrError(f"pnr_backward{'_chunked' if chunk_len else ''} returned {rc}: {pnr_last_error()}")
    out.update(workspace=workspace, status=rc, iters=pnr_iters_used(), residual=pnr_last_residual(),
               history=pnr_last_residual_history())
    return out


def scan(kind: int, A: torch.Tensor, b: torch.Tensor, tile_len: int = 0) -> torch.Tensor:
    """Standalone linear scan d_t = A_t d_{t-1} + b_t (kind 1: [R,T]; kind 2: A [R,4,T], b [R,2,T])."""
    R, T = b.shape[0], b.shape[-1]
    shapes = {1: ((R, T), (R, T)), 2: ((R, 4, T), (R, 2, T))}.get(kind)
    if shapes is not None:
        _check(A, "A", torch.float32, shapes[0])
        _check(b, "b", torch.float32, shapes[1])
    d = torch.empty_like(b)
    need = pnr_scan_workspace_bytes(kind, R, T, tile_len)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device=b.device)
    rc = pnr_scan(kind, R, T, _ptr(A), _ptr(b), _ptr(d), tile_len, ws.data_ptr(), ws.numel(), _stream())
    if rc < 0:
        raise PnrError(f"pnr_scan returned {rc}: {pnr_last_error()}")
    return d


# ---- sequence mixing: linear attention with per-head decay, group norm with an activation ------
# A decoded token costs little more than its call, so the checks below are one expression each
# where everything is right, and the descriptors are packed in one go.
_SEQ_DT = {torch.float32: F32, torch.bfloat16: BF16}
_LINATTN = struct.Struct("8i d 9q 3P N")      # the layouts of pnr_linattn and pnr_norm
_NORM = struct.Struct("6i d 3P N")
_SELSCAN = struct.Struct("7i 12q 3P N")        # ... of pnr_selscan, pnr_checkpoint and pnr_conv
_CHECKPOINT = struct.Struct("4i 2q P")
_CONV = struct.Struct("6i 2q 3P N")


def _pack(struct_type, layout: struct.Struct, *fields):
    """A descriptor from its fields in order."""
    try:
        return struct_type.from_buffer_copy(layout.pack(*fields))
    except struct.error:
        raise PnrError(f"a size of the request does not fit in 32 bits, or a stride in 64 (fields {fields})") from None


def _raw_stream(device: int) -> int:
    """torch's current stream of a device, as a hipStream_t."""
    return torch._C._cuda_getCurrentRawStream(device)


def _on(device: int, t: Optional[torch.Tensor], name: str, dtype: torch.dtype, shape: tuple) -> Optional[int]:
    """The pointer of a contiguous tensor on the call's device."""
    if t is None:
        return None
    if not (t.dtype == dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()):
        _arg(t, name, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> None:
    """Names what is wrong with a strided [..., D] operand."""
    _check(t, name, dtype, shape)
    if not t.is_cuda:
        raise ValueError("libpnr takes device tensors")
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")


def _workspace(need: int, workspace: Optional[torch.Tensor], device: int, desc) -> Optional[torch.Tensor]:
    """Points the descriptor at `workspace`, or at a new one where that is missing or too small."""
    if need:
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", device))
        elif workspace.get_device() != device:
            raise ValueError(f"workspace is on {workspace.device}, not on cuda:{device}")
        elif not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        desc.workspace = _ptr(workspace)
        desc.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


def _call(fn, device: int, *args) -> None:
    """One of the calls above on its tensors' device: a launch goes to the current one, and the default
    stream's handle is the same on all."""
    if torch.cuda.current_device() == device:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc < 0:
        raise PnrError(f"{fn.__name__} returned {rc}: {pnr_last_error()}")


def _linattn(q, k, v, log_decay, scale, lens, step: bool) -> tuple:
    """The descriptor of a linear-attention call, the four inputs' pointers, the sizes, the device."""
    dt = q.dtype
    code = _SEQ_DT.get(dt)
    if code is None:
        raise TypeError(f"linear attention takes float32 or bfloat16 (got {dt})")
    qs, ks, vs, dims = q.shape, k.shape, v.shape, 3 if step else 4
    if not len(qs) == len(ks) == len(vs) == dims:
        raise ValueError("q, k, v must be " + ("[B, heads, D]" if step else "[B, T, heads, D]"))
    lead, (H, Dk), (Hkv, Dv) = qs[:-2], qs[-2:], vs[-2:]
    a, b, c, dev = q.stride(), k.stride(), v.stride(), q.get_device()
    if not (k.dtype == dt == v.dtype and dev >= 0 and k.get_device() == dev == v.get_device() and vs[:-2] == lead
            and ks == (*lead, Hkv, Dk) and (a[-1] == 1 or Dk == 1) and (b[-1] == 1 or Dk == 1) and (c[-1] == 1 or Dv == 1)):
        _rows(q, "q", dt, qs, dev)
        _rows(k, "k", dt, (*lead, Hkv, Dk), dev)
        _rows(v, "v", dt, (*lead, Hkv, Dv), dev)
    token = log_decay.dim() != 1
    g = _on(dev, log_decay, "log_decay", torch.float32, (*lead, Hkv) if token else (Hkv,))
    T, qt, kt, vt = (1, 0, 0, 0) if step else (lead[1], a[1], b[1], c[1])
    desc = _pack(
        PnrLinattn, _LINATTN, lead[0], T, H, Hkv, Dk, Dv, code, DECAY_TOKEN if token else DECAY_HEAD, Dk ** -0.5 if scale is None else scale,
        a[0], qt, a[-2], b[0], kt, b[-2], c[0], vt, c[-2], _on(dev, lens, "lens", torch.int32, lead[:1]) or 0,
        _raw_stream(dev), 0, 0)
    return desc, (q.data_ptr(), k.data_ptr(), v.data_ptr(), g), (lead[0], T, H, Hkv, Dk, Dv), dev


def linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
                     scale: Optional[float] = None, state: Optional[torch.Tensor] = None,
                     lens: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                     state_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_linattn_forward: S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t over whole
    sequences.  q [B,T,H,D_k], k [B,T,H_kv,D_k], v [B,T,H_kv,D_v] (float32 or bfloat16, strided as
    they come, last axis contiguous), log_decay float32 [H_kv] or [B,T,H_kv], state (the state
    before the first token, zeros if None) float32 [B,H_kv,D_k,D_v], lens int32 [B] (tokens of
    each row, T if None); scale None is D_k ** -0.5.  Returns dict(o=[B,T,H,D_v], state=the state
    after each row's last token, workspace)."""
    desc, ptrs, (B, T, H, Hkv, Dk, Dv), dev = _linattn(q, k, v, log_decay, scale, lens, False)
    if o is None:
        o = torch.empty(B, T, H, Dv, dtype=q.dtype, device=q.device)
    shape = (B, Hkv, Dk, Dv)
    if state_out is None:
        state_out = torch.empty(shape, dtype=torch.float32, device=q.device)
    args = (_on(dev, state, "state", torch.float32, shape), _on(dev, o, "o", q.dtype, (B, T, H, Dv)),
            _on(dev, state_out, "state_out", torch.float32, shape))
    workspace = _workspace(pnr_linattn_workspace_bytes(desc), workspace, dev, desc)
    _call(pnr_linattn_forward, dev, desc, *ptrs, *args)
    return {"o": o, "state": state_out, "workspace": workspace}


def linear_attention_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                          state: torch.Tensor, *, scale: Optional[float] = None, slots: Optional[torch.Tensor] = None,
                          state_out: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_linattn_step: one token for each of B requests.  q [B,H,D_k], k [B,H_kv,D_k],
    v [B,H_kv,D_v], log_decay float32 [H_kv] or [B,H_kv]; state float32 [n_slots,H_kv,D_k,D_v], the
    pool of running requests' states, of which request b has slot slots[b] (int32 [B]; slot b if
    None; a slot outside the pool marks an idle row).  The pool is updated in place unless
    state_out gives another one of its shape.  Returns dict(o=[B,H,D_v], state=the updated pool)."""
    desc, ptrs, (B, _, H, Hkv, Dk, Dv), dev = _linattn(q, k, v, log_decay, scale, None, True)
    if state_out is None:
        state_out = state
    if o is None:
        o = torch.empty(B, H, Dv, dtype=q.dtype, device=q.device)
    n_slots = state.shape[0] if state.dim() else 0
    shape = (n_slots, Hkv, Dk, Dv)
    _call(pnr_linattn_step, dev, desc, *ptrs, _on(dev, state, "state", torch.float32, shape),
          _on(dev, slots, "slots", torch.int32, (B,)), n_slots, _on(dev, o, "o", q.dtype, (B, H, Dv)),
          _on(dev, state_out, "state_out", torch.float32, shape))
    return {"o": o, "state": state_out}


def linear_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                              grad_o: torch.Tensor, *, scale: Optional[float] = None,
                              state: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
                              grad_state: Optional[torch.Tensor] = None,
                              want=("q", "k", "v", "log_decay", "state"),
                              workspace: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_linattn_backward: gradients through linear_attention of these arguments, given
    grad_o = dL/do [B,T,H,D_v] and grad_state = dL/d(returned state) (zeros if None).  Returns
    {name: gradient} for the names in `want` (q, k, v in their dtype; log_decay and state in
    float32; "state" only where a state is given) and "workspace"."""
    desc, ptrs, (B, T, H, Hkv, Dk, Dv), dev = _linattn(q, k, v, log_decay, scale, lens, False)
    shape = (B, Hkv, Dk, Dv)
    args = (_on(dev, state, "state", torch.float32, shape), _on(dev, grad_o, "grad_o", q.dtype, (B, T, H, Dv)),
            _on(dev, grad_state, "grad_state", torch.float32, shape))
    like = dict(q=(q.shape, q.dtype), k=(k.shape, q.dtype), v=(v.shape, q.dtype),
                log_decay=(log_decay.shape, torch.float32), state=(shape, torch.float32))
    unknown = set(want) - set(like)
    if unknown:
        raise ValueError(f"no gradient named {sorted(unknown)}")
    out = {n: torch.empty(like[n][0], dtype=like[n][1], device=q.device) for n in want
           if n != "state" or state is not None}
    workspace = _workspace(pnr_linattn_workspace_bytes_backward(desc), workspace, dev, desc)
    _call(pnr_linattn_backward, dev, desc, *ptrs, *args, *[_ptr(out.get(n)) for n in ("q", "k", "v", "log_decay", "state")])
    out["workspace"] = workspace
    return out


def _norm(x, groups, weight, bias, gate, act, eps, lens) -> tuple:
    """The descriptor of a group-norm call, the pointers of x, weight, bias and gate, the device."""
    code = _SEQ_DT.get(x.dtype)
    if code is None:
        raise TypeError(f"group norm takes float32 or bfloat16 (got {x.dtype})")
    shape = x.shape
    if len(shape) != 3:
        raise ValueError(f"x must be [N, L, C] (got {tuple(shape)})")
    dev, params = x.get_device(), shape[2:]
    if dev < 0:
        raise ValueError("libpnr takes device tensors")
    ptrs = (_on(dev, x, "x", x.dtype, shape), _on(dev, weight, "weight", torch.float32, params),
            _on(dev, bias, "bias", torch.float32, params), _on(dev, gate, "gate", x.dtype, shape))
    desc = _pack(PnrNorm, _NORM, *shape, groups, code, act, eps, _on(dev, lens, "lens", torch.int32, shape[:1]) or 0,
                 _raw_stream(dev), 0, 0)
    return desc, ptrs, dev


def group_norm(x: torch.Tensor, groups: int, *, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, act: int = ACT_NONE,
               eps: float = 1e-5, lens: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_groupnorm on x [N, L, C], channels last: every run of C / groups channels is normalised
    over itself and the L positions, scaled by weight and bias (float32 [C], both or neither), then
    y = act(z), or z act(gate) with a gate like x.  lens int32 [N]: the positions of each row.
    L = 1 is the norm of N tokens by heads.  Returns dict(y, mean, rstd [N, groups], workspace)."""
    desc, ptrs, dev = _norm(x, groups, weight, bias, gate, act, eps, lens)
    if y is None:
        y = torch.empty_like(x)
    out = _on(dev, y, "y", x.dtype, x.shape)
    mean, rstd = torch.empty(2, x.shape[0], min(max(groups, 1), x.shape[2]), dtype=torch.float32, device=x.device).unbind(0)
    workspace = _workspace(pnr_groupnorm_workspace_bytes(desc), workspace, dev, desc)
    _call(pnr_groupnorm, dev, desc, *ptrs, out, mean.data_ptr(), rstd.data_ptr())
    return {"y": y, "mean": mean, "rstd": rstd, "workspace": workspace}


def group_norm_backward(grad_y: torch.Tensor, x: torch.Tensor, groups: int, mean: torch.Tensor, rstd: torch.Tensor, *,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, act: int = ACT_NONE,
                        lens: Optional[torch.Tensor] = None, want=("x", "weight", "bias", "gate"),
                        workspace: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_groupnorm_backward: gradients through group_norm of these arguments, given grad_y and the
    mean and rstd that it returned.  Returns {name: gradient} for the names in `want` whose
    argument is given (x and gate in x's dtype, weight and bias float32) and "workspace"."""
    desc, ptrs, dev = _norm(x, groups, weight, bias, gate, act, 1e-5, lens)
    args = dict(x=x, weight=weight, bias=bias, gate=gate)
    unknown = set(want) - set(args)
    if unknown:
        raise ValueError(f"no gradient named {sorted(unknown)}")
    stats = (x.shape[0], groups)
    ins = (_on(dev, grad_y, "grad_y", x.dtype, x.shape), _on(dev, mean, "mean", torch.float32, stats),
           _on(dev, rstd, "rstd", torch.float32, stats))
    out = {n: torch.empty_like(args[n]) for n in want if args[n] is not None}
    workspace = _workspace(pnr_groupnorm_workspace_bytes_backward(desc), workspace, dev, desc)
    _call(pnr_groupnorm_backward, dev, desc, *ptrs, *ins, *[_ptr(out.get(n)) for n in ("x", "weight", "bias", "gate")])
    out["workspace"] = workspace
    return out


# ---- selective scan, the causal convolution before it, 8-bit copies of activations ----------------
def _selscan(u, dt, A, B, C, D, z, dt_bias, softplus, lens, step: bool) -> tuple:
    """The descriptor of a selective-scan call, the eight inputs' pointers, the sizes, the device."""
    ty = u.dtype
    code = _SEQ_DT.get(ty)
    if code is None:
        raise TypeError(f"the selective scan takes float32 or bfloat16 (got {ty})")
    us, bs, dims = u.shape, B.shape, 2 if step else 3
    if len(us) != dims or len(bs) != dims + 1:
        raise ValueError("u, dt, z must be [B, E] and B, C [B, G, N]" if step else "u, dt, z must be [B, T, E] and B, C [B, T, G, N]")
    lead, E, (G, N), dev = us[:-1], us[-1], bs[-2:], u.get_device()
    a, b, c, d = u.stride(), dt.stride(), B.stride(), C.stride()
    zs = (0,) * dims if z is None else z.stride()
    if not (dt.dtype == B.dtype == C.dtype == ty and dev >= 0 and dt.get_device() == dev == B.get_device() == C.get_device()
            and dt.shape == us and bs[:-2] == lead and C.shape == bs and (a[-1] == b[-1] == 1 or E == 1)
            and (c[-1] == d[-1] == 1 or N == 1)
            and (z is None or z.dtype == ty and z.get_device() == dev and z.shape == us and (zs[-1] == 1 or E == 1))):
        for t, name, shape in ((u, "u", us), (dt, "dt", us), (z, "z", us), (B, "B", (*lead, G, N)), (C, "C", (*lead, G, N))):
            if t is not None:
                _rows(t, name, ty, shape, dev)
    f32 = torch.float32
    ptrs = (u.data_ptr(), dt.data_ptr(), _on(dev, A, "A", f32, (E, N)), B.data_ptr(), C.data_ptr(),
            _on(dev, D, "D", f32, (E,)), None if z is None else z.data_ptr(), _on(dev, dt_bias, "dt_bias", f32, (E,)))
    if step:
        T, strides = 1, (a[0], 0, b[0], 0, zs[0], 0, c[0], 0, c[1], d[0], 0, d[1])
    else:
        T, strides = us[1], (a[0], a[1], b[0], b[1], zs[0], zs[1], *c[:3], *d[:3])
    desc = _pack(PnrSelscan, _SELSCAN, us[0], T, E, N, G, code, bool(softplus), *strides,
                 _on(dev, lens, "lens", torch.int32, lead[:1]) or 0, _raw_stream(dev), 0, 0)
    return desc, ptrs, (us[0], E, N), dev


def selective_scan(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, *,
                   D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                   dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                   state: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
                   y: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_selscan_forward: h_t = exp(delta_t A) h_{t-1} + delta_t u_t B_t, y_t = (C_t . h_t + D u_t)
    silu(z_t) over whole sequences, delta = softplus(dt + dt_bias), or dt + dt_bias.  u, dt, z [B,T,E] and
    B, C [B,T,G,N] (float32 or bfloat16, strided as they come, last axis contiguous; a group is E / G
    consecutive channels), A float32 [E,N], D and dt_bias float32 [E], state (before the first token,
    zeros if None) float32 [B,E,N], lens int32 [B] (tokens of each row, T if None).  Returns
    dict(y=[B,T,E], state=the state after each row's last token, workspace)."""
    desc, ptrs, (nb, E, N), dev = _selscan(u, dt, A, B, C, D, z, dt_bias, softplus, lens, False)
    if y is None:
        y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
    shape = (nb, E, N)
    if state_out is None:
        state_out = torch.empty(shape, dtype=torch.float32, device=u.device)
    args = (_on(dev, state, "state", torch.float32, shape), _on(dev, y, "y", u.dtype, u.shape),
            _on(dev, state_out, "state_out", torch.float32, shape))
    workspace = _workspace(pnr_selscan_workspace_bytes(desc), workspace, dev, desc)
    _call(pnr_selscan_forward, dev, desc, *ptrs, *args)
    return {"y": y, "state": state_out, "workspace": workspace}


def selective_scan_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                        state: torch.Tensor, *, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                        dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                        slots: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
                        y: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_selscan_step: one token for each of B requests.  u, dt, z [B,E], B, C [B,G,N]; state float32
    [n_slots,E,N], the pool of running requests' states, of which request b has slot slots[b] (int32
    [B]; slot b if None; a slot outside the pool marks an idle row).  The pool is updated in place
    unless state_out gives another one of its shape.  Returns dict(y=[B,E], state=the updated pool)."""
    desc, ptrs, (nb, E, N), dev = _selscan(u, dt, A, B, C, D, z, dt_bias, softplus, None, True)
    if state_out is None:
        state_out = state
    if y is None:
        y = torch.empty(u.shape, dtype=u.dtype, device=u.device)
    n_slots = state.shape[0] if state.dim() else 0
    shape = (n_slots, E, N)
    _call(pnr_selscan_step, dev, desc, *ptrs, _on(dev, state, "state", torch.float32, shape),
          _on(dev, slots, "slots", torch.int32, (nb,)), n_slots, _on(dev, y, "y", u.dtype, u.shape),
          _on(dev, state_out, "state_out", torch.float32, shape))
    return {"y": y, "state": state_out}


def selective_scan_backward(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                            grad_y: torch.Tensor, *, D: Optional[torch.Tensor] = None,
                            z: Optional[torch.Tensor] = None, dt_bias: Optional[torch.Tensor] = None,
                            softplus: bool = True, state: Optional[torch.Tensor] = None,
                            lens: Optional[torch.Tensor] = None, grad_state: Optional[torch.Tensor] = None,
                            want=("u", "dt", "A", "B", "C", "D", "z", "dt_bias", "state"),
                            workspace: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_selscan_backward: gradients through selective_scan of these arguments, given grad_y = dL/dy
    [B,T,E] and grad_state = dL/d(returned state) (zeros if None).  Returns {name: gradient} for the
    names in `want` whose argument is given (u, dt, B, C, z in their dtype, the others float32) and
    "workspace"."""
    desc, ptrs, (nb, E, N), dev = _selscan(u, dt, A, B, C, D, z, dt_bias, softplus, lens, False)
    shape = (nb, E, N)
    args = (_on(dev, state, "state", torch.float32, shape), _on(dev, grad_y, "grad_y", u.dtype, u.shape),
            _on(dev, grad_state, "grad_state", torch.float32, shape))
    given = dict(u=u, dt=dt, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias, state=state)
    unknown = set(want) - set(given)
    if unknown:
        raise ValueError(f"no gradient named {sorted(unknown)}")
    out = {n: torch.empty(given[n].shape, dtype=given[n].dtype, device=u.device) for n in want if given[n] is not None}
    workspace = _workspace(pnr_selscan_workspace_bytes_backward(desc), workspace, dev, desc)
    _call(pnr_selscan_backward, dev, desc, *ptrs, *args, *[_ptr(out.get(n)) for n in given])
    out["workspace"] = workspace
    return out


class _Copy(NamedTuple):
    codes: torch.Tensor          # int8 [..., E]
    exponents: torch.Tensor      # uint8 [..., ceil(E / 32)]


class Packed(_Copy):
    """An activation in 8 bits, (codes, exponents): value = codes * 2^(exponents - 127), 32 channels an exponent.
    dtype is the type it was made of, None where nobody said."""
    dtype: Optional[torch.dtype] = None

    def __new__(cls, codes: torch.Tensor, exponents: torch.Tensor, dtype: Optional[torch.dtype] = None):
        self = super().__new__(cls, codes, exponents)
        self.dtype = dtype
        return self


def _packed(p: Packed) -> tuple:
    """Shape, device and pointers of a packed activation."""
    shape, dev = p.codes.shape, p.codes.get_device()
    if len(shape) not in (2, 3):
        raise ValueError(f"codes must be [rows, E] or [B, T, E] (got {tuple(shape)})")
    if dev < 0:
        raise ValueError("libpnr takes device tensors")
    return shape, dev, _on(dev, p.codes, "codes", torch.int8, shape), \
        _on(dev, p.exponents, "exponents", torch.uint8, (*shape[:-1], (shape[-1] + 31) // 32))


def checkpoint_pack(x: torch.Tensor) -> Packed:
    """Run pnr_checkpoint_pack: x [rows, E] or [B, T, E] (float32 or bfloat16, strided as it comes, last axis
    contiguous) in 8 bits and an exponent for every 32 channels.  causal_conv and
    causal_conv_backward read the result in place of x; checkpoint_unpack gives the values."""
    code, dims, dev = _SEQ_DT.get(x.dtype), x.dim(), x.get_device()
    if code is None:
        raise TypeError(f"checkpoints are made of float32 or bfloat16 (got {x.dtype})")
    if dims not in (2, 3):
        raise ValueError(f"x must be [rows, E] or [B, T, E] (got {tuple(x.shape)})")
    _rows(x, "x", x.dtype, x.shape, dev)
    E, s = x.shape[-1], x.stride()
    codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    exps = torch.empty(*x.shape[:-1], (E + 31) // 32, dtype=torch.uint8, device=x.device)
    desc = _pack(PnrCheckpoint, _CHECKPOINT, *(x.shape if dims == 3 else (1, *x.shape)), code, s[0] if dims == 3 else 0, s[-2],
                 _raw_stream(dev))
    _call(pnr_checkpoint_pack, dev, desc, x.data_ptr(), codes.data_ptr(), exps.data_ptr())
    return Packed(codes, exps, x.dtype)


def checkpoint_unpack(packed: Packed, dtype: torch.dtype) -> torch.Tensor:
    """Run pnr_checkpoint_unpack: the values of a packed activation (exact in both types)."""
    code = _SEQ_DT.get(dtype)
    if code is None:
        raise TypeError(f"checkpoints are read as float32 or bfloat16 (got {dtype})")
    shape, dev, codes, exps = _packed(packed)
    x = torch.empty(shape, dtype=dtype, device=packed.codes.device)
    desc = _pack(PnrCheckpoint, _CHECKPOINT, *(shape if len(shape) == 3 else (1, *shape)), code, 0, 0, _raw_stream(dev))
    _call(pnr_checkpoint_unpack, dev, desc, codes, exps, x.data_ptr())
    return x


def _conv(x, weight, bias, act, lens, dtype, step: bool) -> tuple:
    """The descriptor of a convolution, the pointers of x, its exponents, weight and bias, the shape of x,
    the taps, the device.  dtype: of y and the states."""
    code = _SEQ_DT.get(dtype)
    if code is None:
        raise TypeError(f"the convolution takes float32 or bfloat16 (got {dtype})")
    if isinstance(x, Packed):
        shape, dev, ptr, exps = _packed(x)
        stride = (0, 0, 1)
    else:
        shape, dev, exps, stride = x.shape, x.get_device(), None, x.stride()
        if not (x.dtype == dtype and dev >= 0 and (stride[-1] == 1 or shape[-1] == 1)):
            _rows(x, "x", dtype, shape, dev)
        ptr = x.data_ptr()
    if len(shape) != (2 if step else 3):
        raise ValueError("x must be " + ("[B, E]" if step else "[B, T, E]"))
    if weight.dim() != 2:
        raise ValueError(f"weight must be [E, W] (got {tuple(weight.shape)})")
    E, W = shape[-1], weight.shape[1]
    ptrs = (ptr, exps, _on(dev, weight, "weight", torch.float32, (E, W)), _on(dev, bias, "bias", torch.float32, (E,)))
    desc = _pack(PnrConv, _CONV, shape[0], 1 if step else shape[1], E, W, code, act, stride[0], 0 if step else stride[1],
                 _on(dev, lens, "lens", torch.int32, shape[:1]) or 0, _raw_stream(dev), 0, 0)
    return desc, ptrs, shape, W, dev


def causal_conv(x: Union[torch.Tensor, Packed], weight: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
                act: int = ACT_SILU, state: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
                dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                state_out: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_conv_forward: y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j}), each channel by itself.
    x [B,T,E] (float32 or bfloat16, strided as it comes, last axis contiguous) or a Packed copy of
    it, weight float32 [E,W], bias float32 [E], state [B,W-1,E] in y's dtype (the inputs before the
    first, zeros if None), lens int32 [B]; dtype is y's, for a packed x (None: what it was made of).  Returns
    dict(y=[B,T,E], state=the last W - 1 inputs of each row)."""
    if dtype is None:
        dtype = x.dtype
        if dtype is None:
            raise ValueError("causal_conv of a packed x whose type is not known needs a dtype")
    desc, ptrs, shape, W, dev = _conv(x, weight, bias, act, lens, dtype, False)
    where, last = weight.device, (shape[0], W - 1, shape[2])
    if y is None:
        y = torch.empty(shape, dtype=dtype, device=where)
    if state_out is None:
        state_out = torch.empty(last, dtype=dtype, device=where)
    _call(pnr_conv_forward, dev, desc, *ptrs, _on(dev, state, "state", dtype, last),
          _on(dev, y, "y", dtype, shape), _on(dev, state_out, "state_out", dtype, last))
    return {"y": y, "state": state_out}


def causal_conv_step(x: torch.Tensor, weight: torch.Tensor, state: torch.Tensor, *, bias: Optional[torch.Tensor] = None,
                     act: int = ACT_SILU, slots: Optional[torch.Tensor] = None,
                     state_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_conv_step: one token for each of B requests.  x [B,E]; state [n_slots,W-1,E] in its dtype, the
    pool of running requests' last inputs, with slots and state_out as in selective_scan_step.
    Returns dict(y=[B,E], state=the updated pool)."""
    if isinstance(x, Packed):
        raise TypeError("a single token's x is a tensor")
    desc, (px, _, pw, pb), shape, W, dev = _conv(x, weight, bias, act, None, x.dtype, True)
    if state_out is None:
        state_out = state
    if y is None:
        y = torch.empty(shape, dtype=x.dtype, device=x.device)
    n_slots = state.shape[0] if state.dim() else 0
    pool = (n_slots, W - 1, shape[1])
    _call(pnr_conv_step, dev, desc, px, pw, pb, _on(dev, state, "state", x.dtype, pool),
          _on(dev, slots, "slots", torch.int32, shape[:1]), n_slots, _on(dev, y, "y", x.dtype, shape),
          _on(dev, state_out, "state_out", x.dtype, pool))
    return {"y": y, "state": state_out}


def causal_conv_backward(x: Union[torch.Tensor, Packed], weight: torch.Tensor, grad_y: torch.Tensor, *,
                         bias: Optional[torch.Tensor] = None, act: int = ACT_SILU,
                         state: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
                         grad_state: Optional[torch.Tensor] = None, want=("x", "weight", "bias", "state"),
                         workspace: Optional[torch.Tensor] = None) -> dict:
    """Run pnr_conv_backward: gradients through causal_conv of these arguments, given grad_y = dL/dy [B,T,E]
    (whose dtype the states have) and grad_state = dL/d(returned state) (zeros if None).  Returns
    {name: gradient} for the names in `want` whose argument is given (x and state in grad_y's
    dtype, weight and bias float32) and "workspace"."""
    desc, ptrs, shape, W, dev = _conv(x, weight, bias, act, lens, grad_y.dtype, False)
    dt, last = grad_y.dtype, (shape[0], W - 1, shape[2])
    args = (_on(dev, state, "state", dt, last), _on(dev, grad_y, "grad_y", dt, shape),
            _on(dev, grad_state, "grad_state", dt, last))
    like = dict(x=(shape, dt), weight=(weight.shape, torch.float32),
                bias=None if bias is None else (bias.shape, torch.float32), state=None if state is None else (last, dt))
    unknown = set(want) - set(like)
    if unknown:
        raise ValueError(f"no gradient named {sorted(unknown)}")
    out = {n: torch.empty(like[n][0], dtype=like[n][1], device=grad_y.device) for n in want if like[n]}
    workspace = _workspace(pnr_conv_workspace_bytes_backward(desc), workspace, dev, desc)
    _call(pnr_conv_backward, dev, desc, *ptrs, *args, *[_ptr(out.get(n)) for n in like])
    out["workspace"] = workspace
    return out
