"""Thin ctypes binding of ``libfs_sinkhorn.so`` (the C ABI in include/fs_sinkhorn.h,
include/fs_attention.h and include/fs_probe.h).

Argument marshalling only: torch tensors provide device memory and the current
HIP stream; every step of the solver runs in the library's kernels.  If the
library has not been built the calls raise; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "FS_OK", "FS_ERR_INVALID_ARG", "FS_ERR_WORKSPACE", "FS_ERR_DEVICE", "FS_ERR_NONFINITE",
    "FS_ERR_NOT_CONVERGED", "PREC_AUTO", "PREC_FP32", "PREC_BF16", "PREC_FP16", "PREC_FP32_VALU",
    "PREC_BF16_REFINE",
    "FsError",
    "Problem", "load", "lib_path", "fs_workspace_bytes", "fs_potentials_init",
    "fs_lse_update_f", "fs_lse_update_g", "fs_marginal_residual", "fs_sinkhorn_solve",
    "fs_apply_transport", "fs_problem_info", "fs_status_string", "fs_last_error", "solve",
    "PROBE_KINDS", "fs_probe_peak", "fs_apply_transport_t", "fs_gradient", "fs_dual_value",
    "fs_hvp", "fs_hvp_workspace_bytes",
    "COST_SQEUCLIDEAN", "COST_COSINE",
    "fs_morton_workspace_bytes", "fs_morton_sort", "fs_unpermute", "fs_bs_workspace_bytes",
    "fs_bs_attach", "fs_bs_lse_update_f", "fs_bs_lse_update_g", "fs_bs_sinkhorn_solve",
    "fs_bs_shape", "fs_bs_read_screen", "fs_centroids", "fs_lift",
    "fs_sampled_marginal_error", "fs_bs_coarse_start", "fs_bs_apply_transport",
    "fs_bs_apply_transport_t", "fs_bs_gradient", "fs_static_scratch_bytes",
    "fs_sinkhorn_solve_static",
    "fs_bucket_edges", "fs_attention_workspace_bytes", "fs_attention_forward",
    "fs_attention_backward", "fs_qk_norm_workspace_bytes", "fs_qk_norm_rotate",
    "fs_qk_norm_rotate_backward",
]

FS_OK, FS_ERR_INVALID_ARG, FS_ERR_WORKSPACE, FS_ERR_DEVICE, FS_ERR_NONFINITE, \
    FS_ERR_NOT_CONVERGED = range(6)
PREC_AUTO, PREC_FP32, PREC_BF16, PREC_FP16, PREC_FP32_VALU, PREC_BF16_REFINE = range(6)
_PREC_NAMES = {"auto": PREC_AUTO, "fp32": PREC_FP32, "bf16": PREC_BF16, "fp16": PREC_FP16,
               "fp32-valu": PREC_FP32_VALU, "bf16-refine": PREC_BF16_REFINE}
COST_SQEUCLIDEAN, COST_COSINE = 0, 1
_COST_NAMES = {"sqeuclidean": COST_SQEUCLIDEAN, "cosine": COST_COSINE}
PROBE_KINDS = {"mfma-bf16": 1, "mfma-fp16": 2, "mfma-fp32": 3, "exp": 4}
PATH_NAMES = {0: "fp32-valu", 1: "fp32-mfma", 2: "bf16-mfma", 3: "fp16-mfma", 4: "fp32-small-mfma",
              5: "bf16-mfma-fp16-refine"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


def lib_path() -> str:
    return os.environ.get("FS_SINKHORN_LIB") or os.path.join(_HERE, "libfs_sinkhorn.so")


class SolveOpts(ctypes.Structure):
    _fields_ = [("n_stages", ctypes.c_int32), ("eps_start", ctypes.c_float),
                ("eps_end", ctypes.c_float), ("iters_per_stage", ctypes.c_int32),
                ("tol", ctypes.c_float), ("check_every", ctypes.c_int32),
                ("warm_start", ctypes.c_int32), ("time_kernels", ctypes.c_int32),
                ("single_launch", ctypes.c_int32), ("refine_iters", ctypes.c_int32)]


class SolveInfo(ctypes.Structure):
    _fields_ = [("iters_done", ctypes.c_int32), ("final_eps", ctypes.c_float),
                ("residual", ctypes.c_float), ("lse_launches", ctypes.c_int32),
                ("lse_ms", ctypes.c_float), ("single_launch", ctypes.c_int32)]


class HvpInfo(ctypes.Structure):
    _fields_ = [("cg_iters", ctypes.c_int32), ("cg_residual", ctypes.c_float)]


class CoarseInfo(ctypes.Structure):
    _fields_ = [("rounds", ctypes.c_int32), ("accepted", ctypes.c_int32),
                ("err_rows", ctypes.c_float), ("err_cols", ctypes.c_float)]


class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride_batch", ctypes.c_int64),
                ("stride_row", ctypes.c_int64), ("stride_head", ctypes.c_int64)]


class AttentionDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("n", ctypes.c_int32),
                ("m", ctypes.c_int32), ("heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dv", ctypes.c_int32), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int32), ("offset", ctypes.c_int32),
                ("offsets", ctypes.c_void_p), ("q_len", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("key_mask", ctypes.c_void_p),
                ("key_mask_stride", ctypes.c_int64), ("bias", ctypes.c_void_p),
                ("edges", ctypes.POINTER(ctypes.c_int32)), ("n_edges", ctypes.c_int32),
                ("two_sided", ctypes.c_int32)]


class QkNormDesc(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("batch", ctypes.c_int32), ("n", ctypes.c_int32),
                ("heads_q", ctypes.c_int32), ("heads_k", ctypes.c_int32), ("d", ctypes.c_int32),
                ("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("eps", ctypes.c_float), ("cos_table", ctypes.c_void_p),
                ("sin_table", ctypes.c_void_p), ("n_pos", ctypes.c_int32),
                ("positions", ctypes.c_void_p), ("positions_stride", ctypes.c_int64),
                ("offset", ctypes.c_int32)]


class FsError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: {_status_name(status)}: {message}")


def _status_name(s: int) -> str:
    lib = _LIB
    if lib is None:
        return str(s)
    return lib.fs_status_string(s).decode()


_vp = ctypes.c_void_p
_fp = ctypes.c_void_p  # device float* passed as an address


def load():
    """Load the HIP library (raises if it is missing)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"HIP library {path} is not built; run __graft_entry__.build() "
                           "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    i64, i32, f32, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    lib.fs_workspace_bytes.restype = sz
    lib.fs_workspace_bytes.argtypes = [i64, i64, i32, i32, ctypes.c_int]
    lib.fs_potentials_init.restype = ctypes.c_int
    lib.fs_potentials_init.argtypes = [_fp, _fp, _fp, _fp, i64, i64, i32, i32, ctypes.c_int,
                                       _vp, sz, _fp, _fp, _vp, ctypes.POINTER(_vp)]
    lib.fs_lse_update_f.restype = ctypes.c_int
    lib.fs_lse_update_f.argtypes = [_vp, f32, _fp, _fp, _fp, _fp, _vp]
    lib.fs_lse_update_g.restype = ctypes.c_int
    lib.fs_lse_update_g.argtypes = [_vp, f32, _fp, _fp, _fp, _fp, _vp]
    lib.fs_marginal_residual.restype = ctypes.c_int
    lib.fs_marginal_residual.argtypes = [_vp, f32, _fp, _fp, _fp, _vp]
    lib.fs_sinkhorn_solve.restype = ctypes.c_int
    lib.fs_sinkhorn_solve.argtypes = [_vp, ctypes.POINTER(SolveOpts), _fp, _fp,
                                      ctypes.POINTER(SolveInfo), _vp]
    lib.fs_apply_transport.restype = ctypes.c_int
    lib.fs_apply_transport.argtypes = [_vp, f32, _fp, _fp, _fp, i32, _fp, i32, _vp]
    lib.fs_destroy.restype = None
    lib.fs_destroy.argtypes = [_vp]
    lib.fs_status_string.restype = ctypes.c_char_p
    lib.fs_status_string.argtypes = [ctypes.c_int]
    lib.fs_last_error.restype = ctypes.c_char_p
    lib.fs_last_error.argtypes = []
    lib.fs_problem_info.restype = ctypes.c_int
    lib.fs_problem_info.argtypes = [_vp] + [ctypes.POINTER(i32)] * 4
    lib.fs_potentials_init_cost.restype = ctypes.c_int
    lib.fs_potentials_init_cost.argtypes = [_fp, _fp, _fp, _fp, i64, i64, i32, i32,
                                            ctypes.c_int, ctypes.c_int, ctypes.c_void_p, sz,
                                            _fp, _fp, _vp, ctypes.POINTER(_vp)]
    lib.fs_apply_transport_t.restype = ctypes.c_int
    lib.fs_apply_transport_t.argtypes = [_vp, f32, _fp, _fp, _fp, i32, _fp, i32, _vp]
    lib.fs_gradient.restype = ctypes.c_int
    lib.fs_gradient.argtypes = [_vp, f32, _fp, _fp, _fp, _fp, _fp, _fp, _vp]
    lib.fs_dual_value.restype = ctypes.c_int
    lib.fs_dual_value.argtypes = [_vp, _fp, _fp, ctypes.c_void_p, _vp]
    lib.fs_hvp_workspace_bytes.restype = ctypes.c_size_t
    lib.fs_hvp_workspace_bytes.argtypes = [_vp]
    lib.fs_hvp.restype = ctypes.c_int
    lib.fs_hvp.argtypes = [_vp, f32, _fp, _fp, _fp, _fp, i32, _fp, _fp, f32, i32,
                           ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(HvpInfo), _vp]
    lib.fs_probe_peak.restype = ctypes.c_int
    lib.fs_probe_peak.argtypes = [ctypes.c_int, _fp, i32, _vp, ctypes.POINTER(ctypes.c_double)]
    lib.fs_morton_workspace_bytes.restype = sz
    lib.fs_morton_workspace_bytes.argtypes = [i64, i32]
    lib.fs_morton_sort.restype = ctypes.c_int
    lib.fs_morton_sort.argtypes = [_fp, _fp, i64, i32, _fp, _fp, _fp, _vp, sz, _vp]
    lib.fs_unpermute.restype = ctypes.c_int
    lib.fs_unpermute.argtypes = [_fp, _fp, i64, i32, _fp, _vp]
    lib.fs_bs_workspace_bytes.restype = sz
    lib.fs_bs_workspace_bytes.argtypes = [_vp]
    lib.fs_bs_attach.restype = ctypes.c_int
    lib.fs_bs_attach.argtypes = [_vp, _vp, sz, _vp]
    for name in ("fs_bs_lse_update_f", "fs_bs_lse_update_g"):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = [_vp, f32, f32, _fp, _fp, _fp, _fp, _vp]
    lib.fs_bs_sinkhorn_solve.restype = ctypes.c_int
    lib.fs_bs_sinkhorn_solve.argtypes = [_vp, ctypes.POINTER(SolveOpts), f32, _fp, _fp,
                                         ctypes.POINTER(SolveInfo), _vp]
    lib.fs_bs_shape.restype = ctypes.c_int
    lib.fs_bs_shape.argtypes = [_vp, i32] + [ctypes.POINTER(i32)] * 3
    lib.fs_bs_read_screen.restype = ctypes.c_int
    lib.fs_bs_read_screen.argtypes = [_vp, i32, _vp, _vp, _vp]
    lib.fs_bs_apply_transport.restype = ctypes.c_int
    lib.fs_bs_apply_transport.argtypes = [_vp, f32, f32, _fp, _fp, _fp, i32, _fp, i32, _vp]
    lib.fs_bs_apply_transport_t.restype = ctypes.c_int
    lib.fs_bs_apply_transport_t.argtypes = [_vp, f32, f32, _fp, _fp, _fp, i32, _fp, i32, _vp]
    lib.fs_bs_gradient.restype = ctypes.c_int
    lib.fs_bs_gradient.argtypes = [_vp, f32, f32, _fp, _fp, _fp, _fp, _vp]
    lib.fs_centroids.restype = ctypes.c_int
    lib.fs_centroids.argtypes = [_fp, _fp, i64, i32, i32, _fp, _fp, _vp]
    lib.fs_lift.restype = ctypes.c_int
    lib.fs_lift.argtypes = [_fp, i64, i32, _fp, _vp]
    lib.fs_sampled_workspace_bytes.restype = sz
    lib.fs_sampled_workspace_bytes.argtypes = [i32, i32]
    lib.fs_sampled_marginal_error.restype = ctypes.c_int
    lib.fs_sampled_marginal_error.argtypes = [_fp, _fp, _fp, _fp, i64, i64, i32, f32, _fp, _fp,
                                              _fp, i32, _fp, i32, _fp, _vp, sz, _vp]
    lib.fs_bs_coarse_start.restype = ctypes.c_int
    lib.fs_bs_coarse_start.argtypes = [_vp, ctypes.POINTER(SolveOpts), i32, f32, _fp, _fp, _fp,
                                       _fp,
                                       i64, i64, i32, i32, f32, i32, _fp, i32, _fp, i32, _fp,
                                       _fp, _fp, _fp, _vp, sz, ctypes.POINTER(CoarseInfo), _vp]
    lib.fs_static_scratch_bytes.restype = sz
    lib.fs_static_scratch_bytes.argtypes = []
    lib.fs_sinkhorn_solve_static.restype = ctypes.c_int
    lib.fs_sinkhorn_solve_static.argtypes = [_fp, _fp, _fp, _fp, i64, i64, i32, ctypes.c_int,
                                             ctypes.POINTER(SolveOpts), _fp, _fp,
                                             ctypes.POINTER(SolveInfo), _vp]
    i32p = ctypes.POINTER(i32)
    desc, norm = ctypes.POINTER(AttentionDesc), ctypes.POINTER(QkNormDesc)
    lib.fs_bucket_edges.restype = ctypes.c_int
    lib.fs_bucket_edges.argtypes = [i32, i32, i32p]
    lib.fs_attention_workspace_bytes.restype = sz
    lib.fs_attention_workspace_bytes.argtypes = [desc, i32]
    lib.fs_attention_forward.restype = ctypes.c_int
    lib.fs_attention_forward.argtypes = [desc] + [Rows] * 4 + [_fp, _vp, sz, _vp]
    lib.fs_attention_backward.restype = ctypes.c_int
    lib.fs_attention_backward.argtypes = [desc] + [Rows] * 4 + [_fp, Rows, _fp] + [Rows] * 3 + \
        [_fp, _vp, sz, _vp]
    lib.fs_qk_norm_workspace_bytes.restype = sz
    lib.fs_qk_norm_workspace_bytes.argtypes = [norm]
    lib.fs_qk_norm_rotate.restype = ctypes.c_int
    lib.fs_qk_norm_rotate.argtypes = [norm, Rows, Rows, _fp, _fp, Rows, Rows, _vp]
    lib.fs_qk_norm_rotate_backward.restype = ctypes.c_int
    lib.fs_qk_norm_rotate_backward.argtypes = [norm, Rows, Rows, _fp, _fp] + [Rows] * 4 + \
        [_fp, _fp, _vp, sz, _vp]
    _LIB = lib
    return lib


def fs_status_string(s: int) -> str:
    return load().fs_status_string(int(s)).decode()


def fs_last_error() -> str:
    return load().fs_last_error().decode()


def _check(status: int, where: str, allow=()):
    if status != FS_OK and status not in allow:
        raise FsError(status, where, fs_last_error())
    return status


def _prec(prec) -> int:
    if isinstance(prec, str):
        return _PREC_NAMES[prec.lower()]
    return int(prec)


def _dev(t: Optional[torch.Tensor], name: str, numel: Optional[int] = None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype != torch.float32 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements (has {t.numel()})")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """torch.empty for a call on `stream`.  The memory comes from that stream's
    pool: a block of the current stream's may still be in use there when it is
    handed out, and only work of the current stream waits for that."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


class Problem:
    """A problem handle plus the workspace tensor it lives in."""

    def __init__(self, handle, workspace: torch.Tensor, n: int, m: int, d: int, dv_max: int):
        self.handle = handle
        self.workspace = workspace
        self.n, self.m, self.d, self.dv_max = n, m, d, dv_max

    def __del__(self):
        if getattr(self, "handle", None) and _LIB is not None:
            _LIB.fs_destroy(self.handle)
            self.handle = None

    @property
    def info(self) -> dict:
        return fs_problem_info(self)


def fs_workspace_bytes(n: int, m: int, d: int, dv_max: int = 0, prec="auto") -> int:
    return int(load().fs_workspace_bytes(n, m, d, dv_max, _prec(prec)))


def fs_potentials_init(X: torch.Tensor, Y: torch.Tensor, a: torch.Tensor, b: torch.Tensor, *,
                       dv_max: int = 0, prec="auto", f: Optional[torch.Tensor] = None,
                       g: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None, cost: str = "sqeuclidean") -> Problem:
    """fs_potentials_init, or fs_potentials_init_cost for cost="cosine"."""
    lib = load()
    n, d = X.shape
    m = Y.shape[0]
    if Y.shape[1] != d:
        raise ValueError("X and Y must have the same number of columns")
    need = lib.fs_workspace_bytes(n, m, d, dv_max, _prec(prec))
    if need == 0:
        _check(FS_ERR_INVALID_ARG, "fs_workspace_bytes")
    if workspace is None:
        workspace = _empty(need + 256, torch.uint8, X.device, stream)
    base = workspace.data_ptr()
    aligned = (base + 255) // 256 * 256
    avail = workspace.numel() - (aligned - base)
    h = _vp()
    if cost not in _COST_NAMES:
        raise ValueError(f"cost must be one of {sorted(_COST_NAMES)}")
    if _COST_NAMES[cost] == COST_SQEUCLIDEAN:
        st = lib.fs_potentials_init(_dev(X, "X", n * d), _dev(Y, "Y", m * d), _dev(a, "a", n),
                                    _dev(b, "b", m), n, m, d, dv_max, _prec(prec), aligned,
                                    avail, _dev(f, "f", n), _dev(g, "g", m), _stream(stream),
                                    ctypes.byref(h))
    else:
        st = lib.fs_potentials_init_cost(_dev(X, "X", n * d), _dev(Y, "Y", m * d),
                                         _dev(a, "a", n), _dev(b, "b", m), n, m, d, dv_max,
                                         _prec(prec), _COST_NAMES[cost], aligned, avail,
                                         _dev(f, "f", n), _dev(g, "g", m), _stream(stream),
                                         ctypes.byref(h))
    _check(st, "fs_potentials_init")
    return Problem(h, workspace, n, m, d, dv_max)


def fs_lse_update_f(p: Problem, eps: float, g, f_out, f_cur=None, row_resid=None, stream=None):
    return _check(load().fs_lse_update_f(p.handle, float(eps), _dev(g, "g", p.m),
                                         _dev(f_out, "f_out", p.n), _dev(f_cur, "f_cur", p.n),
                                         _dev(row_resid, "row_resid", 1), _stream(stream)),
                  "fs_lse_update_f")


def fs_lse_update_g(p: Problem, eps: float, f, g_out, g_cur=None, col_resid=None, stream=None):
    return _check(load().fs_lse_update_g(p.handle, float(eps), _dev(f, "f", p.n),
                                         _dev(g_out, "g_out", p.m), _dev(g_cur, "g_cur", p.m),
                                         _dev(col_resid, "col_resid", 1), _stream(stream)),
                  "fs_lse_update_g")


def fs_marginal_residual(p: Problem, eps: float, f, g, out2, stream=None):
    return _check(load().fs_marginal_residual(p.handle, float(eps), _dev(f, "f", p.n),
                                              _dev(g, "g", p.m), _dev(out2, "out2", 2),
                                              _stream(stream)), "fs_marginal_residual")


def fs_sinkhorn_solve(p: Problem, f, g, *, eps_end: float, iters_per_stage: int,
                      n_stages: int = 1, eps_start: Optional[float] = None, tol: float = 0.0,
                      check_every: int = 10, warm_start: bool = False, stream=None,
                      raise_not_converged: bool = True, time_kernels: bool = False,
                      single_launch: int = 0, refine_iters: int = 0) -> dict:
    opts = SolveOpts(int(n_stages), float(eps_start if eps_start is not None else eps_end),
                     float(eps_end), int(iters_per_stage), float(tol), int(check_every),
                     int(bool(warm_start)), int(bool(time_kernels)), int(single_launch),
                     int(refine_iters))
    info = SolveInfo()
    st = load().fs_sinkhorn_solve(p.handle, ctypes.byref(opts), _dev(f, "f", p.n),
                                  _dev(g, "g", p.m), ctypes.byref(info), _stream(stream))
    allow = () if raise_not_converged else (FS_ERR_NOT_CONVERGED,)
    _check(st, "fs_sinkhorn_solve", allow)
    return {"status": st, "iters_done": info.iters_done, "final_eps": info.final_eps,
            "residual": info.residual, "lse_launches": info.lse_launches,
            "lse_ms": info.lse_ms, "single_launch": bool(info.single_launch)}


def fs_apply_transport(p: Problem, eps: float, f, g, V, U, divide_by_a: bool = False,
                       stream=None):
    dv = V.shape[1]
    return _check(load().fs_apply_transport(p.handle, float(eps), _dev(f, "f", p.n),
                                            _dev(g, "g", p.m), _dev(V, "V", p.m * dv), dv,
                                            _dev(U, "U", p.n * dv), int(bool(divide_by_a)),
                                            _stream(stream)), "fs_apply_transport")


def fs_apply_transport_t(p: Problem, eps: float, f, g, W, U, divide_by_b: bool = False,
                         stream=None):
    dv = W.shape[1]
    return _check(load().fs_apply_transport_t(p.handle, float(eps), _dev(f, "f", p.n),
                                              _dev(g, "g", p.m), _dev(W, "W", p.n * dv), dv,
                                              _dev(U, "U", p.m * dv), int(bool(divide_by_b)),
                                              _stream(stream)), "fs_apply_transport_t")


def fs_gradient(p: Problem, eps: float, f, g, X, Y, grad_x=None, grad_y=None, stream=None):
    return _check(load().fs_gradient(p.handle, float(eps), _dev(f, "f", p.n), _dev(g, "g", p.m),
                                     _dev(X, "X", p.n * p.d), _dev(Y, "Y", p.m * p.d),
                                     _dev(grad_x, "grad_x", p.n * p.d),
                                     _dev(grad_y, "grad_y", p.m * p.d), _stream(stream)),
                  "fs_gradient")


def fs_hvp_workspace_bytes(p: Problem) -> int:
    return int(load().fs_hvp_workspace_bytes(p.handle))


def fs_hvp(p: Problem, eps: float, f, g, X, Y, V, HV, cg_tol: float = 1e-4,
           cg_max_iter: int = 200, workspace=None, stream=None, wrt: str = "x") -> dict:
    """Hessian-vector product of the OT loss with respect to X (wrt="x") or
    Y (wrt="y") into HV; returns the CG iterations and final relative
    residual.  `workspace`: a device tensor of at least
    fs_hvp_workspace_bytes(p) bytes (allocated here if None)."""
    if wrt not in ("x", "y"):
        raise ValueError("wrt must be 'x' or 'y'")
    rows = p.n if wrt == "x" else p.m
    need = fs_hvp_workspace_bytes(p)
    if workspace is None:
        workspace = _empty(max(need, 1), torch.uint8, V.device, stream)
    if not workspace.is_cuda:
        raise TypeError("workspace must be a device tensor")
    info = HvpInfo()
    _check(load().fs_hvp(p.handle, float(eps), _dev(f, "f", p.n), _dev(g, "g", p.m),
                         _dev(X, "X", p.n * p.d), _dev(Y, "Y", p.m * p.d),
                         0 if wrt == "x" else 1, _dev(V, "V", rows * p.d),
                         _dev(HV, "HV", rows * p.d), float(cg_tol),
                         int(cg_max_iter), workspace.data_ptr(),
                         workspace.numel() * workspace.element_size(), ctypes.byref(info),
                         _stream(stream)), "fs_hvp")
    return {"cg_iters": info.cg_iters, "cg_residual": info.cg_residual}


def fs_dual_value(p: Problem, f, g, out=None, stream=None) -> torch.Tensor:
    """<a,f> + <b,g> into a one-element float64 device tensor (returned)."""
    if out is None:
        out = _empty(1, torch.float64, f.device, stream)
    if out.dtype != torch.float64 or not out.is_cuda or out.numel() < 1:
        raise TypeError("out must be a float64 device tensor")
    _check(load().fs_dual_value(p.handle, _dev(f, "f", p.n), _dev(g, "g", p.m), out.data_ptr(),
                                _stream(stream)), "fs_dual_value")
    return out


def fs_problem_info(p: Problem) -> dict:
    vals = [ctypes.c_int32() for _ in range(4)]
    _check(load().fs_problem_info(p.handle, *[ctypes.byref(v) for v in vals]), "fs_problem_info")
    path, dp, fs_, gs = (v.value for v in vals)
    return {"path": PATH_NAMES.get(path, str(path)), "d_pad": dp, "f_splits": fs_,
            "g_splits": gs}


def fs_probe_peak(kind: str, sink, reps: int = 9, stream=None) -> float:
    """Median rate of the unit probe `kind` (a key of PROBE_KINDS): flop/s for
    the matrix-core probes, exponentials/s for "exp".  `sink` is a device
    float tensor of >= 1 element."""
    rate = ctypes.c_double()
    if sink.numel() < 1:
        raise ValueError("sink must have at least one element")
    _check(load().fs_probe_peak(PROBE_KINDS[kind], _dev(sink, "sink"), int(reps),
                                _stream(stream), ctypes.byref(rate)), "fs_probe_peak")
    return rate.value


def _idev(t, name: str, numel: int):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.dtype != torch.int32 or not t.is_contiguous() or t.numel() != numel:
        raise TypeError(f"{name} must be a contiguous int32 tensor of {numel} elements")
    return t.data_ptr()


def fs_morton_workspace_bytes(n: int, d: int) -> int:
    return int(load().fs_morton_workspace_bytes(n, d))


def fs_morton_sort(X, w=None, X_sorted=None, w_sorted=None, perm=None, workspace=None,
                   stream=None):
    """Morton order of the points X (n x d); returns (X_sorted, w_sorted, perm)
    with X_sorted[i] = X[perm[i]] (w_sorted None when w is None)."""
    n, d = X.shape
    dev = X.device
    if X_sorted is None:
        X_sorted = _empty(X.shape, X.dtype, dev, stream)
    if w is not None and w_sorted is None:
        w_sorted = _empty(w.shape, w.dtype, dev, stream)
    if perm is None:
        perm = _empty(n, torch.int32, dev, stream)
    need = fs_morton_workspace_bytes(n, d)
    if need == 0:
        _check(FS_ERR_INVALID_ARG, "fs_morton_workspace_bytes")
    if workspace is None:
        workspace = _empty(need, torch.uint8, dev, stream)
    _check(load().fs_morton_sort(_dev(X, "X", n * d), _dev(w, "w", n), n, d,
                                 _dev(X_sorted, "X_sorted", n * d), _dev(w_sorted, "w_sorted", n),
                                 _idev(perm, "perm", n), workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "fs_morton_sort")
    return X_sorted, w_sorted, perm


def fs_unpermute(src, perm, dst=None, stream=None):
    """dst[perm[i]] = src[i] (rows of src.numel() // n floats)."""
    n = perm.numel()
    width = src.numel() // n
    if dst is None:
        dst = _empty(src.shape, src.dtype, src.device, stream)
    _check(load().fs_unpermute(_dev(src, "src", n * width), _idev(perm, "perm", n), n, width,
                               _dev(dst, "dst", n * width), _stream(stream)), "fs_unpermute")
    return dst


def fs_bs_workspace_bytes(p: Problem) -> int:
    return int(load().fs_bs_workspace_bytes(p.handle))


def fs_bs_attach(p: Problem, workspace=None, stream=None):
    """Enables the block-sparse form; keeps the workspace on the handle."""
    need = fs_bs_workspace_bytes(p)
    if need == 0:
        _check(FS_ERR_INVALID_ARG, "fs_bs_workspace_bytes")
    if workspace is None:
        workspace = _empty(need, torch.uint8, p.workspace.device, stream)
    _check(load().fs_bs_attach(p.handle, workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream(stream)),
           "fs_bs_attach")
    p.bs_workspace = workspace
    return p


def fs_bs_lse_update_f(p: Problem, eps: float, delta: float, g, f_cur, f_out, row_resid=None,
                       stream=None):
    return _check(load().fs_bs_lse_update_f(p.handle, float(eps), float(delta),
                                            _dev(g, "g", p.m), _dev(f_cur, "f_cur", p.n),
                                            _dev(f_out, "f_out", p.n),
                                            _dev(row_resid, "row_resid", 1), _stream(stream)),
                  "fs_bs_lse_update_f")


def fs_bs_lse_update_g(p: Problem, eps: float, delta: float, f, g_cur, g_out, col_resid=None,
                       stream=None):
    return _check(load().fs_bs_lse_update_g(p.handle, float(eps), float(delta),
                                            _dev(f, "f", p.n), _dev(g_cur, "g_cur", p.m),
                                            _dev(g_out, "g_out", p.m),
                                            _dev(col_resid, "col_resid", 1), _stream(stream)),
                  "fs_bs_lse_update_g")


def fs_bs_sinkhorn_solve(p: Problem, f, g, *, eps_end: float, iters_per_stage: int,
                         delta: float, n_stages: int = 1, eps_start: Optional[float] = None,
                         tol: float = 0.0, check_every: int = 10, warm_start: bool = False,
                         stream=None, raise_not_converged: bool = True,
                         time_kernels: bool = False) -> dict:
    opts = SolveOpts(int(n_stages), float(eps_start if eps_start is not None else eps_end),
                     float(eps_end), int(iters_per_stage), float(tol), int(check_every),
                     int(bool(warm_start)), int(bool(time_kernels)))
    info = SolveInfo()
    st = load().fs_bs_sinkhorn_solve(p.handle, ctypes.byref(opts), float(delta),
                                     _dev(f, "f", p.n), _dev(g, "g", p.m), ctypes.byref(info),
                                     _stream(stream))
    allow = () if raise_not_converged else (FS_ERR_NOT_CONVERGED,)
    _check(st, "fs_bs_sinkhorn_solve", allow)
    return {"status": st, "iters_done": info.iters_done, "final_eps": info.final_eps,
            "residual": info.residual, "lse_launches": info.lse_launches,
            "lse_ms": info.lse_ms, "single_launch": bool(info.single_launch)}


def fs_bs_shape(p: Problem, side: int) -> dict:
    vals = [ctypes.c_int32() for _ in range(3)]
    _check(load().fs_bs_shape(p.handle, int(side), *[ctypes.byref(v) for v in vals]),
           "fs_bs_shape")
    return {"row_blocks": vals[0].value, "key_blocks": vals[1].value, "stride": vals[2].value}


def fs_bs_read_screen(p: Problem, side: int, lists: bool = False, stream=None):
    """Kept-block counts per row block of the last screening of `side` (numpy
    int32), and with lists=True the padded lists (row_blocks x stride)."""
    import numpy as np

    sh = fs_bs_shape(p, side)
    counts = np.zeros(sh["row_blocks"], np.int32)
    L = np.zeros((sh["row_blocks"], sh["stride"]), np.int32) if lists else None
    _check(load().fs_bs_read_screen(p.handle, int(side), counts.ctypes.data,
                                    L.ctypes.data if lists else None, _stream(stream)),
           "fs_bs_read_screen")
    return (counts, L) if lists else counts


def fs_bs_apply_transport(p: Problem, eps: float, delta: float, f, g, V, U,
                          divide_by_a: bool = False, stream=None):
    dv = V.shape[1]
    return _check(load().fs_bs_apply_transport(p.handle, float(eps), float(delta),
                                               _dev(f, "f", p.n), _dev(g, "g", p.m),
                                               _dev(V, "V", p.m * dv), dv,
                                               _dev(U, "U", p.n * dv), int(bool(divide_by_a)),
                                               _stream(stream)), "fs_bs_apply_transport")


def fs_bs_apply_transport_t(p: Problem, eps: float, delta: float, f, g, W, U,
                            divide_by_b: bool = False, stream=None):
    dv = W.shape[1]
    return _check(load().fs_bs_apply_transport_t(p.handle, float(eps), float(delta),
                                                 _dev(f, "f", p.n), _dev(g, "g", p.m),
                                                 _dev(W, "W", p.n * dv), dv,
                                                 _dev(U, "U", p.m * dv), int(bool(divide_by_b)),
                                                 _stream(stream)), "fs_bs_apply_transport_t")


def fs_bs_gradient(p: Problem, eps: float, delta: float, f, g, grad_x=None, grad_y=None,
                   stream=None):
    gx = _dev(grad_x, "grad_x", p.n * p.d) if grad_x is not None else None
    gy = _dev(grad_y, "grad_y", p.m * p.d) if grad_y is not None else None
    return _check(load().fs_bs_gradient(p.handle, float(eps), float(delta), _dev(f, "f", p.n),
                                        _dev(g, "g", p.m), gx, gy, _stream(stream)),
                  "fs_bs_gradient")


def fs_centroids(P, w, cell: int, C=None, W=None, stream=None):
    """Centroids and weights of runs of `cell` points; returns (C, W)."""
    n, d = P.shape
    nc = (n + cell - 1) // cell if cell >= 1 else 1  # (the library rejects cell < 1)
    C = _empty((nc, d), P.dtype, P.device, stream) if C is None else C
    W = _empty(nc, P.dtype, P.device, stream) if W is None else W
    _check(load().fs_centroids(_dev(P, "P", n * d), _dev(w, "w", n), n, d, int(cell),
                               _dev(C, "C", nc * d), _dev(W, "W", nc), _stream(stream)),
           "fs_centroids")
    return C, W


def fs_lift(F, n: int, cell: int, f=None, stream=None):
    f = _empty(n, F.dtype, F.device, stream) if f is None else f
    _check(load().fs_lift(_dev(F, "F", (n + cell - 1) // cell), n, int(cell), _dev(f, "f", n),
                          _stream(stream)), "fs_lift")
    return f


def fs_sampled_marginal_error(X, Y, a, b, f, g, eps: float, rows, cols, out2=None,
                              workspace=None, stream=None):
    """(err_rows, err_cols) as a 2-element device tensor."""
    lib = load()
    n, d = X.shape
    m = Y.shape[0]
    nr, nc = rows.numel(), cols.numel()
    out2 = _empty(2, X.dtype, X.device, stream) if out2 is None else out2
    need = lib.fs_sampled_workspace_bytes(nr, nc)
    workspace = _empty(need, torch.uint8, X.device, stream) if workspace is None \
        else workspace
    _check(lib.fs_sampled_marginal_error(
        _dev(X, "X", n * d), _dev(Y, "Y", m * d), _dev(a, "a", n), _dev(b, "b", m), n, m, d,
        float(eps), _dev(f, "f", n), _dev(g, "g", m), _idev(rows, "rows", nr), nr,
        _idev(cols, "cols", nc), nc, _dev(out2, "out2", 2), workspace.data_ptr(),
        workspace.numel(), _stream(stream)), "fs_sampled_marginal_error")
    return out2


def fs_bs_coarse_start(coarse: Problem, X, Y, a, b, cell: int, f, g, F, G, rows, cols, *,
                       eps_end: float, iters_per_stage: int, n_stages: int = 1,
                       eps_start: Optional[float] = None, more_iters: int = 10,
                       check_tol: float = 1e-2, max_rounds: int = 5, coarse_delta: float = 0.0,
                       stream=None) -> dict:
    """The coarse stage (see include/fs_sinkhorn.h); fills F, G (coarse) and
    f, g (lifted); returns rounds, accepted and the last errors.  coarse_delta
    > 0 solves the coarse problem in block-sparse form (attach it first)."""
    lib = load()
    n, d = X.shape
    m = Y.shape[0]
    nr, nc = rows.numel(), cols.numel()
    need = lib.fs_sampled_workspace_bytes(nr, nc) + 256
    ws = _empty(need, torch.uint8, X.device, stream)
    opts = SolveOpts(int(n_stages), float(eps_start if eps_start is not None else eps_end),
                     float(eps_end), int(iters_per_stage), 0.0, 1, 0, 0)
    info = CoarseInfo()
    _check(lib.fs_bs_coarse_start(
        coarse.handle, ctypes.byref(opts), int(more_iters), float(coarse_delta),
        _dev(X, "X", n * d),
        _dev(Y, "Y", m * d), _dev(a, "a", n), _dev(b, "b", m), n, m, d, int(cell),
        float(check_tol), int(max_rounds), _idev(rows, "rows", nr), nr, _idev(cols, "cols", nc),
        nc, _dev(F, "F", coarse.n), _dev(G, "G", coarse.m), _dev(f, "f", n), _dev(g, "g", m),
        ws.data_ptr(), need, ctypes.byref(info), _stream(stream)), "fs_bs_coarse_start")
    return {"rounds": info.rounds, "accepted": bool(info.accepted), "err_rows": info.err_rows,
            "err_cols": info.err_cols}


def fs_static_scratch_bytes() -> int:
    return int(load().fs_static_scratch_bytes())


def fs_sinkhorn_solve_static(X, Y, a, b, f, g, *, eps_end: float, iters_per_stage: int,
                             prec="auto", n_stages: int = 1, eps_start: Optional[float] = None,
                             tol: float = 0.0, check_every: int = 10, warm_start: bool = False,
                             stream=None, raise_not_converged: bool = True,
                             refine_iters: int = 0) -> dict:
    """fs_sinkhorn_solve_static: set-up and solve with the library's static
    device scratch as the workspace (no allocation)."""
    n, d = X.shape
    m = Y.shape[0]
    opts = SolveOpts(int(n_stages), float(eps_start if eps_start is not None else eps_end),
                     float(eps_end), int(iters_per_stage), float(tol), int(check_every),
                     int(bool(warm_start)), 0, 0, int(refine_iters))
    info = SolveInfo()
    st = load().fs_sinkhorn_solve_static(_dev(X, "X", n * d), _dev(Y, "Y", m * d),
                                         _dev(a, "a", n), _dev(b, "b", m), n, m, d, _prec(prec),
                                         ctypes.byref(opts), _dev(f, "f", n), _dev(g, "g", m),
                                         ctypes.byref(info), _stream(stream))
    allow = () if raise_not_converged else (FS_ERR_NOT_CONVERGED,)
    _check(st, "fs_sinkhorn_solve_static", allow)
    return {"status": st, "iters_done": info.iters_done, "final_eps": info.final_eps,
            "residual": info.residual}


def solve(X, Y, a, b, *, eps: float, iters: int, prec="auto", n_stages: int = 1,
          eps_start: Optional[float] = None, tol: float = 0.0, check_every: int = 10,
          dv_max: int = 0, cost: str = "sqeuclidean"):
    """Convenience: init + solve; returns (problem, f, g, info)."""
    dev = X.device
    f = torch.empty(X.shape[0], dtype=torch.float32, device=dev)
    g = torch.empty(Y.shape[0], dtype=torch.float32, device=dev)
    p = fs_potentials_init(X, Y, a, b, dv_max=dv_max, prec=prec, f=f, g=g, cost=cost)
    info = fs_sinkhorn_solve(p, f, g, eps_end=eps, iters_per_stage=iters, n_stages=n_stages,
                             eps_start=eps_start, tol=tol, check_every=check_every,
                             raise_not_converged=False)
    return p, f, g, info


# ---- attention (include/fs_attention.h) -----------------------------------

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_NO_ROWS = Rows(None, 0, 0, 0)


_MAX = 0x7fffffff


def _i32(name: str, *values: int):
    """The values are numbers of 32 bits (ctypes would cut off the rest)."""
    for x in values:
        if not -_MAX - 1 <= x <= _MAX:
            raise ValueError(f"{name} is beyond 32 bits (got {x})")


def fs_bucket_edges(side_buckets: int, max_distance: int) -> list:
    """The edges of one side's buckets: one distance each for the first half,
    then evenly spaced in the logarithm up to max_distance."""
    _i32("side_buckets or max_distance", side_buckets, max_distance)
    out = (ctypes.c_int32 * min(max(side_buckets, 1), 64))()
    _check(load().fs_bucket_edges(side_buckets, max_distance, out), "fs_bucket_edges")
    return list(out[:side_buckets - 1])


def _on(t: torch.Tensor, name: str, dev: int):
    """t is a tensor on device number dev (negative: the host)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, not on {dev} as the others")


def _rows(t: Optional[torch.Tensor], name: str, like: torch.Tensor, dev: int, shape) -> Rows:
    """A [batch, rows, heads, width] tensor of like's type as fs_rows."""
    if t is None:
        return _NO_ROWS
    _on(t, name, dev)
    if t.dtype != like.dtype:
        raise TypeError(f"{name} is {t.dtype}, not {like.dtype} as the others")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)} (is {tuple(t.shape)})")
    b, r, h, w = t.stride()
    if w != 1 and shape[3] != 1:
        raise ValueError(f"{name}'s last axis must be contiguous")
    return Rows(t.data_ptr(), b, r, h)


def _flat(t: Optional[torch.Tensor], name: str, dev: int, dtype, shape) -> Optional[int]:
    """A contiguous tensor of this type and shape, as its address."""
    if t is None:
        return None
    _on(t, name, dev)
    if t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)} (is {tuple(t.shape)})")
    return t.data_ptr()


def _work(workspace: Optional[torch.Tensor], size, like: torch.Tensor, dev: int, stream):
    """Aligned address and size of the workspace, and the tensor to keep: the
    caller's, or one of size() bytes from the memory of the call's stream."""
    if workspace is None:
        workspace = _empty(size() + 256, torch.uint8, like.device, stream)
    else:
        _on(workspace, "workspace", dev)
        if not workspace.is_contiguous():
            raise TypeError("workspace must be contiguous")
    base = workspace.data_ptr()
    aligned = (base + 255) // 256 * 256
    return aligned, max(0, workspace.nbytes - (aligned - base)), workspace


# the current stream's handle without the objects around it, where torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _call(fn, where: str, dev: int, stream, *args):
    """fn(*args, stream handle) with device dev current."""
    if torch.cuda.current_device() == dev:
        st = fn(*args, _raw_stream(dev) if stream is None and _raw_stream else _stream(stream))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(stream))
    return st if st == FS_OK else _check(st, where)


def _needed(fn, where: str, *args):
    need = int(fn(*args))
    if need == 0:
        _check(FS_ERR_INVALID_ARG, where)
    return need


def _attention_desc(q, k, v, scale, causal, offset, offsets, q_len, kv_len, key_mask, bias, edges,
                    two_sided):
    """The description, and q's device number."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a device tensor")
    dtype = _DTYPES.get(q.dtype)
    if dtype is None:
        raise TypeError(f"q must be float32, bfloat16 or float16 (is {q.dtype})")
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k and v must be [batch, rows, heads, width]")
    dev = q.get_device()
    batch, n, heads, d = q.shape
    _, m, kv_heads, _ = k.shape
    dv = v.shape[3]
    lens = (batch,)
    i32 = torch.int32
    if offset or batch > _MAX or n > _MAX or m > _MAX:
        _i32("a size or the offset", batch, n, m, offset)
    a = AttentionDesc(dtype, batch, n, m, heads, kv_heads, d, dv,
                      d ** -0.5 if scale is None else scale, 1 if causal else 0, offset)
    if offsets is not None:
        a.offsets = _flat(offsets, "offsets", dev, i32, lens)
    if q_len is not None:
        a.q_len = _flat(q_len, "q_len", dev, i32, lens)
    if kv_len is not None:
        a.kv_len = _flat(kv_len, "kv_len", dev, i32, lens)
    if key_mask is not None:
        _on(key_mask, "key_mask", dev)
        if key_mask.dtype not in (torch.uint8, torch.bool):
            raise TypeError("key_mask must be uint8 or bool")
        if key_mask.shape != (batch, m) or (m > 1 and key_mask.stride(1) != 1):
            raise ValueError(f"key_mask must be ({batch}, {m}) with a contiguous last axis")
        a.key_mask = key_mask.data_ptr()
        a.key_mask_stride = key_mask.stride(0) if batch > 1 else 0
    if bias is not None:
        e = [] if edges is None else edges
        buckets = (len(e) + 1) * (2 if two_sided else 1)
        a.bias = _flat(bias, "bias", dev, torch.float32, (buckets, heads))
        _i32("an edge", *e)
        a.edges = (ctypes.c_int32 * max(len(e), 1))(*e)
        a.n_edges = len(e)
        a.two_sided = bool(two_sided)
    return a, dev


def fs_attention_workspace_bytes(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, edges=None,
                                 two_sided: bool = True, backward: bool = False) -> int:
    """Bytes that serve the forward call, and the backward call if asked, on
    tensors of these shapes; edges: the bias's (None without a bias)."""
    if q.dtype not in _DTYPES:
        raise TypeError(f"q must be float32, bfloat16 or float16 (is {q.dtype})")
    _i32("a size or an edge", q.shape[0], q.shape[1], k.shape[1], *(edges or ()))
    a = AttentionDesc(_DTYPES[q.dtype], q.shape[0], q.shape[1], k.shape[1], q.shape[2],
                      k.shape[2], q.shape[3], v.shape[3], 1.0)
    if edges is not None:
        a.bias = 1  # only tested against NULL
        a.edges = (ctypes.c_int32 * max(len(edges), 1))(*edges)
        a.n_edges = len(edges)
        a.two_sided = bool(two_sided)
    need = [int(load().fs_attention_workspace_bytes(ctypes.byref(a), b))
            for b in ((0, 1) if backward else (0,))]
    if 0 in need:
        _check(FS_ERR_INVALID_ARG, "fs_attention_workspace_bytes")
    return max(need)


def fs_attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                         lse: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                         causal: bool = False, offset: int = 0, offsets=None, q_len=None,
                         kv_len=None, key_mask=None, bias=None, edges=None,
                         two_sided: bool = True, workspace: Optional[torch.Tensor] = None,
                         stream=None):
    """o <- softmax(scale q.k + bias) v over the visible keys, lse <- the rows'
    log-sum-exps.  q, o: [batch, n, heads, d or dv]; k, v: [batch, m, kv_heads,
    d or dv]; lse: [batch, heads, n] float32; scale: 1/sqrt(d) unless given."""
    lib = load()
    a, dev = _attention_desc(q, k, v, scale, causal, offset, offsets, q_len, kv_len, key_mask, bias,
                             edges, two_sided)
    pa = ctypes.byref(a)
    ws, size, _keep = _work(workspace, lambda: _needed(lib.fs_attention_workspace_bytes,
                                                       "fs_attention_forward", pa, 0), q, dev, stream)
    batch, n, heads, _ = q.shape
    m, kv_heads, dv = a.m, a.kv_heads, a.dv
    return _call(lib.fs_attention_forward, "fs_attention_forward", dev, stream, pa,
                 _rows(q, "q", q, dev, q.shape), _rows(k, "k", q, dev, (batch, m, kv_heads, a.d)),
                 _rows(v, "v", q, dev, (batch, m, kv_heads, dv)),
                 _rows(o, "o", q, dev, (batch, n, heads, dv)),
                 _flat(lse, "lse", dev, torch.float32, (batch, heads, n)), ws, size)


def fs_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                          lse: torch.Tensor, d_o: torch.Tensor, d_q=None, d_k=None, d_v=None, *,
                          d_lse=None, d_bias=None, scale: Optional[float] = None,
                          causal: bool = False, offset: int = 0, offsets=None, q_len=None,
                          kv_len=None, key_mask=None, bias=None, edges=None,
                          two_sided: bool = True, workspace: Optional[torch.Tensor] = None,
                          stream=None):
    """Gradients of fs_attention_forward from those of o (d_o) and lse (d_lse,
    optional): writes d_q, d_k, d_v and d_bias, each of its input's shape;
    None: not wanted."""
    lib = load()
    a, dev = _attention_desc(q, k, v, scale, causal, offset, offsets, q_len, kv_len, key_mask, bias,
                             edges, two_sided)
    pa = ctypes.byref(a)
    ws, size, _keep = _work(workspace, lambda: _needed(lib.fs_attention_workspace_bytes,
                                                       "fs_attention_backward", pa, 1), q, dev, stream)
    if lse is None or o is None or d_o is None:
        raise TypeError("o, lse and d_o must be given")
    f32 = torch.float32
    batch, n, heads, _ = qs = q.shape
    ks, vs = (batch, a.m, a.kv_heads, a.d), (batch, a.m, a.kv_heads, a.dv)
    outs, lses = (batch, n, heads, a.dv), (batch, heads, n)
    return _call(lib.fs_attention_backward, "fs_attention_backward", dev, stream, pa,
                 _rows(q, "q", q, dev, qs), _rows(k, "k", q, dev, ks), _rows(v, "v", q, dev, vs),
                 _rows(o, "o", q, dev, outs), _flat(lse, "lse", dev, f32, lses),
                 _rows(d_o, "d_o", q, dev, outs), _flat(d_lse, "d_lse", dev, f32, lses),
                 _rows(d_q, "d_q", q, dev, qs), _rows(d_k, "d_k", q, dev, ks),
                 _rows(d_v, "d_v", q, dev, vs),
                 _flat(d_bias, "d_bias", dev, f32, bias.shape if bias is not None else ()), ws, size)


def _norm_desc(q, k, eps, cos, sin, positions, offset, interleaved):
    """The description, the tensor whose type and device count, its device number."""
    like = q if q is not None else k
    if not isinstance(like, torch.Tensor) or not like.is_cuda:
        raise TypeError("q or k must be a device tensor")
    dtype = _DTYPES.get(like.dtype)
    if dtype is None:
        raise TypeError(f"q and k must be float32, bfloat16 or float16 (is {like.dtype})")
    if like.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be [batch, rows, heads, d]")
    dev = like.get_device()
    batch, n, _, d = like.shape
    if offset or batch > _MAX or n > _MAX:
        _i32("a size or the offset", batch, n, offset)
    a = QkNormDesc(dtype, batch, n, 0 if q is None else q.shape[2], 0 if k is None else k.shape[2],
                   d, 0, 1 if interleaved else 0, eps)
    if (cos is None) != (sin is None):
        raise TypeError("cos and sin must both be given or both be None")
    if cos is not None:
        if cos.dim() != 2:
            raise ValueError("cos and sin must be [positions, rot / 2]")
        table = cos.shape
        a.rot, a.n_pos = 2 * table[1], table[0]
        a.cos_table = _flat(cos, "cos", dev, torch.float32, table)
        a.sin_table = _flat(sin, "sin", dev, torch.float32, table)
    if positions is not None:
        _on(positions, "positions", dev)
        if positions.dtype != torch.int32 or positions.shape != (batch, n) or \
                (n > 1 and positions.stride(1) != 1):
            raise TypeError(f"positions must be int32 ({batch}, {n}) with a contiguous last axis")
        a.positions = positions.data_ptr()
        a.positions_stride = positions.stride(0) if batch > 1 else 0
    a.offset = offset
    return a, like, dev


def fs_qk_norm_workspace_bytes(q, k) -> int:
    """Bytes of workspace of fs_qk_norm_rotate_backward on tensors of these shapes."""
    a, _, _ = _norm_desc(q, k, 0.0, None, None, None, 0, False)
    return _needed(load().fs_qk_norm_workspace_bytes, "fs_qk_norm_workspace_bytes", ctypes.byref(a))


def fs_qk_norm_rotate(q, k, q_weight, k_weight, q_out, k_out, *, eps: float = 1e-6, cos=None,
                      sin=None, positions=None, offset: int = 0, interleaved: bool = False,
                      stream=None):
    """Norm of every head's row of q and k ([batch, n, heads, d]; either may be
    None) times its weight, and the rotation of the first 2 * cos.shape[1]
    elements by the position's row of cos and sin ([positions, rot / 2])."""
    lib = load()
    a, like, dev = _norm_desc(q, k, eps, cos, sin, positions, offset, interleaved)
    batch, n, _, d = like.shape
    qs, ks = (batch, n, a.heads_q, d), (batch, n, a.heads_k, d)
    f32, w = torch.float32, (d,)
    return _call(lib.fs_qk_norm_rotate, "fs_qk_norm_rotate", dev, stream, ctypes.byref(a),
                 _rows(q, "q", like, dev, qs), _rows(k, "k", like, dev, ks),
                 _flat(q_weight, "q_weight", dev, f32, w), _flat(k_weight, "k_weight", dev, f32, w),
                 _rows(q_out, "q_out", like, dev, qs), _rows(k_out, "k_out", like, dev, ks))


def fs_qk_norm_rotate_backward(q, k, q_weight, k_weight, d_q_out, d_k_out, d_q, d_k,
                               d_q_weight=None, d_k_weight=None, *, eps: float = 1e-6, cos=None,
                               sin=None, positions=None, offset: int = 0,
                               interleaved: bool = False,
                               workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of fs_qk_norm_rotate: writes d_q, d_k and, where given, the
    weights' gradients."""
    lib = load()
    a, like, dev = _norm_desc(q, k, eps, cos, sin, positions, offset, interleaved)
    pa = ctypes.byref(a)
    ws, size, _keep = _work(workspace, lambda: _needed(lib.fs_qk_norm_workspace_bytes,
                                                       "fs_qk_norm_rotate_backward", pa), like, dev,
                            stream)
    batch, n, _, d = like.shape
    qs, ks = (batch, n, a.heads_q, d), (batch, n, a.heads_k, d)
    f32, w = torch.float32, (d,)
    return _call(lib.fs_qk_norm_rotate_backward, "fs_qk_norm_rotate_backward", dev, stream, pa,
                 _rows(q, "q", like, dev, qs), _rows(k, "k", like, dev, ks),
                 _flat(q_weight, "q_weight", dev, f32, w), _flat(k_weight, "k_weight", dev, f32, w),
                 _rows(d_q_out, "d_q_out", like, dev, qs), _rows(d_k_out, "d_k_out", like, dev, ks),
                 _rows(d_q, "d_q", like, dev, qs), _rows(d_k, "d_k", like, dev, ks),
                 _flat(d_q_weight, "d_q_weight", dev, f32, w),
                 _flat(d_k_weight, "d_k_weight", dev, f32, w), ws, size)
