"""ctypes binding of ``libsla.so`` (the C ABI in ``include/sla.h``).

Argument marshalling only: every numerical step runs in the library's HIP
kernels.  Torch tensors supply device memory and the current HIP stream.
torch is imported before the library is loaded so that ``libsla.so`` binds to
the same HIP runtime instance as torch (both carry the soname
``libamdhip64.so.7``).  There is no CPU fallback: if the library is missing or
no GPU is present, the calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
import os
import threading
from typing import Optional, Tuple

import torch  # noqa: F401  (must precede loading libsla.so, see above)

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libsla.so")

SLA_F64, SLA_F32, SLA_BF16, SLA_F16 = 0, 1, 2, 3
SLA_GATE_LINEAR, SLA_GATE_SIGMOID = 0, 1
SLA_ACT_NONE, SLA_ACT_SILU = 0, 1
SLA_GATE_FIRST, SLA_NORM_FIRST = 0, 1
SLA_BUILD_TRANSPOSE, SLA_VALIDATE = 1, 2
STATUS = {0: "SLA_OK", 1: "SLA_NOT_CONVERGED", -1: "SLA_ERR_INVALID_ARG", -2: "SLA_ERR_UNSUPPORTED",
          -3: "SLA_ERR_BREAKDOWN", -4: "SLA_ERR_NONFINITE", -5: "SLA_ERR_HIP", -6: "SLA_ERR_OOM"}
OK, NOT_CONVERGED = 0, 1
ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_BREAKDOWN, ERR_NONFINITE, ERR_HIP, ERR_OOM = -1, -2, -3, -4, -5, -6
PROFILE_CLASSES = {"a_step": 0, "gt_step": 1, "g_step": 2, "spmv": 3}


class SlaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class SolveInfo(ctypes.Structure):
    _fields_ = [("iterations", ctypes.c_int32), ("converged", ctypes.c_int32),
                ("rel_residual", ctypes.c_double), ("bnorm", ctypes.c_double)]


class LinrecShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int64), ("steps", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("d_offsets", ctypes.c_void_p), ("dtype", ctypes.c_int), ("gate", ctypes.c_int)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("d_param", ctypes.c_void_p), ("d_copy", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("dtype", ctypes.c_int), ("grad_dtype", ctypes.c_int)]


class AdamwHyper(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint64)]


class ConvShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int64), ("steps", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("width", ctypes.c_int64), ("d_offsets", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("act", ctypes.c_int)]


class SelscanShape(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int64), ("steps", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("n_state", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("d_offsets", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("softplus", ctypes.c_int32)]


class SelscanIn(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("d_x", "d_dt", "d_z", "d_b", "d_c")] + \
        [(n, ctypes.c_int64) for n in ("x_seq", "x_step", "dt_seq", "dt_step", "z_seq", "z_step",
                                       "b_seq", "b_step", "c_seq", "c_step")] + \
        [(n, ctypes.c_void_p) for n in ("d_a", "d_d", "d_dt_bias", "d_h0")]


class SelscanGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("d_x", "d_dt", "d_z", "d_b", "d_c", "d_a", "d_d",
                                               "d_dt_bias", "d_h0")]


class NormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("stream", ctypes.c_int), ("eps", ctypes.c_double)]


_lib = None
_lock = threading.Lock()


def lib_path() -> str:
    """libsla.so, or with SLA_DEBUG=1 the bounds-checking build libsla_debug.so."""
    if os.environ.get("SLA_DEBUG") == "1":
        return os.path.join(PKG, "libsla_debug.so")
    return LIB_PATH


def lib():
    """Load the library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = lib_path()
            if not os.path.exists(path):
                raise ImportError(f"{path} is missing: build it with "
                                  "preconditioned_cg_solver_amd.build.build()")
            _lib = _declare(ctypes.CDLL(path))
        return _lib


def _declare(L):
    vp, i32, i64, u32, dbl, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                  ctypes.c_double, ctypes.c_size_t)
    st = ctypes.c_int
    sig = {
        "sla_csr_create": ([ctypes.POINTER(vp), i64, i64, vp, vp, vp, ctypes.c_int, u32, vp], st),
        "sla_bsr_create": ([ctypes.POINTER(vp), i64, i64, i32, vp, vp, vp, ctypes.c_int, u32, vp], st),
        "sla_mat_destroy": ([vp], st),
        "sla_mat_info": ([vp, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i32),
                          ctypes.POINTER(i32)], st),
        "sla_mat_transpose_arrays": ([vp, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                      ctypes.POINTER(vp)], st),
        "sla_mat_tiling": ([vp, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)], st),
        "sla_mat_reordered": ([vp, ctypes.POINTER(i32)], st),
        "sla_spmv": ([vp, vp, vp, vp], st),
        "sla_spmv_t": ([vp, vp, vp, vp], st),
        "sla_pcg_workspace_size": ([vp, ctypes.POINTER(sz)], st),
        "sla_precond_apply": ([vp, dbl, vp, vp, vp, sz, vp], st),
        "sla_pcg_solve": ([vp, vp, dbl, vp, vp, dbl, i32, vp, sz, vp, ctypes.POINTER(SolveInfo)],
                          st),
        "sla_pcg_adjoint": ([vp, vp, dbl, vp, vp, vp, vp, dbl, i32, vp, sz, vp,
                             ctypes.POINTER(SolveInfo)], st),
        "sla_spmm": ([vp, vp, vp, i32, vp], st),
        "sla_spmm_t": ([vp, vp, vp, i32, vp], st),
        "sla_pcg_workspace_size_multi": ([vp, i32, ctypes.POINTER(sz)], st),
        "sla_pcg_solve_multi": ([vp, vp, dbl, vp, vp, i32, dbl, i32, vp, sz, vp,
                                 ctypes.POINTER(SolveInfo), ctypes.POINTER(ctypes.c_int)], st),
        "sla_pcg_adjoint_multi": ([vp, vp, dbl, vp, vp, vp, vp, i32, dbl, i32, vp, sz, vp,
                                   ctypes.POINTER(SolveInfo), ctypes.POINTER(ctypes.c_int)], st),
        "sla_lanczos_extremes": ([vp, vp, i32, ctypes.POINTER(dbl), ctypes.POINTER(dbl)], st),
        "sla_sai_loss": ([vp, vp, dbl, vp, i32, dbl, vp, sz, vp, vp], st),
        "sla_pcg_solve_history": ([vp, vp, dbl, vp, vp, dbl, i32, vp, sz, vp, vp, i32, vp,
                                   ctypes.POINTER(SolveInfo)], st),
        "sla_pattern_grad": ([vp, vp, vp, vp, vp], st),
        "sla_init": ([], st),
        "sla_pcg_solve_noalloc": ([vp, vp, dbl, vp, vp, dbl, i32, vp, ctypes.POINTER(SolveInfo)],
                                  st),
        "sla_linrec_sizes": ([vp, ctypes.POINTER(sz), ctypes.POINTER(sz)], st),
        "sla_linrec_forward": ([vp, vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, vp, sz, vp], st),
        "sla_linrec_backward": ([vp, vp, i64, i64, vp, i64, i64, vp, vp, vp, i64, i64, vp, vp, vp,
                                 vp, vp, sz, vp], st),
        "sla_adamw_sizes": ([vp, i32, i32, ctypes.POINTER(sz), ctypes.POINTER(sz),
                             ctypes.POINTER(i64)], st),
        "sla_adamw_create": ([ctypes.POINTER(vp), vp, i32, i32, vp, sz, vp, sz, vp], st),
        "sla_adamw_destroy": ([vp], st),
        "sla_adamw_step": ([vp, vp, vp, vp, vp], st),
        "sla_adamw_get_state": ([vp, vp, vp, vp], st),
        "sla_adamw_set_state": ([vp, vp, vp, vp], st),
        "sla_conv_sizes": ([vp, ctypes.POINTER(sz)], st),
        "sla_rows_clear": ([vp, i64, i64, i64, ctypes.c_int, vp, vp], st),
        "sla_conv_forward": ([vp, vp, i64, i64, vp, vp, vp, vp, vp, vp], st),
        "sla_conv_backward": ([vp, vp, i64, i64, vp, vp, vp, vp, i64, i64, vp, vp, vp, vp, vp, vp,
                               sz, vp], st),
        "sla_selscan_sizes": ([vp, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)],
                              st),
        "sla_selscan_forward": ([vp, vp, vp, vp, vp, vp, sz, vp], st),
        "sla_selscan_backward": ([vp, vp, vp, vp, i64, i64, vp, vp, vp, sz, vp], st),
        "sla_norm_sizes": ([vp, ctypes.POINTER(sz)], st),
        "sla_norm_in_forward": ([vp, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp], st),
        "sla_norm_in_backward": ([vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, sz,
                                  vp], st),
        "sla_norm_out_forward": ([vp, ctypes.c_int, vp, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp],
                                 st),
        "sla_norm_out_backward": ([vp, ctypes.c_int, vp, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp,
                                   vp, vp, sz, vp], st),
        "sla_status_string": ([st], ctypes.c_char_p),
        "sla_last_error": ([], ctypes.c_char_p),
        "sla_set_profiling": ([i32], st),
        "sla_set_profiling_stride": ([i32], st),
        "sla_get_profile": ([i32, ctypes.POINTER(i64), ctypes.POINTER(dbl)], st),
        "sla_reset_profile": ([], st),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    return L


def _check(status: int, allow=(OK,)) -> int:
    if status in allow:
        return status
    msg = lib().sla_last_error().decode(errors="replace")
    raise SlaError(status, msg)


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream) if hasattr(stream, "cuda_stream") else stream


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the library must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _vec(t: torch.Tensor, A: "Mat", numel: int, name: str):
    """Pointer of a vector argument of a call on A: a contiguous tensor on A's
    device, in A's dtype, with exactly `numel` elements (the library reads
    and writes that many from the raw pointer and cannot check it)."""
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must live on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype != A.dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, the matrix has {A.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    if torch.device(t.device) != torch.device(A.device):
        raise ValueError(f"{name} is on {t.device}, the matrix on {A.device}")
    return ctypes.c_void_p(t.data_ptr())


def _work(work: torch.Tensor, A: "Mat"):
    """(pointer, size in bytes) of a workspace tensor on A's device."""
    if not getattr(work, "is_cuda", False) or not work.is_contiguous():
        raise ValueError("the workspace must be a contiguous GPU tensor")
    if torch.device(work.device) != torch.device(A.device):
        raise ValueError(f"the workspace is on {work.device}, the matrix on {A.device}")
    return ctypes.c_void_p(work.data_ptr()), work.numel() * work.element_size()


def _pair(A: "Mat", G: "Mat"):
    if A.n != G.n or A.dtype != G.dtype or A.block_dim != G.block_dim:
        raise ValueError("A and G differ in size, block size or dtype")


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float64:
        return SLA_F64
    if dt == torch.float32:
        return SLA_F32
    raise ValueError(f"unsupported dtype {dt}")


class Mat:
    """A library matrix handle; keeps the borrowed tensors alive."""

    def __init__(self, handle, keep, n, nnz, block_dim, dtype):
        self.handle = handle
        self._keep = keep
        self.n, self.nnz, self.block_dim, self.dtype = n, nnz, block_dim, dtype

    def destroy(self):
        if self.handle:
            lib().sla_mat_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass

    @property
    def device(self):
        return self._keep[0].device


def sla_mat_destroy(A: Mat) -> None:
    A.destroy()


def sla_mat_info(A: Mat) -> Tuple[int, int, int, int]:
    """(n, nnz, block_dim, dtype code) as the library records them."""
    n, nnz = ctypes.c_int64(), ctypes.c_int64()
    bd, dt = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().sla_mat_info(A.handle, ctypes.byref(n), ctypes.byref(nnz), ctypes.byref(bd),
                              ctypes.byref(dt)))
    return n.value, nnz.value, bd.value, dt.value


def sla_last_error() -> str:
    return lib().sla_last_error().decode(errors="replace")


def sla_csr_create(row_ptr: torch.Tensor, col_idx: torch.Tensor, vals: torch.Tensor,
                   build_transpose: bool = False, validate: bool = False, stream=None) -> Mat:
    n = row_ptr.numel() - 1
    nnz = col_idx.numel()
    for t, want in ((row_ptr, torch.int32), (col_idx, torch.int32)):
        if t.dtype != want:
            raise ValueError("index arrays must be int32")
    h = ctypes.c_void_p()
    flags = (SLA_BUILD_TRANSPOSE if build_transpose else 0) | (SLA_VALIDATE if validate else 0)
    _check(lib().sla_csr_create(ctypes.byref(h), n, nnz, _ptr(row_ptr), _ptr(col_idx), _ptr(vals),
                                _dtype_code(vals.dtype), flags, _stream(stream)))
    return Mat(h, (row_ptr, col_idx, vals), n, nnz, 1, vals.dtype)


def sla_bsr_create(brow_ptr: torch.Tensor, bcol_idx: torch.Tensor, bvals: torch.Tensor,
                   block_dim: int = 3, build_transpose: bool = False, validate: bool = False,
                   stream=None) -> Mat:
    nbr = brow_ptr.numel() - 1
    nnzb = bcol_idx.numel()
    if bvals.numel() != nnzb * block_dim * block_dim:
        raise ValueError("bvals must hold nnzb * block_dim^2 values")
    h = ctypes.c_void_p()
    flags = (SLA_BUILD_TRANSPOSE if build_transpose else 0) | (SLA_VALIDATE if validate else 0)
    _check(lib().sla_bsr_create(ctypes.byref(h), nbr, nnzb, block_dim, _ptr(brow_ptr),
                                _ptr(bcol_idx), _ptr(bvals), _dtype_code(bvals.dtype), flags,
                                _stream(stream)))
    return Mat(h, (brow_ptr, bcol_idx, bvals), nbr * block_dim, nnzb * block_dim ** 2, block_dim,
               bvals.dtype)


def sla_mat_tiling(A: Mat, transpose: bool = False) -> Tuple[int, int]:
    nt, nl = ctypes.c_int64(), ctypes.c_int64()
    _check(lib().sla_mat_tiling(A.handle, int(transpose), ctypes.byref(nt), ctypes.byref(nl)))
    return nt.value, nl.value


def sla_mat_reordered(A: Mat) -> bool:
    """True when the solves with A run on its locality ordering."""
    r = ctypes.c_int32()
    _check(lib().sla_mat_reordered(A.handle, ctypes.byref(r)))
    return bool(r.value)


def sla_mat_transpose_arrays(A: Mat):
    """Raw device pointers (row_ptr, col_idx, vals) of the owned transpose."""
    rp, ci, v = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    _check(lib().sla_mat_transpose_arrays(A.handle, ctypes.byref(rp), ctypes.byref(ci),
                                          ctypes.byref(v)))
    return rp.value, ci.value, v.value


def sla_spmv(A: Mat, x: torch.Tensor, y: Optional[torch.Tensor] = None, stream=None,
             transpose: bool = False) -> torch.Tensor:
    px = _vec(x, A, A.n, "x")
    if y is None:
        y = torch.empty(A.n, dtype=A.dtype, device=x.device)
    py = _vec(y, A, A.n, "y")
    f = lib().sla_spmv_t if transpose else lib().sla_spmv
    _check(f(A.handle, px, py, _stream(stream)))
    return y


def sla_spmv_t(A: Mat, x: torch.Tensor, y: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """y = A^T x (the handle must carry its transpose)."""
    return sla_spmv(A, x, y, stream, transpose=True)


def sla_pcg_workspace_size(A: Mat) -> int:
    b = ctypes.c_size_t()
    _check(lib().sla_pcg_workspace_size(A.handle, ctypes.byref(b)))
    return b.value


def workspace(A: Mat, device=None) -> torch.Tensor:
    nbytes = sla_pcg_workspace_size(A)
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device or A.device)


def sla_precond_apply(G: Mat, eps: float, r: torch.Tensor, z: Optional[torch.Tensor] = None,
                      work: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    pr = _vec(r, G, G.n, "r")
    if z is None:
        z = torch.empty_like(r)
    pz = _vec(z, G, G.n, "z")
    if work is None:
        work = workspace(G, r.device)
    pw, nw = _work(work, G)
    _check(lib().sla_precond_apply(G.handle, float(eps), pr, pz, pw, nw, _stream(stream)))
    return z


@dataclasses.dataclass
class Info:
    status: int
    iterations: int
    converged: bool
    rel_residual: float
    bnorm: float


def _info(status, si: SolveInfo) -> Info:
    return Info(status, si.iterations, bool(si.converged), si.rel_residual, si.bnorm)


def sla_pcg_solve(A: Mat, G: Mat, eps: float, b: torch.Tensor, x: Optional[torch.Tensor] = None,
                  rtol: float = 1e-10, maxit: int = 1000, work: Optional[torch.Tensor] = None,
                  stream=None, raise_on_error: bool = True) -> Tuple[torch.Tensor, Info]:
    _pair(A, G)
    pb = _vec(b, A, A.n, "b")
    if x is None:
        x = torch.empty_like(b)
    px = _vec(x, A, A.n, "x")
    if work is None:
        work = workspace(A, b.device)
    pw, nw = _work(work, A)
    si = SolveInfo()
    st = lib().sla_pcg_solve(A.handle, G.handle, float(eps), pb, px, float(rtol), int(maxit), pw,
                             nw, _stream(stream), ctypes.byref(si))
    if raise_on_error:
        _check(st, allow=(OK, NOT_CONVERGED))
    return x, _info(st, si)


def sla_init() -> None:
    """Prepare the current device for sla_pcg_solve_noalloc (resolves the
    library's fixed scratch and reserves a polling record; may allocate)."""
    _check(lib().sla_init())


def sla_pcg_solve_noalloc(A: Mat, G: Mat, eps: float, b: torch.Tensor, x: torch.Tensor,
                          rtol: float = 1e-10, maxit: int = 1000, stream=None,
                          raise_on_error: bool = True) -> Info:
    """sla_pcg_solve with the library's fixed scratch as workspace: allocates
    nothing (x is the caller's output tensor).  Needs sla_init() first."""
    _pair(A, G)
    pb = _vec(b, A, A.n, "b")
    px = _vec(x, A, A.n, "x")
    si = SolveInfo()
    st = lib().sla_pcg_solve_noalloc(A.handle, G.handle, float(eps), pb, px, float(rtol),
                                     int(maxit), _stream(stream), ctypes.byref(si))
    if raise_on_error:
        _check(st, allow=(OK, NOT_CONVERGED))
    return _info(st, si)


def sla_pcg_solve_history(A: Mat, G: Mat, eps: float, b: torch.Tensor,
                          x: Optional[torch.Tensor] = None, rtol: float = 1e-10,
                          maxit: int = 1000, work: Optional[torch.Tensor] = None, stream=None,
                          raise_on_error: bool = True):
    """sla_pcg_solve that also returns the CG coefficients alpha_k (k = 1..iters)
    and beta_k = rho_k / rho_{k-1} (k = 1..iters-1) as CPU float64 tensors."""
    _pair(A, G)
    pb = _vec(b, A, A.n, "b")
    if x is None:
        x = torch.empty_like(b)
    px = _vec(x, A, A.n, "x")
    if work is None:
        work = workspace(A, b.device)
    pw, nw = _work(work, A)
    hist_a = torch.zeros(max(maxit, 1), dtype=torch.float64, device=b.device)
    hist_b = torch.zeros(max(maxit, 1), dtype=torch.float64, device=b.device)
    si = SolveInfo()
    st = lib().sla_pcg_solve_history(A.handle, G.handle, float(eps), pb, px, float(rtol),
                                     int(maxit), pw, nw, _ptr(hist_a), _ptr(hist_b), int(maxit),
                                     _stream(stream), ctypes.byref(si))
    if raise_on_error:
        _check(st, allow=(OK, NOT_CONVERGED))
    k = si.iterations
    return x, _info(st, si), hist_a[:k].cpu(), hist_b[:max(k - 1, 0)].cpu()


def sla_lanczos_extremes(alpha, beta):
    """(lmin, lmax) of the Lanczos tridiagonal from CG's alpha_1..k, beta_1..k-1."""
    a = [float(v) for v in alpha]
    b = [float(v) for v in beta] or [0.0]
    ha = (ctypes.c_double * max(len(a), 1))(*a)
    hb = (ctypes.c_double * len(b))(*b)
    lo, hi = ctypes.c_double(0.0), ctypes.c_double(0.0)
    st = lib().sla_lanczos_extremes(ha, hb, len(a), ctypes.byref(lo), ctypes.byref(hi))
    _check(st)
    return lo.value, hi.value


def sla_sai_loss(A: Mat, G: Mat, eps: float, probes: torch.Tensor, scale: float,
                 work: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Per-probe || A M^-1 w_j / scale - w_j ||^2 for the columns w_j of the
    (n, m) device tensor `probes` (float64 device tensor of length m)."""
    _pair(A, G)
    if probes.dim() != 2 or probes.shape[0] != A.n:
        raise ValueError(f"probes must be ({A.n}, m)")
    n, m = probes.shape
    pt = probes.t().contiguous()  # probe j contiguous at j * n
    pp = _vec(pt, A, n * m, "probes")
    if work is None:
        nb = max(sla_pcg_workspace_size(A), sla_pcg_workspace_size(G), 1)
        work = torch.empty(nb, dtype=torch.uint8, device=probes.device)
    pw, nw = _work(work, A)
    out = torch.empty(max(m, 1), dtype=torch.float64, device=probes.device)
    st = lib().sla_sai_loss(A.handle, G.handle, float(eps), pp, int(m), float(scale), pw, nw,
                            _ptr(out), _stream(stream))
    _check(st)
    return out[:m]


def sla_pcg_adjoint(A: Mat, G: Mat, eps: float, x: torch.Tensor, grad_x: torch.Tensor,
                    rtol: float = 1e-10, maxit: int = 1000, grad_b: Optional[torch.Tensor] = None,
                    grad_vals: Optional[torch.Tensor] = None, work: Optional[torch.Tensor] = None,
                    stream=None, raise_on_error: bool = True):
    _pair(A, G)
    px = _vec(x, A, A.n, "x")
    pgx = _vec(grad_x, A, A.n, "grad_x")
    if grad_b is None:
        grad_b = torch.empty_like(x)
    pgb = _vec(grad_b, A, A.n, "grad_b")
    if grad_vals is None:
        grad_vals = torch.empty(A.nnz, dtype=A.dtype, device=x.device)
    pgv = _vec(grad_vals, A, A.nnz, "grad_vals")
    if work is None:
        work = workspace(A, x.device)
    pw, nw = _work(work, A)
    si = SolveInfo()
    st = lib().sla_pcg_adjoint(A.handle, G.handle, float(eps), px, pgx, pgb, pgv, float(rtol),
                               int(maxit), pw, nw, _stream(stream), ctypes.byref(si))
    if raise_on_error:
        _check(st, allow=(OK, NOT_CONVERGED))
    return grad_b, grad_vals, _info(st, si)


# ----- several right-hand sides (n x k row-major device tensors) -----

def _cols(t: torch.Tensor, A: "Mat" = None) -> int:
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError("expected a contiguous (n, k) tensor")
    if A is not None and t.shape[0] != A.n:
        raise ValueError(f"expected {A.n} rows, got {t.shape[0]}")
    return t.shape[1]


def _block(t: torch.Tensor, A: "Mat", k: int, name: str):
    if t.dim() != 2 or tuple(t.shape) != (A.n, k):
        raise ValueError(f"{name} must be ({A.n}, {k}), got {tuple(t.shape)}")
    return _vec(t, A, A.n * k, name)


def sla_spmm(A: Mat, X: torch.Tensor, Y: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """Y = A X for the k columns of the (n, k) tensor X."""
    k = _cols(X, A)
    px = _block(X, A, k, "X")
    if Y is None:
        Y = torch.empty_like(X)
    py = _block(Y, A, k, "Y")
    _check(lib().sla_spmm(A.handle, px, py, k, _stream(stream)))
    return Y


def sla_spmm_t(A: Mat, X: torch.Tensor, Y: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    k = _cols(X, A)
    px = _block(X, A, k, "X")
    if Y is None:
        Y = torch.empty_like(X)
    py = _block(Y, A, k, "Y")
    _check(lib().sla_spmm_t(A.handle, px, py, k, _stream(stream)))
    return Y


def sla_pcg_workspace_size_multi(A: Mat, k: int) -> int:
    b = ctypes.c_size_t()
    _check(lib().sla_pcg_workspace_size_multi(A.handle, int(k), ctypes.byref(b)))
    return b.value


def workspace_multi(A: Mat, k: int, device=None) -> torch.Tensor:
    return torch.empty(max(sla_pcg_workspace_size_multi(A, k), 1), dtype=torch.uint8,
                       device=device or A.device)


def _multi_out(st, infos, cst, k):
    return [_info(int(cst[c]), infos[c]) for c in range(k)]


def sla_pcg_solve_multi(A: Mat, G: Mat, eps: float, B: torch.Tensor,
                        X: Optional[torch.Tensor] = None, rtol: float = 1e-10, maxit: int = 1000,
                        work: Optional[torch.Tensor] = None, stream=None,
                        raise_on_error: bool = True):
    """Solve A X = B for the k columns of B (n, k) together; returns X and one
    Info per column (its own status, iterations and residual)."""
    _pair(A, G)
    k = _cols(B, A)
    pb = _block(B, A, k, "B")
    if X is None:
        X = torch.empty_like(B)
    px = _block(X, A, k, "X")
    if work is None:
        work = workspace_multi(A, k, B.device)
    pw, nw = _work(work, A)
    infos = (SolveInfo * k)()
    cst = (ctypes.c_int * k)()
    st = lib().sla_pcg_solve_multi(A.handle, G.handle, float(eps), pb, px, k, float(rtol),
                                   int(maxit), pw, nw, _stream(stream), infos, cst)
    if raise_on_error:
        _check(st, allow=(OK, NOT_CONVERGED))
    return X, _multi_out(st, infos, cst, k)


def sla_pcg_adjoint_multi(A: Mat, G: Mat, eps: float, X: torch.Tensor, GX: torch.Tensor,
                          rtol: float = 1e-10, maxit: int = 1000,
                          GB: Optional[torch.Tensor] = None,
                          grad_vals: Optional[torch.Tensor] = None,
                          work: Optional[torch.Tensor] = None, stream=None,
                          raise_on_error: bool = True):
    """Adjoint of k solves sharing A: dL/dB = A^-T dL/dX column by column and
    dL/dA on A's pattern summed over the solves."""
    _pair(A, G)
    k = _cols(X, A)
    px = _block(X, A, k, "X")
    pgx = _block(GX, A, k, "GX")
    if GB is None:
        GB = torch.empty_like(X)
    pgb = _block(GB, A, k, "GB")
    if grad_vals is None:
        grad_vals = torch.empty(A.nnz, dtype=A.dtype, device=X.device)
    pgv = _vec(grad_vals, A, A.nnz, "grad_vals")
    if work is None:
        work = workspace_multi(A, k, X.device)
    pw, nw = _work(work, A)
    infos = (SolveInfo * k)()
    cst = (ctypes.c_int * k)()
    st = lib().sla_pcg_adjoint_multi(A.handle, G.handle, float(eps), px, pgx, pgb, pgv, k,
                                     float(rtol), int(maxit), pw, nw, _stream(stream), infos, cst)
    if raise_on_error:
        _check(st, allow=(OK, NOT_CONVERGED))
    return GB, grad_vals, _multi_out(st, infos, cst, k)


def sla_pattern_grad(A: Mat, lam: torch.Tensor, x: torch.Tensor,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    pl = _vec(lam, A, A.n, "lam")
    px = _vec(x, A, A.n, "x")
    if out is None:
        out = torch.empty(A.nnz, dtype=A.dtype, device=x.device)
    po = _vec(out, A, A.nnz, "out")
    _check(lib().sla_pattern_grad(A.handle, pl, px, po, _stream(stream)))
    return out


def sla_set_profiling(enable) -> None:
    """enable: True (all classes), False, or a bit mask / iterable of class names."""
    if enable is True:
        mask = 15
    elif enable is False or enable is None:
        mask = 0
    elif isinstance(enable, int):
        mask = enable
    else:
        mask = 0
        for c in enable:
            mask |= 1 << (PROFILE_CLASSES[c] if isinstance(c, str) else int(c))
    _check(lib().sla_set_profiling(int(mask)))


def sla_set_profiling_stride(every: int) -> None:
    """Time only the launches of iterations k with k % every == 0."""
    _check(lib().sla_set_profiling_stride(int(every)))


def sla_reset_profile() -> None:
    _check(lib().sla_reset_profile())


def sla_get_profile(kernel_class) -> Tuple[int, float]:
    if isinstance(kernel_class, str):
        kernel_class = PROFILE_CLASSES[kernel_class]
    n, ms = ctypes.c_int64(), ctypes.c_double()
    _check(lib().sla_get_profile(int(kernel_class), ctypes.byref(n), ctypes.byref(ms)))
    return n.value, ms.value


def sla_status_string(status: int) -> str:
    return lib().sla_status_string(int(status)).decode()


# ----- recurrences along a sequence, and the AdamW step -----

_DTYPES = {torch.float64: SLA_F64, torch.float32: SLA_F32, torch.bfloat16: SLA_BF16,
           torch.float16: SLA_F16}
_GATES = {"linear": SLA_GATE_LINEAR, "sigmoid": SLA_GATE_SIGMOID}


def _device_of(named) -> torch.device:
    """The one GPU that all the given (name, tensor) pairs live on."""
    dev = None
    for name, t in named:
        if t is None:
            continue
        if not getattr(t, "is_cuda", False):
            raise ValueError(f"{name} must live on the GPU")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, others on {dev}")
    return dev


def _enter(dev: torch.device, stream):
    """(raw stream, context in which to allocate, stream on which to record what
    the call uses): results and scratch belong to the stream that the kernels run
    on.  Kernels are launched on the current device, which has to be the tensors'.

    Tensors that are used on a given torch.cuda.Stream are recorded on it, so
    that their memory is not reused before the call's work is done.  A stream
    given by its raw pointer (or as ExternalStream) may not live that long: there
    the caller keeps the tensors until then."""
    current = torch.cuda.current_device()
    if dev.index is not None and dev.index != current:
        raise ValueError(f"the tensors are on {dev}, the current device is cuda:{current}")
    if stream is None:
        # current_stream() would make an object of it: 2.5 us of a serving step's 17
        return torch._C._cuda_getCurrentRawStream(current), _SAME_STREAM, None
    if not hasattr(stream, "cuda_stream"):
        raw = stream.value if isinstance(stream, ctypes.c_void_p) else stream
        stream = torch.cuda.ExternalStream(raw or 0, device=dev)
    lasts = not isinstance(stream, torch.cuda.ExternalStream)
    return stream.cuda_stream, torch.cuda.stream(stream), stream if lasts else None


_SAME_STREAM = contextlib.nullcontext()


def _record(stream, *tensors):
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


# Tells autograd that tensors were written, so that a backward pass that has
# saved one raises instead of using its new values.
_written = torch.autograd.graph.increment_version


def _raw(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _linrec_shape(x, gate, offsets, mode) -> Tuple[LinrecShape, torch.dtype]:
    if mode not in _GATES:
        raise ValueError(f"mode must be one of {sorted(_GATES)}, got {mode!r}")
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if offsets is None:
        if x.dim() != 3:
            raise ValueError("x must be (sequences, steps, channels), or give offsets")
        n, t, d = x.shape
    else:
        if x.dim() != 2:
            raise ValueError("packed x must be (steps, channels)")
        if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 1 \
                or not offsets.is_contiguous():
            raise ValueError("offsets must be a contiguous int64 vector of sequences + 1 entries")
        n, (t, d) = offsets.numel() - 1, x.shape
    if tuple(gate.shape) != tuple(x.shape) or gate.dtype != x.dtype:
        raise ValueError("gate must have x's shape and dtype")
    q = LinrecShape(n, t, d, None if offsets is None else offsets.data_ptr(), _DTYPES[x.dtype],
                    _GATES[mode])
    return q, torch.float64 if x.dtype == torch.float64 else torch.float32


def _steps_in(t, name: str, x):
    """(pointer, sequence stride, step stride) of an input shaped like x."""
    if t is None:
        return None, 0, 0
    if tuple(t.shape) != tuple(x.shape) or t.dtype != x.dtype:
        raise ValueError(f"{name} must have x's shape and dtype")
    st = t.stride()
    if t.shape[-1] > 1 and st[-1] != 1 and t.numel():
        raise ValueError(f"{name}'s channels must be adjacent (last stride 1)")
    return t.data_ptr(), (st[0] if len(st) == 3 else 0), st[-2]


def _states(t, name: str, q: LinrecShape, dtype):
    if t is None:
        return None
    if tuple(t.shape) != (q.n_seq, q.dim) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous ({q.n_seq}, {q.dim}) tensor of {dtype}")
    return t.data_ptr()


def _like(x):
    """A dense tensor of x's shape, dtype and device."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def sla_linrec_sizes(x, gate, offsets=None, mode: str = "sigmoid") -> Tuple[int, int]:
    """Bytes of (the states kept for the backward pass, the workspace)."""
    q, _ = _linrec_shape(x, gate, offsets, mode)
    return _linrec_sizes(q)


def _linrec_sizes(q: LinrecShape) -> Tuple[int, int]:
    saved, work = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().sla_linrec_sizes(ctypes.byref(q), ctypes.byref(saved), ctypes.byref(work)))
    return saved.value, work.value


def sla_linrec_forward(x: torch.Tensor, gate: torch.Tensor, h0: Optional[torch.Tensor] = None,
                       offsets: Optional[torch.Tensor] = None, mode: str = "sigmoid",
                       save: bool = False, h_last: Optional[torch.Tensor] = None, stream=None):
    """h_t = a_t h_{t-1} + b_t along each sequence: a = gate, b = x ("linear"),
    or a = sigmoid(gate), b = (1 - a) x ("sigmoid").

    x and gate: (sequences, steps, channels), or (steps, channels) with
    `offsets` (int64, on the device) marking where each of the packed
    sequences begins; slices of a wider tensor and expanded ones are taken as
    they are.  h0 and h_last: (sequences, channels) float32 (float64 for
    float64); h_last may be given, h0 itself included, to be overwritten.
    `stream` (a torch stream or a raw pointer) has to be ordered after what made
    the inputs; given as a raw pointer, the caller keeps them until it is done.
    Returns (h, h_last, saved); `saved` (None unless save) is what the
    backward pass needs."""
    q, sdt = _linrec_shape(x, gate, offsets, mode)
    px, pg = _steps_in(x, "x", x), _steps_in(gate, "gate", x)
    p0, pl = _states(h0, "h0", q, sdt), _states(h_last, "h_last", q, sdt)
    dev = _device_of((("x", x), ("gate", gate), ("h0", h0), ("offsets", offsets),
                      ("h_last", h_last)))
    raw, ctx, used = _enter(dev, stream)
    n_saved, n_work = _linrec_sizes(q)
    with ctx:
        h = _like(x)
        given = h_last
        if h_last is None:
            h_last = _like(h0) if h0 is not None else \
                torch.empty((q.n_seq, q.dim), dtype=sdt, device=dev)
            pl = _raw(h_last)
        saved = torch.empty(n_saved // sdt.itemsize, dtype=sdt, device=dev) if save else None
        work = torch.empty(n_work, dtype=torch.uint8, device=dev) if n_work else None
    _check(lib().sla_linrec_forward(ctypes.byref(q), *px, *pg, p0, _raw(h), pl, _raw(saved),
                                    _raw(work), n_work, raw))
    if used is not None:
        _record(used, x, gate, h0, offsets, given)
    if given is not None:
        _written(given)
    return h, h_last, saved


def sla_linrec_backward(x: torch.Tensor, gate: torch.Tensor, saved: torch.Tensor,
                        grad_h: Optional[torch.Tensor],
                        grad_last: Optional[torch.Tensor] = None,
                        h0: Optional[torch.Tensor] = None,
                        offsets: Optional[torch.Tensor] = None, mode: str = "sigmoid",
                        stream=None):
    """Gradients (of x, of gate, of h0 or None) from those of h and h_last
    (None: zero); the other arguments are the forward call's, and `stream` is
    taken as there."""
    q, sdt = _linrec_shape(x, gate, offsets, mode)
    px, pg = _steps_in(x, "x", x), _steps_in(gate, "gate", x)
    pd = _steps_in(grad_h, "grad_h", x)
    p0, pl = _states(h0, "h0", q, sdt), _states(grad_last, "grad_last", q, sdt)
    dev = _device_of((("x", x), ("gate", gate), ("saved", saved), ("grad_h", grad_h),
                      ("grad_last", grad_last), ("h0", h0), ("offsets", offsets)))
    n_saved, n_work = _linrec_sizes(q)
    if saved.dtype != sdt or not saved.is_contiguous() or \
            saved.numel() * sdt.itemsize != n_saved:
        raise ValueError("saved must be the forward call's")
    raw, ctx, used = _enter(dev, stream)
    with ctx:
        dx, dg = _like(x), _like(x)
        dh0 = _like(h0) if h0 is not None else None
        work = torch.empty(n_work, dtype=torch.uint8, device=dev) if n_work else None
    _check(lib().sla_linrec_backward(ctypes.byref(q), *px, *pg, p0, _raw(saved), *pd, pl,
                                     _raw(dx), _raw(dg), _raw(dh0), _raw(work), n_work, raw))
    if used is not None:
        _record(used, x, gate, saved, grad_h, grad_last, h0, offsets)
    return dx, dg, dh0


class Adamw:
    """A handle of the AdamW step; keeps what it borrows alive.  `state` holds
    the states as bytes (see include/sla.h for the layout): copy it to save a
    run, copy it back to resume."""

    def __init__(self, handle, params, copies, grad_dtypes, state_bits, state, table, padded):
        self.handle = handle
        self.params, self.copies, self.grad_dtypes = params, copies, grad_dtypes
        self.state_bits, self.state, self._table, self.padded = state_bits, state, table, padded
        self.starts, at = [], 0
        for p in params:
            self.starts.append(at)
            at += -(-p.numel() // 256) * 256
        self._want = [(p.numel(), dt) for p, dt in zip(params, grad_dtypes)]
        self._ptrs = (ctypes.c_void_p * max(len(params), 1))()
        self._streams = set()  # on which what the handle holds is known to be used
        self._writes = [state, *params, *(c for c in copies if c is not None)]

    @property
    def device(self):
        return self.state.device

    def _use(self, raw, used, stream):
        """Record what the handle holds on a stream that is not in _streams yet."""
        if stream is None:
            used = torch.cuda.current_stream()
            used = None if isinstance(used, torch.cuda.ExternalStream) else used
        if used is not None:
            _record(used, *self._writes, self._table)
            self._streams.add(raw)

    def views(self, flat: torch.Tensor):
        """The parts of a padded array that belong to each parameter, in its shape."""
        return [flat[a:a + p.numel()].view(p.shape) for a, p in zip(self.starts, self.params)]

    def destroy(self):
        if self.handle:
            lib().sla_adamw_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def _adamw_list(params, grad_dtype, copies):
    n = len(params)
    gd = list(grad_dtype) if isinstance(grad_dtype, (list, tuple)) else \
        [grad_dtype or p.dtype for p in params]
    copies = list(copies) if copies is not None else [None] * n
    if len(gd) != n or len(copies) != n:
        raise ValueError("grad_dtype and copies must have one entry per parameter")
    ts = (AdamwTensor * max(n, 1))()
    for i, (p, g, c) in enumerate(zip(params, gd, copies)):
        if p.dtype not in _DTYPES or g not in _DTYPES:
            raise ValueError(f"unsupported dtypes {p.dtype}, {g}")
        if not p.is_contiguous():
            raise ValueError(f"parameter {i} must be contiguous")
        if c is not None and (c.dtype != torch.bfloat16 or not c.is_contiguous()
                              or tuple(c.shape) != tuple(p.shape)):
            raise ValueError(f"copy {i} must be a contiguous bfloat16 tensor of its "
                             "parameter's shape")
        ts[i] = AdamwTensor(p.data_ptr(), None if c is None else c.data_ptr(), p.numel(),
                            _DTYPES[p.dtype], _DTYPES[g])
    return ts, gd, copies


def sla_adamw_sizes(params, state_bits: int = 32, grad_dtype=None, copies=None):
    """(state bytes, table bytes, padded elements) of a handle for `params`."""
    params = list(params)
    return _adamw_sizes(_adamw_list(params, grad_dtype, copies)[0], len(params), state_bits)


def _adamw_sizes(ts, n, state_bits):
    sb, tb, padded = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_int64()
    _check(lib().sla_adamw_sizes(ts, n, int(state_bits), ctypes.byref(sb), ctypes.byref(tb),
                                 ctypes.byref(padded)))
    return sb.value, tb.value, padded.value


def sla_adamw_create(params, state_bits: int = 32, grad_dtype=None, copies=None,
                     stream=None) -> Adamw:
    """A handle that steps all of `params` (float64, float32 or bfloat16, in
    place) with zero states of 32 or 8 bits.  grad_dtype: one dtype or one per
    parameter (default: the parameter's; bfloat16 is taken for float32
    parameters too).  copies: per parameter None or a bfloat16 tensor that
    each step rewrites from a float32 parameter."""
    params = [p.detach() for p in params]
    ts, gd, copies = _adamw_list(params, grad_dtype, copies)
    sb, tb, padded = _adamw_sizes(ts, len(params), state_bits)
    dev = _device_of([("a parameter", p) for p in params] + [("a copy", c) for c in copies])
    if dev is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    raw, ctx, _ = _enter(dev, stream)
    with ctx:
        state = torch.zeros(sb, dtype=torch.uint8, device=dev)
        table = torch.empty(tb, dtype=torch.uint8, device=dev)
    h = ctypes.c_void_p()
    _check(lib().sla_adamw_create(ctypes.byref(h), ts, len(params), int(state_bits), _raw(state),
                                  sb, _raw(table), tb, raw))
    opt = Adamw(h, params, copies, gd, int(state_bits), state, table, padded)
    if stream is None:
        opt._streams.add(raw)
    return opt


def sla_adamw_destroy(opt: Adamw) -> None:
    opt.destroy()


def sla_adamw_step(opt: Adamw, grads, step: int, lr: float, beta1: float = 0.9,
                   beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
                   grad_scale: Optional[torch.Tensor] = None, seed: int = 0, stream=None) -> None:
    """One step (number `step`, from 1) of every parameter from its gradient
    (None leaves a parameter and its states alone; of parameters that share
    memory, tied weights given twice, one at most can have one).  grad_scale: a float32
    device number that multiplies the gradients; one that is not finite makes
    the step change nothing.  seed: of the stochastic rounding.  stream: as in
    sla_linrec_forward; the handle, too, is kept until a raw stream is done."""
    if len(grads) != len(opt.params):
        raise ValueError(f"{len(grads)} gradients for {len(opt.params)} parameters")
    dev, ptrs, writes, missing = opt.device, opt._ptrs, opt._writes, False
    on, at = dev.index, []
    for g, (n, dt) in zip(grads, opt._want):
        if g is None:
            at.append(None)
            missing = True
            continue
        if g.dtype is not dt or g.numel() != n or g.get_device() != on or not g.is_contiguous():
            raise ValueError(f"gradient {len(at)} must be a contiguous {dt} tensor of {n} "
                             f"elements on {dev}")
        at.append(g.data_ptr())
    ptrs[:len(at)] = at
    if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1
                                   or grad_scale.device != dev):
        raise ValueError("grad_scale must be one float32 number on the parameters' device")
    hyper = AdamwHyper(lr, beta1, beta2, eps, weight_decay, step, seed & 0xFFFFFFFFFFFFFFFF)
    raw, _, used = _enter(dev, stream)
    _check(lib().sla_adamw_step(opt.handle, ptrs, ctypes.byref(hyper), _raw(grad_scale), raw))
    if raw not in opt._streams:
        opt._use(raw, used, stream)
    if used is not None:
        _record(used, *grads, grad_scale)
    if missing:
        own = [t for g, *t in zip(grads, opt.params, opt.copies) if g is not None]
        writes = [opt.state, *(t for ts in own for t in ts if t is not None)]
    _written(writes)


def sla_adamw_get_state(opt: Adamw, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The values of m and v over the padded elements (see Adamw.views): the
    handle's own buffers for 32-bit states, bfloat16 arrays (exact) for 8-bit."""
    if opt.state_bits == 32:
        f = opt.state.view(torch.float32)
        return f[:opt.padded], f[opt.padded:]
    raw, ctx, used = _enter(opt.device, stream)
    with ctx:
        m = torch.empty(opt.padded, dtype=torch.bfloat16, device=opt.device)
        v = torch.empty(opt.padded, dtype=torch.bfloat16, device=opt.device)
    _check(lib().sla_adamw_get_state(opt.handle, _raw(m), _raw(v), raw))
    if raw not in opt._streams:
        opt._use(raw, used, stream)
    return m, v


def sla_adamw_set_state(opt: Adamw, m: torch.Tensor, v: torch.Tensor, stream=None) -> None:
    """Set the states from float32 values over the padded elements (zeros in
    the padding); 8-bit states take the nearest level."""
    for name, t in (("m", m), ("v", v)):
        if t.dtype != torch.float32 or t.numel() != opt.padded or not t.is_contiguous() \
                or t.device != opt.device:
            raise ValueError(f"{name} must be a contiguous float32 tensor of {opt.padded} "
                             f"elements on {opt.device}")
    raw, _, used = _enter(opt.device, stream)
    _check(lib().sla_adamw_set_state(opt.handle, _raw(m), _raw(v), raw))
    if raw not in opt._streams:
        opt._use(raw, used, stream)
    if used is not None:
        _record(used, m, v)
    _written(opt.state)


# ----- operators of a sequence block: convolution, selective scan, norms -----

_ACTS = {"none": SLA_ACT_NONE, "silu": SLA_ACT_SILU}
_ORDERS = {"gate_first": SLA_GATE_FIRST, "norm_first": SLA_NORM_FIRST}


def _sequences(x, offsets, name: str = "x"):
    """(sequences, steps, channels) of a dense or a packed tensor."""
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if offsets is None:
        if x.dim() != 3:
            raise ValueError(f"{name} must be (sequences, steps, channels), or give offsets")
        return tuple(x.shape)
    if x.dim() != 2:
        raise ValueError(f"packed {name} must be (steps, channels)")
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 1 \
            or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int64 vector of sequences + 1 entries")
    return (offsets.numel() - 1, *x.shape)


def _param_dtype(x) -> torch.dtype:
    return torch.float64 if x.dtype == torch.float64 else torch.float32


def _dense(t, name: str, shape, dtype) -> Optional[int]:
    """Pointer of an optional contiguous tensor of a given shape and dtype."""
    if t is None:
        return None
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor of {dtype}")
    return t.data_ptr()


def _scratch(n: int, dev):
    return torch.empty(n, dtype=torch.uint8, device=dev) if n else None


def _conv_shape(x, weight, offsets, act) -> ConvShape:
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    n, t, d = _sequences(x, offsets)
    if weight.dim() != 2 or weight.shape[0] != d:
        raise ValueError("weight must be (channels, taps)")
    return ConvShape(n, t, d, weight.shape[1], None if offsets is None else offsets.data_ptr(),
                     _DTYPES[x.dtype], _ACTS[act])


def _conv_sizes(q: ConvShape) -> int:
    work = ctypes.c_size_t()
    _check(lib().sla_conv_sizes(ctypes.byref(q), ctypes.byref(work)))
    return work.value


def _clear_rows(q, y, raw):
    _check(lib().sla_rows_clear(q.d_offsets, q.n_seq, q.steps, q.dim, q.dtype, _raw(y), raw))


def sla_rows_clear(y: torch.Tensor, offsets: torch.Tensor, stream=None) -> None:
    """Zeros in the rows of a packed, dense y (steps, channels) that are of no sequence:
    before the first offset and behind the last."""
    if offsets is None:
        raise ValueError("offsets must be given")
    n, t, d = _sequences(y, offsets)
    if not y.is_contiguous():
        raise ValueError("y must be dense")
    dev = _device_of((("y", y), ("offsets", offsets)))
    raw, ctx, used = _enter(dev, stream)
    _check(lib().sla_rows_clear(offsets.data_ptr(), n, t, d, _DTYPES[y.dtype], _raw(y), raw))
    if used is not None:
        _record(used, y, offsets)
    _written(y)


def sla_conv_sizes(x, weight, offsets=None, act: str = "silu") -> int:
    """Bytes of the backward pass's workspace."""
    return _conv_sizes(_conv_shape(x, weight, offsets, act))


def sla_conv_forward(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                     state: Optional[torch.Tensor] = None,
                     offsets: Optional[torch.Tensor] = None, act: str = "silu",
                     last: Optional[torch.Tensor] = None, stream=None):
    """y_t = act(bias + sum_k weight[:, k] x_{t - taps + 1 + k}) along each sequence, per
    channel, with 2 to 4 taps and act "silu" or "none".

    x as in sla_linrec_forward, strided or packed; weight (channels, taps) and bias
    (channels) float32 (float64 for float64).  state (sequences, taps - 1, channels), of
    x's dtype: the inputs before each sequence, oldest first (None: zeros); last, of the same
    form, receives what follows needs, and may be state itself.  Packed rows before the first
    offset or behind the last count as nothing and give zeros.  `stream` as in
    sla_linrec_forward.  Returns (y, last)."""
    q = _conv_shape(x, weight, offsets, act)
    pt = _param_dtype(x)
    held = (q.n_seq, q.width - 1, q.dim)
    px = _steps_in(x, "x", x)
    pw, pb = _dense(weight, "weight", (q.dim, q.width), pt), _dense(bias, "bias", (q.dim,), pt)
    ps, pl = _dense(state, "state", held, x.dtype), _dense(last, "last", held, x.dtype)
    dev = _device_of((("x", x), ("weight", weight), ("bias", bias), ("state", state),
                      ("offsets", offsets), ("last", last)))
    raw, ctx, used = _enter(dev, stream)
    given = last
    with ctx:
        y = _like(x)
        if last is None:
            last = torch.empty(held, dtype=x.dtype, device=dev)
            pl = _raw(last)
    if offsets is not None:
        _clear_rows(q, y, raw)
    _check(lib().sla_conv_forward(ctypes.byref(q), *px, pw, pb, ps, _raw(y), pl, raw))
    if used is not None:
        _record(used, x, weight, bias, state, offsets, given)
    if given is not None:
        _written(given)
    return y, last


def sla_conv_backward(x: torch.Tensor, weight: torch.Tensor, grad_y: Optional[torch.Tensor],
                      bias: Optional[torch.Tensor] = None, state: Optional[torch.Tensor] = None,
                      grad_last: Optional[torch.Tensor] = None,
                      offsets: Optional[torch.Tensor] = None, act: str = "silu", stream=None):
    """Gradients (of x, weight, bias or None, state or None) from those of y and last
    (None: zero); the other arguments are the forward call's."""
    q = _conv_shape(x, weight, offsets, act)
    pt = _param_dtype(x)
    held = (q.n_seq, q.width - 1, q.dim)
    px, pd = _steps_in(x, "x", x), _steps_in(grad_y, "grad_y", x)
    pw, pb = _dense(weight, "weight", (q.dim, q.width), pt), _dense(bias, "bias", (q.dim,), pt)
    ps, pl = _dense(state, "state", held, x.dtype), _dense(grad_last, "grad_last", held, x.dtype)
    dev = _device_of((("x", x), ("weight", weight), ("grad_y", grad_y), ("bias", bias),
                      ("state", state), ("grad_last", grad_last), ("offsets", offsets)))
    n_work = _conv_sizes(q)
    raw, ctx, used = _enter(dev, stream)
    with ctx:
        dx, dw = _like(x), _like(weight)
        db = _like(bias) if bias is not None else None
        dstate = _like(state) if state is not None else None
        work = _scratch(n_work, dev)
    _check(lib().sla_conv_backward(ctypes.byref(q), *px, pw, pb, ps, *pd, pl, _raw(dx), _raw(dw),
                                   _raw(db), _raw(dstate), _raw(work), n_work, raw))
    if used is not None:
        _record(used, x, weight, grad_y, bias, state, grad_last, offsets)
    return dx, dw, db, dstate


def _shared_in(t, name: str, x, q):
    """(pointer, sequence stride, step stride) of B or C."""
    want = (*x.shape[:-1], q.groups, q.n_state)
    if tuple(t.shape) != want or t.dtype != x.dtype:
        raise ValueError(f"{name} must be {want} of x's dtype")
    st = t.stride()
    if t.numel() and (t.shape[-1] > 1 and st[-1] != 1 or
                      t.shape[-2] > 1 and st[-2] != t.shape[-1]):
        raise ValueError(f"{name}'s groups and states must be adjacent")
    return t.data_ptr(), (st[0] if len(st) == 4 else 0), st[-3]


class _Selscan:
    """The checked arguments of a selective scan."""
    __slots__ = ("q", "pt", "held", "given", "tensors")

    def __init__(self, x, dt, A, B, C, D, z, dt_bias, h0, offsets, softplus):
        n, t, d = _sequences(x, offsets)
        if B.dim() != x.dim() + 1 or A.dim() != 2:
            raise ValueError("B and C must be (.., groups, states), A (channels, states)")
        self.q = q = SelscanShape(n, t, d, B.shape[-1], B.shape[-2],
                                  None if offsets is None else offsets.data_ptr(),
                                  _DTYPES[x.dtype], 1 if softplus else 0)
        self.pt = pt = _param_dtype(x)
        px, pu, pz = _steps_in(x, "x", x), _steps_in(dt, "dt", x), _steps_in(z, "z", x)
        pb, pc = _shared_in(B, "B", x, q), _shared_in(C, "C", x, q)
        self.held = (n, d, q.n_state)
        self.given = SelscanIn(
            px[0], pu[0], pz[0], pb[0], pc[0], *px[1:], *pu[1:], *pz[1:], *pb[1:], *pc[1:],
            _dense(A, "A", (d, q.n_state), pt), _dense(D, "D", (d,), pt),
            _dense(dt_bias, "dt_bias", (d,), pt), _dense(h0, "h0", self.held, pt))
        self.tensors = (x, dt, A, B, C, D, z, dt_bias, h0, offsets)

    def device(self, *more):
        return _device_of((*zip(_Selscan.NAMES, self.tensors), *more))

    def sizes(self):
        s, f, b = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
        _check(lib().sla_selscan_sizes(ctypes.byref(self.q), ctypes.byref(s), ctypes.byref(f),
                                       ctypes.byref(b)))
        return s.value, f.value, b.value


_Selscan.NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0", "offsets")


def sla_selscan_sizes(x, dt, A, B, C, D=None, z=None, dt_bias=None, h0=None, offsets=None,
                      softplus: bool = True) -> Tuple[int, int, int]:
    """Bytes of (the states kept for the backward pass, the forward pass's workspace, the
    backward pass's)."""
    return _Selscan(x, dt, A, B, C, D, z, dt_bias, h0, offsets, softplus).sizes()


def sla_selscan_forward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                        C: torch.Tensor, D: Optional[torch.Tensor] = None,
                        z: Optional[torch.Tensor] = None,
                        dt_bias: Optional[torch.Tensor] = None,
                        h0: Optional[torch.Tensor] = None,
                        offsets: Optional[torch.Tensor] = None, softplus: bool = True,
                        save: bool = False, h_last: Optional[torch.Tensor] = None, stream=None):
    """A selective scan along each sequence: with delta = softplus(dt + dt_bias) (or
    dt + dt_bias), per channel and state
        h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,
    and y_t = (C_t . h_t + D x_t) silu(z_t), without the last factor if z is None.

    x, dt, z as x in sla_linrec_forward, strided or packed; B and C (.., groups, states) of
    x's dtype, at most 16 states, channels in equal groups of neighbours; A (channels,
    states), D and dt_bias (channels) and the states h0, h_last (sequences, channels,
    states) float32 (float64 for float64).  h_last may be given to be overwritten, for dense
    sequences h0 itself.  Packed rows before the first offset or behind the last count as
    nothing and give zeros.  `stream` as in sla_linrec_forward.  Returns (y, h_last, saved);
    `saved` (None unless save) is what the backward pass needs."""
    a = _Selscan(x, dt, A, B, C, D, z, dt_bias, h0, offsets, softplus)
    pl = _dense(h_last, "h_last", a.held, a.pt)
    dev = a.device(("h_last", h_last))
    # a step or two need neither
    n_saved, n_work, _ = a.sizes() if save or a.q.steps > 2 else (0, 0, 0)
    raw, ctx, used = _enter(dev, stream)
    given = h_last
    with ctx:
        y = _like(x)
        if h_last is None:
            h_last = torch.empty(a.held, dtype=a.pt, device=dev)
            pl = _raw(h_last)
        saved = torch.empty(n_saved // a.pt.itemsize, dtype=a.pt, device=dev) if save else None
        work = _scratch(n_work, dev)
    if offsets is not None:
        _clear_rows(a.q, y, raw)
    _check(lib().sla_selscan_forward(ctypes.byref(a.q), ctypes.byref(a.given), _raw(y), pl,
                                     _raw(saved), _raw(work), n_work, raw))
    if used is not None:
        _record(used, *a.tensors, given)
    if given is not None:
        _written(given)
    return y, h_last, saved


def sla_selscan_backward(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                         C: torch.Tensor, saved: torch.Tensor, grad_y: torch.Tensor,
                         grad_last: Optional[torch.Tensor] = None,
                         D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                         dt_bias: Optional[torch.Tensor] = None,
                         h0: Optional[torch.Tensor] = None,
                         offsets: Optional[torch.Tensor] = None, softplus: bool = True,
                         stream=None):
    """Gradients of (x, dt, A, B, C, D, z, dt_bias, h0), None for those not given, from
    those of y and of h_last (None: zero); the other arguments are the forward call's."""
    a = _Selscan(x, dt, A, B, C, D, z, dt_bias, h0, offsets, softplus)
    pd = _steps_in(grad_y, "grad_y", x)
    pl = _dense(grad_last, "grad_last", a.held, a.pt)
    dev = a.device(("saved", saved), ("grad_y", grad_y), ("grad_last", grad_last))
    n_saved, _, n_work = a.sizes()
    if saved.dtype != a.pt or not saved.is_contiguous() or \
            saved.numel() * a.pt.itemsize != n_saved:
        raise ValueError("saved must be the forward call's")
    raw, ctx, used = _enter(dev, stream)
    with ctx:
        out = [None if t is None else _like(t) for t in (x, dt, A, B, C, D, z, dt_bias, h0)]
        work = _scratch(n_work, dev)
    dx, ddt, dA, dB, dC, dD, dz, dbias, dh0 = (_raw(t) for t in out)
    grads = SelscanGrads(dx, ddt, dz, dB, dC, dA, dD, dbias, dh0)
    _check(lib().sla_selscan_backward(ctypes.byref(a.q), ctypes.byref(a.given), _raw(saved), *pd,
                                      pl, ctypes.byref(grads), _raw(work), n_work, raw))
    if used is not None:
        _record(used, *a.tensors, saved, grad_y, grad_last)
    return tuple(out)


def _rows_of(t, name: str, dim: int):
    """(pointer, rows, elements from row to row) of a tensor of rows, its last dimension."""
    if t is None:
        return None, 0, 0
    if t.dim() < 1 or t.shape[-1] != dim:
        raise ValueError(f"{name} must have {dim} elements in its last dimension")
    rows = t.numel() // dim if dim else 0
    if t.is_contiguous():
        return t.data_ptr(), rows, dim
    if dim > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}'s elements must be adjacent (last stride 1)")
    step = want = None
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if step is None:
            step = want = s
        elif s != want:
            raise ValueError(f"{name}'s rows must lie evenly spaced")
        want *= n
    return t.data_ptr(), rows, dim if step is None else step


def _norm_shape(x, stream_dtype, eps) -> NormShape:
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    if x.dim() < 1:
        raise ValueError("x must have rows")
    if stream_dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {stream_dtype}")
    d = x.shape[-1]
    return NormShape(x.numel() // d if d else 0, d, _DTYPES[x.dtype], _DTYPES[stream_dtype], eps)


def _norm_sizes(q: NormShape) -> int:
    work = ctypes.c_size_t()
    _check(lib().sla_norm_sizes(ctypes.byref(q), ctypes.byref(work)))
    return work.value


def sla_norm_sizes(x, residual=None) -> int:
    """Bytes of the backward passes' workspace."""
    return _norm_sizes(_norm_shape(x, x.dtype if residual is None else residual.dtype, 0.0))


def _like_x(t, name: str, x, dtype):
    if t is not None and (tuple(t.shape) != tuple(x.shape) or t.dtype != dtype):
        raise ValueError(f"{name} must have x's shape and dtype {dtype}")
    return t


def sla_norm_in_forward(x: torch.Tensor, weight: torch.Tensor,
                        residual: Optional[torch.Tensor] = None,
                        scale: Optional[torch.Tensor] = None, eps: float = 1e-5, stream=None):
    """The norm before a block: r = residual + scale x (without residual: scale x; without
    both: x itself), y = weight r / sqrt(mean(r^2) + eps) along the last dimension.

    weight and scale: (dim) float32 (float64 for float64); residual has x's dtype or, where
    that has 16 bits, float32, and r has the same.  x and residual may be slices of wider
    tensors whose rows lie evenly spaced.  `stream` as in sla_linrec_forward.  Returns (y, r,
    rstd); rstd is what the backward pass needs."""
    _like_x(residual, "residual", x, x.dtype if residual is None else residual.dtype)
    rt = x.dtype if residual is None else residual.dtype
    q = _norm_shape(x, rt, eps)
    pt = _param_dtype(x)
    px, pr = _rows_of(x, "x", q.dim), _rows_of(residual, "residual", q.dim)
    pw, ps = _dense(weight, "weight", (q.dim,), pt), _dense(scale, "scale", (q.dim,), pt)
    dev = _device_of((("x", x), ("weight", weight), ("residual", residual), ("scale", scale)))
    raw, ctx, used = _enter(dev, stream)
    same = residual is None and scale is None
    with ctx:
        y = _like(x)
        r = x if same else torch.empty(x.shape, dtype=rt, device=dev)
        rstd = torch.empty(x.shape[:-1], dtype=pt, device=dev)
    _check(lib().sla_norm_in_forward(ctypes.byref(q), px[0], px[2], pr[0], pr[2], ps, pw, _raw(y),
                                     None if same else _raw(r), _raw(rstd), raw))
    if used is not None:
        _record(used, x, weight, residual, scale)
    return y, r, rstd


def sla_norm_in_backward(grad_y: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                         rstd: torch.Tensor, residual: Optional[torch.Tensor] = None,
                         scale: Optional[torch.Tensor] = None,
                         grad_r: Optional[torch.Tensor] = None, stream=None):
    """Gradients of (x, residual, weight, scale or None) from those of y and r (None: zero);
    the other arguments are the forward call's.  The residual's gradient is that of r by
    both uses; where that of x is the same (no scale, one dtype) they are one tensor."""
    _like_x(residual, "residual", x, x.dtype if residual is None else residual.dtype)
    rt = x.dtype if residual is None else residual.dtype
    q = _norm_shape(x, rt, 0.0)
    pt = _param_dtype(x)
    px, pr = _rows_of(x, "x", q.dim), _rows_of(residual, "residual", q.dim)
    pw, ps = _dense(weight, "weight", (q.dim,), pt), _dense(scale, "scale", (q.dim,), pt)
    py, pg = _dense(grad_y, "grad_y", x.shape, x.dtype), _dense(grad_r, "grad_r", x.shape, rt)
    pd = _dense(rstd, "rstd", x.shape[:-1], pt)
    dev = _device_of((("grad_y", grad_y), ("x", x), ("weight", weight), ("rstd", rstd),
                      ("residual", residual), ("scale", scale), ("grad_r", grad_r)))
    n_work = _norm_sizes(q)
    raw, ctx, used = _enter(dev, stream)
    apart = scale is not None or rt != x.dtype
    with ctx:
        dx, dw = _like(x), _like(weight)
        dres = torch.empty(x.shape, dtype=rt, device=dev) if apart else dx
        dscale = _like(scale) if scale is not None else None
        work = _scratch(n_work, dev)
    _check(lib().sla_norm_in_backward(ctypes.byref(q), py, pg, px[0], px[2], pr[0], pr[2], ps, pw,
                                      pd, _raw(dx), _raw(dres) if apart else None, _raw(dw),
                                      _raw(dscale), _raw(work), n_work, raw))
    if used is not None:
        _record(used, grad_y, x, weight, rstd, residual, scale, grad_r)
    return dx, dres, dw, dscale


def sla_norm_out_forward(x: torch.Tensor, weight: torch.Tensor,
                         gate: Optional[torch.Tensor] = None,
                         residual: Optional[torch.Tensor] = None,
                         scale: Optional[torch.Tensor] = None, order: str = "gate_first",
                         eps: float = 1e-5, stream=None):
    """The norm after a block with its gate: n = weight u / sqrt(mean(u^2) + eps) with
    u = x silu(gate) ("gate_first"), or that of x, times silu(gate) ("norm_first"); out =
    residual + scale n.  gate, residual and scale are optional; gate has x's dtype,
    residual, scale, weight and `stream` are as in sla_norm_in_forward, and out has the
    residual's dtype (else x's).  Returns (out, rstd)."""
    if order not in _ORDERS:
        raise ValueError(f"order must be one of {sorted(_ORDERS)}, got {order!r}")
    _like_x(gate, "gate", x, x.dtype)
    _like_x(residual, "residual", x, x.dtype if residual is None else residual.dtype)
    rt = x.dtype if residual is None else residual.dtype
    q = _norm_shape(x, rt, eps)
    pt = _param_dtype(x)
    px, pg = _rows_of(x, "x", q.dim), _rows_of(gate, "gate", q.dim)
    pr = _rows_of(residual, "residual", q.dim)
    pw, ps = _dense(weight, "weight", (q.dim,), pt), _dense(scale, "scale", (q.dim,), pt)
    dev = _device_of((("x", x), ("weight", weight), ("gate", gate), ("residual", residual),
                      ("scale", scale)))
    raw, ctx, used = _enter(dev, stream)
    with ctx:
        out = torch.empty(x.shape, dtype=rt, device=dev)
        rstd = torch.empty(x.shape[:-1], dtype=pt, device=dev)
    _check(lib().sla_norm_out_forward(ctypes.byref(q), _ORDERS[order], px[0], px[2], pg[0], pg[2],
                                      pr[0], pr[2], ps, pw, _raw(out), _raw(rstd), raw))
    if used is not None:
        _record(used, x, weight, gate, residual, scale)
    return out, rstd


def sla_norm_out_backward(grad_out: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                          rstd: torch.Tensor, gate: Optional[torch.Tensor] = None,
                          scale: Optional[torch.Tensor] = None, order: str = "gate_first",
                          stream=None):
    """Gradients of (x, gate or None, weight, scale or None) from that of out, which is the
    residual's as it stands; the other arguments are the forward call's."""
    if order not in _ORDERS:
        raise ValueError(f"order must be one of {sorted(_ORDERS)}, got {order!r}")
    _like_x(gate, "gate", x, x.dtype)
    q = _norm_shape(x, grad_out.dtype, 0.0)
    pt = _param_dtype(x)
    px, pg = _rows_of(x, "x", q.dim), _rows_of(gate, "gate", q.dim)
    pw, ps = _dense(weight, "weight", (q.dim,), pt), _dense(scale, "scale", (q.dim,), pt)
    po = _dense(grad_out, "grad_out", x.shape, grad_out.dtype)
    pd = _dense(rstd, "rstd", x.shape[:-1], pt)
    dev = _device_of((("grad_out", grad_out), ("x", x), ("weight", weight), ("rstd", rstd),
                      ("gate", gate), ("scale", scale)))
    n_work = _norm_sizes(q)
    raw, ctx, used = _enter(dev, stream)
    with ctx:
        dx, dw = _like(x), _like(weight)
        dgate = _like(gate) if gate is not None else None
        dscale = _like(scale) if scale is not None else None
        work = _scratch(n_work, dev)
    _check(lib().sla_norm_out_backward(ctypes.byref(q), _ORDERS[order], po, px[0], px[2], pg[0],
                                       pg[2], ps, pw, pd, _raw(dx), _raw(dgate), _raw(dw),
                                       _raw(dscale), _raw(work), n_work, raw))
    if used is not None:
        _record(used, grad_out, x, weight, rstd, gate, scale)
    return dx, dgate, dw, dscale
