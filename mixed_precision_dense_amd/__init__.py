"""Python binding of ``libmpgemm.so`` (declared in ``include/mpgemm.h``).

Argument marshalling only: every step of D = alpha * op(A) * op(B) + beta * C runs in the HIP
kernels of the library.  PyTorch provides device memory and streams (a tensor argument is
passed as its ``data_ptr()``; a missing stream means torch's current stream).  There is no
CPU fallback: if the library is not built, importing works but every call raises.

The names follow the C ABI: ``mpgemm_create``, ``mpgemm_run``, ``mpgemm_destroy``,
``mpgemm_check``, ``mpgemm_status_string`` and ``mpgemm_tile_shape``; ``Handle`` is a small
owner of one handle.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Union

import torch  # noqa: F401  (loads the HIP runtime the library binds to)

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmpgemm.so")

OP_N, OP_T = 0, 1
R_16F, R_16BF, R_8I, R_32F, R_32I, R_8F_E4M3, R_8F_E5M2 = 0, 1, 2, 3, 4, 5, 6
DTYPES = {"f16": R_16F, "bf16": R_16BF, "i8": R_8I, "f32": R_32F, "i32": R_32I,
          "e4m3": R_8F_E4M3, "e5m2": R_8F_E5M2}
STATUS = {0: "SUCCESS", 1: "NOT_INITIALIZED", 2: "INVALID_VALUE", 3: "NOT_SUPPORTED",
          4: "ALLOC_FAILED", 5: "NO_DEVICE", 6: "LAUNCH_FAILED", 7: "INTERNAL_ERROR",
          8: "WRONG_DEVICE", 9: "SCRATCH_TOO_SMALL"}
SUCCESS = 0
NOALLOC_SCRATCH_BYTES = 64 << 20   # MPGEMM_NOALLOC_SCRATCH_BYTES
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}   # mpgemm_act_t

_lib: Optional[ctypes.CDLL] = None


class MpgemmError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status_string(status)})")


_i64, _i32, _u64, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p
# (restype, argtypes) of every function include/mpgemm.h declares
SIGNATURES = {
    "mpgemm_create": (_i32, [ctypes.POINTER(_vp)]),
    "mpgemm_destroy": (_i32, [_vp]),
    "mpgemm_run": (_i32, [_vp, _i32, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i32,
                          _i64, _vp, _vp, _i32, _i64, _vp, _i32, _vp]),
    "mpgemm_check": (_i32, [_i32, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i32, _i64,
                            _vp, _vp, _i32, _i64, _vp, _i32]),
    "mpgemm_status_string": (ctypes.c_char_p, [_i32]),
    "mpgemm_tile_shape": (_i32, [_i64, _i64, _i32, ctypes.POINTER(_i32), ctypes.POINTER(_i32)]),
    "mpgemm_run_sp24": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i64, _vp,
                               _i32, _i64, _vp, _vp, _i32, _i64, _vp, _i32, _vp]),
    "mpgemm_check_sp24": (_i32, [_i32, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i64, _vp,
                                 _i32, _i64, _vp, _vp, _i32, _i64, _vp, _i32]),
    "mpgemm_run_bf16x3": (_i32, [_vp, _i32, _i32, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64,
                                 _vp, _vp, _i64, _vp, _vp, _u64, _vp]),
    "mpgemm_run_bf16x3_noalloc": (_i32, [_vp, _i32, _i32, _i64, _i64, _i64, _vp, _vp, _i64, _vp,
                                         _i64, _vp, _vp, _i64, _vp, _vp]),
    "mpgemm_check_bf16x3": (_i32, [_i32, _i32, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp,
                                   _vp, _i64, _vp, _vp, _u64]),
    "mpgemm_bf16x3_workspace_size": (_u64, [_i32, _i32, _i64, _i64, _i64]),
    "mpgemm_epilogue_grad_workspace_size": (_u64, [_i64, _i64, _i64]),
    "mpgemm_linear_ce_workspace_size": (_u64, [_i64, _i64, _i64, _i32, _i32]),
}
# Arguments of the products of language models: the check's, and the run's with the handle before
# and the stream after them.
_OPS = {
    "epilogue": [_i32, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _vp,
                 _i32, _i64, _vp, _i32, _i64],
    "epilogue_grad": [_i32, _i32, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i32, _i64, _i32, _vp,
                      _i64, _vp, _i32, _i64, _vp, _vp, _u64],
    "grouped": [_i32, _i64, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _vp, _i32, _i64, _i64, _vp,
                _vp, _i32, _i64],
    "grouped_grad": [_i32, _i64, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _vp, _i32, _i64, _i64,
                     _i32, _vp, _i64, _vp, _i32, _i64, _vp, _vp, _u64],
    "grouped_wgrad": [_i64, _i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _vp,
                      _i32, _i64, _i64],
    "linear_ce": [_i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _u64],
    "linear_ce_grad": [_i64, _i64, _i64, _vp, _vp, _i32, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64,
                       _vp, _i64, _vp, _u64],
}
for _name, _args in _OPS.items():
    SIGNATURES["mpgemm_run_" + _name] = (_i32, [_vp, *_args, _vp])
    SIGNATURES["mpgemm_check_" + _name] = (_i32, _args)


def declare(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Set the C signature of every ABI function the loaded library exports."""
    for name, (res, args) in SIGNATURES.items():
        if hasattr(lib, name):
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
    return lib


def load() -> ctypes.CDLL:
    """Load the built library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run mixed_precision_dense_amd/build.py "
                               "(or __graft_entry__.build())")
        _lib = declare(ctypes.CDLL(LIB_PATH))
    return _lib


# ----------------------------------------------------------------------------- marshalling
def _dtype(t: Union[str, int]) -> int:
    return DTYPES[t] if isinstance(t, str) else int(t)


def _op(t: Union[bool, int, str]) -> int:
    if isinstance(t, str):
        if t.upper() not in ("N", "T"):
            raise ValueError(f"transpose flag {t!r}: expected 'N' or 'T'")
        return OP_T if t.upper() == "T" else OP_N
    return OP_T if t else OP_N


def _ptr(x) -> Optional[int]:
    """Device address of a tensor (which must live on a GPU), or an integer address as is."""
    if x is None:
        return None
    if isinstance(x, torch.Tensor):
        if not x.is_cuda:
            raise ValueError(f"tensor on {x.device}: the kernels read and write device memory")
        return x.data_ptr()
    return int(x)


def _scalar(v, compute_type: int):
    """alpha / beta as the compute type's host scalar (float or int32_t)."""
    if compute_type == R_32I:
        if not -(1 << 31) <= int(v) < (1 << 31):
            raise ValueError(f"integer scalar {v} does not fit in int32")
        return ctypes.c_int32(int(v))
    return ctypes.c_float(float(v))


# torch's current stream as an address, without the stream object that torch.cuda.current_stream()
# makes on every call (2.8 us against 0.3, in calls of about 8 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ----------------------------------------------------------------------------- C ABI
def status_string(status: int) -> str:
    return load().mpgemm_status_string(int(status)).decode()


mpgemm_status_string = status_string


def mpgemm_create() -> int:
    h = ctypes.c_void_p()
    st = load().mpgemm_create(ctypes.byref(h))
    if st != SUCCESS:
        raise MpgemmError(st, "mpgemm_create")
    return h.value


def mpgemm_destroy(handle: int) -> int:
    return load().mpgemm_destroy(handle)


def mpgemm_run(handle, transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb, beta, C,
               c_type, ldc, D, compute_type, stream=None, check: bool = True) -> int:
    """Queue one GEMM.  Pointers may be ints or tensors; types names or enum values."""
    ct = _dtype(compute_type)
    al, be = _scalar(alpha, ct), _scalar(beta, ct)
    st = load().mpgemm_run(handle, _op(transa), _op(transb), m, n, k, ctypes.byref(al),
                           _ptr(A), _dtype(a_type), lda, _ptr(B), _dtype(b_type), ldb,
                           ctypes.byref(be), _ptr(C), _dtype(c_type), ldc, _ptr(D), ct,
                           _stream(stream))
    if check and st != SUCCESS:
        raise MpgemmError(st, "mpgemm_run")
    return st


def mpgemm_run_bf16x3(handle, transa, transb, m, n, k, alpha, A, lda, B, ldb, beta, C, ldc, D,
                      workspace, workspace_bytes, stream=None, check: bool = True) -> int:
    """Queue the FP32 GEMM computed from BF16 pieces (three products); FP32 A, B, C, D."""
    al, be = ctypes.c_float(float(alpha)), ctypes.c_float(float(beta))
    st = load().mpgemm_run_bf16x3(handle, _op(transa), _op(transb), m, n, k, ctypes.byref(al),
                                  _ptr(A), lda, _ptr(B), ldb, ctypes.byref(be), _ptr(C), ldc,
                                  _ptr(D), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream))
    if check and st != SUCCESS:
        raise MpgemmError(st, "mpgemm_run_bf16x3")
    return st


def mpgemm_run_bf16x3_noalloc(handle, transa, transb, m, n, k, alpha, A, lda, B, ldb, beta, C,
                              ldc, D, stream=None, check: bool = True) -> int:
    """mpgemm_run_bf16x3 with the library's fixed scratch buffer in place of a workspace (no
    allocation; calls that overlap on one device race)."""
    al, be = ctypes.c_float(float(alpha)), ctypes.c_float(float(beta))
    st = load().mpgemm_run_bf16x3_noalloc(handle, _op(transa), _op(transb), m, n, k,
                                          ctypes.byref(al), _ptr(A), lda, _ptr(B), ldb,
                                          ctypes.byref(be), _ptr(C), ldc, _ptr(D),
                                          _stream(stream))
    if check and st != SUCCESS:
        raise MpgemmError(st, "mpgemm_run_bf16x3_noalloc")
    return st


def mpgemm_run_sp24(handle, transb, m, n, k, alpha, Ac, a_type, lda, meta, ld_meta, B, b_type,
                    ldb, beta, C, c_type, ldc, D, compute_type="f32", stream=None,
                    check: bool = True) -> int:
    """Queue the GEMM with a 2:4 structured-sparse A given as kept values Ac and metadata
    (alpha and beta are float for F32 compute, int for I32)."""
    ct = _dtype(compute_type)
    al, be = _scalar(alpha, ct), _scalar(beta, ct)
    st = load().mpgemm_run_sp24(handle, _op(transb), m, n, k, ctypes.byref(al), _ptr(Ac),
                                _dtype(a_type), lda, _ptr(meta), ld_meta, _ptr(B), _dtype(b_type),
                                ldb, ctypes.byref(be), _ptr(C), _dtype(c_type), ldc, _ptr(D),
                                ct, _stream(stream))
    if check and st != SUCCESS:
        raise MpgemmError(st, "mpgemm_run_sp24")
    return st


def mpgemm_check_sp24(transb, m, n, k, alpha, Ac, a_type, lda, meta, ld_meta, B, b_type, ldb,
                      beta, C, c_type, ldc, D, compute_type="f32") -> int:
    """Host-only argument check of mpgemm_run_sp24."""
    ct = _dtype(compute_type)
    al, be = _scalar(alpha, ct), _scalar(beta, ct)
    return load().mpgemm_check_sp24(_op(transb), m, n, k, ctypes.byref(al), _ptr(Ac),
                                    _dtype(a_type), lda, _ptr(meta), ld_meta, _ptr(B),
                                    _dtype(b_type), ldb, ctypes.byref(be), _ptr(C), _dtype(c_type),
                                    ldc, _ptr(D), ct)


def mpgemm_check_bf16x3(transa, transb, m, n, k, alpha, A, lda, B, ldb, beta, C, ldc, D,
                        workspace, workspace_bytes) -> int:
    """Host-only argument check of mpgemm_run_bf16x3 (the workspace included)."""
    al, be = ctypes.c_float(float(alpha)), ctypes.c_float(float(beta))
    return load().mpgemm_check_bf16x3(_op(transa), _op(transb), m, n, k, ctypes.byref(al),
                                      _ptr(A), lda, _ptr(B), ldb, ctypes.byref(be), _ptr(C), ldc,
                                      _ptr(D), _ptr(workspace), int(workspace_bytes))


def mpgemm_bf16x3_workspace_size(transa, transb, m: int, n: int, k: int) -> int:
    """Workspace bytes mpgemm_run_bf16x3 needs (host-only)."""
    return int(load().mpgemm_bf16x3_workspace_size(_op(transa), _op(transb), m, n, k))


def mpgemm_check(transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb, beta, C,
                 c_type, ldc, D, compute_type) -> int:
    """Host-only argument check; returns the status mpgemm_run would return before launching."""
    ct = _dtype(compute_type)
    al, be = _scalar(alpha, ct), _scalar(beta, ct)
    return load().mpgemm_check(_op(transa), _op(transb), m, n, k, ctypes.byref(al), _ptr(A),
                               _dtype(a_type), lda, _ptr(B), _dtype(b_type), ldb,
                               ctypes.byref(be), _ptr(C), _dtype(c_type), ldc, _ptr(D), ct)


def mpgemm_tile_shape(m: int, n: int, a_type="f16") -> tuple:
    tm, tn = ctypes.c_int(), ctypes.c_int()
    st = load().mpgemm_tile_shape(m, n, _dtype(a_type), ctypes.byref(tm), ctypes.byref(tn))
    if st != SUCCESS:
        raise MpgemmError(st, "mpgemm_tile_shape")
    return tm.value, tn.value


# ------------------------------------------------------------------- products of language models
# Arguments in the C ABI's order; alpha, beta and the activation as Python values, pointers as
# tensors or integers, types as names or enum values.  Each run has a host-only check beside it
# with the same arguments but the handle and the stream.
class _EpilogueStruct(ctypes.Structure):
    _fields_ = [("act", _i32), ("bias", _vp), ("bias_type", _i32), ("bias_stride", _i64),
                ("aux", _vp), ("ld_aux", _i64)]


class Epilogue:
    """mpgemm_epilogue_t: activation, bias (of ``bias_type``, ``bias_stride`` elements from one
    expert's to the next's) and where the value before the activation is kept.  Holds its tensors."""

    __slots__ = ("struct", "held")

    def __init__(self, act="none", bias=None, bias_type="f32", aux=None, ld_aux=0, bias_stride=0):
        self.held = (bias, aux)
        self.struct = _EpilogueStruct(_act(act), _ptr(bias), _dtype(bias_type), bias_stride, _ptr(aux),
                                      ld_aux)


def _act(act: Union[str, int]) -> int:
    return ACTS[act] if isinstance(act, str) else int(act)


def _f32(v):
    """A scalar argument: the library reads it before the call returns and never writes it."""
    known = _F32.get(v)
    return ctypes.byref(ctypes.c_float(v)) if known is None else known


_F32 = {v: ctypes.byref(ctypes.c_float(v)) for v in (1.0, 0.0)}   # (equal keys: 0.0 stands for -0.0 too)


def _epi(e: Optional[Epilogue]):
    return None if e is None else ctypes.byref(e.struct)


def _run(name: str, handle, args, stream, check: bool) -> int:
    st = getattr(load(), name)(handle, *args, _stream(stream))
    if check and st != SUCCESS:
        raise MpgemmError(st, name)
    return st


def _epilogue_args(transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb, epilogue, beta, C,
                   c_type, ldc, D, d_type, ldd):
    return (_op(transa), _op(transb), m, n, k, _f32(alpha), _ptr(A), _dtype(a_type), lda, _ptr(B),
            _dtype(b_type), ldb, _epi(epilogue), _f32(beta), _ptr(C), _dtype(c_type), ldc, _ptr(D),
            _dtype(d_type), ldd)


def mpgemm_run_epilogue(handle, transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb,
                        epilogue, beta, C, c_type, ldc, D, d_type, ldd, stream=None,
                        check: bool = True) -> int:
    """Queue D = act(alpha op(A) op(B) + bias) + beta C."""
    return _run("mpgemm_run_epilogue", handle,
                _epilogue_args(transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb, epilogue,
                               beta, C, c_type, ldc, D, d_type, ldd), stream, check)


def mpgemm_check_epilogue(*args) -> int:
    return load().mpgemm_check_epilogue(*_epilogue_args(*args))


def _epilogue_grad_args(transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb, act, Z, ldz, D,
                        d_type, ldd, dbias, workspace, workspace_bytes):
    return (_op(transa), _op(transb), m, n, k, _f32(alpha), _ptr(A), _dtype(a_type), lda, _ptr(B),
            _dtype(b_type), ldb, _act(act), _ptr(Z), ldz, _ptr(D), _dtype(d_type), ldd, _ptr(dbias),
            _ptr(workspace), workspace_bytes)


def mpgemm_run_epilogue_grad(handle, transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb,
                             act, Z, ldz, D, d_type, ldd, dbias, workspace, workspace_bytes,
                             stream=None, check: bool = True) -> int:
    """Queue D = alpha op(A) op(B) act'(Z) and dbias, the column sums of D."""
    return _run("mpgemm_run_epilogue_grad", handle,
                _epilogue_grad_args(transa, transb, m, n, k, alpha, A, a_type, lda, B, b_type, ldb, act,
                                    Z, ldz, D, d_type, ldd, dbias, workspace, workspace_bytes),
                stream, check)


def mpgemm_check_epilogue_grad(*args) -> int:
    return load().mpgemm_check_epilogue_grad(*_epilogue_grad_args(*args))


def _grouped_args(transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type, ldb, stride_b,
                  epilogue, D, d_type, ldd):
    return (_op(transb), groups, rows, n, k, _f32(alpha), _ptr(A), _dtype(a_type), lda, _ptr(offsets),
            _ptr(B), _dtype(b_type), ldb, stride_b, _epi(epilogue), _ptr(D), _dtype(d_type), ldd)


def mpgemm_run_grouped(handle, transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type,
                       ldb, stride_b, epilogue, D, d_type, ldd, stream=None, check: bool = True) -> int:
    """Queue D(r) = act(alpha A(r) op(B_e) + bias_e) for the rows r of every expert e."""
    return _run("mpgemm_run_grouped", handle,
                _grouped_args(transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type, ldb,
                              stride_b, epilogue, D, d_type, ldd), stream, check)


def mpgemm_check_grouped(*args) -> int:
    return load().mpgemm_check_grouped(*_grouped_args(*args))


def _grouped_grad_args(transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type, ldb,
                       stride_b, act, Z, ldz, D, d_type, ldd, dbias, workspace, workspace_bytes):
    return (_op(transb), groups, rows, n, k, _f32(alpha), _ptr(A), _dtype(a_type), lda, _ptr(offsets),
            _ptr(B), _dtype(b_type), ldb, stride_b, _act(act), _ptr(Z), ldz, _ptr(D), _dtype(d_type), ldd,
            _ptr(dbias), _ptr(workspace), workspace_bytes)


def mpgemm_run_grouped_grad(handle, transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B,
                            b_type, ldb, stride_b, act, Z, ldz, D, d_type, ldd, dbias, workspace,
                            workspace_bytes, stream=None, check: bool = True) -> int:
    """Queue D(r) = alpha A(r) op(B_e) act'(Z(r)) and dbias(e), the sum of expert e's rows of D."""
    return _run("mpgemm_run_grouped_grad", handle,
                _grouped_grad_args(transb, groups, rows, n, k, alpha, A, a_type, lda, offsets, B, b_type,
                                   ldb, stride_b, act, Z, ldz, D, d_type, ldd, dbias, workspace,
                                   workspace_bytes), stream, check)


def mpgemm_check_grouped_grad(*args) -> int:
    return load().mpgemm_check_grouped_grad(*_grouped_grad_args(*args))


def _grouped_wgrad_args(groups, rows, m, n, alpha, A, a_type, lda, X, x_type, ldx, offsets, beta, D,
                        d_type, ldd, stride_d):
    return (groups, rows, m, n, _f32(alpha), _ptr(A), _dtype(a_type), lda, _ptr(X), _dtype(x_type), ldx,
            _ptr(offsets), _f32(beta), _ptr(D), _dtype(d_type), ldd, stride_d)


def mpgemm_run_grouped_wgrad(handle, groups, rows, m, n, alpha, A, a_type, lda, X, x_type, ldx, offsets,
                             beta, D, d_type, ldd, stride_d, stream=None, check: bool = True) -> int:
    """Queue D_e = alpha A_e^T X_e + beta D_e for every expert e."""
    return _run("mpgemm_run_grouped_wgrad", handle,
                _grouped_wgrad_args(groups, rows, m, n, alpha, A, a_type, lda, X, x_type, ldx, offsets,
                                    beta, D, d_type, ldd, stride_d), stream, check)


def mpgemm_check_grouped_wgrad(*args) -> int:
    return load().mpgemm_check_grouped_wgrad(*_grouped_wgrad_args(*args))


def _linear_ce_args(m, n, k, alpha, X, dtype, ldx, W, ldw, target, loss, lse, workspace,
                    workspace_bytes):
    return (m, n, k, _f32(alpha), _ptr(X), _dtype(dtype), ldx, _ptr(W), ldw, _ptr(target), _ptr(loss),
            _ptr(lse), _ptr(workspace), workspace_bytes)


def mpgemm_run_linear_ce(handle, m, n, k, alpha, X, dtype, ldx, W, ldw, target, loss, lse, workspace,
                         workspace_bytes, stream=None, check: bool = True) -> int:
    """Queue each row's softmax cross entropy (and log-sum-exp) of the logits alpha X W^T."""
    return _run("mpgemm_run_linear_ce", handle,
                _linear_ce_args(m, n, k, alpha, X, dtype, ldx, W, ldw, target, loss, lse, workspace,
                                workspace_bytes), stream, check)


def mpgemm_check_linear_ce(*args) -> int:
    return load().mpgemm_check_linear_ce(*_linear_ce_args(*args))


def _linear_ce_grad_args(m, n, k, alpha, X, dtype, ldx, W, ldw, target, lse, grad, dX, lddx, dW, lddw,
                         workspace, workspace_bytes):
    return (m, n, k, _f32(alpha), _ptr(X), _dtype(dtype), ldx, _ptr(W), ldw, _ptr(target), _ptr(lse),
            _ptr(grad), _ptr(dX), lddx, _ptr(dW), lddw, _ptr(workspace), workspace_bytes)


def mpgemm_run_linear_ce_grad(handle, m, n, k, alpha, X, dtype, ldx, W, ldw, target, lse, grad, dX,
                              lddx, dW, lddw, workspace, workspace_bytes, stream=None,
                              check: bool = True) -> int:
    """Queue the gradients dX and dW (either may be None) of the rows' losses weighted by grad."""
    return _run("mpgemm_run_linear_ce_grad", handle,
                _linear_ce_grad_args(m, n, k, alpha, X, dtype, ldx, W, ldw, target, lse, grad, dX, lddx,
                                     dW, lddw, workspace, workspace_bytes), stream, check)


def mpgemm_check_linear_ce_grad(*args) -> int:
    return load().mpgemm_check_linear_ce_grad(*_linear_ce_grad_args(*args))


def mpgemm_epilogue_grad_workspace_size(groups: int, m: int, n: int) -> int:
    """Workspace bytes of mpgemm_run_epilogue_grad (groups = 1) and mpgemm_run_grouped_grad for dbias."""
    return load().mpgemm_epilogue_grad_workspace_size(groups, m, n)


def mpgemm_linear_ce_workspace_size(m: int, n: int, k: int, dtype, train: bool) -> int:
    """Workspace bytes of mpgemm_run_linear_ce, with train of its gradients too."""
    return load().mpgemm_linear_ce_workspace_size(m, n, k, _dtype(dtype), 1 if train else 0)


class Handle:
    """Owns one library handle bound to the current device."""

    def __init__(self):
        self.h = mpgemm_create()

    def run(self, *args, **kwargs) -> int:
        return mpgemm_run(self.h, *args, **kwargs)

    def close(self):
        if self.h is not None:
            mpgemm_destroy(self.h)
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ----------------------------------------------------------------------------- buffers
def device_buffer(host_array, fmt: str, device="cuda", extra_bytes: int = 0):
    """Copy raw host storage (a numpy array) to a new device tensor holding the same bytes.

    ``extra_bytes`` > 0 appends that many bytes (0xFF-filled) after the data, so reads that
    run past the last row would see them."""
    import numpy as np
    arr = np.ascontiguousarray(host_array)
    flat = torch.from_numpy(arr.view(np.uint8).reshape(-1).copy())
    if extra_bytes:
        flat = torch.cat([flat, torch.full((extra_bytes,), 0xFF, dtype=torch.uint8)])
    dev = flat.to(device)
    return dev


def host_array(dev_buf, fmt: str, shape):
    """Copy a device byte buffer back to numpy raw storage of ``fmt`` with ``shape``."""
    import numpy as np
    storage = {"f16": np.uint16, "bf16": np.uint16, "i8": np.int8, "f32": np.float32,
               "i32": np.int32}[fmt]
    raw = dev_buf.cpu().numpy()
    count = int(np.prod(shape))
    return raw[: count * np.dtype(storage).itemsize].view(storage).reshape(shape)
