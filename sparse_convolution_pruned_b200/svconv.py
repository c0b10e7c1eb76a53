"""Python binding of the svconv C ABI (include/svconv.h).

Argument marshalling only: every step runs in libsvconv.so's CUDA kernels.
PyTorch supplies device memory and the current CUDA stream.  There is no CPU
fallback: if the library is missing or no CUDA device is present, every call
raises.

Function names match the C entry points.  Output tensors may be passed in
(``out=``-style keyword arguments); otherwise they are allocated with torch on
the input's device.

``stream`` is the torch stream to launch on (default: the current one).  Ordering it with the streams that
write the inputs and read the outputs is the caller's part; what a call allocates belongs to that stream.
"""
from __future__ import annotations

import array
import ctypes
import os
import re
from typing import Optional, Sequence, Tuple

import torch

F32, BF16, E4M3 = 0, 1, 2
OK = 0
STATUS_BAD_COORD, STATUS_DUPLICATE, STATUS_BAD_FRAME, STATUS_BAD_OFFSETS = 1, 2, 4, 8
STATUS_TIMEOUT, STATUS_BAD_INDEX, STATUS_CHUNK_OVERFLOW = 16, 32, 64

ROPE_HALF, ROPE_INTERLEAVED = 0, 1

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libsvconv.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "svconv.h")
_lib = None


class CrossAttnDesc(ctypes.Structure):
    """svconv_cross_attn_desc"""
    _fields_ = [("nq", ctypes.c_int), ("nkv", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("d", ctypes.c_int), ("G", ctypes.c_int), ("q_off", ctypes.c_void_p), ("kv_off", ctypes.c_void_p),
                ("max_q", ctypes.c_int), ("max_kv", ctypes.c_int), ("kv_keep", ctypes.c_void_p),
                ("scale", ctypes.c_float)] + \
        [(f, ctypes.c_int64) for f in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head")]


class QkSide(ctypes.Structure):
    """svconv_qk_side"""
    _fields_ = [("x", ctypes.c_void_p), ("x_row", ctypes.c_int64), ("n", ctypes.c_int), ("H", ctypes.c_int),
                ("pos", ctypes.c_void_p), ("w", ctypes.c_void_p), ("y", ctypes.c_void_p), ("dy", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("dw", ctypes.c_void_p)]


class Grad(ctypes.Structure):
    """svconv_grad"""
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int)]


class SvconvError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {code} ({status_str(code)})")
        self.code = code


def lib() -> ctypes.CDLL:
    """Load libsvconv.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m sparse_convolution_pruned_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.svconv_build_index.argtypes = [P, P, I, I, I, I, P, P, P, P]
        L.svconv_fwd.argtypes = [I, P, P, I, I, I, P, P, P, P]
        L.svconv_bwd_data.argtypes = [I, P, P, I, I, I, P, P, P]
        L.svconv_bwd_weight.argtypes = [I, P, P, P, I, I, I, P, P, P, Z, P]
        L.svconv_bwd.argtypes = [I, P, P, P, I, I, I, P, P, P, P, P, Z, P]
        L.svconv_bwd.restype = I
        L.svconv_bwd_single_pass.argtypes = [P, P, P, I, P, P, P, P, P, Z, P]
        L.svconv_bwd_single_pass.restype = I
        L.svconv_bwd_single_pass_workspace_size.argtypes = [I]
        L.svconv_bwd_single_pass_workspace_size.restype = Z
        L.svconv_bwd_workspace_size.argtypes = [I, I, I, I]
        L.svconv_bwd_workspace_size.restype = Z
        L.svconv_bwd_weight_noalloc.argtypes = [I, P, P, P, I, I, I, P, P, P]
        L.svconv_bwd_weight_noalloc.restype = I
        L.svconv_bwd_weight_workspace_size.argtypes = [I, I, I, I]
        L.svconv_bwd_weight_workspace_size.restype = Z
        L.svconv_adapter_fwd.argtypes = [P, P, P, I, I, I, I, P, P, P, P, I, I, P, Z, P, P]
        L.svconv_adapter_workspace_size.argtypes = [I, I]
        L.svconv_adapter_workspace_size.restype = Z
        L.svconv_xattn_aux.argtypes = [P, I, I, P, I, I, P, I, I, P, P, Z, P, P]
        L.svconv_xattn_aux.restype = I
        L.svconv_xattn_workspace_size.argtypes = [I, I, I]
        L.svconv_xattn_workspace_size.restype = Z
        L.svconv_adapter_fwd_xattn.argtypes = [P, P, P, I, I, I, I, P, P, P, P, I, I, P, I, I, P, P, Z, P, P]
        L.svconv_adapter_fwd_xattn.restype = I
        L.svconv_adapter_xattn_workspace_size.argtypes = [I, I, I, I, I]
        L.svconv_adapter_xattn_workspace_size.restype = Z
        L.svconv_cross_attn_fwd.argtypes = [P, P, P, P, P, P, P, Z, P, P]
        L.svconv_cross_attn_fwd.restype = I
        L.svconv_cross_attn_fwd_workspace_size.argtypes = [P]
        L.svconv_cross_attn_fwd_workspace_size.restype = Z
        L.svconv_cross_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, Z, P, P]
        L.svconv_cross_attn_bwd.restype = I
        L.svconv_cross_attn_bwd_workspace_size.argtypes = [P]
        L.svconv_cross_attn_bwd_workspace_size.restype = Z
        L.svconv_qk_norm_rope_fwd.argtypes = [I, I, I, I, P, I, P, ctypes.c_float, P, P, P]
        L.svconv_qk_norm_rope_fwd.restype = I
        L.svconv_qk_norm_rope_bwd.argtypes = [I, I, I, I, P, I, P, ctypes.c_float, P, P, P, Z, P]
        L.svconv_qk_norm_rope_bwd.restype = I
        L.svconv_qk_norm_rope_bwd_workspace_size.argtypes = [I]
        L.svconv_qk_norm_rope_bwd_workspace_size.restype = Z
        L.svconv_clip_grads.argtypes = [P, I, ctypes.c_float, P, P, Z, P]
        L.svconv_clip_grads.restype = I
        L.svconv_clip_grads_workspace_size.argtypes = [P, I]
        L.svconv_clip_grads_workspace_size.restype = Z
        L.svconv_read_error_word.argtypes = [P]
        L.svconv_selftest_timeout.argtypes = [P, I, P]
        L.svconv_status_str.argtypes = [I]
        L.svconv_status_str.restype = ctypes.c_char_p
        L.svconv_version.argtypes = []
        for name in ("svconv_build_index", "svconv_fwd", "svconv_bwd_data", "svconv_bwd_weight",
                     "svconv_adapter_fwd", "svconv_read_error_word", "svconv_selftest_timeout",
                     "svconv_version"):
            getattr(L, name).restype = I
        _lib = L
    return _lib


def declared_symbols() -> list:
    """Entry points declared with SVCONV_API in include/svconv.h."""
    text = open(HEADER_PATH).read()
    return re.findall(r"SVCONV_API\s+[\w\s\*]+?\b(svconv_\w+)\s*\(", text)


def status_str(code: int) -> str:
    try:
        return lib().svconv_status_str(int(code)).decode()
    except Exception:  # pragma: no cover - message formatting only
        return "?"


def svconv_status_str(code: int) -> str:
    return status_str(code)


def svconv_version() -> int:
    return int(lib().svconv_version())


def _check(fn: str, rc: int):
    if rc != OK:
        raise SvconvError(fn, rc)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor, stream=None):
    s = stream if stream is not None else torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(s.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float8_e4m3fn:
        return E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _cuda(*ts):
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("svconv operates on CUDA tensors only")
        if not t.is_contiguous():
            raise ValueError("svconv expects contiguous tensors")


# The current device and raw stream without the Python objects around them, where this torch offers them.
_device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream_now = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _new(shape, dtype, like: torch.Tensor, index: int, stream=None, returned: bool = True) -> torch.Tensor:
    """Memory for a call on `stream` (None: the current one) on cuda:index.  On another stream than the current one it is
    that stream's own memory: what the current stream freed may still be in use there, and what is freed here
    goes back to the stream that works on it.  The current stream may use what is returned to the caller."""
    if stream is None or stream.cuda_stream == _stream_now(index):
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    if returned:
        t.record_stream(torch.cuda.current_stream(index))
    return t


def svconv_build_index(coords: torch.Tensor, frame_off: torch.Tensor, T: int, H: int, W: int, *,
                       nbr: Optional[torch.Tensor] = None, M: Optional[torch.Tensor] = None,
                       want_map: bool = False, status: Optional[torch.Tensor] = None,
                       stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Neighbour table [n, 9] int32 (and the lookup map [T, H, W] if requested)."""
    _cuda(coords, frame_off, nbr, M, status)
    n = coords.shape[0]
    if nbr is None:
        nbr = _new((n, 9), torch.int32, coords, coords.get_device(), stream)
    if M is None and want_map:
        M = _new((T, H, W), torch.int32, coords, coords.get_device(), stream)
    rc = lib().svconv_build_index(_ptr(coords), _ptr(frame_off), int(T), int(H), int(W), int(n), _ptr(nbr),
                                  _ptr(M), _ptr(status), _stream(coords, stream))
    _check("svconv_build_index", rc)
    return nbr, M


def svconv_fwd(X: torch.Tensor, nbr: torch.Tensor, Wt: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
               Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y[k] = bias + sum_j W_j X[N[k, j]]; Wt is [C_out, 9, C_in].  e4m3 X / Wt give a bf16 Y."""
    _cuda(X, nbr, Wt, bias, Y)
    n, Cin = X.shape
    Cout = Wt.shape[0]
    if Y is None:
        ydt = torch.bfloat16 if X.dtype == torch.float8_e4m3fn else X.dtype
        Y = _new((n, Cout), ydt, X, X.get_device(), stream)
    rc = lib().svconv_fwd(_dtype_code(X), _ptr(X), _ptr(nbr), n, Cin, Cout, _ptr(Wt), _ptr(bias), _ptr(Y),
                          _stream(X, stream))
    _check("svconv_fwd", rc)
    return Y


def svconv_bwd_data(dY: torch.Tensor, nbr: torch.Tensor, Wt: torch.Tensor, *, dX: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """dX[k] = sum_j W_j^T dY[N[k, 8-j]]."""
    _cuda(dY, nbr, Wt, dX)
    n, Cout = dY.shape
    Cin = Wt.shape[2]
    if dX is None:
        dX = _new((n, Cin), dY.dtype, dY, dY.get_device(), stream)
    rc = lib().svconv_bwd_data(_dtype_code(dY), _ptr(dY), _ptr(nbr), n, Cin, Cout, _ptr(Wt), _ptr(dX),
                               _stream(dY, stream))
    _check("svconv_bwd_data", rc)
    return dX


def svconv_bwd_weight_workspace_size(dtype: int, n: int, Cin: int, Cout: int) -> int:
    return int(lib().svconv_bwd_weight_workspace_size(int(dtype), int(n), int(Cin), int(Cout)))


def svconv_bwd_weight(dY: torch.Tensor, X: torch.Tensor, nbr: torch.Tensor, *, dW: Optional[torch.Tensor] = None,
                      db: Optional[torch.Tensor] = None, want_db: bool = True,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """(dW [C_out, 9, C_in] fp32, db [C_out] fp32 or None)."""
    _cuda(dY, X, nbr, dW, db, workspace)
    n, Cout = dY.shape
    Cin = X.shape[1]
    dt = _dtype_code(X)
    if dW is None:
        dW = _new((Cout, 9, Cin), torch.float32, X, X.get_device(), stream)
    if db is None and want_db:
        db = _new((Cout,), torch.float32, X, X.get_device(), stream)
    need = svconv_bwd_weight_workspace_size(dt, n, Cin, Cout)
    if workspace is None:
        workspace = _new((max(need, 16),), torch.uint8, X, X.get_device(), stream, returned=False)
    rc = lib().svconv_bwd_weight(dt, _ptr(dY), _ptr(X), _ptr(nbr), n, Cin, Cout, _ptr(dW), _ptr(db),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(X, stream))
    _check("svconv_bwd_weight", rc)
    return dW, db


def svconv_bwd_weight_noalloc(dY: torch.Tensor, X: torch.Tensor, nbr: torch.Tensor, *,
                              dW: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
                              want_db: bool = True, stream=None):
    """As svconv_bwd_weight, with the split partials in the library's fixed device array
    (no workspace; concurrent calls race, see include/svconv.h)."""
    _cuda(dY, X, nbr, dW, db)
    n, Cout = dY.shape
    Cin = X.shape[1]
    if dW is None:
        dW = _new((Cout, 9, Cin), torch.float32, X, X.get_device(), stream)
    if db is None and want_db:
        db = _new((Cout,), torch.float32, X, X.get_device(), stream)
    rc = lib().svconv_bwd_weight_noalloc(_dtype_code(X), _ptr(dY), _ptr(X), _ptr(nbr), n, Cin, Cout, _ptr(dW),
                                         _ptr(db), _stream(X, stream))
    _check("svconv_bwd_weight_noalloc", rc)
    return dW, db


def svconv_bwd_workspace_size(dtype: int, n: int, Cin: int, Cout: int) -> int:
    return int(lib().svconv_bwd_workspace_size(int(dtype), int(n), int(Cin), int(Cout)))


def svconv_bwd(dY: torch.Tensor, X: torch.Tensor, nbr: torch.Tensor, Wt: torch.Tensor, *,
               dX: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
               want_db: bool = True, workspace: Optional[torch.Tensor] = None, stream=None):
    """(dX, dW, db): the data gradient and the weight / bias gradients in one call."""
    _cuda(dY, X, nbr, Wt, dX, dW, db, workspace)
    n, Cout = dY.shape
    Cin = X.shape[1]
    dt = _dtype_code(X)
    if dX is None:
        dX = _new((n, Cin), dY.dtype, dY, dY.get_device(), stream)
    if dW is None:
        dW = _new((Cout, 9, Cin), torch.float32, X, X.get_device(), stream)
    if db is None and want_db:
        db = _new((Cout,), torch.float32, X, X.get_device(), stream)
    need = svconv_bwd_workspace_size(dt, n, Cin, Cout)
    if workspace is None:
        workspace = _new((max(need, 16),), torch.uint8, X, X.get_device(), stream, returned=False)
    rc = lib().svconv_bwd(dt, _ptr(dY), _ptr(X), _ptr(nbr), n, Cin, Cout, _ptr(Wt), _ptr(dX), _ptr(dW), _ptr(db),
                          _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(X, stream))
    _check("svconv_bwd", rc)
    return dX, dW, db


def svconv_bwd_single_pass(dY: torch.Tensor, X: torch.Tensor, nbr: torch.Tensor, Wt: torch.Tensor, *,
                           dX: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                           db: Optional[torch.Tensor] = None, want_db: bool = True,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """(dX, dW, db) at C_in = C_out = 64 (bf16) from one pass over dY."""
    _cuda(dY, X, nbr, Wt, dX, dW, db, workspace)
    n = dY.shape[0]
    if dX is None:
        dX = _new((n, 64), dY.dtype, dY, dY.get_device(), stream)
    if dW is None:
        dW = _new((64, 9, 64), torch.float32, X, X.get_device(), stream)
    if db is None and want_db:
        db = _new((64,), torch.float32, X, X.get_device(), stream)
    need = int(lib().svconv_bwd_single_pass_workspace_size(int(n)))
    if workspace is None:
        workspace = _new((max(need, 16),), torch.uint8, X, X.get_device(), stream, returned=False)
    rc = lib().svconv_bwd_single_pass(_ptr(dY), _ptr(X), _ptr(nbr), n, _ptr(Wt), _ptr(dX), _ptr(dW), _ptr(db),
                                      _ptr(workspace), workspace.numel() * workspace.element_size(),
                                      _stream(X, stream))
    _check("svconv_bwd_single_pass", rc)
    return dX, dW, db


def svconv_adapter_workspace_size(R: int, max_chunk_rows: int) -> int:
    return int(lib().svconv_adapter_workspace_size(int(R), int(max_chunk_rows)))


def svconv_adapter_fwd(X: torch.Tensor, nbr: torch.Tensor, frame_off: torch.Tensor, T: int, Wd: torch.Tensor,
                       Wc: torch.Tensor, Wu: torch.Tensor, bc: Optional[torch.Tensor] = None, *, chunk_T: int,
                       max_chunk_rows: int, workspace: Optional[torch.Tensor] = None,
                       status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """X <- X + Linear_up(GELU(SparseConv(Linear_down(X)))), chunked over frames, in place."""
    _cuda(X, nbr, frame_off, Wd, Wc, Wu, bc, workspace, status)
    n, D = X.shape
    R = Wd.shape[0]
    need = svconv_adapter_workspace_size(R, max_chunk_rows)
    if workspace is None:
        workspace = _new((max(need, 16),), torch.uint8, X, X.get_device(), stream, returned=False)
    rc = lib().svconv_adapter_fwd(_ptr(X), _ptr(nbr), _ptr(frame_off), int(T), n, D, R, _ptr(Wd), _ptr(Wc),
                                  _ptr(bc), _ptr(Wu), int(chunk_T), int(max_chunk_rows), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _ptr(status), _stream(X, stream))
    _check("svconv_adapter_fwd", rc)
    return X


def svconv_xattn_workspace_size(G: int, max_group_rows: int, A: int) -> int:
    return int(lib().svconv_xattn_workspace_size(int(G), int(max_group_rows), int(A)))


def svconv_xattn_aux(H: torch.Tensor, group_off: torch.Tensor, aux: torch.Tensor, *, max_group_rows: int,
                     heads: int = 1, out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """aux [G, A, R] bf16 attending over the rows of H [n, R] of their group -> fp32 [G, A, R]."""
    _cuda(H, group_off, aux, out, workspace, status)
    n, R = H.shape
    G, A, _ = aux.shape
    if out is None:
        out = _new((G, A, R), torch.float32, aux, aux.get_device(), stream)
    need = svconv_xattn_workspace_size(G, max_group_rows, A)
    if workspace is None:
        workspace = _new((max(need, 16),), torch.uint8, aux, aux.get_device(), stream, returned=False)
    rc = lib().svconv_xattn_aux(_ptr(H), n, R, _ptr(group_off), G, int(max_group_rows), _ptr(aux), A, int(heads),
                                _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _ptr(status), _stream(aux, stream))
    _check("svconv_xattn_aux", rc)
    return out


def svconv_adapter_xattn_workspace_size(T: int, R: int, chunk_T: int, max_chunk_rows: int, A: int) -> int:
    return int(lib().svconv_adapter_xattn_workspace_size(int(T), int(R), int(chunk_T), int(max_chunk_rows), int(A)))


def svconv_adapter_fwd_xattn(X: torch.Tensor, nbr: torch.Tensor, frame_off: torch.Tensor, T: int, Wd: torch.Tensor,
                             Wc: torch.Tensor, Wu: torch.Tensor, aux: torch.Tensor, bc: Optional[torch.Tensor] = None, *,
                             chunk_T: int, max_chunk_rows: int, heads: int = 1,
                             aux_out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None, stream=None):
    """The chunked adapter forward (X in place) plus the auxiliary tokens aux [A, R] attending
    over the down-projected rows of the whole sequence -> (X, aux_out fp32 [A, R])."""
    _cuda(X, nbr, frame_off, Wd, Wc, Wu, aux, bc, aux_out, workspace, status)
    n, D = X.shape
    R = Wd.shape[0]
    A = aux.shape[0]
    if aux_out is None:
        aux_out = _new((A, R), torch.float32, X, X.get_device(), stream)
    need = svconv_adapter_xattn_workspace_size(T, R, chunk_T, max_chunk_rows, A)
    if workspace is None:
        workspace = _new((max(need, 16),), torch.uint8, X, X.get_device(), stream, returned=False)
    rc = lib().svconv_adapter_fwd_xattn(_ptr(X), _ptr(nbr), _ptr(frame_off), int(T), n, D, R, _ptr(Wd), _ptr(Wc),
                                        _ptr(bc), _ptr(Wu), int(chunk_T), int(max_chunk_rows), _ptr(aux), A,
                                        int(heads), _ptr(aux_out), _ptr(workspace),
                                        workspace.numel() * workspace.element_size(), _ptr(status),
                                        _stream(X, stream))
    _check("svconv_adapter_fwd_xattn", rc)
    return X, aux_out


def _device_of(t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError("svconv operates on CUDA tensors only")
    return index


def _call(name: str, index: int, fn, *args):
    """fn(*args) with device `index` current (launches and device queries go to the current device)."""
    if _device_now() == index:
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc != OK:
        raise SvconvError(name, rc)


def _like(name: str, t: torch.Tensor, shape, dtype, index: int):
    """`t` is contiguous, of this shape and dtype, on CUDA device `index`."""
    if t.get_device() != index or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {tuple(shape)} {dtype} on cuda:{index} is needed, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}, strides {t.stride()}")


def _same(name: str, t: Optional[torch.Tensor], like: torch.Tensor, index: int, stream=None) -> torch.Tensor:
    """An output of like's shape and dtype, contiguous: checked if given, else allocated."""
    if t is None:
        if stream is None:
            return torch.empty_like(like, memory_format=torch.contiguous_format)
        return _new(like.shape, like.dtype, like, index, stream)
    _like(name, t, like.shape, like.dtype, index)
    return t


def _f32(name: str, t: Optional[torch.Tensor], shape, like: torch.Tensor, index: int, stream=None) -> torch.Tensor:
    if t is None:
        return like.new_empty(shape, dtype=torch.float32) if stream is None else _new(shape, torch.float32, like, index, stream)
    _like(name, t, shape, torch.float32, index)
    return t


def _scratch(ws: Optional[torch.Tensor], need: int, like: torch.Tensor, index: int, stream=None):
    """(tensor to keep until the launch, its address, its bytes)."""
    if ws is None:
        if not need:
            return None, None, 0
        if stream is None:
            ws = like.new_empty((need,), dtype=torch.uint8)
        else:
            ws = _new((need,), torch.uint8, like, index, stream, returned=False)
    elif ws.get_device() != index or not ws.is_contiguous():
        raise ValueError(f"workspace: a contiguous tensor on cuda:{index} is needed")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _status(t: Optional[torch.Tensor], index: int):
    if t is None:
        return None
    if t.get_device() != index or t.dtype is not torch.int32 or t.numel() < 1:
        raise ValueError(f"status: int32 on cuda:{index} is needed")
    return t.data_ptr()


def _attn_desc(Q, K, V, q_off, kv_off, max_q, max_kv, scale, kv_keep) -> Tuple[int, CrossAttnDesc]:
    index = _device_of(Q)
    if Q.dim() != 3 or K.dim() != 3:
        raise ValueError("Q, K and V are [rows, heads, channels]")
    nq, Hq, d = Q.shape
    nkv, Hkv, dk = kshape = K.shape
    if dk != d or V.shape != kshape:
        raise ValueError(f"Q {tuple(Q.shape)}, K {tuple(K.shape)} and V {tuple(V.shape)} do not fit together")
    if (nq | nkv) >> 31:
        raise ValueError("the library counts rows in 32 bits")
    strides = []
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        if t.dtype is not torch.bfloat16:
            raise TypeError(f"{name}: bf16 is needed, got {t.dtype}")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, Q on {Q.device}")
        row, head, one = t.stride()
        if one != 1 and d > 1:
            raise ValueError(f"{name}: contiguous channels are needed (rows and heads may be strided)")
        strides += (row, head)
    offs = q_off.shape
    if q_off.dim() != 1 or offs[0] < 1:
        raise ValueError("q_off: G + 1 offsets are needed")
    _like("q_off", q_off, offs, torch.int32, index)
    _like("kv_off", kv_off, offs, torch.int32, index)
    if kv_keep is not None:
        if kv_keep.dtype not in (torch.uint8, torch.bool):
            raise TypeError(f"kv_keep: uint8 or bool is needed, got {kv_keep.dtype}")
        _like("kv_keep", kv_keep, (nkv,), kv_keep.dtype, index)
        kv_keep = kv_keep.data_ptr()
    return index, CrossAttnDesc(nq, nkv, Hq, Hkv, d, offs[0] - 1, q_off.data_ptr(), kv_off.data_ptr(), min(int(max_q), nq),
                                min(int(max_kv), nkv), kv_keep, d ** -0.5 if scale is None else float(scale), *strides)


def svconv_cross_attn_fwd_workspace_size(desc: CrossAttnDesc) -> int:
    return int(lib().svconv_cross_attn_fwd_workspace_size(ctypes.byref(desc)))


def svconv_cross_attn_bwd_workspace_size(desc: CrossAttnDesc) -> int:
    return int(lib().svconv_cross_attn_bwd_workspace_size(ctypes.byref(desc)))


def svconv_cross_attn_fwd(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, q_off: torch.Tensor,
                          kv_off: torch.Tensor, *, max_q: int, max_kv: int, scale: Optional[float] = None,
                          kv_keep: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Q [nq, Hq, d] attending over K, V [nkv, Hkv, d] of its group -> (O [nq, Hq, d] bf16, lse [nq, Hq] fp32).

    scale defaults to 1 / sqrt(d); kv_keep [nkv] (uint8 or bool) leaves keys out.  Rows of no group
    are not written."""
    index, desc = _attn_desc(Q, K, V, q_off, kv_off, max_q, max_kv, scale, kv_keep)
    out = _same("out", out, Q, index, stream)
    lse = _f32("lse", lse, Q.shape[:2], Q, index, stream)
    L, ref = lib(), ctypes.byref(desc)
    ws, ws_ptr, ws_bytes = _scratch(workspace, L.svconv_cross_attn_fwd_workspace_size(ref), Q, index, stream)
    _call("svconv_cross_attn_fwd", index, L.svconv_cross_attn_fwd, ref, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
          out.data_ptr(), lse.data_ptr(), ws_ptr, ws_bytes, _status(status, index),
          stream.cuda_stream if stream is not None else _stream_now(index))
    return out, lse


def svconv_cross_attn_bwd(dO: torch.Tensor, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
                          lse: torch.Tensor, q_off: torch.Tensor, kv_off: torch.Tensor, *, max_q: int, max_kv: int,
                          scale: Optional[float] = None, kv_keep: Optional[torch.Tensor] = None,
                          dQ: Optional[torch.Tensor] = None, dK: Optional[torch.Tensor] = None,
                          dV: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None, stream=None):
    """(dQ, dK, dV) of svconv_cross_attn_fwd from dO and the forward's O and lse; contiguous bf16."""
    index, desc = _attn_desc(Q, K, V, q_off, kv_off, max_q, max_kv, scale, kv_keep)
    _like("dO", dO, Q.shape, torch.bfloat16, index)
    _like("O", O, Q.shape, torch.bfloat16, index)
    _like("lse", lse, Q.shape[:2], torch.float32, index)
    dQ, dK, dV = _same("dQ", dQ, Q, index, stream), _same("dK", dK, K, index, stream), _same("dV", dV, V, index, stream)
    L, ref = lib(), ctypes.byref(desc)
    ws, ws_ptr, ws_bytes = _scratch(workspace, L.svconv_cross_attn_bwd_workspace_size(ref), Q, index, stream)
    _call("svconv_cross_attn_bwd", index, L.svconv_cross_attn_bwd, ref, dO.data_ptr(), Q.data_ptr(), K.data_ptr(),
          V.data_ptr(), O.data_ptr(), lse.data_ptr(), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), ws_ptr, ws_bytes,
          _status(status, index), stream.cuda_stream if stream is not None else _stream_now(index))
    return dQ, dK, dV


_ROPE_LAYOUTS = {"half": ROPE_HALF, "interleaved": ROPE_INTERLEAVED, ROPE_HALF: ROPE_HALF,
                 ROPE_INTERLEAVED: ROPE_INTERLEAVED}


def _qk_common(Q, K, pq, pk, freq, layout, axis_pairs, wq, wk):
    """Checked sides, and the arguments that both directions share."""
    index, dtype = _device_of(Q), Q.dtype
    code = F32 if dtype is torch.float32 else BF16 if dtype is torch.bfloat16 else None
    if code is None:
        raise TypeError(f"fp32 or bf16 is needed, got {dtype}")
    if layout not in _ROPE_LAYOUTS:
        raise ValueError(f"layout {layout!r}: 'half' or 'interleaved'")
    pairs = freq.numel()
    _like("freq", freq, (pairs,), torch.float64, index)
    axes = pq.shape[1] if pq.dim() == 2 else 1
    split = (pairs,) if axis_pairs is None else axis_pairs
    if len(split) != axes or not 1 <= axes <= 3 or sum(split) != pairs:
        raise ValueError(f"axis_pairs {split}: {axes} counts that add up to {pairs} frequencies are needed, for at most 3 axes")
    d = Q.shape[-1]
    sides = []
    for name, x, pos, w in (("Q", Q, pq, wq), ("K", K, pk, wk)):
        if x.dim() != 3 or x.shape[2] != d or x.dtype is not dtype or x.get_device() != index:
            raise ValueError(f"{name}: [rows, heads, {d}] {dtype} on cuda:{index} is needed")
        n, H, _ = x.shape
        if n >> 31:
            raise ValueError("the library counts rows in 32 bits")
        row, head, one = x.stride()
        if n and ((d > 1 and one != 1) or (H > 1 and head != d)):
            raise ValueError(f"{name}: contiguous heads are needed (rows may be strided)")
        if pos.dim() == 1 and axes != 1:
            raise ValueError("the positions of Q and K have different numbers of axes")
        _like(f"positions of {name}", pos, (n, axes) if pos.dim() == 2 else (n,), torch.int32, index)
        if w is not None:
            _like(f"weight of {name}", w, (d,), torch.float32, index)
            w = w.data_ptr()
        sides.append(QkSide(x.data_ptr(), row if n > 1 else H * d, n, H, pos.data_ptr(), w))
    return index, sides, (code, d, 2 * pairs, _ROPE_LAYOUTS[layout], freq.data_ptr(), axes, (ctypes.c_int32 * 3)(*split))


def svconv_qk_norm_rope_fwd(Q: torch.Tensor, K: torch.Tensor, pos_q: torch.Tensor, pos_k: torch.Tensor,
                            freq: torch.Tensor, *, wq: Optional[torch.Tensor] = None,
                            wk: Optional[torch.Tensor] = None, eps: float = 1e-6, layout="half", axis_pairs=None,
                            Yq: Optional[torch.Tensor] = None, Yk: Optional[torch.Tensor] = None, stream=None):
    """Per-head RMS norm of Q [nq, Hq, d] and K [nk, Hkv, d] (fp32 or bf16) with their tokens' rotary positions.

    pos_* int32 [n] or [n, axes] (the (t, y, x) coords table serves as it is), freq fp64 [rot / 2] radians
    per unit of position (the first 2 * len(freq) channels are rotated), axis_pairs the number of pairs that
    follow each axis.  Yq / Yk may be Q / K themselves when those are contiguous."""
    index, (sq, sk), args = _qk_common(Q, K, pos_q, pos_k, freq, layout, axis_pairs, wq, wk)
    Yq, Yk = _same("Yq", Yq, Q, index, stream), _same("Yk", Yk, K, index, stream)
    sq.y, sk.y = Yq.data_ptr(), Yk.data_ptr()
    _call("svconv_qk_norm_rope_fwd", index, lib().svconv_qk_norm_rope_fwd, *args, float(eps), ctypes.byref(sq),
          ctypes.byref(sk), stream.cuda_stream if stream is not None else _stream_now(index))
    return Yq, Yk


def svconv_qk_norm_rope_bwd_workspace_size(d: int) -> int:
    return int(lib().svconv_qk_norm_rope_bwd_workspace_size(int(d)))


def svconv_qk_norm_rope_bwd(dYq: torch.Tensor, dYk: torch.Tensor, Q: torch.Tensor, K: torch.Tensor,
                            pos_q: torch.Tensor, pos_k: torch.Tensor, freq: torch.Tensor, *,
                            wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6,
                            layout="half", axis_pairs=None, dQ: Optional[torch.Tensor] = None,
                            dK: Optional[torch.Tensor] = None, dwq: Optional[torch.Tensor] = None,
                            dwk: Optional[torch.Tensor] = None, want_dw: bool = True,
                            workspace: Optional[torch.Tensor] = None, stream=None):
    """(dQ, dK, dwq, dwk) of svconv_qk_norm_rope_fwd (dwq, dwk fp32 [d], None unless want_dw)."""
    index, (sq, sk), args = _qk_common(Q, K, pos_q, pos_k, freq, layout, axis_pairs, wq, wk)
    d = Q.shape[2]
    _like("dYq", dYq, Q.shape, Q.dtype, index)
    _like("dYk", dYk, K.shape, K.dtype, index)
    dQ, dK = _same("dQ", dQ, Q, index, stream), _same("dK", dK, K, index, stream)
    if want_dw:
        dwq, dwk = _f32("dwq", dwq, (d,), Q, index, stream), _f32("dwk", dwk, (d,), Q, index, stream)
        sq.dw, sk.dw = dwq.data_ptr(), dwk.data_ptr()
    else:
        dwq = dwk = None
    sq.dy, sq.dx, sk.dy, sk.dx = dYq.data_ptr(), dQ.data_ptr(), dYk.data_ptr(), dK.data_ptr()
    L = lib()
    ws, ws_ptr, ws_bytes = _scratch(workspace, L.svconv_qk_norm_rope_bwd_workspace_size(d), Q, index, stream)
    _call("svconv_qk_norm_rope_bwd", index, L.svconv_qk_norm_rope_bwd, *args, float(eps), ctypes.byref(sq),
          ctypes.byref(sk), ws_ptr, ws_bytes, stream.cuda_stream if stream is not None else _stream_now(index))
    return dQ, dK, dwq, dwk


def svconv_clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *, out: Optional[Sequence[torch.Tensor]] = None,
                      norm: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """Scale the gradients (fp32 or bf16, contiguous, one device) by min(1, max_norm / (norm + 1e-6)), in place
    or into `out`; returns their global norm (fp32 scalar tensor).  max_norm = inf takes the norm alone."""
    T = torch.Tensor
    grads = list(grads)
    count = len(grads)
    if not grads and norm is None:
        raise ValueError("no gradients and no norm tensor: the device is unknown")
    index = _device_of(grads[0] if grads else norm)
    dtypes = [g.dtype for g in grads]
    sizes = list(map(T.numel, grads))
    src = dst = list(map(T.data_ptr, grads))
    every = grads
    if out is not None:
        outs = list(out)
        if [o.dtype for o in outs] != dtypes or list(map(T.numel, outs)) != sizes:
            raise ValueError("outputs of the gradients' sizes and types are needed")
        every = grads + outs
        dst = list(map(T.data_ptr, outs))
    if set(map(T.get_device, every)) - {index} or not all(map(T.is_contiguous, every)):
        raise ValueError(f"contiguous tensors on cuda:{index} are needed")
    # svconv_grad records: src, dst, numel, dtype (the low word of the last 8 bytes)
    flat = array.array("q", bytes(32 * count))
    flat[0::4], flat[1::4], flat[2::4] = array.array("q", src), array.array("q", dst), array.array("q", sizes)
    if dtypes.count(torch.float32) != count:
        if dtypes.count(torch.float32) + dtypes.count(torch.bfloat16) != count:
            raise TypeError(f"fp32 or bf16 gradients are needed, got {set(dtypes)}")
        flat[3::4] = array.array("q", [F32 if t is torch.float32 else BF16 for t in dtypes])
    table = flat.buffer_info()[0] if count else None
    norm = _f32("norm", norm, (), grads[0] if grads else norm, index, stream)
    L = lib()
    ws, ws_ptr, ws_bytes = _scratch(workspace, max(L.svconv_clip_grads_workspace_size(table, count), 16), norm, index, stream)
    _call("svconv_clip_grads", index, L.svconv_clip_grads, table, count, float(max_norm), norm.data_ptr(), ws_ptr, ws_bytes,
          stream.cuda_stream if stream is not None else _stream_now(index))
    return norm


def svconv_read_error_word() -> int:
    out = ctypes.c_int32(0)
    _check("svconv_read_error_word", lib().svconv_read_error_word(ctypes.byref(out)))
    return int(out.value)


def svconv_selftest_timeout(status: torch.Tensor, timeout_us: int, stream=None) -> None:
    _cuda(status)
    _check("svconv_selftest_timeout", lib().svconv_selftest_timeout(_ptr(status), int(timeout_us),
                                                                     _stream(status, stream)))
