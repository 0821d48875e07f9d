"""fp4lin: FP4 (E2M1) quantized linear layer forward on AMD MI355X (gfx950).

Python binding of libfp4lin.so. The functions named ``fp4lin_*`` mirror the C
ABI one to one: they take torch tensors that already live on the GPU, pass
their device pointers, sizes and the current HIP stream, and raise
``Fp4linError`` on a non-zero status. The helpers without the prefix only add
output allocation on top of them. All arithmetic runs in the HIP kernels; there
is no CPU path.
"""
from __future__ import annotations

import contextlib
import ctypes
import itertools
import struct

from . import _lib
from ._lib import BF16, F32, Coo, ForwardOffsets

__all__ = [
    "Fp4linError", "lib", "packed_ld", "quantile_rank", "select_workspace_bytes",
    "weight_workspace_bytes", "workspace_bytes", "forward_layout",
    "fp4lin_outlier_select", "fp4lin_outlier_select_noalloc", "fp4lin_quantize_act", "fp4lin_quantize_weight", "fp4lin_gemm",
    "fp4lin_sparse_add", "fp4lin_forward", "outlier_select", "quantize_act", "quantize_weight", "gemm", "forward",
    "CooBuffers", "mx_scales_ld", "fp4lin_quantize_act_mx", "fp4lin_quantize_weight_mx",
    "fp4lin_gemm_mx", "quantize_act_mx", "quantize_weight_mx", "gemm_mx",
    "fp4lin_forward_mx", "forward_mx", "forward_layout_mx",
    "experts_workspace_bytes", "fp4lin_experts_quantize_weight_mx", "fp4lin_experts_forward_mx",
    "fp4lin_experts_apply_mx", "fp4lin_experts_dgrad_mx", "fp4lin_experts_wgrad_mx",
    "experts_quantize_weight_mx", "experts_forward_mx", "experts_apply_mx", "experts_dgrad_mx",
    "experts_wgrad_mx",
    "head_loss_workspace_bytes", "fp4lin_head_loss", "fp4lin_head_loss_backward", "head_loss",
    "head_loss_backward", "clip_workspace_bytes", "fp4lin_grad_norm", "fp4lin_clip_grads",
    "grad_norm", "clip_grads",
]


class Fp4linError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().fp4lin_status_str(status).decode()
        if status == _lib.ERR_LAUNCH:
            msg += f": {lib().fp4lin_last_hip_error_name().decode()}"
        super().__init__(f"{where}: status {status} ({msg})")
        self.status = status


def lib():
    return _lib.load()


def _check(status: int, where: str):
    if status != _lib.OK:
        raise Fp4linError(status, where)


def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"fp4lin takes float32 or bfloat16 inputs, got {t.dtype}")


def _dev(t, name):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (fp4lin has no CPU path)")
    return ctypes.c_void_p(t.data_ptr())


def _matrix(t, name):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D row-major tensor with unit column stride")
    return t.shape[0], t.shape[1], t.stride(0)


def _stream(stream):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# ---- host helpers --------------------------------------------------------------
def packed_ld(L: int) -> int:
    return int(lib().fp4lin_packed_ld(L))


def quantile_rank(n: int, q: float) -> int:
    return int(lib().fp4lin_quantile_rank(n, q))


def select_workspace_bytes(M: int, K: int, dtype_code: int) -> int:
    return int(lib().fp4lin_select_workspace_bytes(M, K, dtype_code))


def weight_workspace_bytes(K: int, N: int) -> int:
    return int(lib().fp4lin_weight_workspace_bytes(K, N))


def workspace_bytes(M: int, K: int, N: int, dtype_code: int, q: float) -> int:
    return int(lib().fp4lin_workspace_bytes(M, K, N, dtype_code, q))


def forward_layout(M: int, K: int, N: int, dtype_code: int, q: float) -> ForwardOffsets:
    o = ForwardOffsets()
    _check(lib().fp4lin_forward_layout(M, K, N, dtype_code, q, ctypes.byref(o)),
           "fp4lin_forward_layout")
    return o


class CooBuffers:
    """Device arrays of a COO dA (int32 row/col, float32 val, int32 row_ptr)."""

    def __init__(self, row, col, val, row_ptr):
        self.row, self.col, self.val, self.row_ptr = row, col, val, row_ptr

    @property
    def capacity(self) -> int:
        return int(self.row.numel())

    def struct(self) -> Coo:
        return Coo(self.row.data_ptr(), self.col.data_ptr(), self.val.data_ptr(),
                   self.row_ptr.data_ptr(), self.capacity)

    @classmethod
    def empty(cls, M: int, capacity: int, device):
        torch = _torch()
        cap = max(int(capacity), 1)
        return cls(torch.empty(cap, dtype=torch.int32, device=device),
                   torch.empty(cap, dtype=torch.int32, device=device),
                   torch.empty(cap, dtype=torch.float32, device=device),
                   torch.empty(M + 1, dtype=torch.int32, device=device))


# ---- the C ABI, one to one -------------------------------------------------------
def fp4lin_outlier_select(A, q, tau, coo: CooBuffers, ws, stream=None):
    M, K, lda = _matrix(A, "A")
    _dev(tau, "tau"), _dev(ws, "ws"), _dev(coo.row, "coo")
    _check(lib().fp4lin_outlier_select(_dev(A, "A"), _dtype_code(A), M, K, lda, float(q),
                                       _dev(tau, "tau"), coo.struct(), _dev(ws, "ws"),
                                       ws.numel() * ws.element_size(), _stream(stream)),
           "fp4lin_outlier_select")


def fp4lin_outlier_select_noalloc(A, q, tau, coo: CooBuffers, stream=None):
    M, K, lda = _matrix(A, "A")
    _dev(coo.row, "coo")
    _check(lib().fp4lin_outlier_select_noalloc(_dev(A, "A"), _dtype_code(A), M, K, lda,
                                               float(q), _dev(tau, "tau"), coo.struct(),
                                               _stream(stream)),
           "fp4lin_outlier_select_noalloc")


def fp4lin_quantize_act(X, tau, Xq, sX, stream=None):
    M, K, ldx = _matrix(X, "X")
    _check(lib().fp4lin_quantize_act(_dev(X, "X"), _dtype_code(X), M, K, ldx, _dev(tau, "tau"),
                                     _dev(Xq, "Xq"), _dev(sX, "sX"), _stream(stream)),
           "fp4lin_quantize_act")


def fp4lin_quantize_weight(W, Wq, sW, ws, stream=None):
    K, N, ldw = _matrix(W, "W")
    _check(lib().fp4lin_quantize_weight(_dev(W, "W"), _dtype_code(W), K, N, ldw, _dev(Wq, "Wq"),
                                        _dev(sW, "sW"), _dev(ws, "ws"),
                                        ws.numel() * ws.element_size(), _stream(stream)),
           "fp4lin_quantize_weight")


def fp4lin_gemm(Aq, sA, Bq, sB, M, N, K, coo: CooBuffers | None, W, Y, stream=None):
    _, _, ldy = _matrix(Y, "Y")
    if coo is not None:
        _, _, ldw = _matrix(W, "W")
        c = coo.struct()
        cp, wp, wdt = ctypes.byref(c), _dev(W, "W"), _dtype_code(W)
    else:
        cp, wp, wdt, ldw = None, None, F32, 0
    _check(lib().fp4lin_gemm(_dev(Aq, "Aq"), _dev(sA, "sA"), _dev(Bq, "Bq"), _dev(sB, "sB"),
                             M, N, K, cp, wp, wdt, ldw, _dev(Y, "Y"), ldy, _stream(stream)),
           "fp4lin_gemm")


def fp4lin_sparse_add(coo: CooBuffers, W, Y, stream=None):
    """Y += dA . W (Y must already hold the scaled FP4 product)."""
    M, N, ldy = _matrix(Y, "Y")
    K, _, ldw = _matrix(W, "W")
    c = coo.struct()
    _check(lib().fp4lin_sparse_add(ctypes.byref(c), _dev(W, "W"), _dtype_code(W), K, ldw, M, N,
                                   _dev(Y, "Y"), ldy, _stream(stream)),
           "fp4lin_sparse_add")


def fp4lin_forward(A, W, q, Y, ws, stream=None):
    M, K, lda = _matrix(A, "A")
    K2, N, ldw = _matrix(W, "W")
    if K2 != K:
        raise ValueError(f"A is {M}x{K} but W is {K2}x{N}")
    if A.dtype != W.dtype:
        raise TypeError("A and W must have the same dtype")
    _, _, ldy = _matrix(Y, "Y")
    _check(lib().fp4lin_forward(_dev(A, "A"), _dev(W, "W"), _dtype_code(A), M, K, N, lda, ldw,
                                float(q), _dev(Y, "Y"), ldy, _dev(ws, "ws"),
                                ws.numel() * ws.element_size(), _stream(stream)),
           "fp4lin_forward")


def fp4lin_quantize_act_mx(X, tau, Xq, Xs, stream=None):
    M, K, ldx = _matrix(X, "X")
    _check(lib().fp4lin_quantize_act_mx(_dev(X, "X"), _dtype_code(X), M, K, ldx,
                                        _dev(tau, "tau"), _dev(Xq, "Xq"), _dev(Xs, "Xs"),
                                        _stream(stream)),
           "fp4lin_quantize_act_mx")


def fp4lin_quantize_weight_mx(W, Wq, Ws, stream=None):
    K, N, ldw = _matrix(W, "W")
    _check(lib().fp4lin_quantize_weight_mx(_dev(W, "W"), _dtype_code(W), K, N, ldw,
                                           _dev(Wq, "Wq"), _dev(Ws, "Ws"), _stream(stream)),
           "fp4lin_quantize_weight_mx")


def fp4lin_gemm_mx(Aq, As, Bq, Bs, M, N, K, coo: CooBuffers | None, W, Y, stream=None):
    _, _, ldy = _matrix(Y, "Y")
    if coo is not None:
        _, _, ldw = _matrix(W, "W")
        c = coo.struct()
        cp, wp, wdt = ctypes.byref(c), _dev(W, "W"), _dtype_code(W)
    else:
        cp, wp, wdt, ldw = None, None, F32, 0
    _check(lib().fp4lin_gemm_mx(_dev(Aq, "Aq"), _dev(As, "As"), _dev(Bq, "Bq"), _dev(Bs, "Bs"),
                                M, N, K, cp, wp, wdt, ldw, _dev(Y, "Y"), ldy, _stream(stream)),
           "fp4lin_gemm_mx")


def fp4lin_forward_mx(A, W, q, Y, ws, stream=None):
    M, K, lda = _matrix(A, "A")
    K2, N, ldw = _matrix(W, "W")
    if K2 != K:
        raise ValueError(f"A is {M}x{K} but W is {K2}x{N}")
    if A.dtype != W.dtype:
        raise TypeError("A and W must have the same dtype")
    _, _, ldy = _matrix(Y, "Y")
    _check(lib().fp4lin_forward_mx(_dev(A, "A"), _dev(W, "W"), _dtype_code(A), M, K, N, lda, ldw,
                                   float(q), _dev(Y, "Y"), ldy, _dev(ws, "ws"),
                                   ws.numel() * ws.element_size(), _stream(stream)),
           "fp4lin_forward_mx")


# ---- allocating helpers --------------------------------------------------------------
def _empty(shape, dtype, device):
    return _torch().empty(shape, dtype=dtype, device=device)


def outlier_select(A, q, stream=None):
    """Returns (tau[1] float32, CooBuffers)."""
    torch = _torch()
    M, K, _ = _matrix(A, "A")
    k = quantile_rank(M * K, q)
    if k < 0:
        raise Fp4linError(_lib.ERR_QUANTILE, "outlier_select")
    cap = M * K - 1 - k
    tau = _empty((1,), torch.float32, A.device)
    coo = CooBuffers.empty(M, cap, A.device)
    ws = _empty((max(select_workspace_bytes(M, K, _dtype_code(A)), 16),), torch.uint8, A.device)
    fp4lin_outlier_select(A, q, tau, coo, ws, stream)
    return tau, coo


def quantize_act(X, tau=None, stream=None):
    """Returns (Xq uint8 M x packed_ld(K), sX float32 M)."""
    torch = _torch()
    M, K, _ = _matrix(X, "X")
    Xq = _empty((M, packed_ld(K)), torch.uint8, X.device)
    sX = _empty((M,), torch.float32, X.device)
    fp4lin_quantize_act(X, tau, Xq, sX, stream)
    return Xq, sX


def quantize_weight(W, stream=None):
    """Returns (Wq uint8 N x packed_ld(K), sW float32 N)."""
    torch = _torch()
    K, N, _ = _matrix(W, "W")
    Wq = _empty((N, packed_ld(K)), torch.uint8, W.device)
    sW = _empty((N,), torch.float32, W.device)
    ws = _empty((max(weight_workspace_bytes(K, N), 16),), torch.uint8, W.device)
    fp4lin_quantize_weight(W, Wq, sW, ws, stream)
    return Wq, sW


def gemm(Aq, sA, Bq, sB, M, N, K, coo=None, W=None, stream=None):
    """Returns Y float32 M x N."""
    Y = _empty((M, N), _torch().float32, Aq.device)
    fp4lin_gemm(Aq, sA, Bq, sB, M, N, K, coo, W, Y, stream)
    return Y


def forward(A, W, q, stream=None, return_workspace=False):
    """Returns Y float32 M x N (and the workspace holding the intermediates)."""
    torch = _torch()
    M, K, _ = _matrix(A, "A")
    N = W.shape[1]
    nbytes = workspace_bytes(M, K, N, _dtype_code(A), q)
    if nbytes == 0:
        raise Fp4linError(_lib.ERR_SHAPE, "forward")
    ws = _empty((nbytes,), torch.uint8, A.device)
    Y = _empty((M, N), torch.float32, A.device)
    fp4lin_forward(A, W, q, Y, ws, stream)
    return (Y, ws) if return_workspace else Y


def mx_scales_ld(L: int) -> int:
    return lib().fp4lin_mx_scales_ld(L)


def quantize_act_mx(X, tau=None, stream=None):
    """Micro-scaled: returns (Xq uint8 M x packed_ld(K), Xs uint8 (steps, M, 4)),
    the scales step-major: Xs[s, i, j] is the byte of block 4s + j of row i."""
    torch = _torch()
    M, K, _ = _matrix(X, "X")
    Xq = _empty((M, packed_ld(K)), torch.uint8, X.device)
    Xs = _empty((mx_scales_ld(K) // 4, M, 4), torch.uint8, X.device)
    fp4lin_quantize_act_mx(X, tau, Xq, Xs, stream)
    return Xq, Xs


def quantize_weight_mx(W, stream=None):
    """Micro-scaled: returns (Wq uint8 N x packed_ld(K), Ws uint8 (steps, N, 4)),
    the scales step-major as for quantize_act_mx, per column of W."""
    torch = _torch()
    K, N, _ = _matrix(W, "W")
    Wq = _empty((N, packed_ld(K)), torch.uint8, W.device)
    Ws = _empty((mx_scales_ld(K) // 4, N, 4), torch.uint8, W.device)
    fp4lin_quantize_weight_mx(W, Wq, Ws, stream)
    return Wq, Ws


def gemm_mx(Aq, As, Bq, Bs, M, N, K, coo=None, W=None, stream=None):
    """Micro-scaled GEMM; returns Y float32 M x N."""
    Y = _empty((M, N), _torch().float32, Aq.device)
    fp4lin_gemm_mx(Aq, As, Bq, Bs, M, N, K, coo, W, Y, stream)
    return Y


def forward_layout_mx(M: int, K: int, N: int, dtype_code: int, q: float) -> ForwardOffsets:
    o = ForwardOffsets()
    _check(lib().fp4lin_forward_layout_mx(M, K, N, dtype_code, float(q), ctypes.byref(o)),
           "fp4lin_forward_layout_mx")
    return o


def forward_mx(A, W, q, stream=None, return_workspace=False):
    """Micro-scaled forward; returns Y float32 M x N (and the workspace)."""
    torch = _torch()
    M, K, _ = _matrix(A, "A")
    N = W.shape[1]
    nbytes = lib().fp4lin_workspace_bytes_mx(M, K, N, _dtype_code(A), float(q))
    if nbytes == 0:
        raise Fp4linError(_lib.ERR_SHAPE, "forward_mx")
    ws = _empty((nbytes,), torch.uint8, A.device)
    Y = _empty((M, N), torch.float32, A.device)
    fp4lin_forward_mx(A, W, q, Y, ws, stream)
    return (Y, ws) if return_workspace else Y


# ---- products grouped by expert ------------------------------------------------------
# The helpers below are called with a few rows as well, where a call's host time
# is what its user waits for: each argument is looked at once, pointers go to
# ctypes as plain integers, and the device is only switched where it has to be.
_CODES = {}


def _code(t) -> int:
    """_dtype_code from a table."""
    if not _CODES:
        torch = _torch()
        _CODES.update({torch.float32: F32, torch.bfloat16: BF16})
    code = _CODES.get(t.dtype)
    return _dtype_code(t) if code is None else code


def _rows(t, name):
    """(rows, columns, row stride) of a row-major matrix. A single row needs no
    stride and may carry any (hidden[:, -1] of one long sequence): its length is
    taken."""
    size, stride = t.shape, t.stride()
    if len(size) != 2 or (stride[1] != 1 and size[1] > 1):
        raise ValueError(f"{name} must be a 2-D row-major tensor with unit column stride")
    if size[0] <= 1:
        return size[0], size[1], size[1]
    if stride[0] < size[1]:
        raise ValueError(f"{name} must not have overlapping rows")
    return size[0], size[1], stride[0]


def _experts_weight(W, name):
    """(E, K, N, ldw) of a stack of row-major matrices with one row stride throughout
    (that of the experts where they have one row each)."""
    size, stride = W.shape, W.stride()
    if len(size) == 3 and (stride[2] == 1 or size[2] <= 1):
        E, K, N = size
        ldw = stride[1] if K > 1 else stride[0] if E > 1 else N
        if ldw >= N and (E <= 1 or stride[0] == K * ldw):
            return E, K, N, ldw
    raise ValueError(f"{name} must be a 3-D tensor (experts, rows, columns) with unit column "
                     "stride and experts that follow one another at the row stride")


def _gpu(first, *others):
    """The GPU that all of the (name, tensor) pairs are on."""
    device = first[1].get_device()
    if device < 0:
        _dev(first[1], first[0])
    for name, t in others:
        if t.get_device() != device:
            _dev(t, name)
            raise ValueError(f"{name} is on {t.device}, {first[0]} on {first[1].device}")
    return device


def _same_dtype(a, b, names):
    if a.dtype != b.dtype:
        raise TypeError(f"{names} must have the same dtype")


def _row_end(row_end, E):
    if row_end.dtype != _torch().int32 or row_end.dim() != 1 or not row_end.is_contiguous():
        raise TypeError("row_end must be a contiguous int32 vector")
    if row_end.numel() != E:
        raise ValueError(f"row_end has {row_end.numel()} entries for {E} experts")
    return row_end.data_ptr()


def _need(ok, message):
    if not ok:
        raise ValueError(message)


_HERE = contextlib.nullcontext()


def _current():
    """The current GPU."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getDevice", None)  # tensors are there: no set-up to look for
    return torch.cuda.current_device() if raw is None else raw()


def _on(t, stream):
    """A context with the device of t and the stream the call runs on, so that
    what is allocated inside belongs to that stream."""
    device = t.get_device()
    if device < 0 or (stream is None and device == _current()):
        return _HERE
    torch = _torch()
    both = contextlib.ExitStack()
    both.enter_context(torch.cuda.device(device))
    if stream is not None:
        both.enter_context(torch.cuda.stream(stream))
    return both


def _queue(stream, device):
    """The HIP stream of a call on a device (the current one there if none is given)."""
    torch = _torch()
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # without a Stream object
    return torch.cuda.current_stream(device).cuda_stream if raw is None else raw(device)


def _call(device, name, *args):
    """Calls a C entry on `device`: the null stream is that of the current GPU."""
    f = getattr(lib(), name)
    if device == _current():
        _check(f(*args), name)
    else:
        with _torch().cuda.device(device):
            _check(f(*args), name)


def _nbytes(ws):
    return ws.numel() * ws.element_size()


def experts_workspace_bytes(which: int, E: int, M: int, K: int, N: int) -> int:
    return int(lib().fp4lin_experts_workspace_bytes(which, E, M, K, N))


def _experts_ws(which, E, M, K, N, device, where):
    n = lib().fp4lin_experts_workspace_bytes(which, E, M, K, N)
    if n == 0:
        raise Fp4linError(_lib.ERR_SHAPE, where)
    torch = _torch()
    return torch.empty(n, dtype=torch.uint8, device=device)


def _packed_bytes(Wq, Ws, E, K, N):
    """(name, tensor, bytes) of the codes and scales of E matrices of K x N."""
    steps = (K + 127) // 128  # of 64 bytes of codes and 4 scales
    return ("Wq", Wq, E * N * steps * 64), ("Ws", Ws, E * N * steps * 4)


def fp4lin_experts_quantize_weight_mx(W, Wq, Ws, stream=None):
    E, K, N, ldw = _experts_weight(W, "W")
    device = _gpu(("W", W), ("Wq", Wq), ("Ws", Ws))
    for name, t, want in _packed_bytes(Wq, Ws, E, K, N):
        _need(t.is_contiguous(), f"{name} must be contiguous")
        _need(_nbytes(t) >= want, f"{name} holds {_nbytes(t)} bytes, not {want}")
    _call(device, "fp4lin_experts_quantize_weight_mx", W.data_ptr(), _code(W), E, K, N, ldw,
          Wq.data_ptr(), Ws.data_ptr(), _queue(stream, device))


def fp4lin_experts_forward_mx(A, W, row_end, Y, ws, stream=None):
    M, K, lda = _rows(A, "A")
    E, K2, N, ldw = _experts_weight(W, "W")
    My, Ny, ldy = _rows(Y, "Y")
    device = _gpu(("A", A), ("W", W), ("row_end", row_end), ("Y", Y), ("ws", ws))
    _same_dtype(A, W, "A and W")
    if K2 != K:
        raise ValueError(f"A is {M}x{K} but the weights are {K2}x{N}")
    if My != M or Ny != N:
        raise ValueError(f"Y is {My}x{Ny}, not {M}x{N}")
    _call(device, "fp4lin_experts_forward_mx", A.data_ptr(), W.data_ptr(), _code(A),
          _row_end(row_end, E), E, M, K, N, lda, ldw, Y.data_ptr(), _code(Y), ldy, ws.data_ptr(),
          _nbytes(ws), _queue(stream, device))


def fp4lin_experts_apply_mx(A, Wq, Ws, row_end, Y, ws, stream=None):
    M, K, lda = _rows(A, "A")
    My, N, ldy = _rows(Y, "Y")
    E = row_end.numel()
    device = _gpu(("A", A), ("Wq", Wq), ("Ws", Ws), ("row_end", row_end), ("Y", Y), ("ws", ws))
    if My != M:
        raise ValueError(f"Y has {My} rows, A {M}")
    byte = _torch().uint8
    for name, t, want in _packed_bytes(Wq, Ws, E, K, N):
        if t.dtype != byte or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous uint8 tensor")
        if t.numel() != want:
            raise ValueError(f"{name} holds {t.numel()} bytes, not {want}")
    _call(device, "fp4lin_experts_apply_mx", A.data_ptr(), _code(A), Wq.data_ptr(), Ws.data_ptr(),
          _row_end(row_end, E), E, M, K, N, lda, Y.data_ptr(), _code(Y), ldy, ws.data_ptr(),
          _nbytes(ws), _queue(stream, device))


def fp4lin_experts_dgrad_mx(dY, W, row_end, dX, ws, stream=None):
    M, N, lddy = _rows(dY, "dY")
    E, K, N2, ldw = _experts_weight(W, "W")
    Mx, Kx, lddx = _rows(dX, "dX")
    device = _gpu(("dY", dY), ("W", W), ("row_end", row_end), ("dX", dX), ("ws", ws))
    _same_dtype(dY, W, "dY and W")
    if N2 != N:
        raise ValueError(f"dY is {M}x{N} but the weights are {K}x{N2}")
    if Mx != M or Kx != K:
        raise ValueError(f"dX is {Mx}x{Kx}, not {M}x{K}")
    _call(device, "fp4lin_experts_dgrad_mx", dY.data_ptr(), W.data_ptr(), _code(dY),
          _row_end(row_end, E), E, M, K, N, lddy, ldw, dX.data_ptr(), _code(dX), lddx,
          ws.data_ptr(), _nbytes(ws), _queue(stream, device))


def fp4lin_experts_wgrad_mx(A, dY, row_end, dW, ws, stream=None):
    M, K, lda = _rows(A, "A")
    My, N, lddy = _rows(dY, "dY")
    E, Kw, Nw, lddw = _experts_weight(dW, "dW")
    device = _gpu(("A", A), ("dY", dY), ("row_end", row_end), ("dW", dW), ("ws", ws))
    _same_dtype(A, dY, "A and dY")
    if My != M:
        raise ValueError(f"dY has {My} rows, A {M}")
    if Kw != K or Nw != N:
        raise ValueError(f"dW holds {Kw}x{Nw} matrices, not {K}x{N}")
    _call(device, "fp4lin_experts_wgrad_mx", A.data_ptr(), dY.data_ptr(), _code(A),
          _row_end(row_end, E), E, M, K, N, lda, lddy, dW.data_ptr(), _code(dW), lddw,
          ws.data_ptr(), _nbytes(ws), _queue(stream, device))


def experts_quantize_weight_mx(W, stream=None):
    """Weights (E, K, N) for experts_apply_mx. Returns (Wq uint8 (E, N,
    packed_ld(K)), Ws uint8 (steps, E, N, 4)), the scales step-major."""
    torch = _torch()
    E, K, N, _ = _experts_weight(W, "W")
    with _on(W, stream):
        Wq = torch.empty((E, N, packed_ld(K)), dtype=torch.uint8, device=W.device)
        Ws = torch.empty((mx_scales_ld(K) // 4, E, N, 4), dtype=torch.uint8, device=W.device)
        fp4lin_experts_quantize_weight_mx(W, Wq, Ws)
    return Wq, Ws


def experts_forward_mx(A, W, row_end, out_dtype=None, stream=None):
    """Y (M, N) = the rows of A (M, K), sorted by expert, times their expert's
    weight of W (E, K, N), both quantized to micro-scaled FP4. Expert e owns
    the rows row_end[e-1] .. row_end[e] - 1 (int32, on the GPU); rows past
    row_end[-1] give zeros. out_dtype: float32 (default) or bfloat16."""
    torch = _torch()
    M, K, _ = _rows(A, "A")
    E, _, N, _ = _experts_weight(W, "W")
    with _on(A, stream):
        Y = torch.empty((M, N), dtype=out_dtype or torch.float32, device=A.device)
        ws = _experts_ws(_lib.EXPERTS_FORWARD, E, M, K, N, A.device, "experts_forward_mx")
        fp4lin_experts_forward_mx(A, W, row_end, Y, ws)
    return Y


def experts_apply_mx(A, Wq, Ws, row_end, out_dtype=None, stream=None):
    """experts_forward_mx with weights from experts_quantize_weight_mx."""
    torch = _torch()
    M, K, _ = _rows(A, "A")
    _need(Wq.dim() == 3, "Wq must be (experts, columns, packed bytes)")
    E, N, _ = Wq.shape
    with _on(A, stream):
        Y = torch.empty((M, N), dtype=out_dtype or torch.float32, device=A.device)
        ws = _experts_ws(_lib.EXPERTS_APPLY, E, M, K, N, A.device, "experts_apply_mx")
        fp4lin_experts_apply_mx(A, Wq, Ws, row_end, Y, ws)
    return Y


def experts_dgrad_mx(dY, W, row_end, out_dtype=None, stream=None):
    """dX (M, K) = the rows of dY (M, N) times their expert's weight transposed."""
    torch = _torch()
    M, N, _ = _rows(dY, "dY")
    E, K, _, _ = _experts_weight(W, "W")
    with _on(dY, stream):
        dX = torch.empty((M, K), dtype=out_dtype or torch.float32, device=dY.device)
        ws = _experts_ws(_lib.EXPERTS_DGRAD, E, M, K, N, dY.device, "experts_dgrad_mx")
        fp4lin_experts_dgrad_mx(dY, W, row_end, dX, ws)
    return dX


def experts_wgrad_mx(A, dY, row_end, out_dtype=None, stream=None):
    """dW (E, K, N): each expert's rows of A (M, K) transposed times its rows of
    dY (M, N); zeros for an expert without rows."""
    torch = _torch()
    M, K, _ = _rows(A, "A")
    _, N, _ = _rows(dY, "dY")
    E = row_end.numel()
    with _on(A, stream):
        dW = torch.empty((E, K, N), dtype=out_dtype or torch.float32, device=A.device)
        ws = _experts_ws(_lib.EXPERTS_WGRAD, E, M, K, N, A.device, "experts_wgrad_mx")
        fp4lin_experts_wgrad_mx(A, dY, row_end, dW, ws)
    return dW


# ---- head loss -------------------------------------------------------------------------
def head_loss_workspace_bytes(dtype_code, by_vocab, T, H, V, ldx, ldw, backward=False) -> int:
    f = lib().fp4lin_head_loss_backward_workspace_bytes if backward else \
        lib().fp4lin_head_loss_workspace_bytes
    return int(f(dtype_code, int(bool(by_vocab)), T, H, V, ldx, ldw))


def _head_sizes(X, W, target, by_vocab):
    """(T, H, V, ldx, ldw) of matching X, W and targets."""
    T, H, ldx = _rows(X, "X")
    r, c, ldw = _rows(W, "W")
    _same_dtype(X, W, "X and W")
    if (c if by_vocab else r) != H:
        raise ValueError(f"X is {T}x{H} but W is {r}x{c}" + (" (vocabulary first)" if by_vocab else ""))
    if target.dtype != _torch().int32 or target.dim() != 1 or not target.is_contiguous():
        raise TypeError("target must be a contiguous int32 vector")
    if target.numel() != T:
        raise ValueError(f"{target.numel()} targets for {T} rows")
    return T, H, r if by_vocab else c, ldx, ldw


def _row_floats(t, T, name):
    if t.dtype != _torch().float32 or t.dim() != 1 or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 vector")
    if t.numel() != T:
        raise ValueError(f"{name} has {t.numel()} entries for {T} rows")
    return t.data_ptr()


def fp4lin_head_loss(X, W, target, loss, lse, ws, by_vocab=False, stream=None):
    T, H, V, ldx, ldw = _head_sizes(X, W, target, by_vocab)
    device = _gpu(("X", X), ("W", W), ("target", target), ("loss", loss), ("lse", lse), ("ws", ws))
    _call(device, "fp4lin_head_loss", X.data_ptr(), W.data_ptr(), _code(X), int(bool(by_vocab)),
          target.data_ptr(), T, H, V, ldx, ldw, _row_floats(loss, T, "loss"),
          _row_floats(lse, T, "lse"), ws.data_ptr(), _nbytes(ws), _queue(stream, device))


def fp4lin_head_loss_backward(X, W, target, lse, dloss, dX, dW, ws, by_vocab=False, stream=None):
    T, H, V, ldx, ldw = _head_sizes(X, W, target, by_vocab)
    device = _gpu(("X", X), ("W", W), ("target", target), ("lse", lse), ("dloss", dloss), ("dX", dX),
                  ("dW", dW), ("ws", ws))
    _same_dtype(X, dX, "X and dX")
    _same_dtype(X, dW, "X and dW")
    Tx, Hx, lddx = _rows(dX, "dX")
    r, c, lddw = _rows(dW, "dW")
    if Tx != T or Hx != H:
        raise ValueError(f"dX is {Tx}x{Hx}, not {T}x{H}")
    if dW.shape != W.shape:
        raise ValueError(f"dW is {r}x{c}, W {W.shape[0]}x{W.shape[1]}")
    _call(device, "fp4lin_head_loss_backward", X.data_ptr(), W.data_ptr(), _code(X),
          int(bool(by_vocab)), target.data_ptr(), _row_floats(lse, T, "lse"),
          _row_floats(dloss, T, "dloss"), T, H, V, ldx, ldw, dX.data_ptr(), lddx, dW.data_ptr(),
          lddw, ws.data_ptr(), _nbytes(ws), _queue(stream, device))


def _aligned(t):
    """t, or a copy of it where its first element is not 16-byte aligned."""
    return t if t.data_ptr() % 16 == 0 else t.clone(memory_format=_torch().contiguous_format)


def _head_ws(X, sizes, by_vocab, backward, where):
    torch = _torch()
    n = head_loss_workspace_bytes(_code(X), by_vocab, *sizes, backward)
    if n == 0:
        raise Fp4linError(_lib.ERR_SHAPE, where)
    return torch.empty(n, dtype=torch.uint8, device=X.device)


def head_loss(X, W, target, by_vocab=False, stream=None):
    """Cross entropy of the rows' logits X W against target (int32), without
    keeping the logits. X is (T, H), W (H, V) or with by_vocab (V, H); float32 or
    bfloat16. Returns (loss, lse), float32 of T entries; a row whose target
    lies outside [0, V) has loss 0."""
    torch = _torch()
    _gpu(("X", X), ("W", W))
    with _on(X, stream):
        X, W = _aligned(X), _aligned(W)
        sizes = _head_sizes(X, W, target, by_vocab)
        ws = _head_ws(X, sizes, by_vocab, False, "head_loss")
        loss = torch.empty(sizes[0], dtype=torch.float32, device=X.device)
        lse = torch.empty(sizes[0], dtype=torch.float32, device=X.device)
        fp4lin_head_loss(X, W, target, loss, lse, ws, by_vocab)
    return loss, lse


def head_loss_backward(X, W, target, lse, dloss, by_vocab=False, stream=None):
    """Gradients of sum(dloss * loss) of head_loss: (dX, dW), of X's and W's
    shape and dtype. lse is head_loss's, dloss float32 of T entries."""
    torch = _torch()
    _gpu(("X", X), ("W", W))
    with _on(X, stream):
        X, W = _aligned(X), _aligned(W)
        sizes = _head_sizes(X, W, target, by_vocab)
        ws = _head_ws(X, sizes, by_vocab, True, "head_loss_backward")
        dX = torch.empty((sizes[0], sizes[1]), dtype=X.dtype, device=X.device)
        dW = torch.empty(tuple(W.shape), dtype=W.dtype, device=W.device)
        fp4lin_head_loss_backward(X, W, target, lse, dloss, dX, dW, ws, by_vocab)
    return dX, dW


# ---- gradient norm and clipping ----------------------------------------------------------
def clip_workspace_bytes(count: int, elements: int) -> int:
    return int(lib().fp4lin_clip_workspace_bytes(count, elements))


def _dense(t, name):
    """A tensor whose elements fill its memory without gaps or overlaps."""
    at = 1
    for stride, size in sorted((t.stride(d), t.shape[d]) for d in range(t.dim()) if t.shape[d] > 1):
        if stride != at and t.numel() > 0:
            raise ValueError(f"{name} must be dense in memory")
        at *= size


def _grads(tensors, out):
    """The C array of a list of gradients and its outputs, their number and
    elements, and the GPU they are on."""
    torch = _torch()
    T = torch.Tensor
    tensors = list(tensors)
    own = out is None
    out = tensors if own else list(out)
    count = len(tensors)
    _need(count > 0, "no gradients")
    _need(len(out) == count, f"{len(out)} outputs for {count} gradients")
    both = tensors if own else tensors + out
    # whole lists at once: a call on many small tensors spends its time here
    devices = set(map(T.get_device, both))
    if len(devices) != 1 or min(devices) < 0:
        for t in both:
            _dev(t, "gradient")
        raise ValueError("the gradients and outputs must be on one GPU")
    codes = list(map(_code, tensors))
    if not own and codes != list(map(_code, out)):
        raise TypeError("an output must have its gradient's dtype")
    if not own and list(map(T.size, tensors)) != list(map(T.size, out)):
        raise ValueError("an output must have its gradient's shape")
    if not all(map(T.is_contiguous, both)):
        for i, (g, o) in enumerate(zip(tensors, out)):
            _dense(g, f"gradient {i}")
            _need(g.stride() == o.stride() or (g.is_contiguous() and o.is_contiguous()),
                  f"output {i} must have the strides of gradient {i}")
    sizes = list(map(T.numel, tensors))
    pointers = list(map(T.data_ptr, tensors))
    rows = zip(pointers, pointers if own else map(T.data_ptr, out), sizes, codes)
    data = struct.pack("QQqi4x" * count, *itertools.chain.from_iterable(rows))
    return (_lib.Grad * count).from_buffer_copy(data), count, sum(sizes), devices.pop()


def _norm_out(norm, ws, device):
    """Checks that norm can take the call's float32 and that norm and ws are on the
    gradients' GPU."""
    if _gpu(("norm", norm), ("ws", ws)) != device:
        raise ValueError(f"norm and ws are on {norm.device}, the gradients on cuda:{device}")
    if norm.dtype != _torch().float32:
        raise TypeError("norm must be float32")
    _need(norm.numel() == 1, f"norm has {norm.numel()} elements, not one")


def fp4lin_grad_norm(tensors, norm, ws, stream=None):
    array, count, _, device = _grads(tensors, None)
    _norm_out(norm, ws, device)
    _call(device, "fp4lin_grad_norm", array, count, norm.data_ptr(), ws.data_ptr(), _nbytes(ws),
          _queue(stream, device))


def fp4lin_clip_grads(tensors, max_norm, norm, ws, out=None, stream=None):
    array, count, _, device = _grads(tensors, out)
    _norm_out(norm, ws, device)
    _call(device, "fp4lin_clip_grads", array, count, float(max_norm), norm.data_ptr(),
          ws.data_ptr(), _nbytes(ws), _queue(stream, device))


def _clip(tensors, max_norm, out, stream):
    torch = _torch()
    tensors = list(tensors)
    array, count, elements, device = _grads(tensors, out)
    with _on(tensors[0], stream):
        n = lib().fp4lin_clip_workspace_bytes(count, elements)
        ws = torch.empty(n, dtype=torch.uint8, device=tensors[0].device)
        norm = torch.empty((), dtype=torch.float32, device=tensors[0].device)
        args = (norm.data_ptr(), ws.data_ptr(), n, _queue(None, device))
        if max_norm is None:
            _check(lib().fp4lin_grad_norm(array, count, *args), "grad_norm")
        else:
            _check(lib().fp4lin_clip_grads(array, count, float(max_norm), *args), "clip_grads")
    return norm


def grad_norm(tensors, stream=None):
    """2-norm of all elements of a list of float32 or bfloat16 tensors (a
    float32 scalar on the GPU)."""
    return _clip(tensors, None, None, stream)


def clip_grads(tensors, max_norm, out=None, stream=None):
    """Scales the tensors by min(1, max_norm / (norm + 1e-6)), norm their global
    2-norm, in place or into the list `out`; returns norm (on the GPU). No output may
    overlap another tensor of the lists but its own gradient: a gradient that two
    weights share is listed once."""
    return _clip(tensors, max_norm, out, stream)
