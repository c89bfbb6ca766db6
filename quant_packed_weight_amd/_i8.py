"""ctypes binding of libgemmq's int8 half (include/gemmq_i8.h).

Matrices are torch tensors whose rows may lie further apart than they are wide
(a slice of columns of a wider buffer): the last dimension has stride 1.  int8
matrices have rows that start 16 bytes apart or a multiple of it; `quantize_i8`
allocates such a matrix for any width.  Every call runs on the device of its
tensors, on `stream` or that device's current stream, and allocates what it is
not given on that stream.

No call records an autograd graph: the gradients are calls of their own
(`linear_i8_grad`, `loss_i8_grad`), from a torch.autograd.Function's backward or by
hand.  A call on tensors that require a gradient, with grad mode on, is refused
rather than cut the graph unseen; `quantize_i8` takes parameters (leaves) all the
same, whose int8 copy is a constant.
"""
from __future__ import annotations

import ctypes

from . import _lib
from ._lib import GemmqError, _check  # noqa: F401

F32, BF16, F16 = 0, 1, 2  # GEMMQ_F32, GEMMQ_BF16, GEMMQ_F16
I8_ABI_VERSION = 1
I8_MAX_K = 131071
I8_MAX_ROWS = 1 << 24
I8_MAX_PITCH = 1 << 20
I8_MAX_OUTPUTS = 1 << 36

_P, _I, _I64, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
# every entry point include/gemmq_i8.h declares: name -> (restype, argtypes)
EXPORTS_I8 = {
    "gemmq_i8_abi_version": (_I, []),
    "gemmq_quantize_i8": (_I, [_I, _P, _I64, _P, _I64, _P, _I64, _I64, _P]),
    "gemmq_gemm_i8": (_I, [_P, _I64, _P, _P, _I64, _P, _P, _I, _P, _I64, _I64, _I64, _I64, _P]),
    "gemmq_linear_i8": (_I, [_P, _I64, _P, _I, _P, _I64, _P, _I64, _P, _P, _I, _P, _I64, _I64,
                             _I64, _I64, _P]),
    "gemmq_linear_i8_grad_workspace": (_S, [_I, _I64, _I64, _I64]),
    "gemmq_linear_i8_grad": (_I, [_P, _I64, _P, _I, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _S,
                                  _P]),
    "gemmq_loss_i8_workspace": (_S, [_I64, _I64, _I64]),
    "gemmq_loss_i8": (_I, [_P, _I64, _P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _I64, _P, _S, _P]),
    "gemmq_loss_i8_grad_workspace": (_S, [_I, _I64, _I64, _I64]),
    "gemmq_loss_i8_grad": (_I, [_P, _I64, _P, _P, _I64, _P, _P, _P, _P, _I, _P, _I64, _I64, _I64,
                                _I64, _P, _S, _P]),
}

_fns = None
_torch = None  # torch, imported with the library


def lib_i8():
    """libgemmq with the int8 entry points' types set (loaded once)."""
    global _fns, _torch
    if _fns is None:
        import torch

        L = _lib.lib()
        for name, (res, args) in EXPORTS_I8.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        if L.gemmq_i8_abi_version() != I8_ABI_VERSION:
            raise GemmqError(-101, "libgemmq int8 ABI %d, binding expects %d"
                             % (L.gemmq_i8_abi_version(), I8_ABI_VERSION))
        _types.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
        _torch = torch
        _fns = L
    return _fns


_types = {}


def _type(dtype, name):
    t = _types.get(dtype)
    if t is None:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, dtype))
    return t


def _refuse(t, name, dtype, shape, index):
    """Raises for a tensor that is not what the call needs."""
    if t.get_device() != index:
        raise ValueError("%s is on %s, not on device %s" % (name, t.device, index))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    raise ValueError("%s must be %s, got %s" % (name, shape, tuple(t.shape)))


def _matrix(t, name, dtype, rows, cols, index):
    """The row pitch of a [rows, cols] tensor on device `index`, in elements."""
    if (t.get_device() != index or t.shape != (rows, cols)
            or (dtype is not None and t.dtype != dtype)):
        _refuse(t, name, dtype, (rows, cols), index)
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("%s must have consecutive values in its rows" % name)
    # a single row has no next one: any pitch describes it, one of eight values allows
    # 16-byte accesses in every type
    return ld if rows > 1 else -(-cols // 8) * 8


def _i8_matrix(t, name, rows, cols, index):
    """The row pitch of an int8 matrix; its rows lie multiples of 16 bytes apart,
    and each row's bytes up to a multiple of 16 belong to the tensor's memory."""
    if t.get_device() != index or t.shape != (rows, cols) or t.dtype != _torch.int8:
        _refuse(t, name, _torch.int8, (rows, cols), index)
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("%s must have consecutive values in its rows" % name)
    row = -(-cols // 16) * 16
    if rows <= 1:
        ld = max(row, 16)
    if rows and (ld % 16 or t.data_ptr() % 16
                 or (row != cols and t.storage_offset() + (rows - 1) * ld + row
                     > t.untyped_storage().nbytes())):
        raise ValueError("%s: the rows of an int8 matrix start on multiples of 16 bytes and have "
                         "their last 16 bytes in memory (quantize_i8 allocates one)" % name)
    return ld


def _vector(t, name, dtype, n, index):
    if t.get_device() != index or t.shape != (n,) or t.dtype != dtype:
        _refuse(t, name, dtype, (n,), index)
    if n > 1 and t.stride(0) != 1:
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _untracked():
    """Raises where autograd would record a graph of the call."""
    if _torch.is_grad_enabled():
        raise ValueError("the int8 calls record no gradient: call them under torch.no_grad() or "
                         "on detached tensors, and linear_i8_grad or loss_i8_grad for it")


def _elsewhere(t, index, stream):
    """None where a call on tensors of t's device runs on the current stream of the
    current device; else a context in which it does: the tensors' device and
    `stream`, so that what the call allocates belongs to the stream that uses it."""
    if stream is None and index >= 0 and _torch._C._cuda_getDevice() == index:
        return None
    if index < 0:
        raise TypeError("the tensors must be device tensors")
    if stream is None:
        return _torch.cuda.device(index)
    if not isinstance(stream, _torch.cuda.Stream):
        h = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = (_torch.cuda.ExternalStream(h, t.device) if h
                  else _torch.cuda.default_stream(t.device))
    if stream.device != t.device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, t.device))
    return _torch.cuda.stream(stream)  # enters the stream's device too


def _here(index):
    """The current stream of the current device, as the C side takes it (the same
    handle as torch.cuda.current_stream's, without building a Stream for it)."""
    return _torch._C._cuda_getCurrentRawStream(index) or None


def _new_i8(rows, cols, device):
    pitch = -(-max(cols, 1) // 16) * 16
    return _torch.empty((rows, pitch), dtype=_torch.int8, device=device)[:, :cols]


def _workspace(ws, need, device):
    """A workspace of `need` bytes: the given one, or a new one"""
    if ws is None:
        return _torch.empty(max(need, 16), dtype=_torch.uint8, device=device)
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % (device,))
    return ws


def _result(out, out_dtype, default, shape, device):
    if out is None:
        return _torch.empty(shape, dtype=out_dtype or default, device=device)
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
    return out


def quantize_i8(x, out=None, scale=None, stream=None):
    """Rows of x (f32, bf16 or f16 [M, K]) to int8 with one f32 scale each
    (gemmq_quantize_i8): returns (int8 [M, K], f32 [M]).  Activations per token,
    or weights [N, K] per output channel."""
    L = _fns or lib_i8()
    ty = _type(x.dtype, "x")
    if not x.is_leaf:
        _untracked()
    at = _elsewhere(x, x.get_device(), stream)
    if at is not None:
        with at:
            return quantize_i8(x, out, scale)
    M, K = x.shape
    dev = x.get_device()
    if out is None:
        out = _new_i8(M, K, x.device)
    if scale is None:
        scale = _torch.empty(M, dtype=_torch.float32, device=x.device)
    _check(L.gemmq_quantize_i8(ty, x.data_ptr(), _matrix(x, "x", None, M, K, dev), out.data_ptr(),
                               _i8_matrix(out, "out", M, K, dev),
                               _vector(scale, "scale", _torch.float32, M, dev), M, K, _here(dev)),
           "gemmq_quantize_i8")
    return out, scale


def gemm_i8(w, sw, xq, sx, bias=None, out=None, out_dtype=None, stream=None):
    """y = (sx xq) (sw w)^T + bias for int8 w [N, K], xq [M, K] and their scales
    (gemmq_gemm_i8): f32, bf16 or f16 [M, N] (`out_dtype`, f32 by default)."""
    L = _fns or lib_i8()
    if sw.requires_grad or sx.requires_grad or (bias is not None and bias.requires_grad):
        _untracked()
    dev = w.get_device()
    at = _elsewhere(w, dev, stream)
    if at is not None:
        with at:
            return gemm_i8(w, sw, xq, sx, bias, out, out_dtype)
    N, K = w.shape
    M = xq.shape[0]
    f32 = _torch.float32
    out = _result(out, out_dtype, f32, (M, N), w.device)
    _check(L.gemmq_gemm_i8(
        w.data_ptr(), _i8_matrix(w, "w", N, K, dev), _vector(sw, "sw", f32, N, dev),
        xq.data_ptr(), _i8_matrix(xq, "xq", M, K, dev), _vector(sx, "sx", f32, M, dev),
        None if bias is None else _vector(bias, "bias", f32, N, dev), _type(out.dtype, "out"),
        out.data_ptr(), _matrix(out, "out", None, M, N, dev), M, N, K, _here(dev)),
        "gemmq_gemm_i8")
    return out


def linear_i8(w, sw, x, bias=None, out=None, out_dtype=None, xq=None, sx=None, stream=None):
    """The linear layer on activations x (f32, bf16 or f16 [M, K]): quantize per
    token, then gemm_i8 (gemmq_linear_i8).  Returns [M, N] in `out_dtype` (x's by
    default); xq and sx, when given, receive the quantized activations."""
    L = _fns or lib_i8()
    if sw.requires_grad or x.requires_grad or (bias is not None and bias.requires_grad):
        _untracked()
    dev = w.get_device()
    at = _elsewhere(w, dev, stream)
    if at is not None:
        with at:
            return linear_i8(w, sw, x, bias, out, out_dtype, xq, sx)
    N, K = w.shape
    M = x.shape[0]
    f32 = _torch.float32
    out = _result(out, out_dtype, x.dtype, (M, N), w.device)
    if xq is None:
        xq = _new_i8(M, K, w.device)
    if sx is None:
        sx = _torch.empty(M, dtype=f32, device=w.device)
    _check(L.gemmq_linear_i8(
        w.data_ptr(), _i8_matrix(w, "w", N, K, dev), _vector(sw, "sw", f32, N, dev),
        _type(x.dtype, "x"), x.data_ptr(), _matrix(x, "x", None, M, K, dev), xq.data_ptr(),
        _i8_matrix(xq, "xq", M, K, dev), _vector(sx, "sx", f32, M, dev),
        None if bias is None else _vector(bias, "bias", f32, N, dev), _type(out.dtype, "out"),
        out.data_ptr(), _matrix(out, "out", None, M, N, dev), M, N, K, _here(dev)),
        "gemmq_linear_i8")
    return out


def linear_i8_grad(w, sw, dy, out=None, workspace=None, stream=None):
    """dx = (dy sw) w, the gradient of the linear layer with respect to its
    activations (gemmq_linear_i8_grad): dy [M, N] -> [M, K] of dy's type.
    `workspace`: a tensor of at least linear_i8_grad_workspace bytes, or None."""
    L = _fns or lib_i8()
    if sw.requires_grad or dy.requires_grad:
        _untracked()
    dev = w.get_device()
    at = _elsewhere(w, dev, stream)
    if at is not None:
        with at:
            return linear_i8_grad(w, sw, dy, out, workspace)
    N, K = w.shape
    M = dy.shape[0]
    ty = _type(dy.dtype, "dy")
    if out is None:
        out = _torch.empty((M, K), dtype=dy.dtype, device=w.device)
    ws = _workspace(workspace, L.gemmq_linear_i8_grad_workspace(ty, M, N, K), w.device)
    _check(L.gemmq_linear_i8_grad(
        w.data_ptr(), _i8_matrix(w, "w", N, K, dev), _vector(sw, "sw", _torch.float32, N, dev), ty,
        dy.data_ptr(), _matrix(dy, "dy", None, M, N, dev), out.data_ptr(),
        _matrix(out, "out", dy.dtype, M, K, dev), M, N, K, ws.data_ptr(), ws.nbytes, _here(dev)),
        "gemmq_linear_i8_grad")
    return out


def loss_i8(w, sw, xq, sx, target, loss=None, lse=None, workspace=None, stream=None):
    """Softmax cross-entropy of the logits (sx xq) (sw w)^T over the vocabulary w
    [N, K], the logits never in memory (gemmq_loss_i8): returns (loss, lse), f32
    [M]; target int64 [M], negative where a position is ignored (loss 0)."""
    L = _fns or lib_i8()
    if sw.requires_grad or sx.requires_grad:
        _untracked()
    dev = w.get_device()
    at = _elsewhere(w, dev, stream)
    if at is not None:
        with at:
            return loss_i8(w, sw, xq, sx, target, loss, lse, workspace)
    N, K = w.shape
    M = xq.shape[0]
    f32 = _torch.float32
    if loss is None:
        loss = _torch.empty(M, dtype=f32, device=w.device)
    if lse is None:
        lse = _torch.empty(M, dtype=f32, device=w.device)
    ws = _workspace(workspace, L.gemmq_loss_i8_workspace(M, N, K), w.device)
    _check(L.gemmq_loss_i8(
        w.data_ptr(), _i8_matrix(w, "w", N, K, dev), _vector(sw, "sw", f32, N, dev),
        xq.data_ptr(), _i8_matrix(xq, "xq", M, K, dev), _vector(sx, "sx", f32, M, dev),
        _vector(target, "target", _torch.int64, M, dev), _vector(loss, "loss", f32, M, dev),
        _vector(lse, "lse", f32, M, dev), M, N, K, ws.data_ptr(), ws.nbytes, _here(dev)),
        "gemmq_loss_i8")
    return loss, lse


def loss_i8_grad(w, sw, xq, sx, target, lse, dloss, out=None, out_dtype=None, workspace=None,
                 stream=None):
    """The gradient of sum(dloss * loss) with respect to the dequantized hidden
    states sx xq (gemmq_loss_i8_grad): [M, K] in `out_dtype` (bf16 by default);
    lse from loss_i8."""
    L = _fns or lib_i8()
    if sw.requires_grad or sx.requires_grad or lse.requires_grad or dloss.requires_grad:
        _untracked()
    dev = w.get_device()
    at = _elsewhere(w, dev, stream)
    if at is not None:
        with at:
            return loss_i8_grad(w, sw, xq, sx, target, lse, dloss, out, out_dtype, workspace)
    N, K = w.shape
    M = xq.shape[0]
    f32 = _torch.float32
    out = _result(out, out_dtype, _torch.bfloat16, (M, K), w.device)
    ty = _type(out.dtype, "out")
    ws = _workspace(workspace, L.gemmq_loss_i8_grad_workspace(ty, M, N, K), w.device)
    _check(L.gemmq_loss_i8_grad(
        w.data_ptr(), _i8_matrix(w, "w", N, K, dev), _vector(sw, "sw", f32, N, dev),
        xq.data_ptr(), _i8_matrix(xq, "xq", M, K, dev), _vector(sx, "sx", f32, M, dev),
        _vector(target, "target", _torch.int64, M, dev), _vector(lse, "lse", f32, M, dev),
        _vector(dloss, "dloss", f32, M, dev), ty, out.data_ptr(),
        _matrix(out, "out", None, M, K, dev), M, N, K, ws.data_ptr(), ws.nbytes, _here(dev)),
        "gemmq_loss_i8_grad")
    return out


def linear_i8_grad_workspace(dtype, M, N, K):
    """Bytes of linear_i8_grad's workspace for a dy of `dtype` [M, N] and K columns."""
    L = lib_i8()
    return L.gemmq_linear_i8_grad_workspace(_type(dtype, "dtype"), M, N, K)


def loss_i8_workspace(M, N, K):
    """Bytes of loss_i8's workspace for M positions, N vocabulary rows, K columns."""
    return lib_i8().gemmq_loss_i8_workspace(M, N, K)


def loss_i8_grad_workspace(dtype, M, N, K):
    """Bytes of loss_i8_grad's workspace for a result of `dtype`."""
    L = lib_i8()
    return L.gemmq_loss_i8_grad_workspace(_type(dtype, "dtype"), M, N, K)
