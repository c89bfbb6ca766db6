"""ctypes binding of libgemmq's int8 half (include/gemmq_i8.h).

Matrices are torch tensors whose rows may lie further apart than they are wide
(a slice of columns of a wider buffer): the last dimension has stride 1.  int8
matrices have rows that start 16 bytes apart or a multiple of it; `quantize_i8`
allocates such a matrix for any width.  Every call runs on the device of its
tensors, on `stream` or that device's current stream, and allocates what it is
not given on that stream.
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


def lib_i8():
    """libgemmq with the int8 entry points' types set (loaded once)."""
    global _fns
    if _fns is None:
        L = _lib.lib()
        for name, (res, args) in EXPORTS_I8.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        if L.gemmq_i8_abi_version() != I8_ABI_VERSION:
            raise GemmqError(-101, "libgemmq int8 ABI %d, binding expects %d"
                             % (L.gemmq_i8_abi_version(), I8_ABI_VERSION))
        import torch

        _types.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
        _fns = L
    return _fns


_types = {}


def _type(dtype, name):
    t = _types.get(dtype)
    if t is None:
        raise TypeError("%s must be float32, bfloat16 or float16, got %s" % (name, dtype))
    return t


def _matrix(t, name, dtype, shape, device):
    """The row pitch of a 2-d device tensor, in elements."""
    if not t.is_cuda:
        raise TypeError("%s must be a device tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != shape):
        raise ValueError("%s must be %s, got %s"
                         % (name, "2-d" if shape is None else shape, tuple(t.shape)))
    rows, cols = t.shape
    s = t.stride()
    if cols > 1 and s[1] != 1:
        raise ValueError("%s must have consecutive values in its rows" % name)
    # a single row has no next one: any pitch describes it
    return s[0] if rows > 1 else -(-cols // 4) * 4


def _i8_matrix(t, name, shape, device):
    """The row pitch of an int8 matrix; its rows lie multiples of 16 bytes apart,
    and each row's bytes up to a multiple of 16 belong to the tensor's memory."""
    import torch

    ld = _matrix(t, name, torch.int8, shape, device)
    rows, cols = t.shape
    if rows == 1:
        ld = -(-cols // 16) * 16
    if rows == 0:
        return -(-max(cols, 1) // 16) * 16
    end = t.storage_offset() + (rows - 1) * ld + -(-cols // 16) * 16
    if ld % 16 or t.data_ptr() % 16 or end > t.untyped_storage().nbytes():
        raise ValueError("%s: the rows of an int8 matrix start on multiples of 16 bytes and have "
                         "their last 16 bytes in memory (quantize_i8 allocates one)" % name)
    return ld


def _vector(t, name, dtype, n, device):
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError("%s must have shape (%d,), got %s" % (name, n, tuple(t.shape)))
    if n > 1 and t.stride(0) != 1:
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


class _On:
    """The device and stream of one call: enters the tensors' device where it is
    not the current one, and `stream` where one is given, so that what the call
    allocates belongs to the stream that uses it."""

    __slots__ = ("dev", "arg", "handle", "_a", "_b")

    def __init__(self, device, stream):
        if device.type != "cuda":
            raise TypeError("the tensors must be device tensors")
        self.dev, self.arg, self._a, self._b = device, stream, None, None

    def __enter__(self):
        import torch

        if torch.cuda.current_device() != self.dev.index:
            self._a = torch.cuda.device(self.dev)
            self._a.__enter__()
        if self.arg is not None:
            s = self.arg
            if not isinstance(s, torch.cuda.Stream):
                h = s.cuda_stream if hasattr(s, "cuda_stream") else int(s)
                s = torch.cuda.ExternalStream(h, self.dev) if h else torch.cuda.default_stream(self.dev)
            if s.device != self.dev:
                if self._a is not None:
                    self._a.__exit__(None, None, None)
                raise ValueError("stream is on %s, the tensors on %s" % (s.device, self.dev))
            self._b = torch.cuda.stream(s)
            self._b.__enter__()
        self.handle = torch.cuda.current_stream().cuda_stream or None
        return self

    def __exit__(self, *e):
        if self._b is not None:
            self._b.__exit__(*e)
        if self._a is not None:
            self._a.__exit__(*e)


def _new_i8(rows, cols, device):
    import torch

    pitch = -(-max(cols, 1) // 16) * 16
    return torch.empty((rows, pitch), dtype=torch.int8, device=device)[:, :cols]


def _workspace(ws, need, device):
    """(pointer, bytes, owner) of the given or a new workspace"""
    import torch

    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    elif not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % (device,))
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def quantize_i8(x, out=None, scale=None, stream=None):
    """Rows of x (f32, bf16 or f16 [M, K]) to int8 with one f32 scale each
    (gemmq_quantize_i8): returns (int8 [M, K], f32 [M]).  Activations per token,
    or weights [N, K] per output channel."""
    import torch

    L = lib_i8()
    ty = _type(x.dtype, "x")
    ldx = _matrix(x, "x", None, None, None)
    M, K = x.shape
    with _On(x.device, stream) as on:
        if out is None:
            out = _new_i8(M, K, x.device)
        if scale is None:
            scale = torch.empty(M, dtype=torch.float32, device=x.device)
        _check(L.gemmq_quantize_i8(ty, x.data_ptr(), ldx, out.data_ptr(),
                                   _i8_matrix(out, "out", (M, K), x.device),
                                   _vector(scale, "scale", torch.float32, M, x.device), M, K,
                                   on.handle), "gemmq_quantize_i8")
    return out, scale


def gemm_i8(w, sw, xq, sx, bias=None, out=None, out_dtype=None, stream=None):
    """y = (sx xq) (sw w)^T + bias for int8 w [N, K], xq [M, K] and their scales
    (gemmq_gemm_i8): f32, bf16 or f16 [M, N] (`out_dtype`, f32 by default)."""
    import torch

    L = lib_i8()
    dev = w.device
    N, K = w.shape
    M = xq.shape[0]
    with _On(dev, stream) as on:
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype or torch.float32, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
        _check(L.gemmq_gemm_i8(
            w.data_ptr(), _i8_matrix(w, "w", None, dev), _vector(sw, "sw", torch.float32, N, dev),
            xq.data_ptr(), _i8_matrix(xq, "xq", (M, K), dev),
            _vector(sx, "sx", torch.float32, M, dev),
            None if bias is None else _vector(bias, "bias", torch.float32, N, dev),
            _type(out.dtype, "out"), out.data_ptr(), _matrix(out, "out", None, (M, N), dev), M, N,
            K, on.handle), "gemmq_gemm_i8")
    return out


def linear_i8(w, sw, x, bias=None, out=None, out_dtype=None, xq=None, sx=None, stream=None):
    """The linear layer on activations x (f32, bf16 or f16 [M, K]): quantize per
    token, then gemm_i8 (gemmq_linear_i8).  Returns [M, N] in `out_dtype` (x's by
    default); xq and sx, when given, receive the quantized activations."""
    import torch

    L = lib_i8()
    dev = w.device
    N, K = w.shape
    M = x.shape[0]
    with _On(dev, stream) as on:
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype or x.dtype, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
        if xq is None:
            xq = _new_i8(M, K, dev)
        if sx is None:
            sx = torch.empty(M, dtype=torch.float32, device=dev)
        _check(L.gemmq_linear_i8(
            w.data_ptr(), _i8_matrix(w, "w", None, dev), _vector(sw, "sw", torch.float32, N, dev),
            _type(x.dtype, "x"), x.data_ptr(), _matrix(x, "x", None, (M, K), dev),
            xq.data_ptr(), _i8_matrix(xq, "xq", (M, K), dev),
            _vector(sx, "sx", torch.float32, M, dev),
            None if bias is None else _vector(bias, "bias", torch.float32, N, dev),
            _type(out.dtype, "out"), out.data_ptr(), _matrix(out, "out", None, (M, N), dev), M, N,
            K, on.handle), "gemmq_linear_i8")
    return out


def linear_i8_grad(w, sw, dy, out=None, workspace=None, stream=None):
    """dx = (dy sw) w, the gradient of the linear layer with respect to its
    activations (gemmq_linear_i8_grad): dy [M, N] -> [M, K] of dy's type.
    `workspace`: a tensor of at least linear_i8_grad_workspace bytes, or None."""
    import torch

    L = lib_i8()
    dev = w.device
    N, K = w.shape
    M = dy.shape[0]
    ty = _type(dy.dtype, "dy")
    with _On(dev, stream) as on:
        if out is None:
            out = torch.empty((M, K), dtype=dy.dtype, device=dev)
        lddy = _matrix(dy, "dy", None, (M, N), dev)
        ldx = _matrix(out, "out", dy.dtype, (M, K), dev)
        p, n, own = _workspace(workspace, L.gemmq_linear_i8_grad_workspace(ty, M, N, K), dev)
        _check(L.gemmq_linear_i8_grad(
            w.data_ptr(), _i8_matrix(w, "w", None, dev), _vector(sw, "sw", torch.float32, N, dev),
            ty, dy.data_ptr(), lddy, out.data_ptr(), ldx, M, N, K, p, n, on.handle),
            "gemmq_linear_i8_grad")
        del own
    return out


def loss_i8(w, sw, xq, sx, target, loss=None, lse=None, workspace=None, stream=None):
    """Softmax cross-entropy of the logits (sx xq) (sw w)^T over the vocabulary w
    [N, K], the logits never in memory (gemmq_loss_i8): returns (loss, lse), f32
    [M]; target int64 [M], negative where a position is ignored (loss 0)."""
    import torch

    L = lib_i8()
    dev = w.device
    N, K = w.shape
    M = xq.shape[0]
    with _On(dev, stream) as on:
        if loss is None:
            loss = torch.empty(M, dtype=torch.float32, device=dev)
        if lse is None:
            lse = torch.empty(M, dtype=torch.float32, device=dev)
        p, n, own = _workspace(workspace, L.gemmq_loss_i8_workspace(M, N, K), dev)
        _check(L.gemmq_loss_i8(
            w.data_ptr(), _i8_matrix(w, "w", None, dev), _vector(sw, "sw", torch.float32, N, dev),
            xq.data_ptr(), _i8_matrix(xq, "xq", (M, K), dev),
            _vector(sx, "sx", torch.float32, M, dev),
            _vector(target, "target", torch.int64, M, dev),
            _vector(loss, "loss", torch.float32, M, dev),
            _vector(lse, "lse", torch.float32, M, dev), M, N, K, p, n, on.handle),
            "gemmq_loss_i8")
        del own
    return loss, lse


def loss_i8_grad(w, sw, xq, sx, target, lse, dloss, out=None, out_dtype=None, workspace=None,
                 stream=None):
    """The gradient of sum(dloss * loss) with respect to the dequantized hidden
    states sx xq (gemmq_loss_i8_grad): [M, K] in `out_dtype` (bf16 by default);
    lse from loss_i8."""
    import torch

    L = lib_i8()
    dev = w.device
    N, K = w.shape
    M = xq.shape[0]
    with _On(dev, stream) as on:
        if out is None:
            out = torch.empty((M, K), dtype=out_dtype or torch.bfloat16, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
        ty = _type(out.dtype, "out")
        p, n, own = _workspace(workspace, L.gemmq_loss_i8_grad_workspace(ty, M, N, K), dev)
        _check(L.gemmq_loss_i8_grad(
            w.data_ptr(), _i8_matrix(w, "w", None, dev), _vector(sw, "sw", torch.float32, N, dev),
            xq.data_ptr(), _i8_matrix(xq, "xq", (M, K), dev),
            _vector(sx, "sx", torch.float32, M, dev),
            _vector(target, "target", torch.int64, M, dev),
            _vector(lse, "lse", torch.float32, M, dev),
            _vector(dloss, "dloss", torch.float32, M, dev), ty, out.data_ptr(),
            _matrix(out, "out", None, (M, K), dev), M, N, K, p, n, on.handle),
            "gemmq_loss_i8_grad")
        del own
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
