"""ctypes binding of what stands between the int8 products of a decoder (the second
part of include/gemmq_i8.h).  Tensors, streams and autograd are as in the int8
product's own calls: rows may lie further apart than they are wide, every call runs on
the device of its tensors and on `stream` or that device's current stream, and records
no gradient (the `_grad` calls compute it)."""
from __future__ import annotations

from . import _i8
from ._i8 import (_check, _elsewhere, _here, _i8_matrix, _matrix, _new_i8, _type, _untracked,
                  _vector, _workspace, lib_i8)


def _tracked(*tensors):
    """Refuses tensors that a graph would have to be recorded for."""
    for t in tensors:
        if t is not None and t.requires_grad:
            _untracked()


def _optional(t, name, dtype, rows, cols, index):
    """Pointer and pitch of a matrix that may be left out"""
    return (None, 0) if t is None else (t.data_ptr(), _matrix(t, name, dtype, rows, cols, index))


def rms_i8(x, w, eps=1e-6, residual=None, hidden=None, out=None, scale=None, stream=None):
    """h = x + residual and the root-mean-square norm of h's rows, times w, as int8 rows
    with one f32 scale each (gemmq_rms_i8): x, residual f32, bf16 or f16 [M, K], w f32
    [K].  Returns (int8 [M, K], f32 [M], h); h goes to `hidden`, which may be x or
    residual, to a new tensor without one, and is x where there is no residual."""
    L = _i8._fns or lib_i8()
    _tracked(x, w, residual)
    dev = x.get_device()
    at = _elsewhere(x, dev, stream)
    if at is not None:
        with at:
            return rms_i8(x, w, eps, residual, hidden, out, scale)
    M, K = x.shape
    torch = _i8._torch
    dt = x.dtype
    if out is None:
        out = _new_i8(M, K, x.device)
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=x.device)
    if hidden is None and residual is not None:
        hidden = torch.empty((M, K), dtype=dt, device=x.device)
    r, ldr = _optional(residual, "residual", dt, M, K, dev)
    h, ldh = _optional(hidden, "hidden", dt, M, K, dev)
    _check(L.gemmq_rms_i8(
        _type(dt, "x"), x.data_ptr(), _matrix(x, "x", None, M, K, dev), r, ldr, h, ldh,
        _vector(w, "w", torch.float32, K, dev), eps, out.data_ptr(),
        _i8_matrix(out, "out", M, K, dev), _vector(scale, "scale", torch.float32, M, dev), M, K,
        _here(dev)), "gemmq_rms_i8")
    return out, scale, x if hidden is None else hidden


def rms_i8_grad(h, w, dy, dh=None, eps=1e-6, out=None, dw=None, weight_grad=True, workspace=None,
                stream=None):
    """The gradient of the norm of h's rows times w (gemmq_rms_i8_grad): dy [M, K] of h's
    type, dh (or None) what arrives at h by the residual path.  Returns (dx, dw): dx of
    h's type, which is the gradient of both x and the residual, and dw f32 [K], None
    with weight_grad=False.  `workspace`: at least rms_i8_grad_workspace bytes, or None."""
    L = _i8._fns or lib_i8()
    _tracked(h, w, dy, dh)
    dev = h.get_device()
    at = _elsewhere(h, dev, stream)
    if at is not None:
        with at:
            return rms_i8_grad(h, w, dy, dh, eps, out, dw, weight_grad, workspace)
    M, K = h.shape
    torch = _i8._torch
    dt, f32 = h.dtype, torch.float32
    ty = _type(dt, "h")
    if out is None:
        out = torch.empty((M, K), dtype=dt, device=h.device)
    ws = None
    if dw is None and weight_grad:
        dw = torch.empty(K, dtype=f32, device=h.device)
    if dw is not None:
        ws = _workspace(workspace, L.gemmq_rms_i8_grad_workspace(ty, M, K), h.device)
    d, ldd = _optional(dh, "dh", dt, M, K, dev)
    _check(L.gemmq_rms_i8_grad(
        ty, h.data_ptr(), _matrix(h, "h", None, M, K, dev), _vector(w, "w", f32, K, dev), eps,
        dy.data_ptr(), _matrix(dy, "dy", dt, M, K, dev), d, ldd, out.data_ptr(),
        _matrix(out, "out", dt, M, K, dev),
        None if dw is None else _vector(dw, "dw", f32, K, dev), M, K,
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes, _here(dev)),
        "gemmq_rms_i8_grad")
    return out, dw


def rms_i8_grad_workspace(dtype, M, K):
    """Bytes of rms_i8_grad's workspace for rows of `dtype` [M, K] with a dw."""
    L = lib_i8()
    return L.gemmq_rms_i8_grad_workspace(_type(dtype, "dtype"), M, K)
