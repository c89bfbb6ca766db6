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


def _needed(workspace, need, device):
    """The workspace of a call that may need none"""
    return None if workspace is None and not need else _workspace(workspace, need, device)


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
        ws = _needed(workspace, L.gemmq_rms_i8_grad_workspace(ty, M, K), h.device)
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
    """Bytes of rms_i8_grad's workspace for rows of `dtype` [M, K] with a dw (0: none)."""
    L = lib_i8()
    return L.gemmq_rms_i8_grad_workspace(_type(dtype, "dtype"), M, K)


ACT_NONE, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU = range(5)  # GEMMQ_ACT_*


def _act_product(name, w, sw, pair, x, xq, sx, bias, act, residual, pre, up, out, out_dtype):
    """The product of gemm_i8_act (x None) or linear_i8_act, or with pair = (wu, swu, bias_up)
    of their gated forms, on the current stream."""
    L = _i8._fns
    dev = w.get_device()
    N, K = w.shape
    M = (xq if x is None else x).shape[0]
    torch = _i8._torch
    f32 = torch.float32
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or (f32 if x is None else x.dtype), device=w.device)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise TypeError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
    dt = out.dtype
    args = [w.data_ptr(), _i8_matrix(w, "w", N, K, dev), _vector(sw, "sw", f32, N, dev)]
    if pair is not None:
        wu, swu, bias_up = pair
        args += [wu.data_ptr(), _i8_matrix(wu, "wu", N, K, dev), _vector(swu, "swu", f32, N, dev)]
    if x is not None:
        if xq is None:
            xq = _new_i8(M, K, w.device)
        if sx is None:
            sx = torch.empty(M, dtype=f32, device=w.device)
        args += [_type(x.dtype, "x"), x.data_ptr(), _matrix(x, "x", None, M, K, dev)]
    args += [xq.data_ptr(), _i8_matrix(xq, "xq", M, K, dev), _vector(sx, "sx", f32, M, dev),
             None if bias is None else _vector(bias, "bias", f32, N, dev)]
    if pair is not None:
        args += [None if bias_up is None else _vector(bias_up, "bias_up", f32, N, dev), act]
    else:
        args += [act, *_optional(residual, "residual", dt, M, N, dev)]
    args += [_type(dt, "out"), out.data_ptr(), _matrix(out, "out", None, M, N, dev),
             *_optional(pre, "pre", dt, M, N, dev)]
    if pair is not None:
        args += _optional(up, "up", dt, M, N, dev)
    _check(getattr(L, name)(*args, M, N, K, _here(dev)), name)
    return out


def gemm_i8_act(w, sw, xq, sx, act, bias=None, residual=None, pre=None, out=None, out_dtype=None,
                stream=None):
    """act(z) + residual with z = (sx xq) (sw w)^T + bias (gemmq_gemm_i8_act), act one of
    ACT_*: f32, bf16 or f16 [M, N] (`out_dtype`, f32 by default).  residual and pre are of
    the result's type; residual may be `out` itself, and pre, when given, receives z."""
    _i8._fns or lib_i8()
    _tracked(sw, sx, bias, residual)
    at = _elsewhere(w, w.get_device(), stream)
    if at is not None:
        with at:
            return gemm_i8_act(w, sw, xq, sx, act, bias, residual, pre, out, out_dtype)
    return _act_product("gemmq_gemm_i8_act", w, sw, None, None, xq, sx, bias, act, residual, pre,
                        None, out, out_dtype)


def linear_i8_act(w, sw, x, act, bias=None, residual=None, pre=None, out=None, out_dtype=None,
                  xq=None, sx=None, stream=None):
    """gemm_i8_act on activations x (f32, bf16 or f16 [M, K]), quantized per token
    (gemmq_linear_i8_act): [M, N] in `out_dtype` (x's by default).  out and pre may lie in
    x's place."""
    _i8._fns or lib_i8()
    _tracked(sw, x, bias, residual)
    at = _elsewhere(w, w.get_device(), stream)
    if at is not None:
        with at:
            return linear_i8_act(w, sw, x, act, bias, residual, pre, out, out_dtype, xq, sx)
    return _act_product("gemmq_linear_i8_act", w, sw, None, x, xq, sx, bias, act, residual, pre,
                        None, out, out_dtype)


def gemm_i8_gate(w, sw, wu, swu, xq, sx, act=ACT_SILU, bias=None, bias_up=None, pre=None, up=None,
                 out=None, out_dtype=None, stream=None):
    """act(z) u for the products z and u of two int8 matrices [N, K] with the same
    activations (gemmq_gemm_i8_gate); pre and up, when given, receive z and u."""
    _i8._fns or lib_i8()
    _tracked(sw, swu, sx, bias, bias_up)
    at = _elsewhere(w, w.get_device(), stream)
    if at is not None:
        with at:
            return gemm_i8_gate(w, sw, wu, swu, xq, sx, act, bias, bias_up, pre, up, out, out_dtype)
    return _act_product("gemmq_gemm_i8_gate", w, sw, (wu, swu, bias_up), None, xq, sx, bias, act,
                        None, pre, up, out, out_dtype)


def linear_i8_gate(w, sw, wu, swu, x, act=ACT_SILU, bias=None, bias_up=None, pre=None, up=None,
                   out=None, out_dtype=None, xq=None, sx=None, stream=None):
    """gemm_i8_gate on activations x (f32, bf16 or f16 [M, K]), quantized per token
    (gemmq_linear_i8_gate): the gate and up projections of a feed-forward block.  out, pre
    and up may lie in x's place."""
    _i8._fns or lib_i8()
    _tracked(sw, swu, x, bias, bias_up)
    at = _elsewhere(w, w.get_device(), stream)
    if at is not None:
        with at:
            return linear_i8_gate(w, sw, wu, swu, x, act, bias, bias_up, pre, up, out, out_dtype,
                                  xq, sx)
    return _act_product("gemmq_linear_i8_gate", w, sw, (wu, swu, bias_up), x, xq, sx, bias, act,
                        None, pre, up, out, out_dtype)


def act_grad(act, z, dy, up=None, out=None, dup=None, dbias=None, dbias_up=None, workspace=None,
             stream=None):
    """The gradients behind linear_i8_act and, with `up`, linear_i8_gate (gemmq_act_grad):
    dz = dy act'(z), or dz = dy up act'(z) and dup = dy act(z), for linear_i8_grad to take
    on.  z, dy and up [M, N] of one type.  Returns (dz, dup), dup None without `up`; dbias
    and dbias_up, when given, f32 [N], receive the sums of dz and dup over the rows.
    `workspace`: at least act_grad_workspace bytes, or None."""
    L = _i8._fns or lib_i8()
    _tracked(z, dy, up)
    dev = z.get_device()
    at = _elsewhere(z, dev, stream)
    if at is not None:
        with at:
            return act_grad(act, z, dy, up, out, dup, dbias, dbias_up, workspace)
    M, N = z.shape
    torch = _i8._torch
    dt, f32 = z.dtype, torch.float32
    ty = _type(dt, "z")
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=z.device)
    if dup is None and up is not None:
        dup = torch.empty((M, N), dtype=dt, device=z.device)
    ws = None
    if dbias is not None or dbias_up is not None:
        ws = _needed(workspace, L.gemmq_act_grad_workspace(ty, M, N), z.device)
    u, ldu = _optional(up, "up", dt, M, N, dev)
    du, lddu = _optional(dup, "dup", dt, M, N, dev)
    _check(L.gemmq_act_grad(
        act, ty, z.data_ptr(), _matrix(z, "z", dt, M, N, dev), u, ldu, dy.data_ptr(),
        _matrix(dy, "dy", dt, M, N, dev), out.data_ptr(), _matrix(out, "out", dt, M, N, dev), du,
        lddu, None if dbias is None else _vector(dbias, "dbias", f32, N, dev),
        None if dbias_up is None else _vector(dbias_up, "dbias_up", f32, N, dev), M, N,
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes, _here(dev)),
        "gemmq_act_grad")
    return out, dup


def act_grad_workspace(dtype, M, N):
    """Bytes of act_grad's workspace for [M, N] of `dtype`, with a bias's gradient (0: none)."""
    L = lib_i8()
    return L.gemmq_act_grad_workspace(_type(dtype, "dtype"), M, N)


def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, out=None, logprob=None,
           workspace=None, stream=None):
    """One token a row of logits (f32, bf16 or f16 [M, N]; gemmq_sample) from the random
    numbers u, f32 [M] in [0, 1).  Each row's settings, or None: temperature (<= 0 greedy),
    top_p and min_p f32 [M], top_k int32 [M].  Returns (token int64 [M], logprob f32 [M]):
    the logarithm of the token's share of what the settings leave; -1 and NaN for a row
    without a token to draw.  `workspace`: at least sample_workspace bytes, or None."""
    L = _i8._fns or lib_i8()
    _tracked(logits, u, temperature, top_p, min_p)
    dev = logits.get_device()
    at = _elsewhere(logits, dev, stream)
    if at is not None:
        with at:
            return sample(logits, u, temperature, top_k, top_p, min_p, out, logprob, workspace)
    M, N = logits.shape
    torch = _i8._torch
    f32 = torch.float32
    if out is None:
        out = torch.empty(M, dtype=torch.int64, device=logits.device)
    if logprob is None:
        logprob = torch.empty(M, dtype=f32, device=logits.device)
    ws = _needed(workspace, L.gemmq_sample_workspace(M, N), logits.device)
    _check(L.gemmq_sample(
        _type(logits.dtype, "logits"), logits.data_ptr(), _matrix(logits, "logits", None, M, N, dev),
        None if temperature is None else _vector(temperature, "temperature", f32, M, dev),
        None if top_k is None else _vector(top_k, "top_k", torch.int32, M, dev),
        None if top_p is None else _vector(top_p, "top_p", f32, M, dev),
        None if min_p is None else _vector(min_p, "min_p", f32, M, dev), _vector(u, "u", f32, M, dev),
        _vector(out, "out", torch.int64, M, dev), _vector(logprob, "logprob", f32, M, dev), M, N,
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes, _here(dev)),
        "gemmq_sample")
    return out, logprob


def sample_workspace(M, N):
    """Bytes of sample's workspace for logits [M, N] (0: none)."""
    return lib_i8().gemmq_sample_workspace(M, N)
