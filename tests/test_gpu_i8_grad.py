"""The gradients of the int8 half beyond the shapes of test_gpu_i8.py, against
their definitions in 64 bits: factors larger than one piece of the workspace.

u = 2^-24 is half a step of f32, HALF half a step of the result's type.
"""
import math

import pytest
import torch

import quant_packed_weight_amd as gq
from test_gpu_i8 import FLOOR, HALF, U, Guarded, gen, i8, scales, split_error

pytestmark = pytest.mark.gpu

PLANES = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAMES = {F32: "f32", BF16: "bf16", F16: "f16"}


@pytest.fixture(scope="module", autouse=True)
def _device():
    import gpu_util

    gpu_util.device()


def names(cases):
    return ["-".join(NAMES.get(v, str(v)) for v in c) for c in cases]


def planes_of(dtype, M):
    """bf16 numbers for each value of the factor in the workspace"""
    return 2 if dtype == BF16 and M <= 8 else PLANES[dtype]


def pieces(N, step=8192):
    return [(a, min(N, a + step)) for a in range(0, N, step)]


def several(need, dtype, M, N):
    """Whether a workspace is too small for the factor of all N columns at once."""
    return need < 2 * planes_of(dtype, M) * M * N


def norm_error(dtype, M, N):
    """The error's norm relative to the result's.  The result's own rounding and one
    of the factor's that averages out: half a step each at most (f32: 16 u).  And f32
    additions: a range of columns adds sixteen at a time, each sum of n random terms
    of size sqrt(n), and a range is half of the columns at most."""
    own = 16 * U if dtype == F32 else HALF[dtype]
    return own + math.sqrt(N / 32) * U


# More bytes of factor than the 384 MB that one piece holds: two pieces or more, in
# the last case one with fewer steps (one) than the ranges that a piece is cut into.
SEVERAL = [(BF16, 2050, 100003, 40), (F16, 1030, 100003, 40), (F32, 800, 100003, 40),
           (BF16, 5000, 130001, 130), (F32, 32768, 16404, 40)]


@pytest.mark.parametrize("dtype,M,N,K", SEVERAL + [(BF16, 8, 12600001, 16)],
                         ids=names(SEVERAL + [(BF16, 8, 12600001, 16)]))
def test_linear_grad_in_several_pieces(dtype, M, N, K):
    g = gen(M + N)
    w, sw = i8(N, K, g, full=True), scales(N, g, 0.01)
    dy = torch.empty((M, N), dtype=dtype, device="cuda")
    for a, b in pieces(N, 1 << 18):
        dy[:, a:b] = torch.randn((M, b - a), generator=g, device="cuda")
    need = gq.linear_i8_grad_workspace(dtype, M, N, K)
    assert several(need, dtype, M, N)
    ws = torch.full((need + 64,), 173, dtype=torch.uint8, device="cuda")
    out = Guarded(M, K, dtype, extra=N % 4)
    dx = gq.linear_i8_grad(w, sw, dy, out=out.t, workspace=ws[:need])
    torch.cuda.synchronize()
    out.check()
    assert bool((ws[need:] == 173).all())
    ref = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(ref)
    for a, b in pieces(N):
        f, wd = dy[:, a:b].double() * sw[a:b].double(), w[a:b].double()
        ref += f @ wd
        mag += f.abs() @ wd.abs()
    # as in test_linear_grad: dy sw, its expansion, the additions, the result's rounding
    split = 2.0 ** -16 if planes_of(dtype, M) == 2 else split_error(dtype)
    tol = ((1 + planes_of(dtype, M) * N + 64) * U + split) * mag
    tol = tol + HALF[dtype] * (ref.abs() + tol) + FLOOR[dtype]
    assert bool(((dx.double() - ref).abs() <= tol).all())
    assert float((dx.double() - ref).norm() / ref.norm()) <= norm_error(dtype, M, N)
    assert torch.equal(gq.linear_i8_grad(w, sw, dy), dx)


def far_targets(M, N, g):
    """Targets on both sides of every multiple of 256, where pieces begin, as far as
    the rows reach; others anywhere, some ignored and some past the vocabulary."""
    t = torch.randint(0, N, (M,), generator=g, device="cuda")
    at = torch.arange(256, N, 256, device="cuda")
    at = torch.cat([at, at - 1])[:M]
    t[:len(at)] = at
    t = t[torch.randperm(M, generator=g, device="cuda")]
    t[5::97] = -100
    t[7::101] = N
    return t


@pytest.mark.parametrize("even", [False, True], ids=["peaked", "even"])
@pytest.mark.parametrize("dtype,M,N,K", SEVERAL + [(F32, 40, 1700003, 48), (BF16, 8, 12600001, 16)],
                         ids=names(SEVERAL + [(F32, 40, 1700003, 48), (BF16, 8, 12600001, 16)]))
def test_loss_grad_in_several_pieces(dtype, M, N, K, even):
    g = gen(M + N + 1)
    w, sw, t = i8(N, K, g), scales(N, g, K ** -0.5 / 64), far_targets(M, N, g)
    x = torch.randn((M, K), generator=g, device="cuda")
    r = w[t.clamp(0, N - 1)].float()
    x += torch.rand((M, 1), generator=g, device="cuda") * 12 * r / r.norm(dim=1, keepdim=True)
    xq, sx = gq.quantize_i8(x)
    if even:  # nearly equal logits: the target's part is most of a row's gradient
        sx = sx * 1e-3
    gw = 0.5 + torch.rand(M, generator=g, device="cuda")
    xd = xq.double() * sx.double()[:, None]
    lse = torch.full((M,), -math.inf, dtype=torch.float64, device="cuda")
    for a, b in pieces(N):
        z = xd @ (w[a:b].double() * sw[a:b].double()[:, None]).t()
        lse = torch.logaddexp(lse, torch.logsumexp(z, 1))
    need = gq.loss_i8_grad_workspace(dtype, M, N, K)
    assert several(need, dtype, M, N)
    ws = torch.full((need + 64,), 173, dtype=torch.uint8, device="cuda")
    out = Guarded(M, K, dtype, extra=N % 4)
    dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse.float(), gw, out=out.t, workspace=ws[:need])
    torch.cuda.synchronize()
    out.check()
    assert bool((ws[need:] == 173).all())
    ref = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    for a, b in pieces(N):
        wd = w[a:b].double() * sw[a:b].double()[:, None]
        p = torch.exp(xd @ wd.t() - lse.float().double()[:, None])
        here = torch.nonzero((t >= a) & (t < b))[:, 0]
        p[here, t[here] - a] -= 1.0
        ref += p @ wd
    ref *= gw.double()[:, None]
    assert bool(torch.isnan(dx[t >= N]).all()) and not bool(dx[t < 0].any())
    keep = (t >= 0) & (t < N)
    dx, ref = dx[keep].double(), ref[keep]
    off = (dx - ref).norm(dim=1) / ref.norm(dim=1)
    # a row by itself: as the layer's, and the probabilities' own error, the logit's 7 u
    # of itself, |z| <= 16
    assert float((dx - ref).norm() / ref.norm()) <= norm_error(dtype, M, N) + 112 * U
    # no row may lack its target: a row's factor of one rounding in a few large values
    # does not average out, and is at most half a step off in each
    assert float(off.max()) <= 2 * norm_error(dtype, M, N) + 224 * U
    if even and dtype == BF16:
        # the target's factor is not rounded to bf16, and the others are about 1 / N
        # each: the result's own rounding is the error
        own = (ref.bfloat16().double() - ref).norm()
        assert float((dx - ref).norm() / own) <= 1.05
    assert torch.equal(gq.loss_i8_grad(w, sw, xq, sx, t, lse.float(), gw, out_dtype=dtype)[keep].double(), dx)


# ------------------------------------------------------------------ bf16 rows as they lie
@pytest.mark.parametrize("M", [1, 2, 5, 8])
@pytest.mark.parametrize("N,K", [(8, 40), (64, 128), (520, 1000), (1000, 515), (4104, 300), (72, 20000),
                                 (12296, 515), (20000, 130)])
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "odd"])
def test_linear_grad_of_few_rows_rounds_once(M, N, K, aligned):
    # dy sw is two bf16 numbers up to eight rows, however dy lies: 2^-16 of each value is
    # left at most, beside which the result's own rounding, 2^-9.3 in the norm, is all
    g = gen(5 * M + N + K)
    w, sw = i8(N, K, g, full=True), scales(N, g, 0.01)
    dy = torch.zeros((M, N + (8 if aligned else 1)), dtype=BF16, device="cuda")[:, :N]
    dy.copy_(torch.randn((M, N), generator=g, device="cuda"))
    out = Guarded(M, K, BF16, extra=N % 4)
    dx = gq.linear_i8_grad(w, sw, dy, out=out.t)
    torch.cuda.synchronize()
    out.check()
    ref = (dy.double() * sw.double()) @ w.double()
    mag = (dy.double() * sw.double()).abs() @ w.double().abs()
    tol = ((1 + 2 * N + 64) * U + 2.0 ** -16) * mag
    assert bool(((dx.double() - ref).abs() <= tol + HALF[BF16] * (ref.abs() + tol)).all())
    # a value may lie near the middle of two bf16 numbers: 2^-16 sqrt(N) random parts of
    # the result's size sqrt(N) move the error's norm by 2^-13 of the result's at most
    own = float((ref.bfloat16().double() - ref).norm())
    assert float((dx.double() - ref).norm()) <= own + 2.0 ** -13 * float(ref.norm())
    dy[0, N - 1] = math.inf
    if M > 1:
        dy[1, 0] = math.nan
    dz = gq.linear_i8_grad(w, sw, dy)
    # an infinity stays one where the weight is not zero
    want = torch.where(w[N - 1] == 0, math.nan, w[N - 1].double() * math.inf)
    assert torch.equal(dz[0].double().nan_to_num(7.0), want.nan_to_num(7.0))
    assert M == 1 or bool(torch.isnan(dz[1]).all())
    assert torch.equal(dz[2:], dx[2:])


# The taller tiles of the product that scales W (by 64 and 128 tokens): several ranges and
# one, a last step of eight columns (N % 64 == 8) and whole ones, K off the tile's 128
@pytest.mark.parametrize("M,N,K", [(128, 12288, 4096), (96, 4096, 4096), (100, 8200, 2050),
                                   (128, 20000, 1030), (65, 4104, 11000), (100, 72, 20000),
                                   (128, 8, 20000), (64, 4104, 11000), (33, 8200, 2050),
                                   (128, 12296, 515), (64, 72, 20000), (100, 1032, 9000)])
def test_linear_grad_of_aligned_rows_in_taller_tiles(M, N, K):
    g = gen(M + N + K)
    w, sw = i8(N, K, g, full=True), scales(N, g, 0.01)
    wide = torch.full((M, N + 8 * (M % 3)), math.nan, dtype=BF16, device="cuda")
    dy = wide[:, :N]
    dy.copy_(torch.randn((M, N), generator=g, device="cuda"))
    need = gq.linear_i8_grad_workspace(BF16, M, N, K)
    ws = torch.full((need + 64,), 173, dtype=torch.uint8, device="cuda")
    out = Guarded(M, K, BF16, extra=N % 3)
    dx = gq.linear_i8_grad(w, sw, dy, out=out.t, workspace=ws[:need])
    torch.cuda.synchronize()
    out.check()
    assert bool((ws[need:] == 173).all())
    a = dy.double() * sw.double()
    ref = a @ w.double()
    mag = a.abs() @ w.double().abs()
    # as in test_linear_grad_of_aligned_rows
    tol = ((2 + N + 64) * U + 2.0 ** -8) * mag
    tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((dx.double() - ref).abs() <= tol).all())
    # one rounding of sw w, whose parts of N values average out, and one of the result
    assert float((dx.double() - ref).norm() / ref.norm()) <= norm_error(BF16, M, N)
    dy[1, N - 1], dy[2, 0] = math.nan, math.inf
    dz = gq.linear_i8_grad(w, sw, dy)
    assert bool(torch.isnan(dz[1]).all()) and not bool(torch.isfinite(dz[2]).any())
    assert torch.equal(dz[3:], dx[3:]) and torch.equal(dz[0], dx[0])


@pytest.mark.parametrize("M", [3, 20, 60, 128, 200])
@pytest.mark.parametrize("N,K", [(72, 130), (72, 20000), (200, 515), (4104, 300)])
@pytest.mark.parametrize("extra", [0, 1])
def test_linear_grad_with_an_infinite_last_scale(M, N, K, extra):
    # the last channel's scale belongs to no column past it, where the factor is zero
    g = gen(M + N)
    w, sw = i8(N, K, g, full=True), scales(N, g, 0.01)
    sw[N - 1] = math.inf
    dy = torch.zeros((M, N + extra), dtype=BF16, device="cuda")[:, :N]
    dy.copy_(torch.randn((M, N), generator=g, device="cuda"))
    dx = gq.linear_i8_grad(w, sw, dy).double()
    # infinite with the sign of dy w in the last channel; NaN where either is zero
    ref = (dy[:, N - 1:].double() * math.inf) * w[N - 1].double()
    assert torch.equal(dx.nan_to_num(7.0), ref.nan_to_num(7.0))


# ------------------------------------------------------------------ under autograd
def test_in_a_function_of_autograd():
    # the calls run where autograd records nothing: in a Function's forward and backward;
    # a tensor that would lose its gradient unseen is refused
    class Layer(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, sw):
            ctx.save_for_backward(w, sw)
            return gq.linear_i8(w, sw, x)

        @staticmethod
        def backward(ctx, dy):
            return gq.linear_i8_grad(*ctx.saved_tensors, dy.contiguous()), None, None

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, w, sw, t):
            hq, sh = gq.quantize_i8(h)
            loss, lse = gq.loss_i8(w, sw, hq, sh, t)
            ctx.save_for_backward(w, sw, hq, sh, t, lse)
            ctx.dtype = h.dtype
            return loss

        @staticmethod
        def backward(ctx, dloss):
            return (gq.loss_i8_grad(*ctx.saved_tensors, dloss.contiguous(), out_dtype=ctx.dtype),
                    None, None, None)

    g = gen(3)
    M, D, N, V = 20, 200, 320, 3001
    p1 = torch.nn.Parameter(torch.randn((N, D), generator=g, device="cuda") * D ** -0.5)
    w1, s1 = gq.quantize_i8(p1)  # a parameter's int8 copy is a constant
    w2, s2 = gq.quantize_i8(torch.randn((V, N), generator=g, device="cuda") * N ** -0.5)
    x = torch.randn((M, D), generator=g, device="cuda").bfloat16().requires_grad_()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    loss = Loss.apply(Layer.apply(x, w1, s1), w2, s2, t)
    (loss / M).sum().backward()
    with torch.no_grad():
        h = gq.linear_i8(w1, s1, x)
        hq, sh = gq.quantize_i8(h)
        l2, lse = gq.loss_i8(w2, s2, hq, sh, t)
        dh = gq.loss_i8_grad(w2, s2, hq, sh, t, lse, torch.full((M,), 1.0 / M, device="cuda"))
        assert torch.equal(loss, l2) and torch.equal(x.grad, gq.linear_i8_grad(w1, s1, dh))
    for call in (lambda: gq.linear_i8(w1, s1, x), lambda: gq.quantize_i8(2 * x),
                 lambda: gq.linear_i8(w1, s1, x.detach(), bias=p1[:, 0].contiguous())):
        with pytest.raises(ValueError, match="record no gradient"):
            call()
