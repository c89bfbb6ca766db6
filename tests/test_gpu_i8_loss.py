"""The vocabulary loss and its gradient where the target is nearly certain and its
logit is large: what the f32 steps on the way to lse and to the target's factor leave.

u = 2^-24 is half a step of f32.
"""
import math

import pytest
import torch

import quant_packed_weight_amd as gq
from test_gpu_i8 import FLOOR, HALF, U, gen, i8, loss_reference, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import gpu_util

    gpu_util.device()


def certain(M, N, K, size, near, seed, negative=False):
    """Rows that point to their target, whose logit is about `size`; the next row of the
    vocabulary has the target's weights but for a part `near` of them."""
    g = gen(seed)
    w, sw = i8(N, K, g), scales(N, g, 0.01)
    t = 2 * torch.randperm(N // 2, generator=g, device="cuda")[:M]
    other = w[t].clone()
    other[torch.rand((M, K), generator=g, device="cuda") < near] = 0
    w[t + 1], sw[t + 1] = other, sw[t]
    xq = i8(M, K, g)
    xq.copy_(-w[t] if negative else w[t])
    dot = (xq.double() * w[t].double()).sum(1)
    sx = (size * (0.8 + 0.2 * torch.rand(M, generator=g, device="cuda").double()) / (dot * sw[t].double())).float()
    return w, sw, xq, sx, t


# sums of 1.4 10^7 and of 4.3 10^7 to 7 10^8: past 2^24 they are no f32
@pytest.mark.parametrize("M,N,K", [(1, 500, 2600), (8, 500, 8000), (5, 3000, 8000), (40, 500, 8000),
                                   (150, 3000, 8000), (20, 70000, 6000), (3, 200, 131071), (33, 200, 131071)])
def test_loss_grad_of_a_certain_target_with_a_large_sum(M, N, K):
    # nothing else has a probability above 10^-20: the gradient is the target's factor,
    # exp(z - lse) - 1 with z and lse of about 60 and their difference below 2^-18.  The
    # exponent is the sum of r = v sx - lse, rounded once (v is sw dot in f32), and of what
    # v leaves of z: dot's rounding and the product's, u |z| each, so at most 2 u 64 = 2^-17,
    # known to u of itself.  |r| <= |z - lse| + 2^-17: where the two nearly cancel, u (2^-17
    # + 2^-17) = 2^-40 remains beside u of the result and what expm1 and the factors round.
    w, sw, xq, sx, t = certain(M, N, K, 60.0, 0.9, M + K)
    z = (xq.double() * w[t].double()).sum(1) * sx.double() * sw[t].double()
    lse = z.float()
    f = torch.expm1(z - lse.double())
    wd = w[t].double() * sw[t].double()[:, None]
    ref = f[:, None] * wd
    dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse, torch.ones(M, device="cuda"), out_dtype=torch.float32)
    # the others' gradients, below 10^-20 of a weight each, are no part of f
    assert bool(((dx.double() - ref).abs() <= 16 * U * ref.abs() + 2.0 ** -40 * wd.abs() + 1e-15).all())


CERTAIN = [(1, 500, 1000), (8, 500, 8000), (5, 16000, 2048), (40, 500, 1000), (150, 3000, 8000), (20, 70000, 515),
           (300, 9000, 2048), (33, 200, 131071)]


@pytest.mark.parametrize("negative", [False, True], ids=["", "negative"])
@pytest.mark.parametrize("M,N,K", CERTAIN)
def test_lse_of_a_certain_target_is_rounded_once(M, N, K, negative):
    # logits of 96 to 120, whose half step is 2^-18; the others' e^-80 of them
    w, sw, xq, sx, t = certain(M, N, K, 120.0, 0.9, M + K, negative)
    assert bool((sx < 0).all()) == negative
    z = (xq.double() * w[t].double()).sum(1) * sx.double() * sw[t].double()
    loss, lse = gq.loss_i8(w, sw, xq, sx, t)
    # the product's remainder is exact, the sum and the loss of one term are 1 and 0
    assert float((lse.double() - z).abs().max()) <= 2.0 ** -18 * (1 + 2.0 ** -10)
    assert float(loss.abs().max()) <= 1e-12
    # without the target's sum in hand the largest sw dot is known to two roundings more
    for other in (torch.full_like(t, -100), (t + 2) % N):
        loss, lse = gq.loss_i8(w, sw, xq, sx, other)
        assert float((lse.double() - z).abs().max()) <= 2.0 ** -18 * (1 + 2.0 ** -10) + 2 * U * 120
        zo = (xq.double() * w[other.clamp(min=0)].double()).sum(1) * sx.double() * sw[other.clamp(min=0)].double()
        ref = torch.where(other < 0, torch.zeros_like(z), z - zo)
        # both logits' v and their difference, and the product
        assert bool(((loss.double() - ref).abs() <= 2 * U * (z.abs() + zo.abs()) + 2 * U * ref.abs()).all())


@pytest.mark.parametrize("negative", [False, True], ids=["", "negative"])
@pytest.mark.parametrize("M,N,K", CERTAIN)
def test_gradient_of_a_nearly_certain_row_from_the_loss_s_own_lse(M, N, K, negative):
    # logits of 80 to 100 and one other token within about 8: 1 - p of 10^-4, which the
    # half step of lse, 2^-18, moves by some per cent and nothing else by more than that
    w, sw, xq, sx, t = certain(M, N, K, 100.0, 0.09, 3 * M + K, negative)
    z, _, loss_r = loss_reference(w, sw, xq, sx, t)
    loss, lse = gq.loss_i8(w, sw, xq, sx, t)
    dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse, torch.ones(M, device="cuda"), out_dtype=torch.float32)
    rows = torch.arange(M, device="cuda")
    p = torch.softmax(z, 1)
    a = p.clone()
    a[rows, t] = torch.expm1(-loss_r)
    wd = w.double() * sw.double()[:, None]
    ref = a @ wd
    # lse by its half step and, where the others' probability is p', by p' (their v's
    # two roundings); the others' factors by that and their own roundings, the
    # additions by a few u of all
    e = 2.0 ** -18 * (1 + 2.0 ** -10) + (1 - p[rows, t]) * 4 * U * 100
    other = p.clone()
    other[rows, t] = 0
    tol = (e + 4 * U)[:, None] * wd[t].abs() + (other * (e + 6 * U * 100)[:, None]) @ wd.abs()
    # (where w is 0 in both, only factors of 2^-115 are left, whose last parts lie below f32's
    # smallest normal number, 2^-126, and may be lost: N of them, times w < 2^7)
    tol = tol + 32 * U * (a.abs() @ wd.abs()) + N * 2.0 ** -119
    assert bool(((dx.double() - ref).abs() <= tol).all())
    # 1 + p': a sum near one, rounded by a few u
    assert bool(((loss.double() - loss_r).abs() <= 8 * U + (1 - p[rows, t]) * 8 * U * 100).all())


@pytest.mark.parametrize("M,N,K", [(1, 98305, 64), (5, 100001, 260), (17, 98304, 130), (20, 100001, 140),
                                   (32, 99999, 515), (33, 100001, 140)])
def test_few_rows_over_a_large_vocabulary(M, N, K):
    # on both sides of the number of channels from which workgroups take 128 of them
    g = gen(M + N)
    w, sw, xq, sx = i8(N, K, g, full=True), scales(N, g, K ** -0.5 / 64), i8(M, K, g), scales(M, g, 0.05)
    t = torch.randint(0, N, (M,), generator=g, device="cuda")
    t[M - 1] = N - 1
    z, lse_r, loss_r = loss_reference(w, sw, xq, sx, t)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        y = gq.gemm_i8(w, sw, xq, sx, out_dtype=dt)
        # the sum to f32 and two scalings, the result's type
        assert bool(((y.double() - z).abs() <= (4 * U + HALF[dt]) * z.abs() + FLOOR[dt]).all())
    loss, lse = gq.loss_i8(w, sw, xq, sx, t)
    # a logit's two roundings (v, and its difference with the maximum), the exponentials' 2 u
    # and the additions, a term in 300 at most
    tol = 3 * U * z.abs().amax(1) + (302 + 3) * U + U * lse_r.abs()
    assert bool(((lse.double() - lse_r).abs() <= tol).all())
    assert bool(((loss.double() - loss_r).abs() <= tol + 3 * U * z.abs().amax(1)).all())
    p = torch.softmax(z, 1)
    p[torch.arange(M, device="cuda"), t] = torch.expm1(-loss_r)
    ref = p @ (w.double() * sw.double()[:, None])
    dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse, torch.ones(M, device="cuda"), out_dtype=torch.float32)
    assert float((dx.double() - ref).norm() / ref.norm()) <= 2.0 ** -18
