"""The vocabulary loss and its gradient where the target is nearly certain and its
logit is large: what the f32 steps on the way to lse and to the target's factor leave.

u = 2^-24 is half a step of f32.
"""
import math

import pytest
import torch

import quant_packed_weight_amd as gq
from test_gpu_i8 import U, gen, i8, scales

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
