"""The int8 product with an activation and a residual, the gated pair, and their gradient
on the GPU, against their definitions in 64 bits."""
import math

import pytest
import torch

import quant_packed_weight_amd as gq
from block_util import FLOOR, HALF, IDS, TYPES, U, Guarded, gen, i8, normal, scales, within

pytestmark = pytest.mark.gpu

ACTS = [gq.ACT_NONE, gq.ACT_SILU, gq.ACT_GELU, gq.ACT_GELU_TANH, gq.ACT_RELU]
NAMES = ["none", "silu", "gelu", "gelu_tanh", "relu"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    import gpu_util

    gpu_util.device()


def argument(act, z):
    """arg and its derivative where act(z) = z sigma(arg)"""
    if act == gq.ACT_SILU:
        return z, torch.ones_like(z)
    c = 2 * math.sqrt(2 / math.pi)
    return c * (z + 0.044715 * z ** 3), c * (1 + 3 * 0.044715 * z * z)


def function(act, z):
    """act(z), act'(z) in 64 bits, and what f32 arithmetic is off by in them for this z"""
    if act in (gq.ACT_SILU, gq.ACT_GELU_TANH):
        a, d = argument(act, z)
        p, q = torch.sigmoid(a), torch.sigmoid(-a)
        # p: the argument by 3 roundings and 2 constants' and the product with log2 e, as |arg|
        # times as much; exp2, 1 +, the reciprocal (one step each) and z
        rel = (6 * a.abs() + 6) * U
        tiny = 2.0 ** -120  # exp2 past its range
        t = z * p * q * d
        return (z * p, p + t, rel * (z * p).abs() + tiny * z.abs(),
                # p, and z p (1 - p) arg' with 1 - p off by as much as p and a rounding
                rel * p + (rel + 5 * U) * t.abs() + (z * p * d).abs() * (rel * p + U)
                + U * (p + t).abs() + tiny * (1 + (z * d).abs()))
    if act == gq.ACT_GELU:
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        n = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        # erf's argument (slope times argument stays below 1/2) and 2 steps of erf, halved, a
        # rounding: 4 u; n's exponent by 2.5 roundings, exp2 and the constant
        return (z * cdf, cdf + z * n, 4 * U * z.abs() + U * (z * cdf).abs(),
                4 * U + (z * n).abs() * (1.25 * z * z + 5) * U + U * (cdf + z * n).abs())
    if act == gq.ACT_RELU:
        z0 = torch.zeros_like(z)
        return torch.where(z < 0, z0, z), torch.where(z <= 0, z0, torch.ones_like(z)), z0, z0
    return z, torch.ones_like(z), torch.zeros_like(z), torch.zeros_like(z)


def product(w, sw, xq, sx, bias):
    """z in 64 bits and its error in f32: the sum to f32, two scalings, the bias"""
    s = (xq.double() @ w.double().t()) * sx.double()[:, None] * sw.double()
    z = s if bias is None else s + bias.double()
    return z, 3 * U * s.abs() + U * z.abs() * (1 + 2.0 ** -10)


def check(got, ref, err, what):
    t = got.dtype
    within(got, ref, err + HALF[t] * (ref.abs() + err) + FLOOR[t], what)


def check_act(y, z, ze, act, r, what):
    v, _, own, _ = function(act, z)
    # act's slope is at most 1.13
    err = 1.13 * ze + own * 1.01
    ref = v if r is None else v + r.double()
    check(y, ref, err + U * ref.abs(), what)


def check_gate(y, z, ze, u, ue, act, what):
    v, _, own, _ = function(act, z)
    err = 1.13 * ze + own * 1.01
    check(y, v * u, err * (u.abs() + ue) + v.abs() * ue + U * (v * u).abs(), what)


# every tile and every split of K that the library chooses from
SHAPES = [(1, 1, 1), (1, 4096, 4096), (1, 37, 100), (2, 16, 16), (3, 129, 127), (7, 1000, 129),
          (8, 65, 2050), (15, 48, 515), (16, 512, 1024), (17, 33, 63), (31, 255, 4000), (32, 64, 128),
          (33, 130, 300), (48, 640, 1111), (64, 512, 2048), (65, 257, 128), (100, 31, 4100),
          (127, 128, 129), (129, 513, 640), (255, 255, 255), (256, 256, 256), (257, 4099, 1025),
          (333, 777, 96), (512, 1536, 2048), (1000, 264, 136), (1, 40000, 1030), (1, 300, 16384),
          (2, 16400, 300), (3, 20000, 256), (16, 70000, 130), (20, 70001, 260), (20, 110001, 100),
          (20, 4100, 1100),
          (30, 40000, 300), (48, 4096, 4100), (64, 70000, 100), (128, 4096, 640), (300, 4100, 1300),
          (513, 2052, 2200), (512, 12300, 300), (700, 2000, 600), (2048, 4100, 500),
          (4100, 4200, 200), (530, 13500, 40), (780, 7760, 36), (641, 4430, 40), (99, 12340, 36),
          (66, 11700, 140), (560, 11030, 140), (282, 13580, 1100)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_act(M, N, K, dtype):
    g = gen(M * 31 + N * 17 + K)
    w, xq = i8(N, K, g), i8(M, K, g)
    sw, sx = scales(N, g, 1.0 / (74 * math.sqrt(K))), scales(M, g, 1.0 / 37)  # z near 1
    bias = torch.randn(N, generator=g, device="cuda") if N % 2 else None
    z, ze = product(w, sw, xq, sx, bias)
    # each activation in turn over the shapes, each shape with and without the rest
    act = ACTS[(M + N + K) % 5]
    r = normal(M, N, g, dtype, 2.0, extra=M % 3)
    out, pre = Guarded(M, N, dtype, extra=M % 5), Guarded(M, N, dtype, extra=8 - M % 3)
    y = gq.gemm_i8_act(w, sw, xq, sx, act, bias=bias, residual=r, pre=pre.t, out=out.t)
    torch.cuda.synchronize()
    out.check()
    pre.check()
    check_act(y, z, ze, act, r, "y")
    check(pre.t, z, ze, "z")
    act = ACTS[(M + N + K + 1) % 5]
    y = gq.gemm_i8_act(w, sw, xq, sx, act, bias=bias, out_dtype=dtype)
    check_act(y, z, ze, act, None, "y alone")
    # the residual's own place, at a pitch of its own
    held = Guarded(M, N, dtype, extra=M % 4)
    held.t.copy_(r)
    a = gq.gemm_i8_act(w, sw, xq, sx, act, bias=bias, residual=r, out_dtype=dtype)
    b = gq.gemm_i8_act(w, sw, xq, sx, act, bias=bias, residual=held.t, out=held.t)
    assert torch.equal(a, b)
    held.check()


@pytest.mark.parametrize("M,N,K", [(M, (N + 1) // 2 if N > 2000 else N, K) for M, N, K in SHAPES])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gate(M, N, K, dtype):
    g = gen(M * 37 + N * 13 + K)
    w, wu, xq = i8(N, K, g), i8(N, K, g), i8(M, K, g)
    size = 1.0 / (74 * math.sqrt(K))
    sw, swu, sx = scales(N, g, size), scales(N, g, size), scales(M, g, 1.0 / 37)
    bias = torch.randn(N, generator=g, device="cuda") if N % 2 else None
    biasu = torch.randn(N, generator=g, device="cuda") if N % 3 else None
    (z, ze), (u, ue) = product(w, sw, xq, sx, bias), product(wu, swu, xq, sx, biasu)
    act = ACTS[(M + N + K) % 5]
    out, pre = Guarded(M, N, dtype, extra=M % 5), Guarded(M, N, dtype, extra=8 - M % 3)
    up = Guarded(M, N, dtype, extra=M % 2)
    y = gq.gemm_i8_gate(w, sw, wu, swu, xq, sx, act, bias=bias, bias_up=biasu, pre=pre.t, up=up.t,
                        out=out.t)
    torch.cuda.synchronize()
    for o in (out, pre, up):
        o.check()
    check_gate(y, z, ze, u, ue, act, "y")
    check(pre.t, z, ze, "z")
    check(up.t, u, ue, "u")
    act = ACTS[(M + N + K + 1) % 5]
    y = gq.gemm_i8_gate(w, sw, wu, swu, xq, sx, act, bias=bias, bias_up=biasu, out_dtype=dtype)
    check_gate(y, z, ze, u, ue, act, "y alone")
    y2 = gq.gemm_i8_gate(w, sw, wu, swu, xq, sx, act, bias=bias, bias_up=biasu, out_dtype=dtype,
                         up=up.t)
    assert torch.equal(y2, y)


@pytest.mark.parametrize("act", ACTS, ids=NAMES)
@pytest.mark.parametrize("M", [1, 40])
def test_far_and_special_values(act, M):
    # z from an identity: every size of the argument, infinities among them
    N = 96
    w = torch.zeros((N, N), dtype=torch.int8, device="cuda")
    w.fill_diagonal_(1)
    xq = torch.full((M, N), 1, dtype=torch.int8, device="cuda")
    sx = torch.ones(M, device="cuda")
    size = torch.cat([torch.logspace(-30, 30, 46), torch.tensor([0.0, math.inf])])
    sw = torch.cat([size, -size]).cuda()
    y = gq.gemm_i8_act(w, sw, xq, sx, act)
    z = sw.double()[None].repeat(M, 1)
    v, _, own, _ = function(act, z)
    fine = torch.isfinite(z)
    # a weight row of zeros and one with an infinite scale: 0 inf = NaN
    within(y[fine], v[fine], 1.01 * own[fine] + 2 * U * v[fine].abs() + 2.0 ** -120, "y")
    # a row of activations that is not finite spoils its own results only
    sx[0] = math.nan
    y2 = gq.gemm_i8_act(w, sw, xq, sx, act, residual=torch.ones((M, N), device="cuda"))
    assert bool(torch.isnan(y2[0]).all())
    y3 = gq.gemm_i8_act(w, sw, xq, torch.ones_like(sx), act, residual=torch.ones((M, N), device="cuda"))
    assert torch.equal(y2[1:].nan_to_num(), y3[1:].nan_to_num())


LIMITS = {gq.ACT_NONE: (math.inf, -math.inf, 1.0, 1.0), gq.ACT_RELU: (math.inf, 0.0, 1.0, 0.0),
          **{a: (math.inf, 0.0, 1.0, 0.0) for a in (gq.ACT_SILU, gq.ACT_GELU, gq.ACT_GELU_TANH)}}


@pytest.mark.parametrize("act", ACTS, ids=NAMES)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_infinite_arguments(act, dtype):
    # at +inf and -inf: act and its slope are their limits; a NaN stays one
    high, low, up, down = LIMITS[act]
    N = 40
    bias = torch.zeros(N, device="cuda")
    bias[0::4], bias[1::4], bias[2::4] = math.inf, -math.inf, math.nan
    want = torch.zeros(N, device="cuda")
    want[0::4], want[1::4], want[2::4] = high, low, math.nan
    w, sw = torch.zeros((N, 32), dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    for M in (1, 40):
        xq, sx = torch.zeros((M, 32), dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
        pre = torch.empty((M, N), dtype=dtype, device="cuda")
        y = gq.gemm_i8_act(w, sw, xq, sx, act, bias=bias, pre=pre, out_dtype=dtype)
        same = lambda a, b: torch.equal(a.float().nan_to_num(7.0, 8.0, 9.0), b.expand(a.shape).nan_to_num(7.0, 8.0, 9.0))  # noqa: E731,E501
        assert same(y, want) and same(pre, bias)
        two = torch.full((N,), 2.0, device="cuda")
        y = gq.gemm_i8_gate(w, sw, w, sw, xq, sx, act, bias=bias, bias_up=two, out_dtype=dtype)
        assert same(y, 2 * want)
        # the gradients from the z that was kept
        dy = torch.full((M, N), 3.0, dtype=dtype, device="cuda")
        slope = torch.zeros(N, device="cuda")
        slope[0::4], slope[1::4] = up, down
        at = [n for n in range(N) if n % 4 < 2]
        dz, _ = gq.act_grad(act, pre, dy)
        assert torch.equal(dz[:, at].float(), (3 * slope[at]).expand(M, -1))
        if act in (gq.ACT_SILU, gq.ACT_GELU, gq.ACT_GELU_TANH):
            assert bool(torch.isnan(dz[:, 2::4]).all())
        dz, du = gq.act_grad(act, pre, dy, up=torch.full_like(dy, 2.0))
        assert torch.equal(dz[:, at].float(), (6 * slope[at]).expand(M, -1))
        assert same(du, 3 * want)


@pytest.mark.parametrize("act", ACTS, ids=NAMES)
def test_kept_products_past_f16(act):
    # z of 10^5 is kept in f16 as an infinity: the slope is that of a large z, 1 or 0
    w = torch.tensor([[100], [-100]], dtype=torch.int8, device="cuda").repeat(1, 16)
    sw, xq = torch.ones(2, device="cuda"), torch.full((3, 16), 100, dtype=torch.int8, device="cuda")
    sx, pre = torch.ones(3, device="cuda"), torch.empty((3, 2), dtype=torch.float16, device="cuda")
    gq.gemm_i8_act(w, sw, xq, sx, act, pre=pre, out_dtype=torch.float16)
    assert bool(torch.isinf(pre).all())
    dz, du = gq.act_grad(act, pre, torch.ones_like(pre), up=torch.ones_like(pre))
    assert dz.tolist() == [list(LIMITS[act][2:])] * 3
    assert du.tolist() == [list(LIMITS[act][:2])] * 3


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (1, 100, 77), (2, 64, 4096), (5, 321, 333),
                                   (16, 256, 12288), (33, 100, 512), (300, 512, 640), (1, 9000, 100),
                                   (1, 40000, 515), (1, 64, 16384), (1, 64, 16400), (2, 10000, 257),
                                   (2, 5000, 130), (2, 40, 8192), (2, 40, 8300)])
@pytest.mark.parametrize("xt", TYPES, ids=IDS)
@pytest.mark.parametrize("yt", TYPES, ids=IDS)
def test_linear_is_quantize_then_gemm(M, N, K, xt, yt):
    g = gen(M + 3 * N + 5 * K)
    w, sw, wu, swu = i8(N, K, g), scales(N, g, 0.01), i8(N, K, g), scales(N, g, 0.01)
    bias = torch.randn(N, generator=g, device="cuda") if M % 2 else None
    r = normal(M, N, g, yt)
    x = normal(M, K, g, xt, extra=N % 12)
    q, s = gq.quantize_i8(x)
    pre = [torch.empty((M, N), dtype=yt, device="cuda") for _ in range(6)]
    q2 = torch.full((M, -(-K // 16) * 16), 55, dtype=torch.int8, device="cuda")
    s2 = torch.empty(M, device="cuda")
    for act in (gq.ACT_SILU, gq.ACT_GELU):
        ref = gq.gemm_i8_act(w, sw, q, s, act, bias=bias, residual=r, pre=pre[0], out_dtype=yt)
        q2.fill_(55)
        y = gq.linear_i8_act(w, sw, x, act, bias=bias, residual=r, pre=pre[1], out_dtype=yt,
                             xq=q2[:, :K], sx=s2)
        assert torch.equal(y, ref) and torch.equal(pre[0], pre[1])
        assert torch.equal(q2[:, :K], q) and torch.equal(s2, s) and bool((q2[:, K:] == 55).all())
        ref = gq.gemm_i8_gate(w, sw, wu, swu, q, s, act, bias=bias, pre=pre[2], up=pre[3], out_dtype=yt)
        q2.fill_(55)
        y = gq.linear_i8_gate(w, sw, wu, swu, x, act, bias=bias, pre=pre[4], up=pre[5], out_dtype=yt,
                              xq=q2[:, :K], sx=s2)
        assert torch.equal(y, ref) and torch.equal(pre[2], pre[4]) and torch.equal(pre[3], pre[5])
        assert torch.equal(q2[:, :K], q) and torch.equal(s2, s) and bool((q2[:, K:] == 55).all())
    assert gq.linear_i8_act(w, sw, x, gq.ACT_SILU).dtype == xt
    assert gq.linear_i8_gate(w, sw, wu, swu, x).dtype == xt


@pytest.mark.parametrize("M,N,K", [(1, 512, 512), (2, 640, 640), (3, 640, 640), (40, 512, 512),
                                   (1, 40000, 1024), (2, 16000, 1000), (1, 1000, 16384)])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_results_in_the_place_of_x(M, N, K, dtype):
    # x, and a result in the same memory: all of it, its beginning, or around it; with one and
    # two rows, where the quantizer is in the product's launch otherwise, as with more
    g = gen(M + N + K)
    w, sw, wu, swu = i8(N, K, g), scales(N, g, 0.01), i8(N, K, g), scales(N, g, 0.01)
    x, r = normal(M, K, g, dtype), normal(M, N, g, dtype)
    width = max(N, K)

    def held(v):  # v and the place of a result, from the same address on
        b = torch.zeros((M, width), dtype=dtype, device="cuda")
        b[:, :v.shape[1]] = v
        return b[:, :K], b[:, :N]

    ref = gq.linear_i8(w, sw, x)
    a, out = held(x)
    assert torch.equal(gq.linear_i8(w, sw, a, out=out), ref)
    pre, up = torch.empty((M, N), dtype=dtype, device="cuda"), torch.empty((M, N), dtype=dtype, device="cuda")
    ref = gq.linear_i8_act(w, sw, x, gq.ACT_SILU, residual=r, pre=pre)
    a, out = held(x)
    assert torch.equal(gq.linear_i8_act(w, sw, a, gq.ACT_SILU, residual=r, out=out), ref)
    a, out = held(x)
    assert torch.equal(gq.linear_i8_act(w, sw, a, gq.ACT_SILU, residual=r, pre=out), ref)
    assert torch.equal(out, pre)
    if N == K:  # x, the residual and the result in one place
        ref = gq.linear_i8_act(w, sw, x, gq.ACT_NONE, residual=x)
        a, out = held(x)
        assert torch.equal(gq.linear_i8_act(w, sw, a, gq.ACT_NONE, residual=a, out=a), ref)
    ref = gq.linear_i8_gate(w, sw, wu, swu, x, pre=pre, up=up)
    for name, want in (("out", ref), ("pre", pre), ("up", up)):
        a, out = held(x)
        assert torch.equal(gq.linear_i8_gate(w, sw, wu, swu, a, **{name: out}), ref)
        assert torch.equal(out, want), name
    # a result of another type whose second row begins inside x
    if dtype == torch.float32:
        b = torch.zeros(M * width + 8 * N, device="cuda")
        a = b[:M * K].view(M, K).copy_(x)
        out = b.view(torch.bfloat16)[K:K + M * N].view(M, N)
        assert torch.equal(gq.linear_i8_act(w, sw, a, gq.ACT_GELU, out=out),
                           gq.linear_i8_act(w, sw, x, gq.ACT_GELU, out_dtype=torch.bfloat16))
    # side by side in one buffer they share nothing
    b = torch.zeros((M, K + N), dtype=dtype, device="cuda")
    b[:, :K] = x
    assert torch.equal(gq.linear_i8_act(w, sw, b[:, :K], gq.ACT_NONE, out=b[:, K:]), gq.linear_i8(w, sw, x))
    assert torch.equal(b[:, :K], x)


def test_without_an_activation_it_is_the_plain_product():
    g = gen(9)
    for M, N, K in ((1, 300, 500), (9, 300, 500), (200, 300, 500)):
        w, sw, xq, sx = i8(N, K, g), scales(N, g, 0.01), i8(M, K, g), scales(M, g, 0.01)
        b = torch.randn(N, generator=g, device="cuda")
        for t in TYPES:
            assert torch.equal(gq.gemm_i8_act(w, sw, xq, sx, gq.ACT_NONE, bias=b, out_dtype=t),
                               gq.gemm_i8(w, sw, xq, sx, bias=b, out_dtype=t))


def test_empty_products():
    x, one = torch.zeros((3, 32), device="cuda"), torch.zeros(0, device="cuda")
    w = torch.zeros((0, 32), dtype=torch.int8, device="cuda")
    sx = torch.full((3,), 7.0, device="cuda")
    assert gq.linear_i8_act(w, one, x, gq.ACT_SILU, sx=sx).shape == (3, 0)
    assert not bool(sx.any())  # quantized all the same
    sx.fill_(7.0)
    assert gq.linear_i8_gate(w, one, w, one, x, sx=sx).shape == (3, 0)
    assert not bool(sx.any())
    w, s = torch.zeros((5, 32), dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda")
    assert gq.linear_i8_act(w, s, x[:0], gq.ACT_SILU).shape == (0, 5)
    assert gq.linear_i8_gate(w, s, w, s, x[:0]).shape == (0, 5)


# ------------------------------------------------------------------ the gradient
GRADS = [(1, 1), (3, 7), (1, 4096), (2, 255), (5, 512), (9, 513), (77, 1037), (300, 2050),
         (1000, 130), (33, 12289), (4099, 64), (2048, 300), (7, 100000), (16, 520), (17, 520)]


@pytest.mark.parametrize("M,N", GRADS)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("act", ACTS, ids=NAMES)
def test_act_grad(M, N, dtype, act):
    g = gen(M * 3 + N)
    extra = (M + N) % 4 * 4
    z, dy, up = (normal(M, N, g, dtype, s, extra) for s in (2.0, 0.3, 1.0))
    v, d, ve, de = function(act, z.double())
    y, u = dy.double(), up.double()

    def sums(got, ref, err):
        # one rounding for each row more, in whatever order
        within(got, ref.sum(0), err.sum(0) + (M + 1) * U * (ref.abs() + err).sum(0) + 2.0 ** -149, "sum")

    for pair in (False, True):
        dz, du = Guarded(M, N, dtype, extra=extra + 1), Guarded(M, N, dtype, extra=extra)
        db, dbu = torch.full((N + 8,), 3.0, device="cuda"), torch.full((N,), 3.0, device="cuda")
        kw = dict(up=up, dup=du.t, dbias_up=dbu) if pair else {}
        a, b = gq.act_grad(act, z, dy, out=dz.t, dbias=db[4:N + 4], **kw)
        torch.cuda.synchronize()
        dz.check()
        du.check()
        assert bool((db[:4] == 3).all()) and bool((db[N + 4:] == 3).all())
        ref, err = y * d, y.abs() * (1.01 * de) + U * (y * d).abs()
        if pair:
            ref, err = ref * u, err * u.abs() + U * (ref * u).abs()
            uref, uerr = y * v, y.abs() * (1.01 * ve) + U * (y * v).abs()
            check(b, uref, uerr, "du")
            sums(dbu, uref, uerr)
        else:
            assert b is None
        check(a, ref, err, "dz")
        sums(db[4:N + 4], ref, err)
        # without the sums, and in the inputs' own places: the same bits
        a2, b2 = gq.act_grad(act, z, dy, up=up if pair else None)
        assert torch.equal(a2, a) and (b2 is None or torch.equal(b2, b))
        for where in (0, 1):
            c = [z.clone(), dy.clone(), up.clone()]
            a3, b3 = gq.act_grad(act, c[0], c[1], up=c[2] if pair else None, out=c[where],
                                 dup=c[2] if pair else None)
            assert a3 is c[where] and torch.equal(a3, a) and (b3 is None or torch.equal(b3, b))
        if pair:
            c = [z.clone(), dy.clone(), up.clone()]
            a3, b3 = gq.act_grad(act, c[0], c[1], up=c[2], out=c[0], dup=c[1])
            assert torch.equal(a3, a) and torch.equal(b3, b)
            # one of the two sums alone
            one = torch.empty(N, device="cuda")
            gq.act_grad(act, z, dy, up=up, dbias_up=one)
            assert torch.equal(one, dbu)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,N", [(1, 40), (5, 513), (16, 40), (17, 40), (255, 12289), (2048, 300),
                                 (4099, 64), (70001, 40)])
def test_act_grad_sums_every_row(M, N, dtype):
    # whole numbers, none of them zero, without an activation: the sums over rows are exact in
    # any order, and a row that is missing or counted twice shows
    g = gen(M + N)
    whole = lambda: ((2.0 * torch.randint(0, 2, (M, N), generator=g, device="cuda") - 1)  # noqa: E731
                     * torch.randint(1, 5, (M, N), generator=g, device="cuda")).to(dtype)
    z, dy, up = whole(), whole(), whole()
    db, dbu = (torch.empty(N, device="cuda") for _ in range(2))
    gq.act_grad(gq.ACT_NONE, z, dy, dbias=db)
    assert torch.equal(db.double(), dy.double().sum(0))
    gq.act_grad(gq.ACT_NONE, z, dy, up=up, dbias=db, dbias_up=dbu)
    assert torch.equal(db.double(), (dy.double() * up.double()).sum(0))
    assert torch.equal(dbu.double(), (dy.double() * z.double()).sum(0))


def test_act_grad_without_rows():
    z = torch.zeros((0, 9), device="cuda")
    db, dbu = torch.full((9,), 3.0, device="cuda"), torch.full((9,), 3.0, device="cuda")
    gq.act_grad(gq.ACT_SILU, z, z, up=z, dbias=db, dbias_up=dbu)
    assert not bool(db.any()) and not bool(dbu.any())


@pytest.mark.parametrize("act", ACTS, ids=NAMES)
def test_act_grad_far_values(act):
    size = torch.cat([torch.logspace(-30, 30, 61), torch.tensor([0.0])])
    z = torch.cat([size, -size]).cuda()[None]
    one = torch.ones_like(z)
    dz, du = gq.act_grad(act, z, one, up=one)
    v, d, ve, de = function(act, z.double())
    within(dz, d, 1.01 * de + 3 * U * d.abs() + 2.0 ** -120, "dz")
    within(du, v, 1.01 * ve + 2 * U * v.abs() + 2.0 ** -120, "du")


@pytest.mark.parametrize("act", ACTS, ids=NAMES)
def test_block_gradient_against_differences(act):
    # x -> gated pair -> y, back to x: dz and du through linear_i8_grad, against differences
    # of the definition (the quantizer's rounding taken as the identity: x = xq sx)
    g = gen(21)
    M, N, K = 6, 40, 64
    w, wu, xq = i8(N, K, g), i8(N, K, g), i8(M, K, g)
    sw, swu, sx = scales(N, g, 1 / 600), scales(N, g, 1 / 600), scales(M, g, 1 / 37)
    dy = torch.randn((M, N), generator=g, device="cuda")
    z, u = torch.empty((M, N), device="cuda"), torch.empty((M, N), device="cuda")
    gq.gemm_i8_gate(w, sw, wu, swu, xq, sx, act, pre=z, up=u)
    dz, du = gq.act_grad(act, z, dy, up=u)
    dx = gq.linear_i8_grad(w, sw, dz).double() + gq.linear_i8_grad(wu, swu, du).double()
    wd, wud = w.double() * sw.double()[:, None], wu.double() * swu.double()[:, None]
    x = xq.double() * sx.double()[:, None]

    def value(x):
        return (function(act, x @ wd.t())[0] * (x @ wud.t()) * dy.double()).sum()

    for _ in range(5):
        v = torch.randn((M, K), generator=g, device="cuda").double()
        step = 1e-6
        d = float((value(x + step * v) - value(x - step * v)) / (2 * step))
        got = float((dx * v).sum())
        # relu's kink: a product within the step of zero counts for step times its slope's jump
        assert abs(d - got) <= 1e-5 * float((dx * v).abs().sum()) + 1e-5


def test_offsets_past_32_bits():
    # results, a residual and kept products of 2.6 10^9 values each
    g = gen(12)
    M, N, K = 40000, 65536, 64
    w, sw, xq, sx = i8(N, K, g), scales(N, g, 0.01), i8(M, K, g), scales(M, g, 0.01)
    rows = torch.tensor([0, 1, 127, 128, 20000, 32767, 32768, M - 129, M - 1], device="cuda")
    z, ze = product(w, sw, xq[rows], sx[rows], None)
    big = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    big[rows] = 1.0
    pre = torch.empty_like(big)
    gq.gemm_i8_act(w, sw, xq, sx, gq.ACT_SILU, residual=big, pre=pre, out=big)
    check_act(big[rows], z, ze, gq.ACT_SILU, torch.ones_like(z), "y")
    check(pre[rows], z, ze, "z")
    assert bool((big[100] != 0).any())
    y = gq.gemm_i8_gate(w, sw, w, sw, xq, sx, pre=pre, out=big)
    check_gate(y[rows], z, ze, z, ze, gq.ACT_SILU, "gate")
    dy = y[rows].double()
    du = torch.empty_like(big)
    gq.act_grad(gq.ACT_SILU, pre, big, up=pre, out=big, dup=du)
    p = pre[rows].double()
    v, d, ve, de = function(gq.ACT_SILU, p)
    check(du[rows], dy * v, dy.abs() * ve * 1.01 + U * (dy * v).abs(), "du")
    check(big[rows], dy * d * p, (dy * p).abs() * de * 1.01 + 2 * U * (dy * d * p).abs(), "dz")
