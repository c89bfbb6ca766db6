"""The norm between two int8 products and its gradient on the GPU, against their
definitions in 64 bits."""
import math

import pytest
import torch

import quant_packed_weight_amd as gq
from block_util import FLOOR, HALF, IDS, TYPES, U, Guarded, gen, normal, scales, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import gpu_util

    gpu_util.device()


def reference(x, r, w, eps):
    """h, the integers, and the scale in 64 bits"""
    h = x if r is None else (x.double() + r.double()).float().to(x.dtype)
    p = h.float() * w
    s0 = (p.double().abs().amax(1) / 127).float()
    live = (s0 > 0)[:, None]
    q = (p.double() / torch.where(live, s0[:, None], 1.0).double()).float().round().clamp(-127, 127)
    q = torch.where(live, q, 0.0)
    s = s0.double() / torch.sqrt(h.double().square().mean(1) + eps)
    return h, q, torch.where(s0 == 0, 0.0, s)


def check(got, x, r, w, eps):
    q, s, h = got
    hr, qr, sr = reference(x, r, w, eps)
    assert torch.equal(h, hr)
    assert torch.equal(q.float(), qr)
    # the sum of squares in 64 bits: one rounding, that of the scale
    within(s, sr, (U + 2.0 ** -48) * sr + 2.0 ** -149, "scale")


SHAPES = [(1, 1), (1, 16), (3, 17), (5, 255), (2, 256), (7, 1000), (4, 4096), (2, 12289), (1, 8193),
          (300, 64), (2, 8192), (3, 4097), (2, 16384), (2, 16385), (3, 40001),
          (1, 131071)]


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("extra", [0, 3, 8])
def test_rms(M, K, dtype, extra):
    g = gen(M * 7919 + K)
    x, r = normal(M, K, g, dtype, 3, extra), normal(M, K, g, dtype, 2, extra)
    w = torch.randn(K + extra, generator=g, device="cuda")[extra:]  # off 16 bytes at 3
    out, hid = Guarded(M, K, torch.int8, extra=(-K) % 16 + 16), Guarded(M, K, dtype, extra=extra + 1)
    got = gq.rms_i8(x, w, eps=1e-5, residual=r, hidden=hid.t, out=out.t)
    torch.cuda.synchronize()
    out.check()
    hid.check()
    check(got, x, r, w, 1e-5)
    # without a residual, and without a place for h
    q, s, h = gq.rms_i8(x, w, eps=1e-5)
    assert h is x
    check((q, s, h), x, None, w, 1e-5)
    # the residual's sum without a place for h (the C call; the binding always keeps it)
    q2, s2 = torch.zeros_like(got[0].contiguous()), torch.zeros_like(got[1])
    q2 = gq.quantize_i8(torch.zeros((M, K), device="cuda"))[0]
    L = gq.lib_i8()
    ty = {torch.float32: gq.F32, torch.bfloat16: gq.BF16, torch.float16: gq.F16}[dtype]
    st = torch.cuda.current_stream().cuda_stream
    assert L.gemmq_rms_i8(ty, x.data_ptr(), K + extra, r.data_ptr(), K + extra, None, 0, w.data_ptr(),
                          1e-5, q2.data_ptr(), -(-K // 16) * 16, s2.data_ptr(), M, K, st) == 0
    assert torch.equal(q2, got[0]) and torch.equal(s2, got[1])
    # h in the place of x, and of the residual
    for where in (0, 1):
        a = [x.clone(), r.clone()]
        q3, s3, h3 = gq.rms_i8(a[0], w, eps=1e-5, residual=a[1], hidden=a[where])
        assert h3 is a[where]
        assert torch.equal(h3, got[2]) and torch.equal(q3, got[0]) and torch.equal(s3, got[1])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rms_extreme_rows(dtype):
    fi = torch.finfo(dtype)
    K = 300
    x = torch.ones((8, K), device="cuda", dtype=dtype)
    x[0] = 0                       # an empty row
    x[1] = -0.0
    x[2, 7] = math.inf
    x[3, 299] = -math.inf
    x[4, 0] = math.nan
    x[5, 100] = fi.max             # its square passes f32, and f64's sum holds it
    x[6] = fi.smallest_normal      # squares below f32
    x[7, 3] = -5
    w = torch.ones(K, device="cuda")
    for eps in (0.0, 1e-6):
        q, s, _ = gq.rms_i8(x, w, eps=eps)
        fine = torch.tensor([0, 1, 5, 6, 7], device="cuda")
        check((q[fine], s[fine], x[fine]), x[fine], None, w, eps)
        for m in (2, 3, 4):
            assert math.isnan(float(s[m])) and not bool(q[m].any())
    # a sum that leaves the type, and a product that leaves f32, are not finite either
    q, s, h = gq.rms_i8(x[5:6], w, residual=x[5:6].clone())
    assert math.isinf(float(h[0, 100])) and math.isnan(float(s[0])) and not bool(q.any())
    if dtype != torch.float16:
        q, s, _ = gq.rms_i8(x[5:6], 2 * w)
        assert math.isnan(float(s[0])) and not bool(q.any())
    # a weight that is not finite counts, one of zero leaves zeros
    w[9] = math.nan
    q, s, _ = gq.rms_i8(x[7:], w)
    assert math.isnan(float(s[0])) and not bool(q.any())
    q, s, _ = gq.rms_i8(x[7:], torch.zeros(K, device="cuda"))
    assert float(s[0]) == 0.0 and not bool(q.any())


def test_rms_no_rows():
    w = torch.ones(40, device="cuda")
    q, s, h = gq.rms_i8(torch.zeros((0, 40), device="cuda"), w, residual=torch.zeros((0, 40), device="cuda"))
    assert q.shape == (0, 40) and s.shape == (0,) and h.shape == (0, 40)
    z = torch.zeros((0, 40), device="cuda")
    dw = torch.full((40,), 3.0, device="cuda")
    dx, dw = gq.rms_i8_grad(z, w, z, dw=dw)
    assert dx.shape == (0, 40) and not bool(dw.any())


def gradient(h, w, dy, dh, eps):
    """dx, dw in 64 bits and the sums of sizes that their errors are measured by"""
    h, w, dy = h.double(), w.double(), dy.double()
    rstd = (h.square().mean(1, keepdim=True) + eps) ** -0.5
    n, d = h * rstd, dy * w
    mean = (d * n).mean(1, keepdim=True)
    dx = rstd * (d - n * mean)
    size = rstd * (d.abs() + (n * mean).abs())
    # d * h enters the mean with d's rounding
    slack = rstd * n.abs() * (d * n).abs().mean(1, keepdim=True)
    if dh is not None:
        dx, size = dx + dh.double(), size + dh.double().abs()
    return dx, size, slack, (dy * n).sum(0), (dy * n).abs().sum(0)


def check_grad(got, h, w, dy, dh, eps):
    dx, dw = got
    ref, size, slack, refw, sizew = gradient(h, w, dy, dh, eps)
    # roundings on the way of n mean: rstd, n, mean, the fma, rstd, the product, the sum; of
    # d's: itself, the fma, rstd, the product, the sum; and the mean's own by d's
    tol = 8 * U * size + 2 * U * slack
    t = h.dtype
    within(dx, ref, HALF[t] * (ref.abs() + tol) + tol + FLOOR[t], "dx")
    if dw is not None:
        # rstd, n, the product; one for each further row, in whatever order
        within(dw, refw, (4 + h.shape[0]) * U * sizew + 2.0 ** -149, "dw")


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", SHAPES + [(513, 130), (1100, 40), (2, 2049), (5, 4097), (300, 5000), (600, 16400),
                                          (4, 6144), (4, 6145), (6, 4100)])
@pytest.mark.parametrize("extra", [0, 3, 8])
def test_rms_grad(M, K, dtype, extra):
    g = gen(M * 31 + K)
    h, dy = normal(M, K, g, dtype, 2, extra), normal(M, K, g, dtype, 0.3, extra)
    dh = normal(M, K, g, dtype, 0.2, extra)
    w = torch.randn(K + extra, generator=g, device="cuda")[extra:]
    out, dwall = Guarded(M, K, dtype, extra=extra + 1), torch.full((K + 9,), 5.0, device="cuda")
    got = gq.rms_i8_grad(h, w, dy, dh=dh, eps=1e-5, out=out.t, dw=dwall[4:K + 4])
    torch.cuda.synchronize()
    out.check()
    assert bool((dwall[:4] == 5).all()) and bool((dwall[K + 4:] == 5).all())
    check_grad(got, h, w, dy, dh, 1e-5)
    dx, dw = gq.rms_i8_grad(h, w, dy, eps=1e-5)
    check_grad((dx, dw), h, w, dy, None, 1e-5)
    # without dw: the same dx; and in the place of each of the three
    dx2, none = gq.rms_i8_grad(h, w, dy, eps=1e-5, weight_grad=False)
    assert none is None and torch.equal(dx2, dx)
    for where in (0, 1):
        a = [dy.clone(), dh.clone()]
        dx3, dw3 = gq.rms_i8_grad(h, w, a[0], dh=a[1], eps=1e-5, out=a[where])
        assert torch.equal(dx3, got[0]) and torch.equal(dw3, got[1])
    c = h.clone()
    dx3, dw3 = gq.rms_i8_grad(c, w, dy, dh=dh, eps=1e-5, out=c)
    assert torch.equal(dx3, got[0]) and torch.equal(dw3, got[1])


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.5])
def test_rms_grad_against_differences(eps):
    g = gen(77)
    M, K = 9, 200
    h, w = normal(M, K, g, torch.float32, 1.5), torch.randn(K, generator=g, device="cuda")
    dy = normal(M, K, g, torch.float32)

    def value(h, w):
        return (dy.double() * h * (h.square().mean(1, keepdim=True) + eps) ** -0.5 * w).sum()

    dx, dw = gq.rms_i8_grad(h, w, dy, eps=eps)
    step = 1e-5  # the difference is off by about step^2 and 2^-52 / step
    for _ in range(5):
        v = torch.randn((M, K), generator=g, device="cuda").double()
        u = torch.randn(K, generator=g, device="cuda").double()
        for d, got in (((v, 0 * u), (dx.double() * v).sum()), ((0 * v, u), (dw.double() * u).sum())):
            a = value(h.double() + step * d[0], w.double() + step * d[1])
            b = value(h.double() - step * d[0], w.double() - step * d[1])
            assert abs(float((a - b) / (2 * step) - got)) <= 1e-4


def test_rms_grad_special_rows():
    g = gen(5)
    K = 500
    w = torch.randn(K, generator=g, device="cuda")
    h, dy = normal(6, K, g, torch.float32), normal(6, K, g, torch.float32)
    h[0] = 0
    h[1] *= 1e30                  # squares past f32
    h[2] *= 1e-30
    fine = torch.tensor([0, 1, 2, 3, 5], device="cuda")
    dx, dw = gq.rms_i8_grad(h, w, dy, eps=1e-6)
    check_grad((dx, dw), h, w, dy, None, 1e-6)
    # a row that is not finite spoils its own gradient and the sum over rows, not the others
    h[4, 9] = math.inf
    dx2, dw2 = gq.rms_i8_grad(h, w, dy, eps=1e-6)
    assert torch.equal(dx2[fine], dx[fine]) and bool(torch.isnan(dx2[4]).any())
    assert bool(torch.isnan(dw2[9]))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", [(3, 500), (40, 500), (6, 5000), (5, 12288), (5, 20000)])
def test_rms_grad_without_eps(M, K, dtype):
    # a row of zeros is finite forward (scale 0), and takes nothing from the other rows back
    g = gen(M + K)
    w = torch.randn(K, generator=g, device="cuda")
    h, dy = normal(M, K, g, dtype, 2), normal(M, K, g, dtype, 0.3)
    dh = normal(M, K, g, dtype, 0.2)
    h[1], h[M - 1] = 0, -0.0
    kept = torch.tensor([m for m in range(M) if m not in (1, M - 1)], device="cuda")
    for add in (None, dh):
        dx, dw = gq.rms_i8_grad(h, w, dy, dh=add, eps=0.0)
        check_grad((dx[kept], dw), h[kept], w, dy[kept], None if add is None else add[kept], 0.0)
        for m in (1, M - 1):
            assert torch.equal(dx[m], torch.zeros_like(dx[m]) if add is None else add[m])
        assert torch.equal(gq.rms_i8_grad(h, w, dy, dh=add, eps=0.0, weight_grad=False)[0], dx)
    if dtype == torch.float16:
        return
    # a row of subnormal values: 1 / rms is past f32, dx is not; dw has the row as any other
    h[1], dy[1] = normal(1, K, g, dtype)[0] * 1e-40, normal(1, K, g, dtype)[0] * 1e-5
    h[M - 1, 7] = 1e-40
    dy[M - 1] = 0
    assert bool(h[1].any()) and bool(h[M - 1].any())
    check_grad(gq.rms_i8_grad(h, w, dy, eps=0.0), h, w, dy, None, 0.0)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_rms_many_rows(dtype):
    # more rows than a grid dimension of 32768 takes, and not a multiple of it
    g = gen(13)
    M, K = 70001, 40
    x, r, w = normal(M, K, g, dtype), normal(M, K, g, dtype), torch.randn(K, generator=g, device="cuda")
    got = gq.rms_i8(x, w, residual=r)
    check(got, x, r, w, 1e-6)
    check_grad(gq.rms_i8_grad(got[2], w, r, dh=x), got[2], w, r, x, 1e-6)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", [(1, 40), (4, 40), (5, 40), (255, 4096), (513, 4097), (1025, 8192),
                                 (1500, 8200), (700, 12288), (777, 16400), (70001, 40)])
def test_rms_grad_sums_every_row(M, K, dtype):
    # h of +-1 and eps = 3: rstd is 1/2 and n +-1/2, and with whole numbers for dy, none of them
    # zero, dw's sums are exact in any order: a row that is missing or counted twice shows
    g = gen(M + K)
    sign = lambda: 2.0 * torch.randint(0, 2, (M, K), generator=g, device="cuda") - 1  # noqa: E731
    h = sign().to(dtype)
    dy = (sign() * torch.randint(1, 9, (M, K), generator=g, device="cuda")).to(dtype)
    w = torch.ones(K, device="cuda")
    _, dw = gq.rms_i8_grad(h, w, dy, eps=3.0)
    assert torch.equal(dw.double(), (dy.double() * h.double()).sum(0) / 2)
    # and without an eps, rstd 1
    _, dw = gq.rms_i8_grad(h, w, dy, eps=0.0)
    assert torch.equal(dw.double(), (dy.double() * h.double()).sum(0))


def test_rms_offsets_past_32_bits():
    # rows 1.2 10^9 elements apart: element offsets pass 2^31, byte offsets 2^32
    g = gen(3)
    M, K, pitch = 4, 1000, 1200000000 // 8 * 8
    big = torch.empty(3 * pitch + K, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((M, K), (pitch, 1))
    x.copy_(normal(M, K, g, torch.bfloat16))
    near = x.clone()
    w = torch.randn(K, generator=g, device="cuda")
    q, s, _ = gq.rms_i8(x, w)
    check((q, s, near), near, None, w, 1e-6)
    dx, dw = gq.rms_i8_grad(x, w, x, dh=x)
    check_grad((dx, dw), near, w, near, near, 1e-6)
    out = big.as_strided((M, K), (pitch, 1), 0)
    dx2, _ = gq.rms_i8_grad(near, w, near.clone(), dh=x, out=out)
    assert torch.equal(dx2, dx)
