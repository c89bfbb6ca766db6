"""The int8 linear layer, its gradient, and the vocabulary loss with its gradient
on the GPU, against their definitions in 64 bits.

Tolerances count roundings.  u = 2^-24 is half a step of f32, h(t) half a step of
the result's type relative to its value (f32 2^-24, f16 2^-11, bf16 2^-8); f16
results below 2^-14 are rounded to steps of 2^-24, so by at most 2^-25.
"""
import math

import pytest
import torch

import quant_packed_weight_amd as gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FLOOR = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]


@pytest.fixture(scope="module", autouse=True)
def _device():
    import gpu_util

    gpu_util.device()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def i8(rows, cols, g, pitch=None, full=False):
    """Random int8 rows of `cols` values, `pitch` bytes apart; the bytes behind
    each row hold other values, which must not matter."""
    pitch = pitch or -(-cols // 16) * 16
    lo = -128 if full else -127
    return torch.randint(lo, 128, (rows, pitch), generator=g, device="cuda",
                         dtype=torch.int8)[:, :cols]


def scales(n, g, size=1.0):
    return (0.2 + torch.rand(n, generator=g, device="cuda")) * size


class Guarded:
    """A [rows, cols] tensor inside a wider buffer whose other values are known:
    rows above, rows below and columns to the right of it."""

    def __init__(self, rows, cols, dtype, extra=5, fill=7):
        self.all = torch.full((rows + 2, cols + extra), fill, dtype=dtype, device="cuda")
        self.t = self.all[1:rows + 1, :cols]
        self.fill = fill
        self.rows, self.cols = rows, cols

    def check(self):
        a = self.all.clone()
        a[1:self.rows + 1, :self.cols] = self.fill
        assert bool((a == self.fill).all()), "written outside the result"


def product(w, sw, xq, sx):
    """sum and value in 64 bits"""
    s = xq.double() @ w.double().t()
    return s, s * sx.double()[:, None] * sw.double()


# ------------------------------------------------------------------ quantize
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (3, 17), (5, 255), (2, 256), (7, 1000), (4, 4096),
                                 (2, 12289), (1, 131071), (300, 64), (2, 8193)])
@pytest.mark.parametrize("extra", [0, 3, 8])
def test_quantize(M, K, dtype, extra):
    g = gen(M * 7919 + K)
    x = torch.zeros((M, K + extra), dtype=dtype, device="cuda")[:, :K]
    x.copy_(torch.randn((M, K), generator=g, device="cuda") * 3)
    out = Guarded(M, K, torch.int8, extra=(-K) % 16 + 16)
    q, s = gq.quantize_i8(x, out=out.t)
    torch.cuda.synchronize()
    out.check()
    xd = x.double()
    sr = (xd.abs().amax(1) / 127).float()
    assert torch.equal(s, sr)
    qr = (xd / sr.double()[:, None]).float().round().clamp(-127, 127)
    assert torch.equal(q.float(), qr)
    q2, s2 = gq.quantize_i8(x)
    assert torch.equal(q2, q) and torch.equal(s2, s)


def test_quantize_ties():
    # values on and one step beside the ties between two integers, at scales of all
    # sizes: the rounded quotient decides
    g = gen(15)
    half = torch.arange(-127, 127, device="cuda").float() + 0.5
    rows = []
    for e in range(-120, 118, 7):
        s = float(2.0 ** e * (1 + torch.rand(1, generator=g, device="cuda")))
        top = torch.tensor([127.0 * s], device="cuda")
        v = (half.double() * (top / 127).double()).float()
        rows.append(torch.cat([top, v, torch.nextafter(v, top), torch.nextafter(v, -top)]))
    x = torch.stack(rows)
    q, s = gq.quantize_i8(x)
    sr = (x.double().abs().amax(1) / 127).float()
    assert torch.equal(s, sr)
    assert torch.equal(q.float(), (x.double() / sr.double()[:, None]).float().round().clamp(-127, 127))
    # the one-launch layer quantizes by the same steps
    w, sw = i8(48, x.shape[1], g), scales(48, g)
    for m in range(0, x.shape[0], 5):
        y = gq.linear_i8(w, sw, x[m:m + 1], out_dtype=torch.float32)
        assert torch.equal(y, gq.gemm_i8(w, sw, q[m:m + 1], s[m:m + 1]))


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_quantize_extreme_rows(dtype):
    fi = torch.finfo(dtype)
    K = 300
    x = torch.ones((9, K), device="cuda", dtype=dtype)
    x[0] = 0                      # an empty row
    x[1] = -0.0
    x[2, 7] = math.inf
    x[3, 299] = -math.inf
    x[4, 0] = math.nan
    x[5, 100] = fi.max            # everything else rounds to zero
    x[6] = fi.smallest_normal     # a scale below the type's range, or an f32 subnormal
    x[7] = 0
    x[7, 1] = fi.tiny * fi.eps    # the smallest subnormal: s underflows in f32 for f32 and bf16
    x[8, 3] = -5
    q, s = gq.quantize_i8(x)
    xd = x.double().cpu()
    for m in range(9):
        if m in (2, 3, 4):
            assert math.isnan(float(s[m])) and not bool(q[m].any())
            continue
        sr = float((xd[m].abs().max() / 127).float())
        assert float(s[m]) == sr
        ref = torch.zeros(K)
        if sr > 0:
            ref = (xd[m] / sr).float().round().clamp(-127, 127)
        assert torch.equal(q[m].float().cpu(), ref), m
    # and they show in the product: NaN there, finite elsewhere
    w = i8(20, K, gen(1))
    y = gq.gemm_i8(w, torch.ones(20, device="cuda"), q, s)
    bad = torch.isnan(y).all(1).cpu()
    assert bad.tolist() == [m in (2, 3, 4) for m in range(9)]
    assert not bool(torch.isnan(y[~bad.cuda()]).any())


# ------------------------------------------------------------------ product
SHAPES = [(1, 1, 1), (1, 4096, 4096), (1, 37, 100), (2, 16, 16), (3, 129, 127), (7, 1000, 129),
          (8, 65, 2050), (15, 48, 515), (16, 512, 1024), (17, 33, 63), (31, 255, 4000), (32, 64, 128),
          (33, 130, 300), (48, 640, 1111), (64, 512, 2048), (65, 257, 128), (100, 31, 4100),
          (127, 128, 129), (128, 1024, 512), (129, 513, 640), (255, 255, 255), (256, 256, 256),
          (257, 4099, 1025), (333, 777, 96), (512, 1536, 2048), (1000, 264, 136)]
# larger ones: every tile and every split of K that the library chooses from
WIDE = [(1, 40000, 1030), (1, 300, 16384), (1, 130, 20000), (2, 16400, 300), (2, 5000, 8192),
        (2, 100, 8200), (3, 20000, 256), (4, 70000, 129), (5, 16384, 700), (6, 16400, 400),
        (16, 70000, 130), (20, 70001, 260), (20, 4100, 1100), (32, 9000, 1000), (30, 40000, 300),
        (48, 4096, 4100), (64, 70000, 100), (90, 5000, 900), (128, 4096, 640), (300, 4100, 1300),
        (513, 2052, 2200), (512, 12300, 300), (700, 2000, 600), (1030, 6200, 200),
        (2048, 4100, 500), (2050, 8200, 130), (4100, 4200, 200), (530, 13500, 40), (780, 7760, 36),
        (641, 4430, 40), (99, 12340, 36), (33, 8420, 40), (66, 11700, 140), (36, 8230, 140),
        (560, 11030, 140), (560, 11030, 1100), (282, 13580, 1100), (641, 4430, 1100)]


@pytest.mark.parametrize("M,N,K", SHAPES + WIDE)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_gemm(M, N, K, dtype):
    g = gen(M * 31 + N * 17 + K)
    w, xq = i8(N, K, g, full=True), i8(M, K, g, pitch=-(-K // 16) * 16 + 32, full=True)
    sw, sx = scales(N, g, 0.01), scales(M, g, 0.02)
    bias = torch.randn(N, generator=g, device="cuda") if N % 2 else None
    out = Guarded(M, N, dtype, extra=M % 5)
    y = gq.gemm_i8(w, sw, xq, sx, bias=bias, out=out.t)
    torch.cuda.synchronize()
    out.check()
    s, ref = product(w, sw, xq, sx)
    scaled = ref
    if bias is not None:
        ref = ref + bias.double()
    # the i32 sum to f32, two scalings (3 u of the scaled sum), the sum with the
    # bias (u of the result), the result's type
    tol = 3 * U * scaled.abs() + (U + HALF[dtype]) * ref.abs() * (1 + 2.0 ** -7) + FLOOR[dtype]
    assert bool(((y.double() - ref).abs() <= tol).all())


def test_gemm_extreme_sums():
    # all -128 over the longest row: 2^14 * 131071 fits an int32, and f32 exactly
    K = gq.I8_MAX_K
    w = torch.full((33, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    xq = torch.full((40, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    one = torch.ones(40, device="cuda")
    for M in (1, 40):
        y = gq.gemm_i8(w, one[:33], xq[:M], one[:M])
        assert bool((y.double() == float(2 ** 14 * K)).all())


def test_gemm_scales_of_any_size():
    g = gen(5)
    w, xq = i8(70, 200, g), i8(40, 200, g)
    sw = torch.tensor([1e-30, 1e30, 0.0, 1.0, -2.0], device="cuda").repeat(14)
    sx = torch.tensor([1.0, 0.0, math.nan, 1e-5], device="cuda").repeat(10)
    y = gq.gemm_i8(w, sw, xq, sx)
    ref = (xq.double() @ w.double().t()) * sx.double()[:, None] * sw.double()
    nan = torch.isnan(sx)
    assert bool(torch.isnan(y[nan]).all())
    d = (y[~nan].double() - ref[~nan]).abs()
    assert bool((d <= 4 * U * ref[~nan].abs() + 2.0 ** -126).all())


def test_rows_do_not_depend_on_their_neighbours():
    # each row of a batch has the bits that it has in any batch of the same size
    g = gen(11)
    w, sw = i8(500, 777, g), scales(500, g)
    for M in (8, 40, 200):
        xq, sx = i8(M, 777, g), scales(M, g)
        y = gq.gemm_i8(w, sw, xq, sx)
        other = i8(M, 777, g)
        other[M // 2] = xq[M // 2]
        sx2 = scales(M, g)
        sx2[M // 2] = sx[M // 2]
        assert torch.equal(gq.gemm_i8(w, sw, other, sx2)[M // 2], y[M // 2])


# ------------------------------------------------------------------ linear
@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (1, 100, 77), (2, 64, 4096), (5, 321, 333),
                                   (16, 256, 12288), (33, 100, 512), (130, 260, 515),
                                   (300, 512, 640), (1, 9000, 100), (1, 40000, 515), (1, 64, 16384),
                                   (1, 64, 16400), (2, 10000, 257), (2, 17000, 130), (2, 40, 8192),
                                   (2, 40, 8300), (3, 100, 100)])
@pytest.mark.parametrize("xt", TYPES, ids=IDS)
@pytest.mark.parametrize("yt", TYPES, ids=IDS)
def test_linear_is_quantize_then_gemm(M, N, K, xt, yt):
    g = gen(M + 3 * N + 5 * K)
    w, sw = i8(N, K, g), scales(N, g, 0.01)
    bias = torch.randn(N, generator=g, device="cuda") if M % 2 else None
    wide = torch.randn((M, K + 11), generator=g, device="cuda").to(xt)
    for x in (wide[:, :K], wide[:, 11:], wide[:, :K].contiguous()):
        q, s = gq.quantize_i8(x)
        ref = gq.gemm_i8(w, sw, q, s, bias=bias, out_dtype=yt)
        q2 = torch.full((M, -(-K // 16) * 16), 55, dtype=torch.int8, device="cuda")
        s2 = torch.empty(M, device="cuda")
        y = gq.linear_i8(w, sw, x, bias=bias, out_dtype=yt, xq=q2[:, :K], sx=s2)
        assert torch.equal(y, ref)
        assert torch.equal(q2[:, :K], q) and torch.equal(s2, s)
        assert bool((q2[:, K:] == 55).all())
    assert gq.linear_i8(w, sw, x).dtype == xt


def test_linear_rows_with_nan():
    g = gen(3)
    w, sw = i8(300, 400, g), scales(300, g)
    for M in (1, 2, 20, 140):
        x = torch.randn((M, 400), generator=g, device="cuda")
        x[0, 5] = math.inf
        if M > 1:
            x[M - 1, 399] = math.nan
        y = gq.linear_i8(w, sw, x)
        assert bool(torch.isnan(y[0]).all()) and bool(torch.isnan(y[M - 1]).all())
        assert not bool(torch.isnan(y[1:M - 1]).any())


# ------------------------------------------------------------------ gradient of the layer
def split_error(dtype):
    """Relative error of the bf16 expansion of an f32 value: rounded at once to 8
    bits; 8 bits cut off, then the rest (below 2^-7) rounded to 8; exact."""
    return {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -15, torch.float32: 0.0}[dtype]


GRADS = [(1, 1, 1), (1, 64, 64), (1, 1000, 300), (2, 63, 130), (5, 65, 33), (8, 4096, 1024),
         (16, 127, 128), (17, 129, 1), (31, 640, 515), (32, 512, 512), (33, 200, 129),
         (64, 1111, 640), (77, 1037, 515), (128, 128, 128), (129, 2000, 255), (200, 50, 1000),
         (256, 1024, 512), (300, 333, 777), (513, 640, 264), (16, 20000, 200), (40, 9000, 600),
         (100, 30000, 130), (700, 3001, 2050), (2050, 130, 4100), (1500, 70, 5000), (4, 64, 100000),
         (1400, 3001, 70), (500, 4097, 1030), (1030, 1100, 4090), (1030, 2300, 4090),
         (2050, 777, 4100), (270, 3716, 7555)]


@pytest.mark.parametrize("M,N,K", GRADS)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_linear_grad(M, N, K, dtype):
    g = gen(M * 3 + N * 5 + K * 7)
    w, sw = i8(N, K, g, full=True), scales(N, g, 0.01)
    dy = torch.zeros((M, N + M % 3), dtype=dtype, device="cuda")[:, :N]
    dy.copy_(torch.randn((M, N), generator=g, device="cuda"))
    out = Guarded(M, K, dtype, extra=N % 4)
    need = gq.linear_i8_grad_workspace(dtype, M, N, K)
    ws = torch.full((need + 64,), 173, dtype=torch.uint8, device="cuda")
    dx = gq.linear_i8_grad(w, sw, dy, out=out.t, workspace=ws[:need])
    torch.cuda.synchronize()
    out.check()
    assert bool((ws[need:] == 173).all())
    a = dy.double() * sw.double()
    ref = a @ w.double()
    mag = a.abs() @ w.double().abs()
    # dy * sw in f32 (u), its bf16 expansion, N f32 additions per expansion in any
    # order (exact products), the additions of the partial sums
    planes = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}[dtype]
    tol = ((1 + planes * N + 64) * U + split_error(dtype)) * mag
    tol = tol + HALF[dtype] * (ref.abs() + tol) + FLOOR[dtype]
    assert bool(((dx.double() - ref).abs() <= tol).all())
    # the error as a whole, where the additions' errors average out: far below the
    # worst case, and small against the result
    rel = float((dx.double() - ref).norm() / ref.norm())
    assert rel <= {torch.float32: 16 * U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[dtype]
    assert torch.equal(gq.linear_i8_grad(w, sw, dy), dx)


@pytest.mark.parametrize("M", [1, 5, 32, 33, 64, 65, 128, 129, 300, 1030])
@pytest.mark.parametrize("N,K", [(8, 40), (64, 128), (72, 515), (1000, 256), (4104, 300), (640, 2050)])
def test_linear_grad_of_aligned_rows(M, N, K):
    # bf16 rows on 16 bytes are read as they lie up to 128 tokens; what lies behind
    # them is no part of the result, be it NaN
    g = gen(M + N + K)
    w, sw = i8(N, K, g, full=True), scales(N, g, 0.01)
    wide = torch.full((M, N + 8 * (M % 3)), math.nan, dtype=torch.bfloat16, device="cuda")
    dy = wide[:, :N]
    dy.copy_(torch.randn((M, N), generator=g, device="cuda"))
    out = Guarded(M, K, torch.bfloat16, extra=N % 4)
    dx = gq.linear_i8_grad(w, sw, dy, out=out.t)
    torch.cuda.synchronize()
    out.check()
    a = dy.double() * sw.double()
    ref = a @ w.double()
    mag = a.abs() @ w.double().abs()
    # one rounding of sw w (or of dy sw) to bf16, N additions in f32, the result's
    tol = ((2 + N + 64) * U + 2.0 ** -8) * mag
    tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(((dx.double() - ref).abs() <= tol).all())
    odd = torch.zeros((M, N + 1), dtype=torch.bfloat16, device="cuda")[:, :N]
    odd.copy_(dy)
    dx2 = gq.linear_i8_grad(w, sw, odd)
    assert bool(((dx2.double() - ref).abs() <= tol).all())
    # rows with NaN and infinities stay apart from the others
    if M > 4:
        dy[1, N - 1], dy[2, 0], dy[3, N // 2] = math.nan, math.inf, -math.inf
        dz = gq.linear_i8_grad(w, sw, dy)
        assert bool(torch.isnan(dz[1]).all()) and not bool(torch.isfinite(dz[2:4]).any())
        keep = [0] + list(range(4, M))
        assert torch.equal(dz[keep], dx[keep])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_linear_grad_is_the_adjoint(dtype):
    # <dy, w x> = <dx, x> for the layer as a linear map of the dequantized x
    g = gen(9)
    M, N, K = 40, 300, 200
    w, sw, xq, sx = i8(N, K, g), scales(N, g, 0.01), i8(M, K, g), scales(M, g, 0.01)
    dy = torch.randn((M, N), generator=g, device="cuda").to(dtype)
    _, y = product(w, sw, xq, sx)
    dx = gq.linear_i8_grad(w, sw, dy).double()
    x = xq.double() * sx.double()[:, None]
    mag = float((dx.abs() * x.abs()).sum() + (dy.double().abs() * y.abs()).sum())
    # every element of dx is off by its rounding and its sum's, see test_linear_grad
    a = dy.double() * sw.double()
    slack = (split_error(dtype) + 3 * N * U) * float(((a.abs() @ w.double().abs()) * x.abs()).sum())
    assert abs(float((dx * x).sum() - (dy.double() * y).sum())) <= HALF[dtype] * mag + slack


def test_linear_grad_empty_and_special():
    g = gen(2)
    w, sw = i8(50, 70, g), scales(50, g)
    out = torch.full((6, 70), 9.0, device="cuda")
    gq.linear_i8_grad(w[:0], sw[:0], torch.zeros((6, 0), device="cuda"), out=out)
    assert not bool(out.any())
    dy = torch.randn((6, 50), generator=g, device="cuda")
    dy[2, 3] = math.inf
    dy[4, 49] = math.nan
    for dt in TYPES:
        dx = gq.linear_i8_grad(w, sw, dy.to(dt))
        assert bool(torch.isnan(dx[4]).all())
        assert not bool(torch.isfinite(dx[2]).any())
        assert bool(torch.isfinite(dx[[0, 1, 3, 5]]).all())


# ------------------------------------------------------------------ the loss
def head(M, N, K, seed, sharp=20.0, pitch=None):
    """Weights and hidden states whose target logits run from chance to certainty."""
    g = gen(seed)
    w = i8(N, K, g)
    sw = scales(N, g, K ** -0.5 / 64)
    t = torch.randint(0, N, (M,), generator=g, device="cuda")
    x = torch.randn((M, K), generator=g, device="cuda")
    r = w[t].float()
    x += torch.rand((M, 1), generator=g, device="cuda") * sharp * r / r.norm(dim=1, keepdim=True).clamp(min=1e-3)
    q, sx = gq.quantize_i8(x)
    xq = i8(M, K, g, pitch=pitch)
    xq.copy_(q)
    return w, sw, xq, sx, t


def loss_reference(w, sw, xq, sx, t):
    _, z = product(w, sw, xq, sx)
    lse = torch.logsumexp(z, 1)
    hit = z.gather(1, t.clamp(0, z.shape[1] - 1)[:, None])[:, 0]
    return z, lse, torch.where(t >= 0, lse - hit, torch.zeros_like(lse))


def logit_error(z):
    """Base-2 logits from the exact sum: its conversion, sx log2 e (and log2 e's own
    rounding), two scalings, and back to base e: 7 u of the largest logit."""
    return 7 * U * z.abs().amax(1)


LOSSES = [(1, 1, 1), (1, 1000, 64), (1, 32003, 515), (2, 127, 100), (5, 128, 128), (8, 4097, 1024),
          (16, 129, 33), (17, 1000, 200), (32, 3000, 256), (33, 255, 129), (64, 5000, 300),
          (128, 256, 512), (130, 1111, 640), (257, 2050, 255), (500, 513, 64), (3, 16390, 200),
          (12, 16384, 600), (20, 70001, 260), (48, 4096, 1000), (100, 20000, 130), (300, 9000, 300),
          (600, 12300, 140), (2050, 8200, 130), (530, 13500, 40), (780, 7760, 36), (641, 4430, 40),
          (66, 11700, 140), (36, 8230, 140), (99, 12340, 36), (282, 13580, 300), (641, 4430, 700),
          (50, 70000, 60)]


@pytest.mark.parametrize("M,N,K", LOSSES)
def test_loss(M, N, K):
    w, sw, xq, sx, t = head(M, N, K, M + N + K, pitch=-(-K // 16) * 16 + 16)
    if M > 2:
        t[::3] = -100
    out = Guarded(2, M, torch.float32)
    need = gq.loss_i8_workspace(M, N, K)
    ws = torch.full((need + 64,), 173, dtype=torch.uint8, device="cuda")
    loss, lse = gq.loss_i8(w, sw, xq, sx, t, loss=out.t[0], lse=out.t[1], workspace=ws[:need])
    torch.cuda.synchronize()
    out.check()
    assert bool((ws[need:] == 173).all())
    z, lse_r, loss_r = loss_reference(w, sw, xq, sx, t)
    # each term's exponent carries the logit's error, twice (the maximum's too); the
    # exponentials are good to 2 u, and no term passes more than 300 additions
    tol = 3 * logit_error(z) + (302 + 3) * U + 3 * U * lse_r.abs()
    assert bool(((lse.double() - lse_r).abs() <= tol).all())
    assert bool(((loss.double() - loss_r).abs() <= tol + logit_error(z) + 2 * U * loss_r.abs()).all())
    assert not bool(loss[t < 0].any())
    l2, e2 = gq.loss_i8(w, sw, xq, sx, t)
    assert torch.equal(l2, loss) and torch.equal(e2, lse)


def test_loss_special_targets_and_rows():
    for M in (1, 6, 40, 150):
        w, sw, xq, sx, t = head(M, 1000, 96, M)
        t[M - 1] = 1000              # one past the vocabulary
        if M > 3:
            t[0] = -1
            t[1] = -(1 << 40)
            t[2] = 1 << 40
            sx[3] = math.nan
        loss, lse = gq.loss_i8(w, sw, xq, sx, t)
        assert math.isnan(float(loss[M - 1])) and math.isfinite(float(lse[M - 1]))
        if M > 3:
            assert float(loss[0]) == 0 and float(loss[1]) == 0
            assert math.isnan(float(loss[2])) and math.isnan(float(loss[3]))
            assert math.isnan(float(lse[3]))
            keep = [m for m in range(M) if m not in (2, 3, M - 1)]
            assert bool(torch.isfinite(loss[keep]).all())
        every = gq.loss_i8(w, sw, xq, sx, torch.full_like(t, -100))[0]
        assert not bool(every.any())


def test_loss_of_equal_logits():
    # no row stands out: lse = log N exactly, whatever the tiles
    for N in (1, 127, 128, 129, 5000):
        w = torch.zeros((N, 64), dtype=torch.int8, device="cuda")
        for M in (3, 40, 140):
            q = torch.ones((M, 64), dtype=torch.int8, device="cuda")
            one = torch.ones(max(N, M), device="cuda")
            loss, lse = gq.loss_i8(w, one[:N], q, one[:M], torch.zeros(M, dtype=torch.int64, device="cuda"))
            assert float((lse.double() - math.log(N)).abs().max()) <= 4 * U * max(1.0, math.log(N))
            assert torch.equal(loss, lse)


def test_loss_of_far_apart_logits():
    # logits from -6 10^5 to 6 10^5: no overflow, and the largest one decides
    g = gen(4)
    w, xq = i8(700, 64, g), i8(140, 64, g)
    one = torch.ones(700, device="cuda")
    for M in (2, 20, 140):
        z = xq[:M].double() @ w.double().t()
        top, at = z.max(1)
        loss, lse = gq.loss_i8(w, one, xq[:M], one[:M], at)
        assert float((lse.double() - torch.logsumexp(z, 1)).abs().max()) <= 12 * U * float(z.abs().max())
        far = gq.loss_i8(w, one, xq[:M], one[:M], z.argmin(1))[0]
        assert float((far.double() - (top - z.amin(1))).abs().max()) <= 24 * U * float(z.abs().max())


# ------------------------------------------------------------------ gradient of the loss
@pytest.mark.parametrize("M,N,K", LOSSES + [(3, 140000, 96), (40, 70000, 40)])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_loss_grad(M, N, K, dtype):
    w, sw, xq, sx, t = head(M, N, K, M + N + K, pitch=-(-K // 16) * 16 + 16)
    if M > 2:
        t[::3] = -100
    g = gen(77)
    gw = torch.randn(M, generator=g, device="cuda")
    z, lse_r, _ = loss_reference(w, sw, xq, sx, t)
    lse = lse_r.float()
    out = Guarded(M, K, dtype, extra=N % 4)
    need = gq.loss_i8_grad_workspace(dtype, M, N, K)
    ws = torch.full((need + 64,), 173, dtype=torch.uint8, device="cuda")
    dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse, gw, out=out.t, workspace=ws[:need])
    torch.cuda.synchronize()
    out.check()
    assert bool((ws[need:] == 173).all())
    p = torch.exp(z - lse.double()[:, None])
    f = p.clone()
    keep = (t >= 0).double()[:, None]
    rows = torch.arange(M, device="cuda")
    f[rows, t.clamp(min=0)] -= 1.0
    a = f * sw.double() * keep
    wd = w.double()
    gd = gw.double()[:, None]
    ref = gd * (a @ wd)
    # p is off by its exponent's error (the logit's and lse's) and the exponential's
    # 2 u; the difference with 1, the product with sw and the factor gw by u each;
    # then the expansion and the additions, as in test_linear_grad
    ep = (logit_error(z) + 3 * U * lse_r.abs() + 4 * U)[:, None]
    planes = {torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}[dtype]
    mag = a.abs() @ wd.abs()
    tol = gd.abs() * (((planes * N + 70) * U + split_error(dtype)) * mag
                      + ep * ((p * sw.double() * keep) @ wd.abs()))
    tol = tol + HALF[dtype] * (ref.abs() + tol) + FLOOR[dtype]
    assert bool(((dx.double() - ref).abs() <= tol).all())
    assert not bool(dx[t < 0].any())
    assert torch.equal(gq.loss_i8_grad(w, sw, xq, sx, t, lse, gw, out_dtype=dtype), dx)


@pytest.mark.parametrize("M,N,K", [(1, 2000, 256), (2, 3137, 768), (16, 16000, 100),
                                   (17, 4000, 515), (70, 30000, 200), (300, 9000, 300)])
def test_loss_grad_where_the_target_is_most_of_it(M, N, K):
    # nearly equal logits: a row's factor is -1 at its target and about 1 / N elsewhere.
    # The target's part is not rounded to bf16: beside the result's own rounding there
    # is that of the others, whose sum over N random rows is about sqrt(N) / N of the
    # target's, six times that where its scale is 0.2 and theirs 1.2: 0.14 of the result
    # at most, whose rounding adds 0.14^2 / 2 = 1% to the result's own
    w, sw, xq, sx, t = head(M, N, K, 31 * M + N)
    sx = sx * 1e-3
    z = (xq.double() * sx.double()[:, None]) @ (w.double() * sw.double()[:, None]).t()
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    p[torch.arange(M, device="cuda"), t] -= 1.0
    ref = p @ (w.double() * sw.double()[:, None])
    one = torch.ones(M, device="cuda")
    dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse.float(), one)
    own = float((ref.bfloat16().double() - ref).norm())
    assert float((dx.double() - ref).norm()) <= 1.05 * own


@pytest.mark.parametrize("M,N,K", [(1, 2112, 698), (16, 3000, 512), (40, 5000, 300)])
def test_loss_grad_near_certainty(M, N, K):
    # The target's factor is -(1 - p) with 1 - p well below the rounding of its logit;
    # the sum of the others' as large.  z - lse is off by the rounding of its difference
    # (u of it), so the factor by a few u and by the expansion; the others' by u |z| each.
    # What the two of them leave is small against the result where W's rows differ.
    g = gen(M + N)
    w, sw = i8(N, K, g), scales(N, g, K ** -0.5 / 64)
    t = torch.arange(M, device="cuda") * 7
    xq, sx = gq.quantize_i8(w[t].float())
    z = (xq.double() * sx.double()[:, None]) @ (w.double() * sw.double()[:, None]).t()
    gap = z.gather(1, t[:, None])[:, 0] - z.scatter(1, t[:, None], -math.inf).amax(1)
    sx = (sx.double() * (8.0 / gap)).float()  # the target's logit 8 above the next
    z = (xq.double() * sx.double()[:, None]) @ (w.double() * sw.double()[:, None]).t()
    lse = torch.logsumexp(z, 1).float()
    rows = torch.arange(M, device="cuda")
    p = torch.exp(z - lse.double()[:, None])
    p[rows, t] = torch.expm1(z[rows, t] - lse.double())
    wd = w.double() * sw.double()[:, None]
    ref = p @ wd
    dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse, torch.ones(M, device="cuda"),
                         out_dtype=torch.float32)
    tol = (p.abs() * (4 * U + 2 * U * (z.abs() + 1) * (p > 0) + (3 * N + 70) * U)) @ wd.abs()
    tol = tol + 4 * U * (z[rows, t] - lse.double()).abs()[:, None] * wd[t].abs()
    assert bool(((dx.double() - ref).abs() <= tol).all())
    # the target's own logit adds nothing of its size
    assert float((dx.double() - ref).norm()) <= 64 * U * float(ref.norm())


def test_loss_grad_special_rows():
    for M in (6, 40, 150):
        w, sw, xq, sx, t = head(M, 1000, 96, M)
        gw = torch.ones(M, device="cuda")
        t[0], t[1], t[2] = -1, 1000, 1 << 40
        sx[3] = math.nan
        sx[0] = math.nan          # an ignored row stays zero, whatever it holds
        gw[0] = math.nan
        _, lse = gq.loss_i8(w, sw, xq, sx, t)
        for dt in TYPES:
            dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse, gw, out_dtype=dt)
            assert not bool(dx[0].any())
            assert bool(torch.isnan(dx[1:4]).all())
            assert bool(torch.isfinite(dx[4:]).all())
            every = gq.loss_i8_grad(w, sw, xq, sx, torch.full_like(t, -5), lse, gw, out_dtype=dt)
            assert not bool(every.any())


@pytest.mark.parametrize("M,N,K", [(5, 1000, 96), (40, 3001, 200), (150, 777, 130)])
def test_loss_grad_against_differences(M, N, K):
    # d loss / d sx[m] = sum_k dx[m, k] xq[m, k]: a row's scale moves all of its
    # hidden state.  Central differences of the loss itself, in 64 bits.
    w, sw, xq, sx, t = head(M, N, K, 3 * M)
    loss, lse = gq.loss_i8(w, sw, xq, sx, t)
    dx = gq.loss_i8_grad(w, sw, xq, sx, t, lse, torch.ones(M, device="cuda"), out_dtype=torch.float32)
    slope = (dx.double() * xq.double()).sum(1)
    e = 1e-4
    s = xq.double() @ w.double().t() * sw.double()

    def f(scale):
        z = s * scale[:, None]
        return torch.logsumexp(z, 1) - z.gather(1, t[:, None])[:, 0]

    s64 = sx.double()
    num = (f(s64 * (1 + e)) - f(s64 * (1 - e))) / (2 * e * s64)
    # the loss is a log-sum-exp of s * scale: its third derivative is below
    # (max|s| + ...)^3 terms, the centred difference's error below
    # (e scale)^2 / 6 * 8 max|s|^3; and the gradient's f32 roundings
    top = s.abs().amax(1)
    mag = (dx.double().abs() * xq.double().abs()).sum(1)
    tol = (e * s64) ** 2 / 6 * 8 * top ** 3 + 2.0 ** -12 * mag + 1e-9 * top + 40 * U * (top * s64 + 1) * top
    assert bool(((slope - num).abs() <= tol).all())


# ------------------------------------------------------------------ far offsets
def test_offsets_past_32_bits():
    # weights of 4.6 GB: byte offsets of the last rows pass 2^32
    N, K, tail = 140000, 32768, 200
    g = gen(6)
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    w[-tail:] = i8(tail, K, g)
    sw = torch.ones(N, device="cuda")
    for M in (1, 3, 20, 200):
        xq, sx = i8(M, K, g), scales(M, g, 1e-6)
        s, z = product(w[-tail:], sw[-tail:], xq, sx)
        y = gq.gemm_i8(w, sw, xq, sx)
        assert not bool(y[:, :-tail].any())
        assert bool(((y[:, -tail:].double() - z).abs() <= 4 * U * z.abs()).all())
        t = torch.full((M,), N - 1, device="cuda")
        loss, lse = gq.loss_i8(w, sw, xq, sx, t)
        ref = torch.logsumexp(torch.cat([z, torch.full_like(z[:, :1], math.log(N - tail))], 1), 1)
        tol = 3 * logit_error(z) + 320 * U + 3 * U * ref.abs()
        assert bool(((lse.double() - ref).abs() <= tol).all())
        assert bool(((loss.double() - (ref - z[:, -1])).abs() <= 2 * tol).all())
        # only the last rows have weights: their part of the gradient is all of it
        dy = torch.randn((M, N), generator=g, device="cuda")
        dx = gq.linear_i8_grad(w, sw, dy)
        d = dy[:, -tail:].double()
        ref = d @ w[-tail:].double()
        mag = d.abs() @ w[-tail:].double().abs()
        # the zero products add nothing, but their additions may be in any place
        assert bool(((dx.double() - ref).abs() <= (3 * tail + 70) * U * mag).all())
        del dy, dx, y


def test_results_past_32_bits():
    # 2.6 10^9 results: element offsets pass 2^31, and in bytes 2^32
    M, N, K = 40000, 65536, 64
    g = gen(12)
    w, sw, xq, sx = i8(N, K, g), scales(N, g, 0.01), i8(M, K, g), scales(M, g, 0.01)
    y = gq.gemm_i8(w, sw, xq, sx, out_dtype=torch.bfloat16)
    rows = torch.tensor([0, 1, 127, 128, 20000, 32767, 32768, M - 129, M - 1], device="cuda")
    _, ref = product(w, sw, xq[rows], sx[rows])
    assert bool(((y[rows].double() - ref).abs() <= (2.0 ** -8 + 8 * U) * ref.abs()).all())


def test_many_rows():
    # more rows than a grid dimension of 32768 takes, and not a multiple of it
    M, K, N = 70001, 48, 40
    g = gen(13)
    x = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    q, s = gq.quantize_i8(x)
    xd = x.double()
    sr = (xd.abs().amax(1) / 127).float()
    assert torch.equal(s, sr)
    assert torch.equal(q.float(), (xd / sr.double()[:, None]).float().round())
    w, sw = i8(N, K, g), scales(N, g, 0.01)
    t = torch.randint(0, N, (M,), generator=g, device="cuda")
    z, lse_r, loss_r = loss_reference(w, sw, q, s, t)
    loss, lse = gq.loss_i8(w, sw, q, s, t)
    tol = 4 * logit_error(z) + 320 * U + 3 * U * lse_r.abs()
    assert bool(((loss.double() - loss_r).abs() <= tol + 2 * U * loss_r.abs()).all())
    for dt in (torch.float32, torch.bfloat16):
        dx = gq.loss_i8_grad(w, sw, q, s, t, lse, torch.ones(M, device="cuda"), out_dtype=dt)
        f = torch.softmax(z, 1)
        f[torch.arange(M, device="cuda"), t] -= 1.0
        ref = (f * sw.double()) @ w.double()
        assert float((dx.double() - ref).norm() / ref.norm()) <= (2.0 ** -8 if dt != torch.float32 else 2.0 ** -18)
    dy = torch.randn((M, N), generator=g, device="cuda")
    dx = gq.linear_i8_grad(w, sw, dy)
    ref = (dy.double() * sw.double()) @ w.double()
    assert float((dx.double() - ref).norm() / ref.norm()) <= 2.0 ** -21


# ------------------------------------------------------------------ together
def test_layer_and_head_with_their_gradients():
    # hidden -> int8 layer -> int8 head -> loss, and back: each call on what the
    # one before it gave
    g = gen(21)
    M, N, D, V = 70, 384, 256, 5003
    w1, s1 = gq.quantize_i8(torch.randn((N, D), generator=g, device="cuda") * D ** -0.5)
    w2, s2 = gq.quantize_i8(torch.randn((V, N), generator=g, device="cuda") * N ** -0.5)
    x = torch.randn((M, D), generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    t[::7] = -100
    h = gq.linear_i8(w1, s1, x)
    hq, sh = gq.quantize_i8(h)
    loss, lse = gq.loss_i8(w2, s2, hq, sh, t)
    gw = torch.full((M,), 1.0 / int((t >= 0).sum()), device="cuda")
    dh = gq.loss_i8_grad(w2, s2, hq, sh, t, lse, gw)
    dx = gq.linear_i8_grad(w1, s1, dh)
    assert dh.dtype == dx.dtype == torch.bfloat16 and dx.shape == x.shape
    wd1, wd2 = w1.double() * s1.double()[:, None], w2.double() * s2.double()[:, None]
    hd = (hq.double() * sh.double()[:, None]).requires_grad_(True)
    z = hd @ wd2.t()
    ref = torch.nn.functional.cross_entropy(z, t, ignore_index=-100)
    (dhr,) = torch.autograd.grad(ref, hd)
    assert abs(float((loss.double() * gw.double()).sum()) - float(ref.detach())) <= 1e-5
    # bf16 twice: the factor's and the result's roundings, averaged over a row
    assert float((dh.double() - dhr).norm() / dhr.norm()) <= 2.0 ** -8
    dxr = dhr @ wd1
    assert float((dx.double() - dxr).norm() / dxr.norm()) <= 2.0 ** -7


def _step(w1, s1, w2, s2, x, t, gw, b):
    gq.linear_i8(w1, s1, x, out=b["h"], xq=b["xq"], sx=b["sx"])
    gq.quantize_i8(b["h"], out=b["hq"], scale=b["sh"])
    gq.loss_i8(w2, s2, b["hq"], b["sh"], t, loss=b["loss"], lse=b["lse"])
    gq.loss_i8_grad(w2, s2, b["hq"], b["sh"], t, b["lse"], gw, out=b["dh"])
    gq.linear_i8_grad(w1, s1, b["dh"], out=b["dx"])


@pytest.mark.parametrize("M", [1, 16, 100])
def test_captured_and_replayed(M):
    g = gen(M)
    N, D, V = 320, 200, 3001
    w1, s1, w2, s2 = i8(N, D, g), scales(N, g, 1e-3), i8(V, N, g), scales(V, g, 1e-3)
    x = torch.randn((M, D), generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    gw = scales(M, g)

    def buffers():
        e = dict(device="cuda")
        return {"h": torch.empty((M, N), dtype=torch.bfloat16, **e),
                "xq": torch.empty((M, 208), dtype=torch.int8, **e)[:, :D], "sx": torch.empty(M, **e),
                "hq": torch.empty((M, N), dtype=torch.int8, **e), "sh": torch.empty(M, **e),
                "loss": torch.empty(M, **e), "lse": torch.empty(M, **e),
                "dh": torch.empty((M, N), dtype=torch.bfloat16, **e),
                "dx": torch.empty((M, D), dtype=torch.bfloat16, **e)}

    eager, held = buffers(), buffers()
    _step(w1, s1, w2, s2, x, t, gw, eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(w1, s1, w2, s2, x, t, gw, held)
    for n in range(4):
        x.copy_(torch.randn((M, D), generator=g, device="cuda"))
        t.copy_(torch.randint(0, V, (M,), generator=g, device="cuda"))
        _step(w1, s1, w2, s2, x, t, gw, eager)
        graph.replay()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(eager[k], held[k]), (n, k)


def test_other_streams():
    # the same step on two streams at once, each with what the call allocates
    g = gen(8)
    M, N, D, V = 64, 320, 256, 4000
    w1, s1, w2, s2 = i8(N, D, g), scales(N, g, 1e-3), i8(V, N, g), scales(V, g, 1e-3)
    xs = [torch.randn((M, D), generator=g, device="cuda").bfloat16() for _ in range(2)]
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    gw = scales(M, g)

    def step(x, stream):
        h = gq.linear_i8(w1, s1, x, stream=stream)
        hq, sh = gq.quantize_i8(h, stream=stream)
        loss, lse = gq.loss_i8(w2, s2, hq, sh, t, stream=stream)
        dh = gq.loss_i8_grad(w2, s2, hq, sh, t, lse, gw, stream=stream)
        return h, loss, lse, dh, gq.linear_i8_grad(w1, s1, dh, stream=stream)

    ref = [step(x, None) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for n in range(3):
        got = [step(x, s if n < 2 else s.cuda_stream) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_refusals_on_the_device():
    g = gen(1)
    w, sw, xq, sx = i8(40, 64, g), scales(40, g), i8(4, 64, g), scales(4, g)
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    x = torch.zeros((4, 64), device="cuda")
    bad = [
        lambda: gq.gemm_i8(w, sw[:39], xq, sx),                       # scales of another length
        lambda: gq.gemm_i8(w, sw, xq[:, :63], sx),                    # another K
        lambda: gq.gemm_i8(w.t(), sw, xq, sx),                        # columns, not rows
        lambda: gq.gemm_i8(w[:, 8:40], sw, xq[:, 8:40], sx),          # rows off 16 bytes
        lambda: gq.gemm_i8(w, sw.double(), xq, sx),
        lambda: gq.gemm_i8(w, sw, xq, sx, out=torch.empty((4, 41), device="cuda")),
        lambda: gq.gemm_i8(w, sw, xq, sx, bias=sw.bfloat16()),
        lambda: gq.gemm_i8(w, sw, xq, sx, out_dtype=torch.float64),
        lambda: gq.gemm_i8(w, sw, xq, sx, out=torch.empty((40, 4), device="cuda").t()),
        lambda: gq.linear_i8(w, sw, x.double()),
        lambda: gq.linear_i8(w, sw, x.cpu()),
        lambda: gq.linear_i8(w, sw, x, xq=torch.empty((4, 72), dtype=torch.int8, device="cuda")[:, :64]),
        lambda: gq.linear_i8(w, sw, torch.zeros((1, 64), device="cuda").expand(4, 64)),
        lambda: gq.linear_i8_grad(w, sw, torch.zeros((4, 39), device="cuda")),
        lambda: gq.linear_i8_grad(w, sw, torch.zeros((4, 40), device="cuda"),
                                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: gq.linear_i8_grad(w, sw, torch.zeros((4, 40), device="cuda"),
                                  out=torch.empty((4, 64), dtype=torch.bfloat16, device="cuda")),
        lambda: gq.loss_i8(w, sw, xq, sx, t.int()),
        lambda: gq.loss_i8(w, sw, xq, sx, t[:3]),
        lambda: gq.loss_i8(w[:0], sw[:0], xq, sx, t),
        lambda: gq.loss_i8_grad(w, sw, xq, sx, t, sx, sx[:3]),
        lambda: gq.loss_i8_grad(w, sw, xq, sx, t, sx, sx, out_dtype=torch.int8),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, gq.GemmqError)):
            call()
            print("call %d was taken" % i)
    # no rows: no work, and results of the right shape
    assert gq.linear_i8(w, sw, x[:0]).shape == (0, 40)
    assert gq.quantize_i8(x[:0])[0].shape == (0, 64)
    assert gq.linear_i8_grad(w, sw, torch.zeros((0, 40), device="cuda")).shape == (0, 64)
    assert gq.loss_i8(w, sw, xq[:0], sx[:0], t[:0])[0].shape == (0,)
    assert gq.loss_i8_grad(w, sw, xq[:0], sx[:0], t[:0], sx[:0], sx[:0]).shape == (0, 64)
    assert gq.gemm_i8(w[:0], sw[:0], xq, sx).shape == (4, 0)
