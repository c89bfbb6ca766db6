"""Sampling on the GPU against its definition in 64 bits: the vocabulary sorted, the weights
summed in that order."""
import math

import pytest
import torch

import quant_packed_weight_amd as gq
from block_util import IDS, TYPES, U, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import gpu_util

    gpu_util.device()


def reference(z, u, t=None, k=None, p=None, q=None):
    M, N = z.shape
    dev = z.device
    full = lambda v: torch.full((M,), v, dtype=torch.float64, device=dev)  # noqa: E731
    t = full(1.0) if t is None else t.double()
    k = full(0) if k is None else k
    p = full(1.0) if p is None else torch.where(torch.isnan(p), 1.0, p.double())
    q = full(0.0) if q is None else torch.where(torch.isnan(q), 0.0, q.double()).clamp(max=1)
    u = torch.where(torch.isnan(u), 0.0, u.double()).clamp(0, 1 - 2.0 ** -24)
    bad = torch.isnan(z).any(1) | ((z == math.inf).any(1)) | (z == -math.inf).all(1)
    bad |= torch.isnan(t) | (t == math.inf)
    v, order = torch.sort(torch.where(bad[:, None], 0.0, z.double()), dim=1, descending=True, stable=True)
    place = torch.arange(N, device=dev)[None]
    greedy = (t <= 0)[:, None]
    e = torch.exp((v - v[:, :1]) / torch.where(t > 0, t, 1.0)[:, None])
    keep = (place < 1) | ~greedy
    keep &= (place < k[:, None]) | (k <= 0)[:, None]
    e = torch.where(keep, e, 0.0)
    total = torch.cumsum(e, 1)
    whole = total[:, -1:]
    before = torch.cat([torch.zeros_like(whole), total[:, :-1]], 1)
    keep &= (before < p[:, None] * whole) | (p >= 1)[:, None] | (place < 1)
    keep &= e >= q[:, None]
    e = torch.where(keep, e, 0.0)
    total = torch.cumsum(e, 1)
    at = (total <= u[:, None] * total[:, -1:]).sum(1, keepdim=True).clamp(max=N - 1)
    token = torch.where(bad, -1, order.gather(1, at)[:, 0])
    # the first token's share by what the others have: log(1 / (1 + others))
    others = e[:, 1:].sum(1)
    drawn = (v.gather(1, at) - v[:, :1])[:, 0] / torch.where(t > 0, t, 1.0)
    logp = torch.where(bad, math.nan, torch.where(greedy[:, 0], 0.0, drawn) - torch.log1p(others))
    return token, logp


def check(z, u, t=None, k=None, p=None, q=None):
    token, logp = gq.sample(z, u, temperature=t, top_k=k, top_p=p, min_p=q)
    rt, rl = reference(z, u, t, k, p, q)
    assert torch.equal(token, rt), torch.nonzero(token != rt)[:5].tolist()
    assert torch.equal(torch.isnan(logp), torch.isnan(rl))
    fine = ~torch.isnan(rl)
    # in 64 bits, with sums of weights to 2^-38 of the largest, rounded once
    assert bool(((logp.double() - rl).abs()[fine] <= (U * (1 + 1e-6) * rl.abs() + 1e-10)[fine]).all())
    return token, logp


def settings(M, g):
    r = lambda: torch.rand(M, generator=g, device="cuda")  # noqa: E731
    t = torch.where(r() < 0.1, 0.0, 0.3 + 1.5 * r())
    k = torch.where(r() < 0.5, 0.0, 1 + 100 * r() ** 2).to(torch.int32)
    p = torch.where(r() < 0.4, 1.0, 0.02 + 0.97 * r())
    q = torch.where(r() < 0.6, 0.0, 0.5 * r() ** 3)
    return t, k, p, q


def logits(kind, M, N, g):
    z = torch.randn((M, N), generator=g, device="cuda")
    if kind == "peaked":
        z = 3 * z
        at = torch.randint(0, N, (M, 8), generator=g, device="cuda")
        return z.scatter_(1, at, 12 + 3 * torch.randn((M, 8), generator=g, device="cuda"))
    if kind == "flat":      # as of a model before training
        return 0.05 * z
    if kind == "ties":      # few distinct values, many equal
        return (2 * z).round()
    if kind == "masked":
        z = torch.where(torch.rand((M, N), generator=g, device="cuda") < 0.7, -math.inf, 2 * z)
        z[:, 0] = 0.5
        return z
    return 1e4 * z          # "far": all but a few weights are zero


# one part and several, both sides of the list, odd sizes
WIDTHS = [1, 2, 3, 17, 255, 256, 257, 1000, 1025, 4095, 4096, 4097, 8193, 16384, 16385, 32003,
          32768, 32769, 151936]


@pytest.mark.parametrize("kind", ["peaked", "flat", "ties", "masked", "far"])
@pytest.mark.parametrize("N", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_sample(N, kind, dtype):
    g = gen(N * 5 + len(kind))
    M = 41
    z = torch.empty((M, N + 3), dtype=dtype, device="cuda")[:, N % 4:N + N % 4]
    z.copy_(logits(kind, M, N, g))
    u = torch.rand(M, generator=g, device="cuda")
    t, k, p, q = settings(M, g)
    check(z, u, t, k, p, q)
    check(z.contiguous(), u)
    check(z, u, t=t)
    check(z, u, k=k)
    check(z, u, p=p)
    check(z, u, t=2 * t, q=q)
    check(z, u, t=t, k=k, p=p)
    check(z[:1], u[:1], k=k[:1], p=p[:1], q=q[:1])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("N", [16385, 32768, 32770, 50001, 65536, 65537])
def test_many_rows(N, dtype):
    # rows of one launch and of four by their number
    g = gen(N)
    for M in (1, 15, 16, 127, 130):
        z = logits("peaked", M, N, g).to(dtype)
        u = torch.rand(M, generator=g, device="cuda")
        t, k, p, q = settings(M, g)
        check(z, u, t, k, p, q)
        check(z, u, p=p)


@pytest.mark.parametrize("N", [7, 5000, 20000, 40000])
def test_equal_logits(N):
    # the order is the index's: every place can be computed
    M = 64
    z = torch.full((M, N), 2.5, device="cuda")
    z[1::2] = torch.tensor([0.0, -0.0], device="cuda").repeat(N)[:N]  # equal as well
    u = torch.arange(M, device="cuda") / M
    token, logp = check(z, u)
    ref = torch.floor(u.double() * N).long()
    assert torch.equal(token, ref)
    assert bool(((logp.double() + math.log(N)).abs() <= U * math.log(N) + 1e-10).all())
    k = torch.arange(1, M + 1, device="cuda").int()
    token, _ = check(z, u, k=k)
    assert torch.equal(token, torch.floor(u.double() * k.clamp(max=N)).long())
    p = torch.full((M,), 0.5, device="cuda")
    token, _ = check(z, u, p=p)
    assert torch.equal(token, torch.floor(u.double() * ((N + 1) // 2)).long())
    check(z, u, k=k * 3, p=p)
    check(z, u, k=k * 100, p=p, q=p, t=p)


@pytest.mark.parametrize("N", [5001, 60000])
@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_many_ties_at_every_place(N, dtype):
    # more tokens share a logit than are sorted, at the places that the limits decide
    g = gen(N)
    M = 48
    z = torch.randint(0, 3, (M, N), generator=g, device="cuda").to(dtype) * 0.5 - 0.25
    z[:, 100:103] = 3.0
    u = torch.rand(M, generator=g, device="cuda")
    t, k, p, q = settings(M, g)
    k = torch.where(k > 0, k * (N // 150), 0).int()
    check(z, u)
    check(z, u, t=t, k=k)
    check(z, u, t=t, p=p)
    check(z, u, t=t, q=q)
    check(z, u, t=t, k=k, p=p, q=q)


@pytest.mark.parametrize("N", [4500, 9000, 30000, 50000])
def test_large_k(N):
    # k beyond what is listed down to the k-th, around the number of tokens with a weight, and
    # more of those than are sorted
    g = gen(N + 1)
    M = 40
    k = torch.cat([torch.arange(2044, 2054), torch.arange(4090, 4100), N - torch.arange(1, 11),
                   torch.randint(2049, N, (10,))]).int().cuda()
    u = torch.rand(M, generator=g, device="cuda")
    u[::4] = 0.99999
    p = torch.where(torch.arange(M, device="cuda") % 3 == 0, 0.97, 1.0)
    q = torch.where(torch.arange(M, device="cuda") % 5 == 0, 0.01, 0.0)
    for kind in ("flat", "ties", "peaked", "far"):
        z = logits(kind, M, N, g)
        check(z, u, k=k)
        check(z, u, k=k, p=p)
        check(z, u, k=k, p=p, q=q, t=p + q)
    # 4200 tokens with a weight and k above that
    z = torch.full((M, N), -1e5, device="cuda")
    z[:, :4200] = torch.randn((M, 4200), generator=g, device="cuda").mul(3).round() / 3
    check(z, u, k=torch.full((M,), 4400, device="cuda").int(), p=p)
    check(z, u, k=torch.full((M,), 4100, device="cuda").int(), p=p)


def test_frequencies():
    # u on a grid: a token's count is its share of the grid, to one point at each end
    g = gen(1)
    z = 2 * torch.randn((1, 300), generator=g, device="cuda")
    n = 20000
    u = ((torch.arange(n, device="cuda").double() + 0.5) / n).float()
    token, logp = gq.sample(z.expand(n, 300).contiguous(), u)
    share = torch.bincount(token, minlength=300).double() / n
    ref = torch.softmax(z[0].double(), 0)
    assert bool(((share - ref).abs() <= 1.0 / n + 1e-6).all())
    assert bool(((logp.double() - torch.log(ref[token])).abs() <= 1e-5).all())


@pytest.mark.parametrize("N", [300, 5000, 40000, 151936])
def test_nearly_certain(N):
    # the logarithm of a share near one is as exact as the others' sum: to a rounding, and
    # to what a sum with 1 in 64 bits leaves; the settings keep all, or lists
    g = gen(N)
    gap = torch.linspace(0, 60, 41, device="cuda")
    z = torch.randn((41, N), generator=g, device="cuda")
    z[:, N // 3] = z.amax(1) + gap
    u = torch.full((41,), 0.3, device="cuda")
    k, q = torch.full((41,), 40, device="cuda").int(), torch.full((41,), 1e-9, device="cuda")
    for kw in (dict(), dict(k=k), dict(q=q), dict(t=torch.full((41,), 0.7, device="cuda"))):
        token, logp = check(z, u, **kw)
        rt, rl = reference(z, u, **kw)
        # (a list leaves out weights below 2^-(62 - 18))
        slack = 2.0 ** -52 * 8 + (40 * 2.0 ** -44 if "k" in kw else 0)
        assert bool(((logp.double() - rl).abs() <= U * (1 + 1e-6) * rl.abs() + slack).all()), kw.keys()


def test_settings_at_their_ends():
    g = gen(4)
    N = 3001
    nan, inf = math.nan, math.inf
    one = dict(t=1.0, k=0, p=1.0, q=0.0, u=0.3)
    rows = [dict(), dict(u=0.0), dict(u=1.0), dict(u=5.0), dict(u=-1.0), dict(u=nan), dict(u=1 - 2.0 ** -24),
            dict(p=0.0), dict(p=-1.0), dict(p=nan), dict(p=2.0), dict(p=1e-30), dict(p=1 - 2.0 ** -24, u=0.99),
            dict(k=-5), dict(k=N), dict(k=N + 1), dict(k=1), dict(k=2 ** 31 - 1), dict(k=N - 1, u=0.999),
            dict(q=1.0), dict(q=7.0), dict(q=nan), dict(q=-1.0), dict(q=1e-40), dict(q=1e-38, u=0.999),
            dict(t=0.0), dict(t=-1.0), dict(t=1e-40), dict(t=1e-6), dict(t=1e6), dict(t=3e38), dict(t=inf),
            dict(t=nan), dict(t=-inf), dict(t=0.0, u=nan, p=nan, q=nan, k=3)]
    rows = [dict(one, **r) for r in rows]
    col = lambda n, d: torch.tensor([r[n] for r in rows], dtype=d, device="cuda")  # noqa: E731
    f = torch.float32
    for kind in ("peaked", "ties"):
        z = logits(kind, len(rows), N, g)
        check(z, col("u", f), col("t", f), col("k", torch.int32), col("p", f), col("q", f))


@pytest.mark.parametrize("N", [3000, 50000])
@pytest.mark.parametrize("t,scale", [(1e-9, 5.0), (1e-7, 5.0), (1e37, 1e38), (1e38, 1e38), (3e38, 1.5e38)])
def test_temperatures_next_to_the_logits_ends(N, t, scale):
    # differences past f32, and a range of weights below a step of the largest logit
    g = gen(N)
    rows = [(k, p, q) for k in (0, 1, 3, 50, 2500) for p in (1.0, 0.7) for q in (0.0, 0.1)]
    M = len(rows)
    z = (torch.randn((M, N), generator=g, device="cuda") * scale).clamp(-3.4e38, 3.4e38)
    z[1::2] = torch.where(z[1::2] > 2 * scale, 2 * scale, z[1::2])  # equal ones at the top
    z[::3, ::7] = -math.inf
    u = torch.rand(M, generator=g, device="cuda")
    k, p, q = (torch.tensor(c, device="cuda") for c in zip(*rows))
    check(z, u, torch.full((M,), t, device="cuda"), k.int(), p, q)


def test_rows_that_cannot_be_drawn_from():
    g = gen(6)
    z = torch.randn((9, 5000), generator=g, device="cuda")
    z[1, 4999] = math.nan
    z[2, 0] = math.inf
    z[3] = -math.inf
    z[4] = -math.inf
    z[4, 4321] = -3.0             # one token is left
    z[5, 17] = 3.4e38
    z[5, 18] = -3.4e38
    z[6] = math.nan
    z[7, :] = math.inf
    for t in (None, torch.zeros(9, device="cuda"), torch.full((9,), 1e30, device="cuda")):
        token, logp = check(z, torch.full((9,), 0.4, device="cuda"), t)
        assert int(token[4]) == 4321 and float(logp[4]) == 0.0
        assert token[[1, 2, 3, 6, 7]].tolist() == [-1] * 5


@pytest.mark.parametrize("M,N", [(1023, 700), (1024, 40000), (1025, 40000), (2500, 34000), (32769, 40)])
def test_more_rows_than_a_set_of_launches(M, N):
    g = gen(M)
    z = logits("peaked", M, N, g)
    u = torch.rand(M, generator=g, device="cuda")
    token = torch.full((M + 2,), 77, device="cuda")
    logp = torch.full((M + 2,), 77.0, device="cuda")
    t, k, p, q = settings(M, g)
    check(z, u, t, k, p, q)
    gq.sample(z, u, t, k, p, q, out=token[1:M + 1], logprob=logp[1:M + 1])
    assert torch.equal(token[1:M + 1], reference(z, u, t, k, p, q)[0])
    assert token[[0, M + 1]].tolist() == [77, 77] and logp[[0, M + 1]].tolist() == [77, 77]


def test_the_longest_row():
    g = gen(9)
    N = gq.I8_MAX_ROWS
    z = logits("peaked", 2, N, g).bfloat16()
    u = torch.rand(2, generator=g, device="cuda")
    p = torch.tensor([0.9, 0.5], device="cuda")
    check(z, u)
    check(z, u, p=p)
    check(z, u, k=torch.tensor([50, 1000000], device="cuda").int(), p=p)


def test_rows_past_32_bits():
    g = gen(3)
    pitch, N = 1400000000, 3000
    big = torch.empty(3 * pitch + N, dtype=torch.bfloat16, device="cuda")
    z = big.as_strided((4, N), (pitch, 1))
    z.copy_(logits("peaked", 4, N, g))
    u = torch.rand(4, generator=g, device="cuda")
    token, _ = gq.sample(z, u)
    assert torch.equal(token, reference(z.contiguous(), u)[0])


def test_without_logprob_and_a_used_workspace():
    # whatever the workspace holds, the results are the same
    g = gen(8)
    M, N = 5, 40000
    z, u = logits("ties", M, N, g), torch.rand(M, generator=g, device="cuda")
    ref = check(z, u)[0]
    L = gq.lib_i8()
    ws = torch.randint(0, 255, (gq.sample_workspace(M, N),), generator=g, device="cuda").to(torch.uint8)
    token = torch.empty(M, dtype=torch.int64, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    for _ in range(3):
        assert L.gemmq_sample(gq.F32, z.data_ptr(), N, None, None, None, None, u.data_ptr(),
                              token.data_ptr(), None, M, N, ws.data_ptr(), ws.numel(), st) == 0
        assert torch.equal(token, ref)
