"""The int8 calls of a decoder's block together on the GPU, as a user runs them: a decode step
down to its token, a training step and back, captured into a graph, on other streams, inside
a Function of autograd; and what is refused."""
import math

import pytest
import torch

import quant_packed_weight_amd as gq
from block_util import HALF, IDS, TYPES, U, gen, i8, normal, scales, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device():
    import gpu_util

    gpu_util.device()


class Model:
    """A feed-forward block, a last norm and a head: int8 weights, f32 norms."""

    def __init__(self, D, F, V, g):
        q = lambda n, k: gq.quantize_i8(torch.randn((n, k), generator=g, device="cuda") * k ** -0.5)  # noqa: E731
        self.w1, self.w2 = (1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2))
        self.gate, self.up, self.down, self.head = q(F, D), q(F, D), q(D, F), q(V, D)


def decode(m, x, r, u, t, k, p, out=None, **kw):
    """One step: x, r -> tokens; what it keeps in `out` goes there."""
    o = out or {}
    q, s, h = gq.rms_i8(x, m.w1, residual=r, hidden=o.get("h"), out=o.get("q"), scale=o.get("s"), **kw)
    y = gq.gemm_i8_gate(*m.gate, *m.up, q, s, out=o.get("y"), out_dtype=x.dtype, **kw)
    h2 = gq.linear_i8_act(*m.down, y, gq.ACT_NONE, residual=h, out=o.get("h2"), **kw)
    q2, s2, _ = gq.rms_i8(h2, m.w2, out=o.get("q2"), scale=o.get("s2"), **kw)
    z = gq.gemm_i8(*m.head, q2, s2, out=o.get("z"), **kw)
    token, logp = gq.sample(z, u, temperature=t, top_k=k, top_p=p, out=o.get("token"),
                            logprob=o.get("logp"), **kw)
    return dict(h=h, q=q, s=s, y=y, h2=h2, q2=q2, s2=s2, z=z, token=token, logp=logp)


def batch(M, D, g, dtype):
    f = lambda: torch.rand(M, generator=g, device="cuda")  # noqa: E731
    return (normal(M, D, g, dtype), normal(M, D, g, dtype, 2.0), f(), 0.5 + f(),
            (1 + 50 * f()).int(), 0.5 + 0.5 * f())


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("M", [1, 2, 9, 40, 300])
def test_decode_step(M, dtype):
    # each stage against 64 bits, from what the stage before it left
    g = gen(M)
    D, F, V = 320, 500, 3001
    m = Model(D, F, V, g)
    x, r, u, t, k, p = batch(M, D, g, dtype)
    o = decode(m, x, r, u, t, k, p)
    h = (x.float() + r.float()).to(dtype)
    assert torch.equal(o["h"], h)
    wd = lambda w: w[0].double() * w[1].double()[:, None]  # noqa: E731
    n = h.double() * (h.double().square().mean(1, keepdim=True) + 1e-6) ** -0.5 * m.w1.double()
    a = o["q"].double() * o["s"].double()[:, None]
    # half a step of the quantizer, and what rounds beside a tie
    assert bool(((a - n).abs() <= 0.5001 * o["s"].double()[:, None] + 1e-6 * n.abs()).all())
    z, up = a @ wd(m.gate).t(), a @ wd(m.up).t()
    y = z * torch.sigmoid(z) * up
    # f32 through the products, SiLU and theirs (the bounds' own tests are elsewhere)
    within(o["y"], y, HALF[dtype] * y.abs() + 2.0 ** -20 * (1 + y.abs()) * (1 + up.abs()), "gate")
    yq, ys = gq.quantize_i8(o["y"])
    h2 = (yq.double() * ys.double()[:, None]) @ wd(m.down).t() + h.double()
    within(o["h2"], h2, HALF[dtype] * h2.abs() + 2.0 ** -20 * (1 + h2.abs()), "down")
    q2, s2, _ = gq.rms_i8(o["h2"], m.w2)
    assert torch.equal(q2, o["q2"]) and torch.equal(s2, o["s2"])
    logits = (q2.double() * s2.double()[:, None]) @ wd(m.head).t()
    within(o["z"], logits, 2.0 ** -20 * (1 + logits.abs()), "logits")
    # the token is one that is kept, with its share
    for i in range(M):
        v, order = torch.sort(o["z"][i].double(), descending=True, stable=True)
        e = torch.exp((v - v[0]) / float(t[i]))[:int(k[i])]
        held = torch.cumsum(e, 0)
        e = e[:1 + int((held < float(p[i]) * held[-1]).sum())]
        at = int(torch.nonzero(order == o["token"][i])[0])
        assert at < len(e)
        assert abs(float(o["logp"][i]) - float(torch.log(e[at] / e.sum()))) <= 1e-5
        before = float(e[:at].sum() / e.sum())
        assert before - 1e-9 <= float(u[i]) <= before + float(e[at] / e.sum()) + 1e-9


def buffers(M, D, F, V, dtype):
    e = dict(device="cuda")
    i = lambda n: torch.empty((M, -(-n // 16) * 16), dtype=torch.int8, **e)[:, :n]  # noqa: E731
    f = lambda n: torch.empty((M, n), dtype=dtype, **e)  # noqa: E731
    return dict(h=f(D), q=i(D), s=torch.empty(M, **e), y=f(F), h2=f(D), q2=i(D),
                s2=torch.empty(M, **e), z=torch.empty((M, V), **e),
                token=torch.empty(M, dtype=torch.int64, **e), logp=torch.empty(M, **e))


@pytest.mark.parametrize("M", [1, 16, 100])
def test_decode_captured_and_replayed(M):
    g = gen(M + 50)
    D, F, V = 320, 500, 9001
    m = Model(D, F, V, g)
    live = batch(M, D, g, torch.bfloat16)
    eager, held = buffers(M, D, F, V, torch.bfloat16), buffers(M, D, F, V, torch.bfloat16)
    decode(m, *live, out=eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode(m, *live, out=held)
    for n in range(4):
        for a, b in zip(live, batch(M, D, g, torch.bfloat16)):
            a.copy_(b)
        if n == 2:
            live[3][0] = 0.0   # greedy from now on
        decode(m, *live, out=eager)
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(eager[name], held[name]), (n, name)


def train(m, x, r, target, dtype, **kw):
    """Forward to the loss, and back to x and the norms' weights."""
    M = x.shape[0]
    F = m.gate[0].shape[0]
    q, s, h = gq.rms_i8(x, m.w1, residual=r, **kw)
    z, up = (torch.empty((M, F), dtype=dtype, device="cuda") for _ in range(2))
    y = gq.gemm_i8_gate(*m.gate, *m.up, q, s, pre=z, up=up, out_dtype=dtype, **kw)
    yq, ys = gq.quantize_i8(y, **kw)
    h2 = gq.gemm_i8_act(*m.down, yq, ys, gq.ACT_NONE, residual=h, out_dtype=dtype, **kw)
    q2, s2, _ = gq.rms_i8(h2, m.w2, **kw)
    loss, lse = gq.loss_i8(*m.head, q2, s2, target, **kw)
    one = torch.full((M,), 1.0 / M, device="cuda")
    dn = gq.loss_i8_grad(*m.head, q2, s2, target, lse, one, out_dtype=dtype, **kw)
    dh2, dw2 = gq.rms_i8_grad(h2, m.w2, dn, **kw)
    dy = gq.linear_i8_grad(*m.down, dh2, **kw)
    dz, du = gq.act_grad(gq.ACT_SILU, z, dy, up=up, **kw)
    da = gq.linear_i8_grad(*m.gate, dz, **kw) + gq.linear_i8_grad(*m.up, du, **kw)
    dx, dw1 = gq.rms_i8_grad(h, m.w1, da, dh=dh2, **kw)
    return dict(loss=loss, dx=dx, dw1=dw1, dw2=dw2, q=q, s=s, h=h, yq=yq, ys=ys, h2=h2, q2=q2, s2=s2)


def reference(m, x, r, target, o):
    """The same in 64 bits through autograd, the quantizers' results taken from `o` and their
    rounding passed through as the identity."""
    wd = lambda w: w[0].double() * w[1].double()[:, None]  # noqa: E731
    fixed = lambda v, q, s: v + (q.double() * s.double()[:, None] - v).detach()  # noqa: E731
    x = x.double().requires_grad_()
    w1, w2 = m.w1.double().requires_grad_(), m.w2.double().requires_grad_()
    norm = lambda h, w: h * (h.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * w  # noqa: E731
    h = x + r.double()
    h = h + (o["h"].double() - h).detach()
    a = fixed(norm(h, w1), o["q"], o["s"])
    z, up = a @ wd(m.gate).t(), a @ wd(m.up).t()
    y = fixed(z * torch.sigmoid(z) * up, o["yq"], o["ys"])
    h2 = y @ wd(m.down).t() + h
    h2 = h2 + (o["h2"].double() - h2).detach()
    n = fixed(norm(h2, w2), o["q2"], o["s2"])
    loss = torch.nn.functional.cross_entropy(n @ wd(m.head).t(), target, reduction="none")
    loss.mean().backward()
    return loss.detach(), x.grad, w1.grad, w2.grad


@pytest.mark.parametrize("M", [3, 40, 200])
def test_training_step(M):
    g = gen(M + 7)
    D, F, V = 192, 320, 1009
    m = Model(D, F, V, g)
    x, r = normal(M, D, g, torch.float32), normal(M, D, g, torch.float32, 2.0)
    target = torch.randint(0, V, (M,), generator=g, device="cuda")
    o = train(m, x, r, target, torch.float32)
    ref = reference(m, x, r, target, o)
    # some ten stages in f32, each off by a few roundings of its terms, which are of both
    # signs: 2^-24 times ten stages, the square root of 1009 terms and a factor of two
    for got, want, name in zip((o["loss"], o["dx"], o["dw1"], o["dw2"]), ref, ("loss", "dx", "dw1", "dw2")):
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 640 * U, (name, off)
    # in bf16: each stage rounds to 2^-8 or less
    o = train(m, x.bfloat16(), r.bfloat16(), target, torch.bfloat16)
    ref = reference(m, x.bfloat16(), r.bfloat16(), target, o)
    for got, want, name in zip((o["dx"], o["dw1"], o["dw2"]), ref[1:], ("dx", "dw1", "dw2")):
        off = float((got.double() - want).norm() / want.norm())
        assert off <= 10 * 2.0 ** -8, (name, off)


def test_training_captured_and_replayed():
    g = gen(99)
    M, D, F, V = 24, 192, 320, 1009
    m = Model(D, F, V, g)
    x, r = normal(M, D, g, torch.float32), normal(M, D, g, torch.float32)
    target = torch.randint(0, V, (M,), generator=g, device="cuda")
    eager = train(m, x, r, target, torch.float32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = train(m, x, r, target, torch.float32)
    for _ in range(3):
        x.copy_(normal(M, D, g, torch.float32))
        eager = train(m, x, r, target, torch.float32)
        graph.replay()
        torch.cuda.synchronize()
        for name in eager:
            assert torch.equal(eager[name], held[name]), name


class Block(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w1, model):
        q, s, h = gq.rms_i8(x, w1)
        z, up = (torch.empty((x.shape[0], model.gate[0].shape[0]), device="cuda") for _ in range(2))
        y = gq.gemm_i8_gate(*model.gate, *model.up, q, s, pre=z, up=up)
        out = gq.linear_i8_act(*model.down, y, gq.ACT_NONE, residual=x)
        ctx.save_for_backward(x, w1, z, up)
        ctx.model = model
        return out

    @staticmethod
    def backward(ctx, dout):
        x, w1, z, up = ctx.saved_tensors
        m = ctx.model
        dz, du = gq.act_grad(gq.ACT_SILU, z, gq.linear_i8_grad(*m.down, dout.contiguous()), up=up)
        da = gq.linear_i8_grad(*m.gate, dz) + gq.linear_i8_grad(*m.up, du)
        dx, dw = gq.rms_i8_grad(x, w1, da, dh=dout.contiguous())
        return dx, dw, None


def test_in_a_function_of_autograd():
    g = gen(31)
    M, D, F = 17, 192, 320
    m = Model(D, F, 64, g)
    x = normal(M, D, g, torch.float32).requires_grad_()
    w1 = m.w1.clone().requires_grad_()
    (Block.apply(x, w1, m) ** 2).sum().backward()
    # by hand
    with torch.no_grad():
        q, s, _ = gq.rms_i8(x, w1)
        z, up = (torch.empty((M, F), device="cuda") for _ in range(2))
        y = gq.gemm_i8_gate(*m.gate, *m.up, q, s, pre=z, up=up)
        out = gq.linear_i8_act(*m.down, y, gq.ACT_NONE, residual=x)
        dz, du = gq.act_grad(gq.ACT_SILU, z, gq.linear_i8_grad(*m.down, 2 * out), up=up)
        da = gq.linear_i8_grad(*m.gate, dz) + gq.linear_i8_grad(*m.up, du)
        dx, dw = gq.rms_i8_grad(x, w1, da, dh=2 * out)
    assert torch.equal(x.grad, dx) and torch.equal(w1.grad, dw)


def test_other_streams():
    # the same steps on two streams at once, each with what the calls allocate
    g = gen(8)
    M, D, F, V = 64, 320, 500, 9001
    m = Model(D, F, V, g)
    live = [batch(M, D, g, torch.bfloat16) for _ in range(2)]
    target = torch.randint(0, V, (M,), generator=g, device="cuda")
    ref = [decode(m, *b) for b in live], [train(m, *b[:2], target, torch.bfloat16) for b in live]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for n in range(3):
        got = [], []
        for b, s in zip(live, streams):
            stream = s if n < 2 else s.cuda_stream
            got[0].append(decode(m, *b, stream=stream))
            with torch.cuda.stream(s):  # (the sum of two gradients is torch's)
                got[1].append(train(m, *b[:2], target, torch.bfloat16))
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            for c, d in zip(a, b):
                for name in c:
                    assert torch.equal(c[name], d[name]), name


def test_refusals_on_the_device():
    g = gen(1)
    w, sw, xq, sx = i8(40, 64, g), scales(40, g), i8(4, 64, g), scales(4, g)
    x, w1 = torch.zeros((4, 64), device="cuda"), torch.ones(64, device="cuda")
    z, u = torch.zeros((4, 40), device="cuda"), torch.zeros(4, device="cuda")
    x9, far = torch.zeros((9, 64), device="cuda"), torch.zeros((1, 50000), device="cuda")
    half = lambda t: t.half()  # noqa: E731
    bad = [
        lambda: gq.rms_i8(x, w1[:63]),                                # a weight of another width
        lambda: gq.rms_i8(x, half(w1)),
        lambda: gq.rms_i8(x, w1, residual=half(x)),                   # another type
        lambda: gq.rms_i8(x, w1, residual=x[:3]),
        lambda: gq.rms_i8(x.t(), w1[:4]),                             # columns, not rows
        lambda: gq.rms_i8(x, w1, eps=-1.0),
        lambda: gq.rms_i8(x, w1, eps=math.nan),
        lambda: gq.rms_i8(x[:1].expand(4, 64), w1),                   # rows on top of each other
        lambda: gq.rms_i8(x, w1, out=xq[:, :60]),
        lambda: gq.rms_i8(x.double(), w1),
        lambda: gq.rms_i8(x.long(), w1),
        lambda: gq.rms_i8_grad(x, w1, half(x)),
        lambda: gq.rms_i8_grad(x, w1, x, dh=x[:3]),
        lambda: gq.rms_i8_grad(x, w1, x, dw=w1[:63]),
        lambda: gq.rms_i8_grad(x9, w1, x9, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        lambda: gq.gemm_i8_act(w, sw, xq, sx, 9),                     # no such activation
        lambda: gq.gemm_i8_act(w, sw, xq, sx, gq.ACT_SILU, residual=half(z)),
        lambda: gq.gemm_i8_act(w, sw, xq, sx, gq.ACT_SILU, pre=z[:, :39]),
        lambda: gq.gemm_i8_act(w, sw, xq, sx, gq.ACT_SILU, bias=sw[:39]),
        lambda: gq.gemm_i8_act(w, sw, xq, sx, gq.ACT_SILU, out=z, out_dtype=torch.float16),
        lambda: gq.gemm_i8_gate(w, sw, w[:39], sw[:39], xq, sx),      # matrices of other heights
        lambda: gq.gemm_i8_gate(w, sw, w, sw, xq, sx, up=half(z)),
        lambda: gq.linear_i8_gate(w, sw, w, sw, x[:, :60]),
        lambda: gq.act_grad(gq.ACT_SILU, z, half(z)),
        lambda: gq.act_grad(gq.ACT_SILU, z, z, up=z[:3]),
        lambda: gq.act_grad(gq.ACT_SILU, z, z, up=z.clone(), out=z, dup=z),  # one place for both
        lambda: gq.act_grad(gq.ACT_SILU, z, z, dup=z.clone()),        # a place, but no pair
        lambda: gq.act_grad(gq.ACT_SILU, z, z, dbias_up=sw.clone()),
        lambda: gq.sample(z, u[:3]),
        lambda: gq.sample(z, u.double()),
        lambda: gq.sample(z, u, top_k=u),                             # not whole numbers
        lambda: gq.sample(z, u, temperature=torch.ones(8, device="cuda")[::2]),
        lambda: gq.sample(z[:, :0], u),                               # no vocabulary
        lambda: gq.sample(z, u, out=torch.zeros(4, dtype=torch.int32, device="cuda")),
        lambda: gq.sample(far, u[:1], workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
        lambda: gq.sample(z, u.cpu()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError, gq.GemmqError)):
            call()
            raise AssertionError("call %d was not refused" % i)
    torch.cuda.synchronize()
    # and the device is as it was
    assert gq.sample(z, u)[0].tolist() == [0, 0, 0, 0]
