"""The int8 linear layer and the loss over a vocabulary that reads the same
weights, as measured work.

Weights are int8 with one f32 scale per output channel, activations int8 with
one f32 scale per token (w = sw[n] * wq[n, k], x = sx[m] * xq[m, k]).  Four
operators:

  linear       x -> quantized per token -> y = x w^T (+ bias)
  linear_grad  dy -> dx = dy w, the gradient with respect to the activations
  loss         the negative log-likelihood of each token's target over the
               vocabulary, and the log-sum-exp of its logits
  loss_grad    the gradient of the weighted sum of those losses with respect to
               the hidden states

`own` chooses between the plain torch form and the package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
IGNORE = -100


def listed():
    return [
        # one token through an attention output projection: latency
        {"name": "linear M1 4096x4096", "op": "linear", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16", "bias": False, "strided": False},
        # one token through a language-model head: a stream of 311 MB of weights, f32 logits
        {"name": "linear M1 head", "op": "linear", "M": 1, "N": 151936, "K": 2048, "dtype": "f32", "bias": False, "strided": False},
        # a decode batch through a gate projection
        {"name": "linear M16 12288x4096", "op": "linear", "M": 16, "N": 12288, "K": 4096, "dtype": "bf16", "bias": False, "strided": False},
        # odd sizes, rows of a wider buffer, a bias
        {"name": "linear ragged", "op": "linear", "M": 333, "N": 4099, "K": 2050, "dtype": "f16", "bias": True, "strided": True},
        # a prompt of 512 tokens through a gate projection
        {"name": "linear M512 12288x4096", "op": "linear", "M": 512, "N": 12288, "K": 4096, "dtype": "bf16", "bias": False, "strided": False},
        # 2048 tokens through a down projection
        {"name": "linear M2048 4096x12288", "op": "linear", "M": 2048, "N": 4096, "K": 12288, "dtype": "bf16", "bias": False, "strided": False},
        # the backward of a gate projection over a training batch
        {"name": "linear_grad M2048", "op": "linear_grad", "M": 2048, "N": 12288, "K": 4096, "dtype": "bf16", "strided": False},
        # a small backward in f32 at odd sizes, the gradient a slice of a wider buffer
        {"name": "linear_grad ragged f32", "op": "linear_grad", "M": 77, "N": 1037, "K": 515, "dtype": "f32", "strided": True},
        # scoring the next token of a decode batch
        {"name": "loss M8 head", "op": "loss", "M": 8, "N": 151936, "K": 2048, "ignored": 0.0},
        # the loss of a training or evaluation batch, some positions ignored
        {"name": "loss M2048 head", "op": "loss", "M": 2048, "N": 151936, "K": 2048, "ignored": 0.15},
        # its gradient with respect to the hidden states
        {"name": "loss_grad M1024 head", "op": "loss_grad", "M": 1024, "N": 151936, "K": 2048, "dtype": "bf16", "ignored": 0.15},
        # a short sequence over a small vocabulary at odd sizes, in f32
        {"name": "loss_grad ragged f32", "op": "loss_grad", "M": 37, "N": 32003, "K": 1000, "dtype": "f32", "ignored": 0.3},
    ]


def _spread(rng, low, high):
    """A size of [low, high], spread over its logarithm; half of them as drawn
    (odd ones among them), half rounded down to a multiple of 64 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and v >= 2 * max(low, 64):
        v -= v % 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "loss", "loss_grad"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op in ("linear", "linear_grad"):
        c = {"op": op, "M": _spread(rng, 1, 2048), "N": _spread(rng, 256, 12288), "K": _spread(rng, 256, 12288), "dtype": dtype}
        while c["M"] * c["N"] * c["K"] > 2048 * 4096 * 12288:
            c["M"] = max(1, c["M"] // 2)
        if op == "linear":
            c["bias"] = rng.random() < 0.3
        c["strided"] = rng.random() < 0.3
        return c
    c = {"op": op, "M": _spread(rng, 1, 2048 if op == "loss" else 1024), "N": _spread(rng, 1000, 151936), "K": _spread(rng, 256, 4096)}
    while c["M"] * c["N"] * c["K"] > (2048 if op == "loss" else 1024) * 151936 * 2048:
        c["M"] = max(1, c["M"] // 2)
    if op == "loss_grad":
        c["dtype"] = rng.choice(["f32", "bf16", "bf16", "f16"])
    c["ignored"] = rng.choice([0.0, 0.15, 0.5])
    return c


def _int8_rows(rows, cols):
    """An uninitialised int8 matrix whose rows start 16 bytes apart or a multiple of it."""
    pitch = -(-cols // 16) * 16
    return torch.zeros((rows, pitch), dtype=torch.int8, device="cuda")[:, :cols]


def _quantized(x):
    """int8 rows and their scales: s = max|x| / 127 in f32, q = x / s rounded to
    the nearest integer, ties to even.  The quotients are taken in 64 bits and
    rounded to f32, which is the correctly rounded f32 quotient."""
    x = x.float()
    s = (x.abs().amax(dim=1).double() / 127.0).float()
    d = torch.where(s > 0, s, torch.ones_like(s)).double()
    q = (x.double() / d[:, None]).float().round().clamp(-127, 127)
    return torch.where(s[:, None] > 0, q, torch.zeros_like(q)), s


def _strided(rows, cols, extra, dtype):
    return torch.zeros((rows, cols + extra), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, N, K = case["M"], case["N"], case["K"]
    # trained weights: normal, with a spread of the channels' magnitudes
    wq, sw = _int8_rows(N, K), torch.empty(N, device="cuda")
    for a in range(0, N, 16384):
        b = min(N, a + 16384)
        w = torch.randn((b - a, K), generator=g, device="cuda") * (K ** -0.5)
        w *= torch.exp(0.3 * torch.randn((b - a, 1), generator=g, device="cuda"))
        q, s = _quantized(w)
        wq[a:b] = q.to(torch.int8)
        sw[a:b] = s
    state = {"op": case["op"], "w": wq, "sw": sw}
    if case["op"] in ("linear", "linear_grad"):
        dt = DTYPES[case["dtype"]]
        cols = K if case["op"] == "linear" else N
        x = torch.randn((M, cols), generator=g, device="cuda")
        if case["op"] == "linear":
            x[:, :: max(1, K // 4)] *= 20.0  # a few outlier channels, as activations have
        else:
            x *= 1e-3
        at = _strided(M, cols, 24 if case["strided"] else 0, dt)
        at.copy_(x)
        state["x"] = at
        state["out"] = torch.empty((M, N if case["op"] == "linear" else K), dtype=dt, device="cuda")
        if case["op"] == "linear":
            state["bias"] = torch.randn(N, generator=g, device="cuda") if case["bias"] else None
            state["xq"], state["sx"] = _int8_rows(M, K), torch.empty(M, device="cuda")
        return state
    # hidden states that point to their token's row more or less clearly, so that
    # the targets' probabilities run from near zero to near one
    target = torch.randint(0, N, (M,), generator=g, device="cuda")
    toward = wq[target].float() * sw[target][:, None]
    toward = toward / toward.norm(dim=1, keepdim=True)
    x = 2.0 * torch.randn((M, K), generator=g, device="cuda")
    x += torch.rand((M, 1), generator=g, device="cuda") * 24.0 * toward
    q, sx = _quantized(x)
    xq = _int8_rows(M, K)
    xq.copy_(q.to(torch.int8))
    target[torch.rand(M, generator=g, device="cuda") < case["ignored"]] = IGNORE
    state.update(xq=xq, sx=sx, target=target)
    if case["op"] == "loss":
        state.update(loss=torch.empty(M, device="cuda"), lse=torch.empty(M, device="cuda"))
    else:
        parts = [torch.logsumexp((xq.float() @ wq[a:a + 16384].float().t()).double() * sw[a:a + 16384] * sx[:, None], 1) for a in range(0, N, 16384)]
        state["lse"] = torch.logsumexp(torch.stack(parts), 0).float()
        # the mean over the positions that count, with weights of their own
        state["dloss"] = (0.5 + torch.rand(M, generator=g, device="cuda")) / (target >= 0).sum().clamp(min=1)
        if case["dtype"] == "f16":  # the loss scale that training in f16 uses
            state["dloss"] *= 1024.0
        state["out"] = torch.empty((M, K), dtype=DTYPES[case["dtype"]], device="cuda")
    return state


def run(s):
    if own:
        return _run_own(s)
    return {"linear": _linear, "linear_grad": _linear_grad, "loss": _loss, "loss_grad": _loss_grad}[s["op"]](s)


def _run_own(s):
    import quant_packed_weight_amd as gq

    if s["op"] == "linear":
        return gq.linear_i8(s["w"], s["sw"], s["x"], bias=s["bias"], out=s["out"], xq=s["xq"], sx=s["sx"])
    if s["op"] == "linear_grad":
        return gq.linear_i8_grad(s["w"], s["sw"], s["x"], out=s["out"])
    if s["op"] == "loss":
        return gq.loss_i8(s["w"], s["sw"], s["xq"], s["sx"], s["target"], loss=s["loss"], lse=s["lse"])
    return gq.loss_i8_grad(s["w"], s["sw"], s["xq"], s["sx"], s["target"], s["lse"], s["dloss"], out=s["out"])


def _linear(s):
    q, sx = _quantized(s["x"])
    y = (q @ s["w"].float().t()) * sx[:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["x"].dtype)


def _linear_grad(s):
    return ((s["x"].float() * s["sw"]) @ s["w"].float()).to(s["x"].dtype)


def _logits(s):
    return (s["xq"].float() @ s["w"].float().t()) * s["sx"][:, None] * s["sw"]


def _loss(s):
    z, t = _logits(s), s["target"]
    top = z.amax(dim=1)
    lse = top + torch.exp(z - top[:, None]).sum(dim=1).log()
    hit = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    return torch.where(t >= 0, lse - hit, torch.zeros_like(lse)), lse


def _loss_grad(s):
    t = s["target"]
    p = torch.exp(_logits(s) - s["lse"][:, None])
    at = t.clamp(min=0)[:, None]
    p.scatter_(1, at, p.gather(1, at) - 1.0)
    d = (p * s["sw"]) @ s["w"].float()
    d = d * torch.where(t >= 0, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    return d.to(s["out"].dtype)


def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    e = SIZES[case.get("dtype", "f32")]
    if case["op"] == "linear":
        return {"bytes": N * K + 4 * N + M * K * e + M * N * e + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    if case["op"] == "linear_grad":
        return {"bytes": N * K + 4 * N + M * N * e + M * K * e, "flops": 2 * M * N * K}
    if case["op"] == "loss":
        return {"bytes": N * K + 4 * N + M * K + 4 * M + 8 * M + 8 * M, "flops": 2 * M * N * K}
    # the logits once more from the hidden states, then the product with the weights
    return {"bytes": N * K + 4 * N + M * K + M * K * e + 20 * M, "flops": 4 * M * N * K}


def exact(case, seed):
    """The definitions in 64 bits, the vocabulary or channels in pieces."""
    s = prepare(case, seed)
    w, sw = s["w"], s["sw"].double()
    N = case["N"]
    cut = [(a, min(N, a + 8192)) for a in range(0, N, 8192)]
    if case["op"] == "linear":
        x = s["x"].double()
        scale = (x.abs().amax(dim=1) / 127.0).float().double()
        live = (scale > 0)[:, None]
        q = torch.where(live, torch.round((x / torch.where(live, scale[:, None], 1.0)).float().double()), 0.0).clamp(-127, 127)
        y = torch.cat([(q * scale[:, None]) @ (w[a:b].double() * sw[a:b, None]).t() for a, b in cut], 1)
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "linear_grad":
        return sum(s["x"][:, a:b].double() @ (w[a:b].double() * sw[a:b, None]) for a, b in cut)
    x, t = s["xq"].double() * s["sx"].double()[:, None], s["target"]
    rows = torch.arange(case["M"], device=t.device)
    if case["op"] == "loss":
        lse = torch.full((case["M"],), -math.inf, dtype=torch.float64, device=t.device)
        for a, b in cut:
            lse = torch.logaddexp(lse, torch.logsumexp(x @ (w[a:b].double() * sw[a:b, None]).t(), 1))
        keep = t >= 0
        hit = (x * w[t.clamp(min=0)].double()).sum(1) * sw[t.clamp(min=0)]
        return torch.where(keep, lse - hit, 0.0), lse
    d = torch.zeros_like(x)
    for a, b in cut:
        wd = w[a:b].double() * sw[a:b, None]
        p = torch.exp(x @ wd.t() - s["lse"].double()[:, None])
        here = (t >= a) & (t < b)
        p[rows[here], t[here] - a] -= 1.0
        d += p @ wd
    return d * torch.where(t >= 0, s["dloss"].double(), 0.0)[:, None]
