"""What stands around the int8 linear layers of a decoder, as measured work.

Weights are int8 with one f32 scale per output channel, activations int8 with
one f32 scale per token (w = sw[n] * wq[n, k], x = sx[m] * xq[m, k]).  Six
operators:

  rms       h = x + r; the root-mean-square norm of h times a weight, quantized
            to int8 with a scale per token: what the next layer's product reads
  rms_grad  the norm's gradient with respect to h and to the weight
  act       x -> quantized -> y = act(x w^T + bias) + residual
  gate      x -> quantized -> y = act(x wg^T + bg) * (x wu^T + bu)
  act_grad  the gradients of act and gate with respect to what is before the
            activation, and to the biases
  sample    logits -> one token a row: temperature, top-k, top-p, min-p, and a
            given random number

`own` chooses between the plain torch form and the package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def listed():
    return [
        # one token into an attention or gate projection: latency
        {"name": "rms M1 4096", "op": "rms", "M": 1, "K": 4096, "dtype": "bf16", "residual": True, "strided": False},
        # a prompt or a training batch of 2048 tokens
        {"name": "rms M2048 4096", "op": "rms", "M": 2048, "K": 4096, "dtype": "bf16", "residual": True, "strided": False},
        # the backward of that norm, the residual path's gradient added to it
        {"name": "rms_grad M2048 4096", "op": "rms_grad", "M": 2048, "K": 4096, "dtype": "bf16", "residual": True, "strided": False},
        # a short sequence at odd sizes, in f32, rows of a wider buffer
        {"name": "rms_grad ragged f32", "op": "rms_grad", "M": 77, "K": 1037, "dtype": "f32", "residual": False, "strided": True},
        # one token through a gate and an up projection
        {"name": "gate M1 12288x4096", "op": "gate", "M": 1, "N": 12288, "K": 4096, "dtype": "bf16", "act": "silu", "bias": False, "pre": False, "strided": False},
        # 2048 tokens through them in training, which keeps both projections for the backward
        {"name": "gate M2048 12288x4096", "op": "gate", "M": 2048, "N": 12288, "K": 4096, "dtype": "bf16", "act": "silu", "bias": False, "pre": True, "strided": False},
        # a decode batch through a down projection, onto the residual stream
        {"name": "act M16 4096x12288", "op": "act", "M": 16, "N": 4096, "K": 12288, "dtype": "bf16", "act": "none", "bias": False, "residual": True, "pre": False, "strided": False},
        # odd sizes, rows of wider buffers, everything that the epilogue has
        {"name": "act ragged", "op": "act", "M": 333, "N": 4099, "K": 2050, "dtype": "f16", "act": "gelu_tanh", "bias": True, "residual": True, "pre": True, "strided": True},
        # the backward of a gated pair over a training batch
        {"name": "act_grad M2048 12288", "op": "act_grad", "M": 2048, "N": 12288, "dtype": "bf16", "act": "silu", "gated": True, "bias": False, "strided": False},
        # a short sequence at odd sizes, in f32, with the bias's gradient
        {"name": "act_grad ragged f32", "op": "act_grad", "M": 77, "N": 1037, "dtype": "f32", "act": "gelu", "gated": False, "bias": True, "strided": True},
        # the next token of one sequence, from a language-model head's f32 logits
        {"name": "sample M1 151936", "op": "sample", "M": 1, "N": 151936, "dtype": "f32", "filters": "chat", "strided": False},
        # a decode batch whose requests have settings of their own, some greedy, some unfiltered, some with masked tokens
        {"name": "sample M128 151936", "op": "sample", "M": 128, "N": 151936, "dtype": "bf16", "filters": "mixed", "strided": False},
    ]


def _spread(rng, low, high):
    """A size of [low, high], spread over its logarithm; half of them as drawn
    (odd ones among them), half rounded down to a multiple of 64 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and v >= 2 * max(low, 64):
        v -= v % 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["rms", "rms_grad", "act", "gate", "act_grad", "sample"])
    c = {"op": op, "M": _spread(rng, 1, 128 if op == "sample" else 2048)}
    if op in ("rms", "rms_grad"):
        c["K"] = _spread(rng, 256, 12288)
        while c["M"] * c["K"] > 2048 * 4096:
            c["M"] = max(1, c["M"] // 2)
        c["residual"] = rng.random() < 0.7
    elif op in ("act", "gate"):
        c["N"], c["K"] = _spread(rng, 256, 12288), _spread(rng, 256, 12288)
        while c["M"] * c["N"] * c["K"] > 2048 * 4096 * (24576 if op == "act" else 12288):
            c["M"] = max(1, c["M"] // 2)
        c["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu", "none"])
        c["bias"] = rng.random() < 0.3
        if op == "act":
            c["residual"] = rng.random() < 0.5
        c["pre"] = rng.random() < 0.4
    elif op == "act_grad":
        c["N"] = _spread(rng, 256, 12288)
        c["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu", "none"])
        c["gated"] = rng.random() < 0.6
        c["bias"] = rng.random() < 0.4
    else:
        c["N"] = _spread(rng, 1000, 151936)
        c["filters"] = rng.choice(["chat", "mixed", "mixed", "none"])
    c["dtype"] = rng.choice(["f32", "bf16", "bf16", "f16"])
    c["strided"] = rng.random() < 0.3
    return c


def _int8_rows(rows, cols):
    """An int8 matrix whose rows start 16 bytes apart or a multiple of it."""
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


def _rows(rows, cols, strided, dtype):
    return torch.zeros((rows, cols + (24 if strided else 0)), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    M, dt, strided = case["M"], DTYPES[case["dtype"]], case["strided"]
    s = {"op": case["op"], "M": M}

    def normal(rows, cols, scale=1.0, outliers=False):
        v = torch.randn((rows, cols), generator=g, device="cuda") * scale
        if outliers:
            v[:, :: max(1, cols // 4)] *= 20.0  # a few outlier channels, as activations have
        at = _rows(rows, cols, strided, dt)
        at.copy_(v)
        return at

    def out(rows, cols):
        return torch.empty((rows, cols), dtype=dt, device="cuda")

    if case["op"] == "rms":
        K = case["K"]
        s["x"] = normal(M, K, 0.7, True)
        s["w"] = 1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")
        s["r"] = normal(M, K, 2.0, True) if case["residual"] else None
        s["h"] = out(M, K) if case["residual"] else None
        s["q"], s["sx"] = _int8_rows(M, K), torch.empty(M, device="cuda")
        s["y"] = torch.empty((M, K), device="cuda")
        return s
    if case["op"] == "rms_grad":
        K = case["K"]
        s["h"] = normal(M, K, 2.0, True)
        s["w"] = 1.0 + 0.2 * torch.randn(K, generator=g, device="cuda")
        s["dy"] = normal(M, K, 1e-3)
        s["dh"] = normal(M, K, 1e-3) if case["residual"] else None
        s["dx"], s["dw"] = out(M, K), torch.empty(K, device="cuda")
        return s
    N = case["N"]
    if case["op"] in ("act", "gate"):
        K = case["K"]
        s["act"] = case["act"]
        for name in ("", "u") if case["op"] == "gate" else ("",):
            # trained weights: normal, with a spread of the channels' magnitudes
            w = torch.randn((N, K), generator=g, device="cuda") * (K ** -0.5)
            w *= torch.exp(0.3 * torch.randn((N, 1), generator=g, device="cuda"))
            q, s["sw" + name] = _quantized(w)
            s["w" + name] = _int8_rows(N, K)
            s["w" + name].copy_(q.to(torch.int8))
            s["b" + name] = 0.5 * torch.randn(N, generator=g, device="cuda") if case["bias"] else None
            s["z" + name] = out(M, N) if case["pre"] else None
        s["x"] = normal(M, K, 1.0, True)
        s["xq"], s["sx"] = _int8_rows(M, K), torch.empty(M, device="cuda")
        s["r"] = normal(M, N, 2.0) if case.get("residual") else None
        s["out"] = out(M, N)
        return s
    if case["op"] == "act_grad":
        s["act"], s["bias"] = case["act"], case["bias"]
        s["z"], s["dy"] = normal(M, N, 1.5), normal(M, N, 1e-3)
        s["u"] = normal(M, N, 1.0) if case["gated"] else None
        s["dz"], s["du"] = out(M, N), out(M, N) if case["gated"] else None
        s["db"] = torch.empty(N, device="cuda") if case["bias"] else None
        s["dbu"] = torch.empty(N, device="cuda") if case["bias"] and case["gated"] else None
        return s
    # logits: a body that most of the vocabulary is in, and a few likely tokens a row
    z = 2.5 * torch.randn((M, N), generator=g, device="cuda")
    at = torch.randint(0, N, (M, 40), generator=g, device="cuda")
    z.scatter_(1, at, 8.0 + 4.0 * torch.randn((M, 40), generator=g, device="cuda"))
    u = lambda: torch.rand(M, generator=g, device="cuda")  # noqa: E731
    s["u"] = u()
    s["t"] = s["k"] = s["p"] = s["mp"] = None
    if case["filters"] == "chat":
        s["t"] = 0.6 + 0.4 * u()
        s["k"] = (20 + 30 * u()).to(torch.int32)
        s["p"] = 0.9 + 0.08 * u()
    elif case["filters"] == "mixed":
        s["t"] = torch.where(u() < 0.1, torch.zeros_like(s["u"]), 0.5 + u())
        s["k"] = torch.where(u() < 0.5, torch.zeros_like(s["u"]), 1 + 200 * u() ** 2).to(torch.int32)
        s["p"] = torch.where(u() < 0.4, torch.ones_like(s["u"]), 0.7 + 0.299 * u())
        s["mp"] = torch.where(u() < 0.6, torch.zeros_like(s["u"]), 0.2 * u() ** 2)
        # a grammar leaves a part of the vocabulary in some rows
        left = torch.where(u() < 0.2, 0.01 + 0.5 * u(), torch.ones_like(s["u"]))
        off = torch.rand((M, N), generator=g, device="cuda") > left[:, None]
        off[:, 0] = False
        z[off] = -math.inf
    s["z"] = _rows(M, N, strided, dt)
    s["z"].copy_(z)
    s["token"] = torch.empty(M, dtype=torch.int64, device="cuda")
    s["logprob"] = torch.empty(M, device="cuda")
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"rms": _rms, "rms_grad": _rms_grad, "act": _act, "gate": _gate, "act_grad": _act_grad, "sample": _sample}[s["op"]](s)


def _run_own(s):
    import quant_packed_weight_amd as gq

    op = s["op"]
    if op == "rms":
        q, sx, h = gq.rms_i8(s["x"], s["w"], eps=EPS, residual=s["r"], hidden=s["h"], out=s["q"], scale=s["sx"])
        return {"h": h, "y": torch.mul(q, sx[:, None], out=s["y"]), "s": sx}
    if op == "rms_grad":
        dx, dw = gq.rms_i8_grad(s["h"], s["w"], s["dy"], dh=s["dh"], eps=EPS, out=s["dx"], dw=s["dw"])
        return {"dx": dx, "dw": dw}
    if op == "sample":
        return gq.sample(s["z"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["mp"], out=s["token"], logprob=s["logprob"])
    act = {"none": gq.ACT_NONE, "silu": gq.ACT_SILU, "gelu": gq.ACT_GELU, "gelu_tanh": gq.ACT_GELU_TANH, "relu": gq.ACT_RELU}[s["act"]]
    if op == "act":
        y = gq.linear_i8_act(s["w"], s["sw"], s["x"], act, bias=s["b"], residual=s["r"], pre=s["z"], out=s["out"], xq=s["xq"], sx=s["sx"])
        return {"y": y, "z": s["z"]}
    if op == "gate":
        y = gq.linear_i8_gate(s["w"], s["sw"], s["wu"], s["swu"], s["x"], act, bias=s["b"], bias_up=s["bu"], pre=s["z"], up=s["zu"], out=s["out"], xq=s["xq"], sx=s["sx"])
        return {"y": y, "z": s["z"], "u": s["zu"]}
    dz, du = gq.act_grad(act, s["z"], s["dy"], up=s["u"], out=s["dz"], dup=s["du"], dbias=s["db"], dbias_up=s["dbu"])
    return {"dz": dz, "du": du, "db": s["db"], "dbu": s["dbu"]}


def _rms(s):
    h = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["x"].dtype)
    v = h.float()
    rstd = 1.0 / torch.sqrt(v.square().mean(dim=1) + EPS)
    # the norm is one factor a row: it leaves the integers alone and enters the scale
    q, scale = _quantized(v * s["w"])
    scale = scale * rstd
    return {"h": h, "y": q * scale[:, None], "s": scale}


def _rms_grad(s):
    h, dy = s["h"].float(), s["dy"].float()
    rstd = 1.0 / torch.sqrt(h.square().mean(dim=1, keepdim=True) + EPS)
    n = h * rstd
    d = dy * s["w"]
    dx = rstd * (d - n * (d * n).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dw": (dy * n).sum(dim=0)}


_C = math.sqrt(2.0 / math.pi)


def _activation(act, z):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_C * (z + 0.044715 * z ** 3)))
    return torch.where(z > 0, z, torch.zeros_like(z)) if act == "relu" else z


def _slope(act, z):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * _C * (1.0 + 3.0 * 0.044715 * z * z)
    return (z > 0).float() if act == "relu" else torch.ones_like(z)


def _product(q, sx, w, sw, bias):
    z = (q @ w.float().t()) * sx[:, None] * sw
    return z if bias is None else z + bias


def _act(s):
    dt = s["x"].dtype
    q, sx = _quantized(s["x"])
    z = _product(q, sx, s["w"], s["sw"], s["b"])
    y = _activation(s["act"], z)
    if s["r"] is not None:
        y = y + s["r"].float()
    return {"y": y.to(dt), "z": None if s["z"] is None else z.to(dt)}


def _gate(s):
    dt = s["x"].dtype
    q, sx = _quantized(s["x"])
    z, u = _product(q, sx, s["w"], s["sw"], s["b"]), _product(q, sx, s["wu"], s["swu"], s["bu"])
    kept = s["z"] is not None
    return {"y": (_activation(s["act"], z) * u).to(dt), "z": z.to(dt) if kept else None, "u": u.to(dt) if kept else None}


def _act_grad(s):
    z, dy, dt = s["z"].float(), s["dy"].float(), s["z"].dtype
    slope = _slope(s["act"], z)
    if s["u"] is None:
        dz, du = dy * slope, None
    else:
        dz, du = dy * s["u"].float() * slope, dy * _activation(s["act"], z)
    return {"dz": dz.to(dt), "du": None if du is None else du.to(dt), "db": dz.sum(dim=0) if s["bias"] else None,
            "dbu": du.sum(dim=0) if s["bias"] and du is not None else None}


def _sample(s):
    # in 64 bits: a random number may lie next to the border between two tokens
    z, M, N = s["z"].double(), s["M"], s["z"].shape[1]
    one = torch.ones(M, dtype=torch.float64, device=z.device)
    t = one if s["t"] is None else s["t"].double()
    greedy = (t <= 0)[:, None]
    z, order = torch.sort(z, dim=1, descending=True, stable=True)
    e = torch.exp((z - z[:, :1]) / torch.where(t > 0, t, one)[:, None])
    place = torch.arange(N, device=z.device)[None, :]
    keep = (place < 1) | ~greedy
    if s["k"] is not None:
        keep &= (place < s["k"][:, None]) | (s["k"][:, None] <= 0)
    e = torch.where(keep, e, torch.zeros_like(e))
    if s["p"] is not None:
        # the fewest tokens that hold the share p: those before which less is held
        total = torch.cumsum(e, dim=1)
        p = s["p"].double()[:, None]
        keep &= (total - e < p * total[:, -1:]) | (p >= 1) | (place < 1)
    if s["mp"] is not None:
        keep &= e >= s["mp"].double()[:, None]
    e = torch.where(keep, e, torch.zeros_like(e))
    total = torch.cumsum(e, dim=1)
    at = (total <= s["u"].double()[:, None] * total[:, -1:]).sum(dim=1, keepdim=True).clamp(max=N - 1)
    token = order.gather(1, at)[:, 0]
    return token, torch.log(e.gather(1, at) / total[:, -1:])[:, 0].float()


def work(case):
    M, e = case["M"], SIZES[case["dtype"]]
    N, K, op = case.get("N", 0), case.get("K", 0), case["op"]
    if op == "rms":
        return {"bytes": M * K * (e * (3 if case["residual"] else 1) + 1) + 4 * K + 4 * M, "flops": 6 * M * K}
    if op == "rms_grad":
        return {"bytes": M * K * e * (4 if case["residual"] else 3) + 8 * K, "flops": 12 * M * K}
    if op in ("act", "gate"):
        pair = 2 if op == "gate" else 1
        wide = 1 + (1 if case.get("residual") else 0) + (pair if case["pre"] else 0)
        return {"bytes": pair * (N * K + 4 * N * (2 if case["bias"] else 1)) + M * K * e + M * N * e * wide, "flops": 2 * pair * M * N * K}
    if op == "act_grad":
        pair = 2 if case["gated"] else 1
        return {"bytes": M * N * e * (1 + 2 * pair) + (4 * N * pair if case["bias"] else 0), "flops": 12 * M * N}
    return {"bytes": M * N * e + 32 * M, "flops": 8 * M * N}


def _function(act, z):
    """act and its derivative in 64 bits."""
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        cdf = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        # (1 + tanh a) / 2 = sigmoid(2 a)
        a = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
        p = torch.sigmoid(a)
        return z * p, p + z * p * (1 - p) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z * z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    return z, torch.ones_like(z)


def exact(case, seed):
    """The definitions in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "rms":
        x = s["x"].double()
        total = x if s["r"] is None else x + s["r"].double()
        h = total.to(s["x"].dtype).double()  # the norm is of the rows as they are kept
        p = h * s["w"].double()
        top = p.abs().amax(dim=1, keepdim=True)
        scale = top / 127 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
        q = torch.where(top > 0, torch.round(127 * p / torch.where(top > 0, top, 1.0)), 0.0)
        return {"h": total, "y": q * scale, "s": scale[:, 0]}
    if op == "rms_grad":
        h, dy, w = s["h"].double(), s["dy"].double(), s["w"].double()
        K = case["K"]
        var = (h * h).sum(dim=1, keepdim=True) / K + EPS
        inner = (dy * w * h).sum(dim=1, keepdim=True) / K
        dx = (dy * w) * var ** -0.5 - h * inner * var ** -1.5
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dw": (dy * h * var ** -0.5).sum(dim=0)}
    if op in ("act", "gate"):
        x = s["x"].double()
        scale = (x.abs().amax(dim=1) / 127.0).float().double()
        live = (scale > 0)[:, None]
        q = torch.where(live, torch.round((x / torch.where(live, scale[:, None], 1.0)).float().double()), 0.0).clamp(-127, 127)
        z = ((q @ s["w"].double().t()) * scale[:, None]) * s["sw"].double()
        z = z if s["b"] is None else z + s["b"].double()
        y, kept = _function(case["act"], z)[0], case["pre"]
        if op == "act":
            return {"y": y if s["r"] is None else y + s["r"].double(), "z": z if kept else None}
        u = ((q @ s["wu"].double().t()) * scale[:, None]) * s["swu"].double()
        u = u if s["bu"] is None else u + s["bu"].double()
        return {"y": y * u, "z": z if kept else None, "u": u if kept else None}
    if op == "act_grad":
        z, dy = s["z"].double(), s["dy"].double()
        f, d = _function(case["act"], z)
        dz = dy * d if s["u"] is None else dy * d * s["u"].double()
        du = None if s["u"] is None else dy * f
        return {"dz": dz, "du": du, "db": dz.sum(dim=0) if case["bias"] else None,
                "dbu": du.sum(dim=0) if case["bias"] and du is not None else None}
    # a row at a time, its tokens from the likeliest on
    token, logprob = [], []
    for m in range(case["M"]):
        z = s["z"][m].double()
        t = 1.0 if s["t"] is None else float(s["t"][m])
        if t <= 0:
            token.append(int(torch.nonzero(z == z.max())[0]))
            logprob.append(0.0)
            continue
        v, order = torch.sort(z, descending=True, stable=True)
        e = torch.exp(v / t - v[0] / t)
        k = 0 if s["k"] is None else int(s["k"][m])
        if k > 0:
            e = e[:k]
        held, n = torch.cumsum(e, 0), len(e)
        p = 1.0 if s["p"] is None else float(s["p"][m])
        if p < 1:
            n = min(n, 1 + int((held < p * held[-1]).sum()))
        if s["mp"] is not None:
            n = min(n, int((e >= float(s["mp"][m])).sum()))
        held = held[:n]
        at = min(int((held <= float(s["u"][m]) * held[-1]).sum()), n - 1)
        token.append(int(order[at]))
        logprob.append(float(v[at] / t - v[0] / t - torch.log(held[-1])))
    return torch.tensor(token, device=s["z"].device), torch.tensor(logprob, dtype=torch.float64, device=s["z"].device)
