"""The entry points of what stands between the int8 products, without a GPU: every
refusal.  The calls below fail validation (or are empty), so none reaches HIP."""
import os

import pytest

import quant_packed_weight_amd as gq

A = 0x10000  # never dereferenced
B = 0x20000
INVALID, SHAPE, ALIGN = -1, -3, -4


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gq.LIB_PATH):
        pytest.fail("libgemmq.so not built: run python -m quant_packed_weight_amd.build")
    return gq.lib_i8()


NAN, INF = float("nan"), float("inf")
RMS = dict(type=1, X=A, ldx=100, R=A, ldr=100, H=B, ldh=100, w=A, eps=1e-6, Q=A, ldq=112, s=A, M=4,
           K=100)
RGRAD = dict(type=1, H=A, ldh=100, w=A, eps=1e-6, dY=A, lddy=100, dH=A, lddh=100, dX=B, lddx=100,
             dw=A, M=40, K=100, ws=A, bytes=1 << 40)
GEMM = dict(W=A, ldw=112, sw=A, Xq=A, ldq=112, sx=A, bias=A, act=1, R=A, ldr=50, ytype=0, Y=B,
            ldy=50, Z=2 * B, ldz=50, M=4, N=50, K=100)
LINEAR = dict(W=A, ldw=112, sw=A, xtype=1, X=A, ldx=100, Xq=A, ldq=112, sx=A, bias=A, act=1, R=A,
              ldr=50, ytype=2, Y=B, ldy=50, Z=2 * B, ldz=50, M=4, N=50, K=100)
GATE = dict(W=A, ldw=112, sw=A, Wu=A, ldwu=112, swu=A, Xq=A, ldq=112, sx=A, bias=A, biasu=A, act=1,
            ytype=0, Y=B, ldy=50, Z=2 * B, ldz=50, U=3 * B, ldu=50, M=4, N=50, K=100)
LGATE = dict(W=A, ldw=112, sw=A, Wu=A, ldwu=112, swu=A, xtype=1, X=A, ldx=100, Xq=A, ldq=112, sx=A,
             bias=A, biasu=A, act=1, ytype=2, Y=B, ldy=50, Z=2 * B, ldz=50, U=3 * B, ldu=50, M=4, N=50,
             K=100)
AGRAD = dict(act=1, type=1, Z=A, ldz=50, U=A, ldu=50, dY=A, lddy=50, dZ=B, lddz=50, dU=2 * B,
             lddu=50, db=A, dbu=3 * B, M=40, N=50, ws=A, bytes=1 << 40)
SAMPLE = dict(type=1, Z=A, ldz=50000, temperature=A, top_k=A, top_p=A, min_p=A, u=A, token=A,
              logprob=A, M=4, N=50000, ws=A, bytes=1 << 40)
ENTRIES = {"sample": SAMPLE, "rms_i8": RMS, "rms_i8_grad": RGRAD, "gemm_i8_act": GEMM, "linear_i8_act": LINEAR,
           "gemm_i8_gate": GATE, "linear_i8_gate": LGATE, "act_grad": AGRAD}
_Y = [("Y", "ldy", "N", False), ("Z", "ldz", "N", True)]
_X = [("X", "ldx", "K", False)]
# matrices of the element type: name, pitch, width, and whether it may be NULL
MATRICES = {"rms_i8": [("X", "ldx", "K", False), ("R", "ldr", "K", True), ("H", "ldh", "K", True)],
            "rms_i8_grad": [("H", "ldh", "K", False), ("dY", "lddy", "K", False),
                            ("dH", "lddh", "K", True), ("dX", "lddx", "K", False)],
            "gemm_i8_act": _Y + [("R", "ldr", "N", True)],
            "linear_i8_act": _X + _Y + [("R", "ldr", "N", True)],
            "gemm_i8_gate": _Y + [("U", "ldu", "N", True)],
            "linear_i8_gate": _X + _Y + [("U", "ldu", "N", True)],
            "sample": [("Z", "ldz", "N", False)],
            "act_grad": [("Z", "ldz", "N", False), ("dY", "lddy", "N", False),
                         ("dZ", "lddz", "N", False), ("U", "ldu", "N", True),
                         ("dU", "lddu", "N", True)]}
_I = [("W", "ldw"), ("Xq", "ldq")]
I8_MATRICES = {"rms_i8": [("Q", "ldq")], "gemm_i8_act": _I, "linear_i8_act": _I,
               "gemm_i8_gate": _I + [("Wu", "ldwu")], "linear_i8_gate": _I + [("Wu", "ldwu")]}
# f32 vectors: name, and whether it may be NULL
_V = [("sw", False), ("sx", False), ("bias", True)]
VECTORS = {"rms_i8": [("w", False), ("s", False)], "rms_i8_grad": [("w", False), ("dw", True)],
           "gemm_i8_act": _V, "linear_i8_act": _V,
           "gemm_i8_gate": _V + [("swu", False), ("biasu", True)],
           "linear_i8_gate": _V + [("swu", False), ("biasu", True)],
           "act_grad": [("db", True), ("dbu", True)],
           "sample": [("temperature", True), ("top_k", True), ("top_p", True), ("min_p", True),
                      ("u", False), ("token", False), ("logprob", True)]}
OWN = {"rms_i8": [(dict(H=A, ldh=104, R=B), INVALID),            # X, but not as X lies
                  (dict(H=B, ldh=104, R=B), INVALID)],
       "rms_i8_grad": [(dict(dX=A, lddx=104, dH=B), INVALID), (dict(dX=B, lddx=104, dH=B), INVALID),
                       (dict(dX=B, lddx=104, H=B), INVALID)],
       "gemm_i8_act": [(dict(R=B, ldr=52), INVALID), (dict(Z=B), INVALID), (dict(Z=A), INVALID)],
       "linear_i8_act": [(dict(R=B, ldr=52), INVALID), (dict(Z=B), INVALID), (dict(Z=A), INVALID)],
       "gemm_i8_gate": [(dict(Z=B), INVALID), (dict(U=B), INVALID), (dict(U=2 * B), INVALID)],
       "linear_i8_gate": [(dict(Z=B), INVALID), (dict(U=B), INVALID), (dict(U=2 * B), INVALID)],
       "sample": [(dict(N=0), SHAPE), (dict(token=A + 4), ALIGN)],
       "act_grad": [(dict(U=None), INVALID), (dict(dU=None), INVALID), (dict(dbu=A), INVALID),
                    (dict(U=None, dU=None), INVALID),   # a dbu without a pair
                    (dict(dZ=A, lddz=52), INVALID), (dict(dU=A, lddu=52), INVALID),
                    (dict(dU=B), INVALID)]}            # dZ's place


def _changes(entry, a):
    yield dict(M=-1), INVALID
    yield dict(M=gq.I8_MAX_ROWS + 1), SHAPE
    for c in ("K", "N"):
        if c in a:
            yield {c: gq.I8_MAX_K + 1 if c == "K" else gq.I8_MAX_ROWS + 1}, SHAPE
    if "K" in a:
        yield dict(K=0), SHAPE
    if "N" in a:
        yield dict(N=-1), INVALID
    for t in ("type", "xtype", "ytype"):
        if t in a:
            yield {t: 3}, INVALID
            yield {t: -1}, INVALID
    if "act" in a:
        yield dict(act=5), INVALID
        yield dict(act=-1), INVALID
    if "eps" in a:
        for v in (-1.0, NAN, INF):
            yield dict(eps=v), INVALID
    for p, ld, width, null in MATRICES[entry]:
        if not null:
            yield {p: None}, INVALID
        yield {p: A + 1}, ALIGN
        yield {ld: a[width] - 1}, SHAPE
        yield {ld: (1 << 40) + 1}, SHAPE
    for p, ld in I8_MATRICES.get(entry, []):
        yield {p: None}, INVALID
        yield {p: A + 8}, ALIGN
        yield {ld: 104}, ALIGN
        yield {ld: 96}, SHAPE
        yield {ld: gq.I8_MAX_PITCH + 16}, SHAPE
    for v, null in VECTORS[entry]:
        if not null:
            yield {v: None}, INVALID
        yield {v: A + 2}, ALIGN
    if "ws" in a:
        yield dict(ws=None), INVALID
        yield dict(ws=A + 8), ALIGN
        yield dict(bytes=16), INVALID
    yield from OWN.get(entry, [])


CASES = [(e, c, s) for e, a in ENTRIES.items() for c, s in _changes(e, a)]


@pytest.mark.parametrize("entry,change,status", CASES,
                         ids=["%s-%s" % (e, "-".join("%s=%s" % i for i in c.items()))
                              for e, c, _ in CASES])
def test_refusals(L, entry, change, status):
    args = dict(ENTRIES[entry], **change)
    assert getattr(L, "gemmq_" + entry)(*args.values(), None) == status


def test_empty_calls(L):
    assert L.gemmq_rms_i8(*dict(RMS, M=0).values(), None) == 0
    # no rows and no sum over them; with one, zeros are written
    assert L.gemmq_rms_i8_grad(*dict(RGRAD, M=0, dw=None).values(), None) == 0
    for entry in ("gemm_i8_act", "linear_i8_act", "gemm_i8_gate", "linear_i8_gate"):
        assert getattr(L, "gemmq_" + entry)(*dict(ENTRIES[entry], M=0).values(), None) == 0
    for entry in ("gemm_i8_act", "gemm_i8_gate"):
        assert getattr(L, "gemmq_" + entry)(*dict(ENTRIES[entry], N=0).values(), None) == 0
    assert L.gemmq_act_grad(*dict(AGRAD, M=0, db=None, dbu=None).values(), None) == 0
    assert L.gemmq_act_grad(*dict(AGRAD, N=0).values(), None) == 0
    assert L.gemmq_sample(*dict(SAMPLE, M=0).values(), None) == 0


def test_products_that_no_launch_holds(L):
    for entry in ("gemm_i8_act", "linear_i8_act", "gemm_i8_gate", "linear_i8_gate"):
        a = dict(ENTRIES[entry], M=1 << 24, N=1 << 24)
        a.update({k: 1 << 24 for k in ("ldy", "ldz", "ldu", "ldr") if k in a})
        assert getattr(L, "gemmq_" + entry)(*a.values(), None) == SHAPE


def test_workspace_sizes(L):
    import torch

    for ty, dtype in enumerate((torch.float32, torch.bfloat16, torch.float16)):
        need = L.gemmq_rms_i8_grad_workspace(ty, 40, 100)
        assert need >= 40 * 100 * 4
        assert L.gemmq_rms_i8_grad_workspace(ty, 4, 100) == 0  # none is needed
        assert L.gemmq_rms_i8_grad(*dict(RGRAD, type=ty, bytes=need - 1).values(), None) == INVALID
        assert gq.rms_i8_grad_workspace(dtype, 40, 100) == need
        need = L.gemmq_act_grad_workspace(ty, 40, 50)
        assert need >= 2 * 50 * 4 and gq.act_grad_workspace(dtype, 40, 50) == need
        assert L.gemmq_act_grad_workspace(ty, 16, 50) == 0
        assert L.gemmq_act_grad(*dict(AGRAD, type=ty, bytes=need - 1).values(), None) == INVALID
        assert L.gemmq_act_grad_workspace(ty, 1 << 20, 12288) < 64 << 20
        # a few rows of partial sums, not one for each row
        assert L.gemmq_rms_i8_grad_workspace(ty, 1 << 20, 4096) < 64 << 20
    for bad in ((3, 40, 100), (0, -1, 100), (0, 40, 0), (0, 0, 100)):
        assert L.gemmq_rms_i8_grad_workspace(*bad) == 0
        assert L.gemmq_act_grad_workspace(*bad) == 0


def test_sample_workspace(L):
    need = L.gemmq_sample_workspace(4, 50000)
    assert need > 0 and gq.sample_workspace(4, 50000) == need
    assert L.gemmq_sample_workspace(4, 5000) == 0  # none is needed
    assert L.gemmq_sample(*dict(SAMPLE, bytes=need - 1).values(), None) == INVALID
    for bad in ((0, 50000), (4, 0), (-1, 50000), (4, -1), (gq.I8_MAX_ROWS + 1, 50000),
                (4, gq.I8_MAX_ROWS + 1)):
        assert L.gemmq_sample_workspace(*bad) == 0
    # bounded for any number of rows
    assert L.gemmq_sample_workspace(1 << 24, 151936) < 64 << 20


def test_binding_refusals(L):
    import torch

    x, w, leaf = torch.zeros((4, 32)), torch.zeros(32), torch.zeros((4, 32), requires_grad=True)
    w1 = w.clone().requires_grad_()
    calls = [lambda: gq.rms_i8(leaf, w), lambda: gq.rms_i8(x, w1), lambda: gq.rms_i8(x, w, residual=leaf),
             lambda: gq.rms_i8_grad(leaf, w, x), lambda: gq.rms_i8_grad(x, w1, x),
             lambda: gq.rms_i8_grad(x, w, leaf), lambda: gq.rms_i8_grad(x, w, x, dh=leaf)]
    i, one, o = torch.zeros((32, 32), dtype=torch.int8), torch.zeros(32), torch.zeros((4, 32))
    i4, o4 = i[:4], one[:4]
    l1 = one.clone().requires_grad_()
    calls += [lambda: gq.gemm_i8_act(i, l1, i4, o4, 1), lambda: gq.gemm_i8_act(i, one, i4, l1[:4], 1),
              lambda: gq.gemm_i8_act(i, one, i4, o4, 1, bias=l1),
              lambda: gq.gemm_i8_act(i, one, i4, o4, 1, residual=leaf),
              lambda: gq.linear_i8_act(i, one, leaf, 1),
              lambda: gq.linear_i8_act(i, one, x, 1, residual=leaf),
              lambda: gq.gemm_i8_gate(i, one, i, l1, i4, o4),
              lambda: gq.gemm_i8_gate(i, one, i, one, i4, o4, bias_up=l1),
              lambda: gq.linear_i8_gate(i, one, i, one, leaf),
              lambda: gq.act_grad(1, leaf, o), lambda: gq.act_grad(1, o, leaf),
              lambda: gq.act_grad(1, o, o, up=leaf), lambda: gq.sample(leaf, o4),
              lambda: gq.sample(o, l1[:4]), lambda: gq.sample(o, o4, temperature=l1[:4])]
    for call in calls:
        with pytest.raises(ValueError, match="record no gradient"):
            call()
        with torch.no_grad(), pytest.raises(TypeError, match="device tensors"):
            call()
    with pytest.raises(TypeError):
        gq.rms_i8_grad_workspace(torch.int8, 4, 4)
    with pytest.raises(TypeError):
        gq.act_grad_workspace(torch.int8, 4, 4)


def test_constants_follow_the_header():
    import re

    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                            "gemmq_i8.h")).read()
    for name, value in [("NONE", gq.ACT_NONE), ("SILU", gq.ACT_SILU), ("GELU", gq.ACT_GELU),
                        ("GELU_TANH", gq.ACT_GELU_TANH), ("RELU", gq.ACT_RELU)]:
        assert int(re.search(r"#define GEMMQ_ACT_%s (\d+)" % name, src).group(1)) == value
