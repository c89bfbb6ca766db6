"""The int8 entry points without a GPU: exports, and every refusal.  The calls
below fail validation (or are empty), so none reaches HIP."""
import os
import re
import subprocess

import pytest

import quant_packed_weight_amd as gq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemmq_i8.h")
A = 0x10000  # never dereferenced
INVALID, SHAPE, ALIGN, DEVICE = -1, -3, -4, -5


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gq.LIB_PATH):
        pytest.fail("libgemmq.so not built: run python -m quant_packed_weight_amd.build")
    return gq.lib_i8()


def test_every_declared_symbol_exported(L):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(gemmq_\w+)\s*\(", src))
    assert names == set(gq.EXPORTS_I8)
    out = subprocess.run(["nm", "-D", "--defined-only", gq.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert names <= set(re.findall(r"\sT\s+(gemmq_\w+)", out))
    assert L.gemmq_i8_abi_version() == gq.I8_ABI_VERSION


def test_an_older_library_is_named(monkeypatch):
    # one of another version, which lacks entry points that this binding has
    from quant_packed_weight_amd import _i8, _lib

    class Older:
        @staticmethod
        def gemmq_i8_abi_version():
            return gq.I8_ABI_VERSION - 1

        @staticmethod
        def gemmq_status_str(status):
            return b"GEMMQ_E_UNKNOWN"

    monkeypatch.setattr(_lib, "lib", Older)
    monkeypatch.setattr(_i8, "_fns", None)
    with pytest.raises(gq.GemmqError, match="int8 ABI %d, binding expects %d"
                       % (gq.I8_ABI_VERSION - 1, gq.I8_ABI_VERSION)):
        gq.lib_i8()
    src = open(HEADER).read()
    assert int(re.search(r"#define GEMMQ_I8_ABI_VERSION (\d+)", src).group(1)) == gq.I8_ABI_VERSION


def test_constants_follow_the_header():
    src = open(HEADER).read()
    for name, value in [("GEMMQ_F32", gq.F32), ("GEMMQ_BF16", gq.BF16), ("GEMMQ_F16", gq.F16),
                        ("GEMMQ_I8_MAX_K", gq.I8_MAX_K), ("GEMMQ_I8_MAX_ROWS", gq.I8_MAX_ROWS),
                        ("GEMMQ_I8_MAX_PITCH", gq.I8_MAX_PITCH)]:
        assert int(re.search(r"#define %s (\d+)" % name, src).group(1)) == value


# one good argument list per entry, and changes to it with the status they give
QUANT = dict(xtype=0, X=A, ldx=100, Q=A, ldq=112, s=A, M=4, K=100)
GEMM = dict(W=A, ldw=112, sw=A, Xq=A, ldq=112, sx=A, bias=None, ytype=0, Y=A, ldy=50, M=4, N=50,
            K=100)
LINEAR = dict(W=A, ldw=112, sw=A, xtype=1, X=A, ldx=100, Xq=A, ldq=112, sx=A, bias=A, ytype=2,
              Y=A, ldy=50, M=4, N=50, K=100)
GRAD = dict(W=A, ldw=112, sw=A, type=1, dY=A, lddy=50, dX=A, lddx=100, M=4, N=50, K=100, ws=A,
            bytes=1 << 40)
LOSS = dict(W=A, ldw=112, sw=A, Xq=A, ldq=112, sx=A, target=A, loss=A, lse=A, M=4, N=50, K=100,
            ws=A, bytes=1 << 40)
LGRAD = dict(W=A, ldw=112, sw=A, Xq=A, ldq=112, sx=A, target=A, lse=A, dloss=A, type=1, dX=A,
             lddx=100, M=4, N=50, K=100, ws=A, bytes=1 << 40)
ENTRIES = {"quantize_i8": QUANT, "gemm_i8": GEMM, "linear_i8": LINEAR, "linear_i8_grad": GRAD,
           "loss_i8": LOSS, "loss_i8_grad": LGRAD}
I8_MATRICES = [("W", "ldw"), ("Xq", "ldq"), ("Q", "ldq")]
FLOAT_MATRICES = [("X", "ldx", "xtype", "K"), ("Y", "ldy", "ytype", "N"),
                  ("dY", "lddy", "type", "N"), ("dX", "lddx", "type", "K")]


def _changes(args):
    yield dict(M=-1), INVALID
    yield dict(K=0), SHAPE
    yield dict(K=gq.I8_MAX_K + 1), SHAPE
    yield dict(M=gq.I8_MAX_ROWS + 1), SHAPE
    if "N" in args:
        yield dict(N=-1), INVALID
        yield dict(N=gq.I8_MAX_ROWS + 1), SHAPE
    for t in ("xtype", "ytype", "type"):
        if t in args:
            yield {t: 3}, INVALID
            yield {t: -1}, INVALID
    for p, ld in I8_MATRICES:
        if p in args:
            yield {p: None}, INVALID
            yield {p: A + 8}, ALIGN
            yield {ld: 104}, ALIGN          # not a multiple of 16
            yield {ld: 96}, SHAPE           # below K
            yield {ld: gq.I8_MAX_PITCH + 16}, SHAPE
    for p, ld, ty, width in FLOAT_MATRICES:
        if p in args:
            yield {p: None}, INVALID
            yield {p: A + 1}, ALIGN
            yield {ld: args[width] - 1}, SHAPE
            yield {ty: 0, p: A + 2}, ALIGN  # f32 on a 2-byte boundary
    for v in ("sw", "sx", "s", "loss", "lse", "dloss", "target"):
        if v in args:
            yield {v: None}, INVALID
            yield {v: A + 2}, ALIGN
    if "target" in args:
        yield dict(target=A + 4), ALIGN
        yield dict(N=0), SHAPE              # no vocabulary
    if args.get("bias") is not None or args is GEMM:
        yield dict(bias=A + 2), ALIGN
    if "ws" in args:
        yield dict(ws=None), INVALID
        yield dict(ws=A + 8), ALIGN
        yield dict(bytes=16), INVALID
    yield dict(M=0), 0                      # empty: nothing is touched


CASES = [(e, c, s) for e, a in ENTRIES.items() for c, s in _changes(a)]


@pytest.mark.parametrize("entry,change,status", CASES,
                         ids=["%s-%s" % (e, "-".join("%s=%s" % i for i in c.items()))
                              for e, c, _ in CASES])
def test_refusals(L, entry, change, status):
    args = dict(ENTRIES[entry], **change)
    assert getattr(L, "gemmq_" + entry)(*args.values(), None) == status


def test_empty_product_is_no_error(L):
    assert L.gemmq_gemm_i8(*dict(GEMM, N=0).values(), None) == 0


def test_grid_limits_are_refused_before_anything_runs(L):
    # 2^24 x 2^24 outputs are more tiles than a grid has
    big = dict(M=gq.I8_MAX_ROWS, N=gq.I8_MAX_ROWS, ldy=gq.I8_MAX_ROWS, lddy=gq.I8_MAX_ROWS)
    for name, args in (("gemm_i8", GEMM), ("linear_i8", LINEAR), ("loss_i8", LOSS)):
        a = dict(args, **{k: v for k, v in big.items() if k in args})
        assert getattr(L, "gemmq_" + name)(*a.values(), None) == SHAPE, name
    assert L.gemmq_loss_i8_workspace(gq.I8_MAX_ROWS, gq.I8_MAX_ROWS, 64) == 0
    # 2^19 x 2^20: 2^23 tiles of 512 threads, one launch's threads pass 2^32
    a = dict(M=1 << 19, N=1 << 20, ldy=1 << 20)
    assert L.gemmq_gemm_i8(*dict(GEMM, **a).values(), None) == SHAPE
    assert L.gemmq_linear_i8(*dict(LINEAR, **a).values(), None) == SHAPE
    assert L.gemmq_loss_i8_workspace(1 << 19, 1 << 20, 64) == 0
    assert L.gemmq_loss_i8_workspace(1 << 18, 1 << 20, 64) > 0  # half of that fits


def test_workspace_sizes(L):
    for f in (L.gemmq_linear_i8_grad_workspace, L.gemmq_loss_i8_grad_workspace):
        for ty in (0, 1, 2):
            assert f(ty, 7, 1000, 100) > 0
            assert f(ty, 0, 1000, 100) == 0
            assert f(ty, 7, 1000, 0) == 0
            assert f(ty, -1, 1000, 100) == 0
        assert f(3, 7, 1000, 100) == 0
    assert L.gemmq_linear_i8_grad_workspace(1, 7, 0, 100) > 0  # writes zeros
    assert L.gemmq_loss_i8_grad_workspace(1, 7, 0, 100) == 0
    assert L.gemmq_loss_i8_workspace(7, 1000, 100) > 0
    assert L.gemmq_loss_i8_workspace(7, 0, 100) == 0
    # the logits of a large head are never held: far less than M * N values
    assert L.gemmq_loss_i8_workspace(2048, 151936, 2048) < 2048 * 151936 * 4 // 10
    assert L.gemmq_loss_i8_grad_workspace(1, 8192, 151936, 2048) < 8192 * 151936 * 4 // 5


def test_workspace_of_a_call_is_what_its_size_says(L):
    need = L.gemmq_linear_i8_grad_workspace(1, 4, 50, 100)
    assert L.gemmq_linear_i8_grad(*dict(GRAD, bytes=need - 1).values(), None) == INVALID
    need = L.gemmq_loss_i8_workspace(4, 50, 100)
    assert L.gemmq_loss_i8(*dict(LOSS, bytes=need - 1).values(), None) == INVALID


def test_tensors_on_the_host_are_refused(L):
    import torch

    w, sw = torch.zeros((32, 32), dtype=torch.int8), torch.zeros(32)
    x = torch.zeros((4, 32))
    t = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: gq.quantize_i8(x), lambda: gq.linear_i8_grad(w, sw, x),
                 lambda: gq.gemm_i8(w, sw, x.to(torch.int8), sw[:4]),
                 lambda: gq.linear_i8(w, sw, x),
                 lambda: gq.loss_i8(w, sw, x.to(torch.int8), sw[:4], t),
                 lambda: gq.loss_i8_grad(w, sw, x.to(torch.int8), sw[:4], t, sw[:4], sw[:4])):
        with pytest.raises((TypeError, ValueError)):
            call()


def test_unknown_element_types_are_refused(L):
    import torch

    with pytest.raises(TypeError):
        gq.quantize_i8(torch.zeros((4, 32), dtype=torch.float64))
    with pytest.raises(TypeError):
        gq.linear_i8_grad_workspace(torch.int8, 4, 4, 4)


def test_a_single_row_allows_wide_accesses_at_any_width():
    # the pitch that the binding names for one row is a multiple of 16 bytes in every type
    import torch

    from quant_packed_weight_amd import _i8

    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        for cols in (1, 7, 8, 12, 515, 1028):
            x = torch.zeros((1, cols + 3), dtype=dtype)[:, :cols]
            ld = _i8._matrix(x, "x", dtype, 1, cols, -1)
            assert ld >= cols and ld * x.element_size() % 16 == 0
            x = torch.zeros((2, cols + 3), dtype=dtype)[:, :cols]
            assert _i8._matrix(x, "x", dtype, 2, cols, -1) == cols + 3


def test_tensors_that_require_a_gradient_are_refused(L):
    # no result has a graph, so none is cut unseen; without grad mode the calls go on (here
    # to the refusal of host tensors)
    import torch

    w, sw = torch.zeros((32, 32), dtype=torch.int8), torch.zeros(32)
    xq, one, t = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(4), torch.zeros(4, dtype=torch.int64)
    x, leaf = torch.zeros((4, 32)), torch.zeros((4, 32), requires_grad=True)
    s1, b1, one1 = sw.clone().requires_grad_(), sw.clone().requires_grad_(), one.clone().requires_grad_()
    calls = [lambda: gq.linear_i8(w, sw, leaf), lambda: gq.linear_i8(w, sw, x, bias=b1),
             lambda: gq.linear_i8(w, s1, x), lambda: gq.linear_i8(w, sw, 2 * leaf),
             lambda: gq.gemm_i8(w, sw, xq, one1), lambda: gq.gemm_i8(w, s1, xq, one),
             lambda: gq.gemm_i8(w, sw, xq, one, bias=b1), lambda: gq.linear_i8_grad(w, sw, leaf),
             lambda: gq.loss_i8(w, sw, xq, one1, t), lambda: gq.loss_i8(w, s1, xq, one, t),
             lambda: gq.loss_i8_grad(w, sw, xq, one, t, one, one1),
             lambda: gq.loss_i8_grad(w, sw, xq, one, t, one1, one),
             lambda: gq.quantize_i8(2 * leaf)]
    for call in calls:
        with pytest.raises(ValueError, match="record no gradient"):
            call()
        with torch.no_grad(), pytest.raises(TypeError, match="device tensors"):
            call()
    # a parameter's int8 copy is a constant
    with pytest.raises(TypeError, match="device tensors"):
        gq.quantize_i8(leaf)


def test_outputs_that_always_fit(L):
    # the header's limits: every shape of up to 2^36 outputs is taken, and a status text names them
    import math
    import random

    src = open(HEADER).read()
    most = int(re.search(r"#define GEMMQ_I8_MAX_OUTPUTS (\d+)", src).group(1))
    assert most == gq.I8_MAX_OUTPUTS == 1 << 36
    r = random.Random(3)

    def size(low, high):
        return int(round(math.exp(r.uniform(math.log(low), math.log(high)))))

    for n in range(6000):
        M = size(1, gq.I8_MAX_ROWS)
        N = min(gq.I8_MAX_ROWS, most // M) if n % 2 else size(1, min(gq.I8_MAX_ROWS, most // M))
        K = min(gq.I8_MAX_K, most // M) if n % 3 else size(1, min(gq.I8_MAX_K, most // M))
        assert L.gemmq_loss_i8_workspace(M, N, size(1, gq.I8_MAX_K)) > 0, (M, N)
        for ty in (0, 1, 2):
            assert L.gemmq_linear_i8_grad_workspace(ty, M, N, K) > 0, (ty, M, N, K)
            assert L.gemmq_loss_i8_grad_workspace(ty, M, N, K) > 0, (ty, M, N, K)
    assert "2^36 outputs" in gq.status_str(SHAPE)
