"""Helpers of the GPU tests of what stands between the int8 products.

Tolerances count roundings.  U = 2^-24 is half a step of f32, HALF[t] half a step of
the type t relative to the value, FLOOR[t] half a step of its subnormals."""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FLOOR = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(rows, cols, g, dtype, scale=1.0, extra=0):
    """Random rows of a buffer `extra` columns wider."""
    x = torch.full((rows, cols + extra), 9.0, dtype=dtype, device="cuda")[:, :cols]
    return x.copy_(torch.randn((rows, cols), generator=g, device="cuda") * scale)


def scales(n, g, size=1.0):
    return (0.2 + torch.rand(n, generator=g, device="cuda")) * size


def i8(rows, cols, g):
    """Random int8 rows; the bytes behind each hold other values, which must not matter."""
    pitch = -(-cols // 16) * 16
    return torch.randint(-127, 128, (rows, pitch), generator=g, device="cuda",
                         dtype=torch.int8)[:, :cols]


class Guarded:
    """A [rows, cols] tensor inside a wider buffer whose other values are known:
    rows above, rows below and columns to the right of it."""

    def __init__(self, rows, cols, dtype, extra=5, fill=7):
        self.all = torch.full((rows + 2, cols + extra), fill, dtype=dtype, device="cuda")
        self.t = self.all[1:rows + 1, :cols]
        self.fill, self.rows, self.cols = fill, rows, cols

    def check(self):
        a = self.all.clone()
        a[1:self.rows + 1, :self.cols] = self.fill
        assert bool((a == self.fill).all()), "written outside the result"


def within(got, ref, tol, what=""):
    """|got - ref| <= tol element by element, `ref` and `tol` in 64 bits; NaN where ref is."""
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), what + ": NaN in other places"
    bad = ((got.double() - ref).abs() > tol) & ~nan
    if bool(bad.any()):
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError("%s: %d of %d off; first at %s: %r, not %r +- %r"
                             % (what, int(bad.sum()), bad.numel(), i, float(got[i]), float(ref[i]),
                                float(tol[i])))
