"""Routings of any content, next to guards that are wider than the near misses drawn
here: what lies around the results stays, and nothing that lies around the inputs,
which is NaN, comes into them."""
import numpy as np
import pytest
import torch

from test_gpu_moe import moe  # noqa: F401  (the fixture)
from test_gpu_mx import mx  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
NEAR = 300                       # rows that an index may lie outside by, half of the time
BF16, F32 = torch.bfloat16, torch.float32


class Guarded:
    """Memory with NEAR rows of its own, and a page, on either side: bytes 255, which is NaN
    in every type here, codes and scales among them."""

    def __init__(self):
        self.around = []

    def matrix(self, dtype, rows, cols):
        size = torch.empty(0, dtype=dtype).element_size()
        guard = -(-(NEAR + 8) * cols * size // 4096) * 4096
        mem = torch.full((rows * cols * size + 2 * guard,), 255, dtype=torch.uint8, device="cuda")
        self.around += [mem[:guard], mem[-guard:]]
        inner = mem[guard:-guard].view(dtype).view(rows, cols)
        return inner.zero_()

    def form(self, mx, fmt, rows, cols):  # noqa: F811
        t = mx.MxTensor.empty(fmt, rows, cols)
        t.codes = self.matrix(torch.uint8, *t.codes.shape)
        t.scales = self.matrix(torch.uint8, t.scales.numel() // 512, 512).view(-1)
        return t

    def intact(self):
        return all(bool((m == 255).all()) for m in self.around)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("C", [264, 135])           # rows on 16 bytes, and off them
def test_near_misses(mx, moe, seed, C):  # noqa: F811
    rng = np.random.default_rng(100 + seed)
    T, k, E = 300, 3, 5
    rows = moe._rows(T, k, E)
    g = Guarded()

    def any_int(*shape):
        v = rng.integers(-2 ** 31, 2 ** 31, size=shape)
        near = rng.integers(-NEAR, rows + NEAR, size=shape)
        return torch.from_numpy(np.where(rng.random(shape) < 0.25, v, near).astype(np.int32)).cuda()

    def values(dtype, *shape):
        m = g.matrix(dtype, *shape)
        return m.copy_(torch.from_numpy(rng.standard_normal(shape).astype(np.float32)))

    r = moe.Routing(T, k, E, any_int(E), any_int(E + 1), any_int(T, k), any_int(rows))
    x, dy, y = values(BF16, T, C), values(BF16, T, C), values(BF16, rows, C)
    w = values(F32, T, k)
    got = []
    for weights in (None, w):
        for fmts in (("e2m1", None), ("e4m3", None), ("e4m3", "e5m2"), (None, "e4m3")):
            row, col = (None if f is None else g.form(mx, f, *s) for f, s in zip(fmts, ((rows, C), (C, rows))))
            moe.dispatch(x, r, row=row, col=col, weights=weights)
            got += [mx.dequantize(t) for t in (row, col) if t is not None]
        got.append(moe.combine(y, r, weights, out=g.matrix(BF16, T, C)))
    got.append(moe.weight_gradient(dy, y, r, out=g.matrix(F32, T, k)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, c = g.form(mx, "e4m3", rows, C), g.form(mx, "e4m3", C, rows)
    mx.quantize(y, row=a, col=c)
    for n in (140, 700):         # tiles by tokens and by weights
        b = mx.MxStack.empty("e4m3", E, n, C)
        b.codes, b.scales = g.matrix(torch.uint8, *b.codes.shape), g.matrix(torch.uint8, b.scales.numel() // 512, 512).view(-1)
        for e in range(E):
            mx.quantize(values(BF16, n, C), row=b[e])
        for dtype in (BF16, F32):
            got.append(moe.expert_matmul(a, b, r, out=g.matrix(dtype, rows, n), status=status))
    out = g.matrix(F32, E * C, C)
    moe.expert_gradient(c, c, r, out=out.view(E, C, C), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and g.intact()
    assert all(bool(torch.isfinite(t).all()) for t in got + [out])
