"""The norm over the range of values that its y is exact in: mean(total^2) + eps, total
weight and y between 2^-96 and 2^127.  Sums and rstd are held to 2^-40 and 64-bit
arithmetic here to (C + 5) 2^-53 < 2^-44, so y is a number within 2^-39 of the 64-bit one,
rounded to FP32 and to BF16; both roundings are monotonic, so that the ends of that
interval say what y may be.  The forms are those of y."""
import numpy as np
import pytest
import torch

import moe_ref
from test_gpu_mx import bits_of, mx, to_dev  # noqa: F401  (mx: the fixture)

pytestmark = pytest.mark.gpu


def scaled(rng, power, *shape):
    """Normal numbers times 2^power, no nearer to zero than 2^(power - 12)."""
    v = rng.standard_normal(shape)
    v = np.where(np.abs(v) < 2.0 ** -12, 2.0 ** -12, v)
    return to_dev(bits_of(torch.from_numpy(np.ldexp(v, power).astype(np.float32)).to(torch.bfloat16)))


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def rounded(y64):
    return f64(torch.from_numpy(y64.astype(np.float32)).to(torch.bfloat16))


@pytest.mark.parametrize("C", [304, 301])
@pytest.mark.parametrize("of_total,of_weight", [(-40, -20), (-40, 60), (0, -70), (0, 90), (57, -57), (57, 60), (30, -70), (-20, 30)])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_y_is_exact(mx, C, of_total, of_weight, eps):  # noqa: F811
    rng = np.random.default_rng(of_total * 1000 + of_weight + C + 10 ** 6)
    T = 40
    x, w = scaled(rng, of_total, T, C), scaled(rng, of_weight, C)
    y = torch.empty_like(x)
    row, col, row_y, col_y = (mx.MxTensor.empty("e4m3", *s) for s in ((T, C), (C, T)) * 2)
    mx.rms_norm(x, w, eps, out=y, row=row, col=col)
    want = f64(x) * f64(w) * moe_ref.rms(f64(x), float(np.float32(eps)))[:, None]
    off = 2.0 ** -39 * np.abs(want)
    assert np.abs(want).min() >= 2.0 ** -96 and np.abs(f64(x) * f64(w)).max() < 2.0 ** 127
    got = f64(y)
    assert ((rounded(want - off) <= got) & (got <= rounded(want + off))).all()
    mx.quantize(y, row=row_y, col=col_y)
    for a, b in ((row, row_y), (col, col_y)):
        assert torch.equal(a.codes, b.codes) and torch.equal(mx.dequantize(a), mx.dequantize(b))
