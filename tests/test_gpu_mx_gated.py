"""The gated unit and its backward pass where they can go wrong beside the
sizes and gates of test_gpu_mx.py."""
import numpy as np
import pytest
import torch

import mx_ref as ref
from test_gpu_mx import bits_of, mx, near, to_dev  # noqa: F401  (mx is the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("u", [1.0, 3.0e4, -2.0e30])
def test_gates_far_below_zero(mx, u):
    """Gates down to where exp(-g) leaves FP32: s = 1 / (1 + exp(-g)) is then a small
    number and no zero; from there on it is zero.  The fast exp of CUDA is off by up
    to 2 + 1.173 |g| units in the last place, under 107 * 2^-23, and the reciprocal
    and products by a few more: together under 2^-15.  Where s has no 24 bits left,
    it is off by up to 2 steps of 2^-149."""
    far = [-89.0, -96.0, -126.0, -200.0, -1e30]
    g = np.concatenate([-np.arange(60, 89, 0.25), far])
    g = np.concatenate([g, np.full(-len(g) % 32, -0.5)])[None, :]
    gb = bits_of(torch.from_numpy(g.astype(np.float32)).to(torch.bfloat16))
    g = ref.bf16_to_f64(gb)
    ub = bits_of(torch.full(g.shape, u).to(torch.bfloat16))
    u64 = ref.bf16_to_f64(ub)
    top = np.log(float(np.finfo(np.float32).max))

    def logistic(x):
        return np.where(x < -top, 0.0, 1 / (1 + np.exp(np.minimum(-x, top))))

    def bound(want, factor):
        return 2.0 ** -15 * np.abs(want) + 2.0 ** -148 * np.abs(factor)

    g8, u8 = mx.MxTensor.empty("e5m2", *g.shape), mx.MxTensor.empty("e5m2", *g.shape)
    h = mx.swiglu(to_dev(gb), to_dev(ub), g8, u8)
    want = g * logistic(g) * u64
    assert near(h, want, np.where(g < -top, 0.0, bound(want, g * u64)))
    # from the checkpoint, whose gates there are -64, -80 and -96: the last above -88.7
    # are kept in E4M3
    for fmt, gates in (("e5m2", (-64.0, -80.0, -96.0)), ("e4m3", (-72.0, -80.0, -88.0))):
        e = np.repeat(np.array(gates), 32)[None, :]
        eb = bits_of(torch.from_numpy(e.astype(np.float32)).to(torch.bfloat16))
        ub = bits_of(torch.full(e.shape, u).to(torch.bfloat16))
        g8, u8 = mx.MxTensor.empty(fmt, *e.shape), mx.MxTensor.empty(fmt, *e.shape)
        mx.swiglu(to_dev(eb), to_dev(ub), g8, u8)
        vg, vu = mx.dequantize(g8).double().cpu().numpy(), mx.dequantize(u8).double().cpu().numpy()
        assert np.array_equal(vg, e)
        d = torch.full(e.shape, 0.75, device="cuda").to(torch.bfloat16)
        dg, du, h = torch.empty_like(d), torch.empty_like(d), torch.empty_like(d)
        mx.swiglu_backward(g8, u8, d, dg, du, h=h)
        s = logistic(vg)
        for got, want, factor in ((h, vg * s * vu, vg * vu), (du, 0.75 * vg * s, vg),
                                  (dg, 0.75 * vu * s * (1 + vg * (1 - s)), vu * (1 + np.abs(vg)))):
            assert near(got, want, np.where(vg < -top, 0.0, bound(want, factor)))
