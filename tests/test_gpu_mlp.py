"""The gated MLP on microscaled operands: every product of its forward and
backward pass against 64-bit arithmetic on the same quantised operands, its
gradients against differences of the loss it then computes, and weights that
come out of the compressed gather."""
import numpy as np
import pytest
import torch

import mx_ref as ref
from test_gpu_mx import U16, U23, bits_of, near, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mlp():
    from lossless_bf16_exponent_codec_gb300 import build
    build.build()
    from lossless_bf16_exponent_codec_gb300 import mlp
    return mlp


def bf16(rng, *shape, scale=1.0):
    return to_dev(bits_of(torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16)))


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def q(x, fmt):
    return ref.quantize(x, fmt)[2]


@pytest.mark.parametrize("T,K,F", [(1, 64, 96), (37, 100, 65), (200, 256, 384)])
def test_step_against_64_bits(mlp, T, K, F):
    """Each stage from the stage before as the GPU rounded it, so that the bounds
    are those of one product: (K + 2) 2^-23 sum|a b| before rounding."""
    from lossless_bf16_exponent_codec_gb300 import mx
    rng = np.random.default_rng(T)
    w1, w2 = bf16(rng, 2 * F, K, scale=0.1), bf16(rng, K, F, scale=0.1)
    x, dy = bf16(rng, T, K), bf16(rng, T, K, scale=1e-3)
    m = mlp.GatedMLP(w1, w2)
    y, kept = m.forward(x)
    dx = m.backward(dy, kept)
    assert int(m.status.item()) == 0

    def product(a, b):
        return a @ b.T, (a.shape[1] + 2) * U23 * (np.abs(a) @ np.abs(b).T)

    # forward: the checkpoint holds the products' results in 8 bits
    x64, w164, w264 = f64(x), f64(w1), f64(w2)
    gu, off = product(q(x64, "e2m1"), q(w164, "e2m1"))
    x4 = mx.MxTensor.empty("e2m1", T, K)
    mx.quantize(x, row=x4)
    gu_gpu = mx.matmul(x4, m.w1)
    assert near(gu_gpu, gu, off)
    g64, u64 = f64(gu_gpu)[:, :F], f64(gu_gpu)[:, F:]
    vg, vu = q(g64, "e4m3"), q(u64, "e4m3")
    assert np.array_equal(f64(mx.dequantize(kept.gate)), vg) and np.array_equal(f64(mx.dequantize(kept.up)), vu)
    assert np.array_equal(f64(mx.dequantize(kept.x)), q(x64.T, "e4m3"))
    h = mx.swiglu(gu_gpu[:, :F], gu_gpu[:, F:], kept.gate, kept.up)
    want = ref.silu_parts(g64)[1] * u64
    assert near(h, want, U16 * np.abs(want))
    assert near(y, *product(q(f64(h), "e2m1"), q(w264, "e2m1")))
    # backward
    dh, off = product(q(f64(dy), "e5m2"), q(w264.T, "e4m3"))
    dy_row = mx.MxTensor.empty("e5m2", T, K)
    mx.quantize(dy, row=dy_row)
    dh_gpu = mx.matmul(dy_row, m.w2t)
    assert near(dh_gpu, dh, off)
    s, a = ref.silu_parts(vg)
    d64 = f64(dh_gpu)
    dgu = torch.empty(T, 2 * F, dtype=torch.bfloat16, device="cuda")
    h2 = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    mx.swiglu_backward(kept.gate, kept.up, dh_gpu, dgu[:, :F], dgu[:, F:], h=h2)
    assert near(h2, a * vu, U16 * np.abs(a * vu))
    assert near(dgu[:, F:], d64 * a, U16 * np.abs(d64 * a))
    assert near(dgu[:, :F], d64 * vu * s * (1 + vg * (1 - s)), U16 * np.abs(d64 * vu) * s * (1 + np.abs(vg) * (1 - s)))
    want, off = product(q(f64(dy).T, "e5m2"), q(f64(h2).T, "e4m3"))
    assert (np.abs(f64(m.d_down) - want) <= off).all()
    want, off = product(q(f64(dgu).T, "e5m2"), q(x64.T, "e4m3"))
    assert (np.abs(f64(m.d_gate_up) - want) <= off).all()
    assert near(dx, *product(q(f64(dgu), "e5m2"), q(w164.T, "e4m3")))
    # a second pass adds the same gradients again, in one FP32 addition each
    first = m.d_down.clone(), m.d_gate_up.clone()
    m.backward(dy, kept)
    assert torch.allclose(m.d_down, 2 * first[0], rtol=2.0 ** -22, atol=0)
    assert torch.allclose(m.d_gate_up, 2 * first[1], rtol=2.0 ** -22, atol=0)
    # without a checkpoint the result is the same
    y2, none = m.forward(x, keep=False)
    assert none is None and torch.equal(y2, y)


def test_gradient_against_differences(mlp):
    """Along the weight gradient itself the exact MLP's loss falls by what the
    gradient promises, up to the 8- and 4-bit operands' relative error (at most
    1/4 for the E2M1 values of the forward pass and 1/8 for the E5M2 gradients):
    the measured slope lies between half and one and a half of |d|^2."""
    rng = np.random.default_rng(3)
    T, K, F = 256, 128, 256
    w1, w2 = bf16(rng, 2 * F, K, scale=0.1), bf16(rng, K, F, scale=0.1)
    x, target = bf16(rng, T, K), bf16(rng, T, K)
    m = mlp.GatedMLP(w1, w2)
    y, kept = m.forward(x)
    m.backward(((y.float() - target.float()) / T).to(torch.bfloat16), kept)
    x64, t64, a, b = f64(x), f64(target), f64(w1), f64(w2)

    def loss(a, b):
        g, u = x64 @ a[:F].T, x64 @ a[F:].T
        return ((ref.silu_parts(g)[1] * u @ b.T - t64) ** 2).sum() / (2 * T)

    for d, at in ((f64(m.d_gate_up), lambda e: (a + e, b)), (f64(m.d_down), lambda e: (a, b + e))):
        e = 1e-4 / np.abs(d).max()
        slope = (loss(*at(e * d)) - loss(*at(-e * d))) / (2 * e)
        assert 0.5 <= slope / (d * d).sum() <= 1.5


@pytest.mark.parametrize("W", [1, 4])
def test_weights_from_the_gather(mlp, W):
    from lossless_bf16_exponent_codec_gb300.codec import Codec
    K, F = 96, 160
    n = 3 * F * K
    shards = bf16(np.random.default_rng(W), n, scale=0.02)
    c = Codec(n, W)
    c.stats(shards)
    c.encode_code3(shards)
    flat = c.gather_decode(*c.exchange())
    assert c.status_word() == 0
    a = mlp.GatedMLP(*mlp.gathered(flat, K, F))
    b = mlp.GatedMLP(shards[:2 * F * K].view(2 * F, K), shards[2 * F * K:].view(K, F))
    x = bf16(np.random.default_rng(9), 33, K)
    assert torch.equal(a.forward(x)[0], b.forward(x)[0])


def test_refuses_other_shapes(mlp):
    with pytest.raises(ValueError, match="gated MLP"):
        mlp.GatedMLP(torch.zeros(64, 32, dtype=torch.bfloat16, device="cuda"),
                     torch.zeros(32, 33, dtype=torch.bfloat16, device="cuda"))


def test_time_outs_are_told(mlp):
    """A pass whose products gave up says so, until the status is cleared."""
    from lossless_bf16_exponent_codec_gb300 import binding as B
    rng = np.random.default_rng(5)
    m = mlp.GatedMLP(bf16(rng, 192, 64, scale=0.1), bf16(rng, 64, 96, scale=0.1))
    x = bf16(rng, 40, 64)
    y, kept = m.forward(x)
    dx = m.backward(y, kept)
    assert m.status_word() == 0
    for step in (lambda: m.forward(x), lambda: m.backward(y, kept)):
        try:
            B.ez_mx_wait_limit(0)
            step()
        finally:
            B.ez_mx_wait_limit()
        assert m.status_word() == 8
        m.forward(x)
        assert m.status_word() == 8
        m.clear_status()
    again, kept = m.forward(x)
    assert torch.equal(again, y) and torch.equal(m.backward(y, kept), dx) and m.status_word() == 0
