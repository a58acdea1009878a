"""Layers of gated experts, and of a gated MLP, with the norm in front: every stage
against 64-bit arithmetic on what the GPU gave it, gradients against differences of
the loss, captured and replayed steps, streams, weights out of the compressed
gather."""
import numpy as np
import pytest
import torch

import moe_ref
import mx_ref as ref
from test_gpu_moe import U24, choices
from test_gpu_mx import U16, U23, bits_of, mx, near, to_dev  # noqa: F401  (mx: the fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe(mx):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import moe
    return moe


@pytest.fixture(scope="module")
def mlp(mx):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import mlp
    return mlp


def bf16(rng, *shape, scale=1.0, mean=0.0):
    return to_dev(bits_of(torch.from_numpy((mean + scale * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16)))


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def q(x, fmt):
    return ref.quantize(x, fmt)[2]


def product(a, b):
    return a @ b.T, (a.shape[1] + 2) * U23 * (np.abs(a) @ np.abs(b).T)


def setting(rng, T, k, E, K, F, kind="some"):
    """gate_up, down, norm, x, residual, ids, weights"""
    ids = torch.from_numpy(choices(rng, T, k, E, kind)).cuda()
    w = torch.softmax(torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)), 1).cuda()
    return (bf16(rng, E, 2 * F, K, scale=0.1), bf16(rng, E, K, F, scale=0.1), bf16(rng, K, scale=0.1, mean=1.0), bf16(rng, T, K),
            bf16(rng, T, K), ids, w)


@pytest.mark.parametrize("T,k,E,K,F", [(1, 2, 4, 64, 96), (70, 3, 5, 100, 65), (300, 2, 3, 256, 160)])
@pytest.mark.parametrize("kind", ["some", "dropped"])
def test_step_against_64_bits(mx, moe, T, k, E, K, F, kind):  # noqa: F811
    rng = np.random.default_rng(T)
    gate_up, down, norm, x, res, ids, w = setting(rng, T, k, E, K, F, kind)
    dy, dtotal = bf16(rng, T, K, scale=1e-3), bf16(rng, T, K, scale=1e-3)
    layer = moe.ExpertMLP(gate_up, down, norm)
    y, kept = layer.forward(x, ids, w, residual=res)
    dx, dw = layer.backward(dy, kept, dtotal=dtotal)
    assert layer.status_word() == 0
    counts, offsets, slots, sources = moe_ref.routing(ids.cpu().numpy(), E)
    used = int(offsets[-1])
    w64, w1, w2 = w.cpu().numpy().astype(np.float64), f64(gate_up), f64(down)
    # the norm
    t64 = ref.round_bf16(f64(x) + f64(res))
    assert np.array_equal(f64(kept.total), t64)
    h0 = torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    mx.rms_norm(x, norm, residual=res, out=h0)
    n64 = f64(h0)
    want = t64 * moe_ref.rms(t64, 1e-6)[:, None] * f64(norm)
    assert near(h0, want, 2.0 ** -20 * np.abs(want))
    # there: forms, products, gated unit
    g = moe_ref.ordered(n64, sources, k)
    assert np.array_equal(f64(mx.dequantize(kept.x))[:, :used], q(g.T, "e4m3")[:, :used])
    vg, vu = f64(mx.dequantize(kept.gate))[:used], f64(mx.dequantize(kept.up))[:used]
    x4 = mx.MxTensor.empty("e2m1", kept.routing.rows, K)
    moe.dispatch(h0, kept.routing, row=x4)
    gu = moe.expert_matmul(x4, layer.w1, kept.routing)
    rows = f64(kept.rows)[:used]
    h = f64(mx.swiglu(gu[:, :F], gu[:, F:], mx.MxTensor.empty("e4m3", kept.routing.rows, F), mx.MxTensor.empty("e4m3", kept.routing.rows, F)))[:used]
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if lo == hi:
            continue
        want, off = product(q(g[lo:hi], "e2m1"), q(w1[e], "e2m1"))
        assert near(gu[lo:hi], want, off)
        g64 = f64(gu[lo:hi])
        assert np.array_equal(vg[lo:hi], q(g64[:, :F], "e4m3")) and np.array_equal(vu[lo:hi], q(g64[:, F:], "e4m3"))
        want = ref.silu_parts(g64[:, :F])[1] * g64[:, F:]
        assert ref.is_rounding_near(h[lo:hi], want, U16 * np.abs(want))
        want, off = product(q(h[lo:hi], "e2m1"), q(w2[e], "e2m1"))
        assert ref.is_rounding_near(rows[lo:hi], want, off)
        assert (rows[lo + counts[e]:hi] == 0).all()
    want, mag = moe_ref.combine(rows, slots, w64)
    assert near(y, want, k * U24 * mag)
    # and back
    d64 = f64(dy)
    for j in range(k):
        some = slots[:, j] >= 0
        terms = d64[some] * rows[slots[some, j]]
        assert (np.abs(f64(dw)[some, j] - terms.sum(axis=1)) <= 16 * U24 * np.abs(terms).sum(axis=1)).all()
        assert (f64(dw)[~some, j] == 0).all()
    dg = torch.from_numpy(moe_ref.ordered(d64, sources, k).astype(np.float32)
                          * np.where(sources >= 0, w.cpu().numpy().reshape(-1)[sources], 1)[:, None]).to(torch.bfloat16).double().numpy()
    row = mx.MxTensor.empty("e5m2", kept.routing.rows, K)
    moe.dispatch(dy, kept.routing, row=row, weights=w)
    dh = moe.expert_matmul(row, layer.w2t, kept.routing)
    R = kept.routing.rows
    dgu, h2 = torch.empty(R, 2 * F, dtype=torch.bfloat16, device="cuda"), torch.empty(R, F, dtype=torch.bfloat16, device="cuda")
    mx.swiglu_backward(kept.gate, kept.up, dh, dgu[:, :F], dgu[:, F:], h=h2)
    dgu64, h64 = f64(dgu)[:used], f64(h2)[:used]
    back = np.zeros((used, K))
    back_off = np.zeros((used, K))
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        want, off = product(q(dg[lo:hi].T, "e5m2"), q(h64[lo:hi].T, "e4m3")) if hi > lo else (np.zeros((K, F)), 0.0)
        assert (np.abs(f64(layer.d_down[e]) - want) <= off).all()
        want, off = product(q(dgu64[lo:hi].T, "e5m2"), q(g[lo:hi].T, "e4m3")) if hi > lo else (np.zeros((2 * F, K)), 0.0)
        assert (np.abs(f64(layer.d_gate_up[e]) - want) <= off).all()
        if hi > lo:
            want, off = product(q(dg[lo:hi], "e5m2"), q(w2[e].T, "e4m3"))
            assert near(dh[lo:hi], want, off)
            back[lo:hi], back_off[lo:hi] = product(q(dgu64[lo:hi], "e5m2"), q(w1[e].T, "e4m3"))
    # the rows' gradients are rounded to BF16 before they are added up, and so is their sum: BF16
    # has 8 significant bits, steps of 2^-7 of a power of two, so a rounding is off by 2^-8 at most
    back_off += 2.0 ** -8 * (np.abs(back) + back_off)
    dn, mag = moe_ref.combine(back, slots)
    off = moe_ref.combine(back_off, slots)[0] + k * U24 * mag
    off += 2.0 ** -8 * (np.abs(dn) + off)
    n, r = t64 * f64(kept.rstd)[:, None], f64(kept.rstd)[:, None]
    want, want_norm = moe_ref.rms_backward(dn, t64, f64(kept.rstd), f64(norm), f64(dtotal))
    gn = np.abs(dn * f64(norm))
    through = off * np.abs(f64(norm))                 # to first order, and 2^-16 for what FP32 does
    off_dx = r * (through + np.abs(n) * (through * np.abs(n)).mean(axis=1, keepdims=True)) \
        + U16 * (r * (gn + np.abs(n) * (gn * np.abs(n)).mean(axis=1, keepdims=True)) + np.abs(f64(dtotal)))
    assert near(dx, want, off_dx)
    assert (np.abs(f64(layer.d_norm) - want_norm) <= ((off + U16 * np.abs(dn)) * np.abs(n)).sum(axis=0)).all()
    # a second pass adds the same gradients again; without a checkpoint the result is the same
    first = layer.d_gate_up.clone(), layer.d_down.clone(), layer.d_norm.clone()
    layer.backward(dy, kept, dtotal=dtotal)
    for got, once in zip((layer.d_gate_up, layer.d_down, layer.d_norm), first):
        assert torch.allclose(got, 2 * once, rtol=2.0 ** -22, atol=0)
    total = torch.empty_like(x)
    y2, none = layer.forward(x, ids, w, keep=False, residual=res, total=total)
    assert none is None and torch.equal(y2, y) and torch.equal(total, kept.total)


def test_experts_gradient_against_differences(moe):
    """As of the gated MLP: along each gradient the exact loss falls by what it promises, up to
    the operands' relative errors: between half and one and a half of |d|^2."""
    rng = np.random.default_rng(3)
    T, k, E, K, F = 300, 2, 3, 128, 160
    gate_up, down, norm, x, res, ids, w = setting(rng, T, k, E, K, F)
    target = bf16(rng, T, K)
    layer = moe.ExpertMLP(gate_up, down, norm)
    y, kept = layer.forward(x, ids, w, residual=res)
    dx, dw = layer.backward(((y.float() - target.float()) / T).to(torch.bfloat16), kept)
    x64, r64, t64, a, b, m, c = (f64(v) for v in (x, res, target, gate_up, down, norm, w))
    idn = ids.cpu().numpy()

    def loss(x=x64, a=a, b=b, m=m, c=c):
        t = x + r64
        h = t * moe_ref.rms(t, 1e-6)[:, None] * m
        out = np.zeros((T, K))
        for e in range(E):
            for j in range(k):
                s = idn[:, j] == e
                g, u = h[s] @ a[e][:F].T, h[s] @ a[e][F:].T
                out[s] += c[s, j, None] * (ref.silu_parts(g)[1] * u @ b[e].T)
        return ((out - t64) ** 2).sum() / (2 * T)

    for d, name, at in ((f64(layer.d_gate_up), "a", a), (f64(layer.d_down), "b", b), (f64(layer.d_norm), "m", m), (f64(dx), "x", x64),
                        (f64(dw), "c", c)):
        e = 1e-4 / np.abs(d).max()
        slope = (loss(**{name: at + e * d}) - loss(**{name: at - e * d})) / (2 * e)
        assert 0.5 <= slope / (d * d).sum() <= 1.5, name


@pytest.mark.parametrize("T,K,F", [(1, 64, 96), (37, 100, 65), (200, 256, 384)])
def test_gated_mlp_with_a_norm(mx, mlp, T, K, F):  # noqa: F811
    """The norm in front of the gated MLP: as the MLP on the norm's result, and the norm's
    gradients of what that gives back."""
    rng = np.random.default_rng(T + 1)
    w1, w2, norm = bf16(rng, 2 * F, K, scale=0.1), bf16(rng, K, F, scale=0.1), bf16(rng, K, scale=0.1, mean=1.0)
    x, res, dy, dt = bf16(rng, T, K), bf16(rng, T, K), bf16(rng, T, K, scale=1e-3), bf16(rng, T, K, scale=1e-3)
    m, plain = mlp.GatedMLP(w1, w2, norm=norm), mlp.GatedMLP(w1, w2)
    h = torch.empty_like(x)
    total, rstd = mx.rms_norm(x, norm, residual=res, out=h)
    y, kept = m.forward(x, residual=res)
    want, plain_kept = plain.forward(h)
    assert torch.equal(y, want) and torch.equal(kept.total, total) and torch.equal(kept.rstd, rstd)
    dx, dh = m.backward(dy, kept, dtotal=dt), plain.backward(dy, plain_kept)
    dnorm = torch.empty(K, device="cuda")
    assert torch.equal(dx, mx.rms_norm_backward(dh, total, rstd, norm, dtotal=dt, dweight=dnorm))
    assert torch.equal(m.d_norm, dnorm) and torch.equal(m.d_gate_up, plain.d_gate_up) and torch.equal(m.d_down, plain.d_down)
    y2, none = m.forward(x, keep=False, residual=res, total=x)         # decoding: the stream in place
    assert none is None and torch.equal(y2, y) and torch.equal(x, total)


def test_captured_step(moe):
    """A step in a graph: replayed on other tokens, other choices and other weights of them, it
    gives what an eager step gives."""
    rng = np.random.default_rng(8)
    T, k, E, K, F = 200, 2, 6, 128, 96
    gate_up, down, norm, x, res, ids, w = setting(rng, T, k, E, K, F)
    dy = bf16(rng, T, K, scale=1e-3)
    layer = moe.ExpertMLP(gate_up, down, norm)

    def step():
        y, kept = layer.forward(x, ids, w, residual=res)
        dx, dw = layer.backward(dy, kept)
        return y, dx, dw

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    sums = layer.d_gate_up, layer.d_down, layer.d_norm
    for seed in (1, 2):
        rng = np.random.default_rng(seed)
        _, _, _, x2, res2, ids2, w2 = setting(rng, T, k, E, K, F, "dropped" if seed == 2 else "some")
        for to, of in ((x, x2), (res, res2), (ids, ids2), (w, w2)):
            to.copy_(of)
        for s in sums:
            s.zero_()
        want = [t.clone() for t in step()] + [s.clone() for s in sums]
        for s in sums:
            s.zero_()
        for o in outs:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for got, exact in zip(list(outs) + list(sums), want):
            assert torch.equal(got, exact)
    assert layer.status_word() == 0


def test_two_layers_on_two_streams(moe):
    """Steps of two layers that overlap on the GPU give what they give alone."""
    rng = np.random.default_rng(9)
    made = []
    for T, k, E, K, F in ((700, 2, 5, 256, 200), (900, 4, 16, 128, 96)):
        gate_up, down, norm, x, res, ids, w = setting(rng, T, k, E, K, F)
        made.append((moe.ExpertMLP(gate_up, down, norm), x, res, ids, w, bf16(rng, T, K, scale=1e-3)))

    def step(layer, x, res, ids, w, dy):
        y, kept = layer.forward(x, ids, w, residual=res)
        return (y,) + layer.backward(dy, kept)

    alone = [step(*m) for m in made]
    sums = [[s.clone() for s in (m[0].d_gate_up, m[0].d_down, m[0].d_norm)] for m in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(5):
        for m in made:
            for s in (m[0].d_gate_up, m[0].d_down, m[0].d_norm):
                s.zero_()
        torch.cuda.synchronize()
        got = []
        for m, stream in zip(made, streams):
            with torch.cuda.stream(stream):
                got.append(step(*m))
        torch.cuda.synchronize()
        for g, a, m, s in zip(got, alone, made, sums):
            assert all(torch.equal(p, q) for p, q in zip(g, a))
            assert all(torch.equal(p, q) for p, q in zip((m[0].d_gate_up, m[0].d_down, m[0].d_norm), s))


@pytest.mark.parametrize("W", [1, 4])
def test_weights_from_the_gather(moe, W):
    from lossless_bf16_exponent_codec_gb300.codec import Codec
    E, K, F = 4, 96, 64
    n = 3 * E * F * K + K
    shards = bf16(np.random.default_rng(W), n, scale=0.02)
    shards[-K:] = 1.0
    c = Codec(n, W)
    c.stats(shards)
    c.encode_code3(shards)
    flat = c.gather_decode(*c.exchange())
    assert c.status_word() == 0
    m = 2 * E * F * K
    a = moe.ExpertMLP(*moe.gathered(flat, E, K, F))
    b = moe.ExpertMLP(shards[:m].view(E, 2 * F, K), shards[m:m + m // 2].view(E, K, F), shards[m + m // 2:])
    rng = np.random.default_rng(9)
    x, ids = bf16(rng, 33, K), torch.from_numpy(choices(rng, 33, 2, E)).cuda()
    w = torch.full((33, 2), 0.5, device="cuda")
    assert torch.equal(a.forward(x, ids, w)[0], b.forward(x, ids, w)[0])


def test_no_tokens(moe):
    """An empty batch: nothing comes out and nothing is added."""
    rng = np.random.default_rng(1)
    gate_up, down, norm, x, res, ids, w = setting(rng, 4, 2, 3, 64, 96)
    layer = moe.ExpertMLP(gate_up, down, norm)
    y, kept = layer.forward(x[:0], ids[:0], w[:0], residual=res[:0])
    dx, dw = layer.backward(y, kept)
    assert y.shape == (0, 64) and dx.shape == (0, 64) and dw.shape == (0, 2) and layer.status_word() == 0
    assert all(bool((s == 0).all()) for s in (layer.d_gate_up, layer.d_down, layer.d_norm))


def test_time_outs_are_told(moe):
    from lossless_bf16_exponent_codec_gb300 import binding as B
    rng = np.random.default_rng(5)
    gate_up, down, norm, x, res, ids, w = setting(rng, 40, 2, 3, 64, 96)
    layer = moe.ExpertMLP(gate_up, down)
    y, kept = layer.forward(x, ids, w)
    dx, _ = layer.backward(y, kept)
    assert layer.status_word() == 0
    for step in (lambda: layer.forward(x, ids, w), lambda: layer.backward(y, kept)):
        try:
            B.ez_mx_wait_limit(0)
            step()
        finally:
            B.ez_mx_wait_limit()
        assert layer.status_word() == 8
        layer.clear_status()
    again, kept = layer.forward(x, ids, w)
    assert torch.equal(again, y) and torch.equal(layer.backward(y, kept)[0], dx) and layer.status_word() == 0


def test_what_goes_with_a_norm(moe, mlp):
    rng = np.random.default_rng(5)
    gate_up, down, norm, x, res, ids, w = setting(rng, 4, 2, 3, 64, 96)
    layer, dense = moe.ExpertMLP(gate_up, down), mlp.GatedMLP(gate_up[0], down[0])
    for call in (lambda: layer.forward(x, ids, w, residual=res), lambda: dense.forward(x, residual=res),
                 lambda: layer.backward(x, None, dtotal=x), lambda: dense.backward(x, None, dtotal=x)):
        with pytest.raises(ValueError, match="norm"):
            call()
    with pytest.raises(ValueError, match="gated experts"):
        moe.ExpertMLP(gate_up, down[:, :, :5])
