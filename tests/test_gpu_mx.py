"""Microscaled operators on the GPU against the plain 64-bit implementation.

Codes, scales and decoded values are compared exactly.  Products: with the
element products exact in FP32 and K sums each off by at most one unit in the
last place of a partial sum (2^-23 of the sum of magnitudes, which also covers
sums that truncate), |error| <= (K + 2) 2^-23 sum|a b| before C is rounded.
The gated unit: exp, the division and the products are off by a few 2^-23 and
the exponent's argument by |g| 2^-23, together under 2^-16 for |g| < 64.  A
BF16 result has to be the rounding of a number within these bounds."""
import numpy as np
import pytest
import torch

import mx_ref as ref

pytestmark = pytest.mark.gpu
U23, U16 = 2.0 ** -23, 2.0 ** -16
FORMATS = ["e2m1", "e4m3", "e5m2"]
PAIRS = [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")]


@pytest.fixture(scope="module")
def mx():
    from lossless_bf16_exponent_codec_gb300 import build
    build.build()
    from lossless_bf16_exponent_codec_gb300 import mx
    return mx


def to_dev(bits: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def bits_of(t: torch.Tensor) -> np.ndarray:
    return t.detach().contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def random_bits(rng, rows, cols, spread=2.0):
    x = rng.standard_normal((rows, cols)) * np.exp(spread * rng.standard_normal((rows, 1)))
    x[:, rng.random(cols) < 0.05] *= 50
    return bits_of(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16))


def fill(mx, fmt, bits):
    """The row form of a BF16 matrix, and its values in 64 bits."""
    t = mx.MxTensor.empty(fmt, *bits.shape)
    mx.quantize(to_dev(bits), row=t)
    return t, ref.quantize(ref.bf16_to_f64(bits), fmt)[2]


def check_form(t, x64, fmt):
    code, scale, value = ref.quantize(x64, fmt)
    assert np.array_equal(t.codes.cpu().numpy(), code)
    assert np.array_equal(t.scales.cpu().numpy(), scale)
    return value


def same(got: torch.Tensor, want: np.ndarray):
    """A BF16 tensor holds exactly these values (NaN where they are NaN)."""
    assert np.array_equal(got.float().cpu().numpy().astype(np.float64), want, equal_nan=True)


def near(got: torch.Tensor, want: np.ndarray, off: np.ndarray) -> bool:
    return ref.is_rounding_near(got.float().cpu().numpy(), want, off)


# ------------------------------------------------------------ quantisation

@pytest.mark.parametrize("R,C", [(1, 1), (1, 31), (1, 5120), (3, 33), (32, 32), (31, 129), (128, 128), (129, 127),
                                 (257, 1000), (640, 96)])
@pytest.mark.parametrize("row,col", [("e2m1", None), (None, "e4m3"), ("e2m1", "e2m1"), ("e2m1", "e4m3"),
                                     ("e4m3", "e5m2"), ("e5m2", "e2m1")])
def test_quantize(mx, R, C, row, col):
    bits = random_bits(np.random.default_rng(R * 7919 + C), R, C)
    x64 = ref.bf16_to_f64(bits)
    r = mx.MxTensor.empty(row, R, C) if row else None
    c = mx.MxTensor.empty(col, C, R) if col else None
    for t in (r, c):          # what is there before does not matter
        if t is not None:
            t.codes.fill_(0xA5)
            t.scales.fill_(0xA5)
    mx.quantize(to_dev(bits), row=r, col=c)
    for t, x, fmt in ((r, x64, row), (c, x64.T, col)):
        if t is not None:
            same(mx.dequantize(t), check_form(t, x, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
def test_every_bf16_amax(mx, fmt):
    """One block per non-negative BF16 bit pattern (infinity and NaNs too), the
    pattern its largest magnitude; the rest of the block smaller."""
    pat = np.arange(0x8000, dtype=np.uint16)
    bits = np.zeros((len(pat), 32), np.uint16)
    bits[:, 5] = pat
    bits[:, 6] = pat | 0x8000
    for j in range(7, 32):
        bits[:, j] = np.maximum(pat.astype(np.int64) - 37 * (j - 6), 0).astype(np.uint16) | (0x8000 * (j & 1))
    t = mx.MxTensor.empty(fmt, len(pat), 32)
    mx.quantize(to_dev(bits), row=t)
    same(mx.dequantize(t), check_form(t, ref.bf16_to_f64(bits), fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("k", [0, -100, 100])
def test_every_value_of_a_block(mx, fmt, k):
    """Every BF16 value not above F 2^k, in blocks whose scale F 2^k fixes: all
    roundings and ties of the format, subnormals among them."""
    F = ref.MAGS[fmt][-1] * 2.0 ** k
    top = int(np.float32(F).view(np.uint32) >> 16)
    vals = np.arange(top + 1, dtype=np.uint16)
    vals = np.concatenate([vals, vals | 0x8000])
    vals = np.concatenate([vals, np.zeros(-len(vals) % 31, np.uint16)]).reshape(-1, 31)
    bits = np.concatenate([np.full((len(vals), 1), top, np.uint16), vals], axis=1)
    r = mx.MxTensor.empty(fmt, *bits.shape)
    mx.quantize(to_dev(bits), row=r)
    c = mx.MxTensor.empty(fmt, *bits.shape)
    mx.quantize(to_dev(bits.T), col=c)
    for t in (r, c):
        same(mx.dequantize(t), check_form(t, ref.bf16_to_f64(bits), fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_infinities_and_nan_mark_their_block(mx, fmt, value):
    bits = random_bits(np.random.default_rng(1), 40, 100)
    x = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).clone()
    x[3, 40] = value
    x[39, 99] = value
    bits = bits_of(x)
    r, c = mx.MxTensor.empty(fmt, 40, 100), mx.MxTensor.empty(fmt, 100, 40)
    mx.quantize(x.cuda(), row=r, col=c)
    v = check_form(r, ref.bf16_to_f64(bits), fmt)
    assert np.isnan(v).sum() == 32 + 4 and np.isnan(v[3, 32:64]).all()
    same(mx.dequantize(r), v)
    same(mx.dequantize(c), check_form(c, ref.bf16_to_f64(bits).T, fmt))


@pytest.mark.parametrize("off,extra", [(0, 0), (1, 0), (0, 1), (3, 5), (7, 2), (5, 8), (8, 16)])
@pytest.mark.parametrize("R,C", [(5, 200), (130, 261), (1, 17)])
def test_any_alignment_and_stride(mx, off, extra, R, C):
    """Rows at every 2-byte alignment and row strides above the width; nothing
    outside the matrix is read into it or written."""
    rng = np.random.default_rng(off * 31 + extra)
    ld = C + extra
    bits = random_bits(rng, R, C)
    buf = torch.full((off + R * ld + 9,), float("nan"), dtype=torch.bfloat16, device="cuda")
    view = buf[off:off + R * ld].as_strided((R, C), (ld, 1))
    view.copy_(to_dev(bits))
    r, c = mx.MxTensor.empty("e2m1", R, C), mx.MxTensor.empty("e4m3", C, R)
    mx.quantize(view, row=r, col=c)
    x64 = ref.bf16_to_f64(bits)
    v = check_form(r, x64, "e2m1")
    check_form(c, x64.T, "e4m3")
    out = torch.full_like(buf, 7.0)
    ov = out[off:off + R * ld].as_strided((R, C), (ld, 1))
    mx.dequantize(r, out=ov)
    same(ov, v)
    ov.fill_(7.0)
    assert bool((out == 7.0).all())


def test_sizes_of_zero(mx):
    for R, C in ((0, 5), (5, 0), (0, 0)):
        x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
        r, c = mx.MxTensor.empty("e2m1", R, C), mx.MxTensor.empty("e4m3", C, R)
        mx.quantize(x, row=r, col=c)
        assert mx.dequantize(r).shape == (R, C)
        h = mx.swiglu(x, x, mx.MxTensor.empty("e4m3", R, C), mx.MxTensor.empty("e4m3", R, C))
        assert h.shape == (R, C)
    a, b = mx.MxTensor.empty("e4m3", 3, 0), mx.MxTensor.empty("e4m3", 40, 0)
    assert bool((mx.matmul(a, b) == 0).all())
    add = torch.randn(3, 40, device="cuda")
    assert torch.equal(mx.matmul(a, b, add=add), add)
    e = mx.MxTensor.empty("e4m3", 0, 64)
    f = mx.MxTensor.empty("e4m3", 5, 64)
    assert mx.matmul(e, f).shape == (0, 5) and mx.matmul(f, e).shape == (5, 0)


def test_more_than_32_bits_of_values(mx):
    """A matrix of over 2^32 values: its last rows and columns are those of the
    same values alone."""
    R, C = 65800, 65600
    x = torch.zeros(R, C, dtype=torch.bfloat16, device="cuda")
    bits = random_bits(np.random.default_rng(8), 200, C)
    x[-200:] = to_dev(bits)
    big = mx.MxTensor.empty("e2m1", R, C)
    mx.quantize(x, row=big)
    code, _, value = ref.quantize(ref.bf16_to_f64(bits), "e2m1")
    assert np.array_equal(big.codes[-200:].cpu().numpy(), code)
    same(mx.dequantize(big, out=x)[-200:], value)
    assert bool((x[:-200:997] == 0).all())


# ------------------------------------------------------------------ product

def check_product(mx, fa, fb, M, N, K, out, add, seed=0, ld=None):
    rng = np.random.default_rng(seed + M * 131 + N * 17 + K)
    A, va = fill(mx, fa, random_bits(rng, M, K, 0.5))
    Bt, vb = fill(mx, fb, random_bits(rng, N, K, 0.5))
    want = va @ vb.T
    mass = np.abs(va) @ np.abs(vb).T
    kind = torch.bfloat16 if out == "bf16" else torch.float32
    ld = ld or N
    buf = torch.full((M, ld), 3.0, dtype=kind, device="cuda")
    c = buf[:, :N]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = None
    if add is not None:
        vals = rng.standard_normal((M, N)).astype(np.float32) * np.float32(np.abs(want).mean() + 1)
        if add == "in place":
            c.copy_(torch.from_numpy(vals))
            d = c
        else:
            d = torch.full((M, ld), 9.0, device="cuda")[:, :N]
            d.copy_(torch.from_numpy(vals))
        want = want + vals
        mass = mass + np.abs(vals)
    mx.matmul(A, Bt, out=c, add=d, status=status)
    assert int(status.item()) == 0
    got = c.float().cpu().numpy().astype(np.float64)
    tol = (K + 2) * U23 * mass
    assert ref.is_rounding_near(got, want, tol) if out == "bf16" else (np.abs(got - want) <= tol).all()
    if ld > N:
        assert bool((buf[:, N:] == 3.0).all())
    return A, Bt, c


@pytest.mark.parametrize("M,N,K", [(1, 64, 32), (1, 512, 4096), (2, 100, 33), (5, 300, 1000), (16, 257, 512),
                                   (31, 129, 160), (48, 640, 768), (65, 128, 128), (100, 1000, 520), (128, 128, 256),
                                   (129, 255, 257), (200, 72, 1), (257, 513, 2048), (1000, 33, 96), (384, 1, 400)])
@pytest.mark.parametrize("fa,fb", PAIRS)
def test_product(mx, fa, fb, M, N, K):
    out, add = [("bf16", None), ("f32", None), ("f32", "apart"), ("f32", "in place")][(M + N + K) % 4]
    check_product(mx, fa, fb, M, N, K, out, add)


@pytest.mark.parametrize("out,add", [("bf16", None), ("f32", None), ("f32", "apart"), ("f32", "in place")])
@pytest.mark.parametrize("M,N,K,ld", [(3, 130, 288, 131), (150, 260, 300, 264), (300, 301, 96, 333), (7, 64, 2049, 64)])
def test_product_outputs(mx, out, add, M, N, K, ld):
    check_product(mx, "e2m1", "e2m1", M, N, K, out, add, ld=ld)
    check_product(mx, "e5m2", "e4m3", M, N, K, out, add, ld=ld)


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (700, 900, 8200), (24, 2048, 16384), (2048, 3000, 1024)])
@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e5m2", "e4m3")])
def test_product_long(mx, fa, fb, M, N, K):
    A, Bt, c = check_product(mx, fa, fb, M, N, K, "f32", None)
    again = mx.matmul(A, Bt, dtype=torch.float32)
    assert torch.equal(again, c)           # the order of the sums is fixed


@pytest.mark.parametrize("M,N,K,ld", [(1600, 1664, 300, 1664), (1411, 1700, 1000, 1701), (2304, 1920, 4400, 1936),
                                      (9000, 300, 129, 304), (257, 10001, 640, 10001), (1792, 1792, 33, 1792)])
@pytest.mark.parametrize("fa,fb", [("e2m1", "e2m1"), ("e5m2", "e4m3"), ("e4m3", "e4m3")])
@pytest.mark.parametrize("out,add", [("bf16", None), ("f32", "in place")])
def test_product_many_tiles(mx, fa, fb, M, N, K, ld, out, add):
    check_product(mx, fa, fb, M, N, K, out, add, ld=ld)


@pytest.mark.parametrize("fa", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(4, 200, 700), (300, 200, 700), (1900, 2000, 700)])
def test_product_carries_nan_blocks(mx, fa, M, N, K):
    """A NaN block makes its row of A (its column of C for B) NaN, no other."""
    rng = np.random.default_rng(4)
    x, y = (torch.from_numpy(random_bits(rng, r, K, 0.5).view(np.int16)).view(torch.bfloat16).clone() for r in (M, N))
    x[2, 100] = float("nan")
    y[150, K - 1] = float("inf")
    a, b = mx.MxTensor.empty(fa, M, K), mx.MxTensor.empty(fa, N, K)
    mx.quantize(x.cuda(), row=a)
    mx.quantize(y.cuda(), row=b)
    c = mx.matmul(a, b, dtype=torch.float32).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[2] = True
    want[:, 150] = True
    assert np.array_equal(np.isnan(c), want) and np.isfinite(c[~want]).all()


def test_product_range_of_scales(mx):
    """Blocks of very large and very small scales in one sum."""
    rng = np.random.default_rng(6)
    M, N, K = 40, 70, 256
    ea = rng.integers(-100, 20, (M, K // 32)).repeat(32, axis=1)
    eb = rng.integers(-20, 60, (N, K // 32)).repeat(32, axis=1)
    for fmt in ("e2m1", "e4m3"):
        xa = bits_of(torch.from_numpy((rng.standard_normal((M, K)) * 2.0 ** ea).astype(np.float32)).to(torch.bfloat16))
        xb = bits_of(torch.from_numpy((rng.standard_normal((N, K)) * 2.0 ** eb).astype(np.float32)).to(torch.bfloat16))
        a, va = fill(mx, fmt, xa)
        b, vb = fill(mx, fmt, xb)
        c = mx.matmul(a, b, dtype=torch.float32).cpu().numpy().astype(np.float64)
        assert (np.abs(c - va @ vb.T) <= (K + 2) * U23 * (np.abs(va) @ np.abs(vb).T) + K * 2.0 ** -149).all()


def test_product_of_more_than_32_bits_of_codes(mx):
    """B of over 2^32 code bytes, and C's rows over 2^31 bytes apart: the last
    results are those of B's last rows alone."""
    N, K = 65700, 65600
    x = torch.zeros(N, K, dtype=torch.bfloat16, device="cuda")
    bits = random_bits(np.random.default_rng(9), 100, K, 0.5)
    x[-100:] = to_dev(bits)
    b = mx.MxTensor.empty("e4m3", N, K)
    mx.quantize(x, row=b)
    del x
    a, va = fill(mx, "e4m3", random_bits(np.random.default_rng(10), 3, K, 0.5))
    vb = ref.quantize(ref.bf16_to_f64(bits), "e4m3")[2]
    ld = 1 << 29
    buf = torch.empty(2 * ld + N, device="cuda")
    c = mx.matmul(a, b, out=buf.as_strided((3, N), (ld, 1)))
    got = c[:, -100:].cpu().numpy().astype(np.float64)
    assert (np.abs(got - va @ vb.T) <= (K + 2) * U23 * (np.abs(va) @ np.abs(vb).T)).all()
    assert bool((c[:, :-100] == 0).all())


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("fmt,M,N,K", [("e2m1", 2, 130, 3_200_017), ("e4m3", 150, 20, 1_100_003),
                                       ("e4m3", 3000, 2100, 70_000)])
def test_product_of_small_integers_is_exact(mx, fmt, M, N, K, out):
    """Sums of products of -1, 0 and 1 are integers below 2^24: every order of
    additions gives them exactly, however many segments they take."""
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    x, y = (torch.randint(-1, 2, (r, K), generator=g, device="cuda", dtype=torch.int8) for r in (M, N))
    a, b = mx.MxTensor.empty(fmt, M, K), mx.MxTensor.empty(fmt, N, K)
    mx.quantize(x.to(torch.bfloat16), row=a)
    mx.quantize(y.to(torch.bfloat16), row=b)
    rows = torch.arange(0, M, max(1, M // 40), device="cuda")
    want = sum(x[rows, i:i + 65536].float() @ y[:, i:i + 65536].float().t() for i in range(0, K, 65536))
    kind = torch.bfloat16 if out == "bf16" else torch.float32
    assert torch.equal(mx.matmul(a, b, dtype=kind)[rows], want.to(kind))


# --------------------------------------------------------------- gated unit

@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("R,C,joined", [(1, 32, False), (1, 2731, True), (33, 100, True), (128, 128, False),
                                        (129, 333, True), (300, 1024, True)])
def test_swiglu_and_backward(mx, fmt, R, C, joined):
    rng = np.random.default_rng(R + C)
    gb, ub, db = (random_bits(rng, R, C, 0.7) for _ in range(3))
    g64, u64, d64 = (ref.bf16_to_f64(b) for b in (gb, ub, db))
    g64, gb = np.clip(g64, -60, 60), bits_of(torch.from_numpy(np.clip(g64, -60, 60)).to(torch.bfloat16))
    g64 = ref.bf16_to_f64(gb)
    if joined:
        gu = torch.cat((to_dev(gb), to_dev(ub)), dim=1)
        gate, up = gu[:, :C], gu[:, C:]
    else:
        gate, up = to_dev(gb), to_dev(ub)
    g8, u8 = mx.MxTensor.empty(fmt, R, C), mx.MxTensor.empty(fmt, R, C)
    h = mx.swiglu(gate, up, g8, u8)
    s, a = ref.silu_parts(g64)
    want = a * u64
    assert near(h, want, U16 * np.abs(want))
    vg, vu = check_form(g8, g64, fmt), check_form(u8, u64, fmt)
    dgu = torch.full((R, 2 * C + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    h2 = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    mx.swiglu_backward(g8, u8, to_dev(db), dgu[:, :C], dgu[:, C:2 * C], h=h2)
    s, a = ref.silu_parts(vg)
    want_h, want_u = a * vu, d64 * a
    want_g = d64 * vu * s * (1 + vg * (1 - s))
    loose = U16 * np.abs(d64 * vu) * s * (1 + np.abs(vg) * (1 - s))
    assert near(h2, want_h, U16 * np.abs(want_h))
    assert near(dgu[:, C:2 * C], want_u, U16 * np.abs(want_u))
    assert near(dgu[:, :C], want_g, loose)
    assert bool((dgu[:, 2 * C:] == 5.0).all())
    # and against central differences of h in 64 bits
    e = 1e-6
    f = lambda g, u: ref.silu_parts(g)[1] * u  # noqa: E731
    num_g = d64 * (f(vg + e, vu) - f(vg - e, vu)) / (2 * e)
    num_u = d64 * (f(vg, vu + e) - f(vg, vu - e)) / (2 * e)
    # the differences' own error: e^2 times the third derivative (under 1) and
    # 2^-52 of h over e
    off = np.abs(d64) * (e * e * (1 + np.abs(vu)) + 2.0 ** -50 * (np.abs(want_h) + np.abs(vg) + np.abs(vu) + 1) / e)
    assert near(dgu[:, :C], num_g, loose + 2 * off)
    assert near(dgu[:, C:2 * C], num_u, U16 * np.abs(num_u) + 2 * off)
    # without h the gradients are the same
    dg2, du2 = torch.empty_like(h2), torch.empty_like(h2)
    mx.swiglu_backward(g8, u8, to_dev(db), dg2, du2)
    assert torch.equal(dg2, dgu[:, :C]) and torch.equal(du2, dgu[:, C:2 * C])


def test_swiglu_far_gates(mx):
    """Gates where exp overflows or vanishes: the limits, no NaN."""
    g = torch.tensor([[1e30, -1e30, 100.0, -100.0, 3e38, -3e38, 0.0, -0.0] * 4], device="cuda").to(torch.bfloat16)
    u = torch.full_like(g, 0.5)
    g8, u8 = mx.MxTensor.empty("e5m2", 1, 32), mx.MxTensor.empty("e5m2", 1, 32)
    h = mx.swiglu(g, u, g8, u8).float()
    assert torch.equal(h, (g.clamp(min=0).float() * 0.5).to(torch.bfloat16).float())
    d = torch.ones_like(g)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    for row in ([1e30] * 32, [-1e30] * 32, [100.0] * 32, [-100.0] * 32):
        gg = torch.tensor([row], device="cuda").to(torch.bfloat16)
        mx.swiglu(gg, u, g8, u8)
        mx.swiglu_backward(g8, u8, d, dg, du)
        v = mx.dequantize(g8).float()
        assert torch.equal(dg.float(), (v > 0).float() * 0.5)
        assert torch.equal(du.float(), v.clamp(min=0))


# ------------------------------------------------------- streams and graphs

def test_another_stream_and_a_graph(mx):
    rng = np.random.default_rng(12)
    M, N, K = 70, 300, 512
    w, vw = fill(mx, "e2m1", random_bits(rng, N, K, 0.5))
    x = to_dev(random_bits(rng, M, K, 0.5))
    x4 = mx.MxTensor.empty("e2m1", M, K)
    c = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mx.quantize(x, row=x4)
    mx.matmul(x4, w, out=c, status=status)
    torch.cuda.synchronize()
    first = c.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.zero_()
    side.wait_stream(torch.cuda.current_stream())
    mx.quantize(x, row=x4, stream=side)
    mx.matmul(x4, w, out=c, status=status, stream=side)
    side.synchronize()
    assert torch.equal(c, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.quantize(x, row=x4)
        mx.matmul(x4, w, out=c, status=status)
    bits = random_bits(rng, M, K, 0.5)
    x.copy_(to_dev(bits))
    graph.replay()
    torch.cuda.synchronize()
    va = ref.quantize(ref.bf16_to_f64(bits), "e2m1")[2]
    want, mass = va @ vw.T, np.abs(va) @ np.abs(vw).T
    assert near(c, want, (K + 2) * U23 * mass)
    assert int(status.item()) == 0
