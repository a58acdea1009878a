"""The norm with the residual's addition on the GPU against 64-bit arithmetic.

total is exact (the sum of two BF16 values, rounded once).  y is total weight rstd,
rounded to FP32 and to BF16: sums and rstd are held to some 2^-40, so that this is the
64-bit y's rounding to FP32 but within 2^-16 of a step from an FP32 border, and seen in
BF16 only if that is next to a border there, which no value here is.  rstd is that number
rounded to FP32: off by 2^-24 and a 2^-40th.  The forms are functions of y.  All compared
exactly.

Back: n = total rstd is off by 2^-24, each of the terms g n of c by two more, the sum
by 32 + 9 roundings and c by one of the division: |c's error| <= 46 2^-24 mean|g n|.
dx: four more roundings of numbers under rstd (|g| + |n c|) + |dtotal|.  dweight:
ceil(rows / 304) terms in a thread, at most 76 partial sums of a column in a slice, 32
slices, n's rounding and the addend's."""
import numpy as np
import pytest
import torch

import moe_ref
import mx_ref as ref
from test_gpu_mx import bits_of, check_form, mx, near, random_bits, same, to_dev  # noqa: F401  (mx: the fixture)

pytestmark = pytest.mark.gpu
U24 = 2.0 ** -24


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def weight_bits(rng, C):
    return bits_of(torch.from_numpy((1 + 0.3 * rng.standard_normal(C)).astype(np.float32)).to(torch.bfloat16))


def wide(bits, ld, shift=0):
    """The matrix on the GPU with a row stride of ld, `shift` values into its memory."""
    R, C = bits.shape
    mem = torch.zeros(R * ld + shift + 8, dtype=torch.bfloat16, device="cuda")
    t = mem[shift:shift + R * ld].view(R, ld)[:, :C]
    t.copy_(to_dev(bits))
    return t


def expected_y(t64, eps, wbits):
    """y of total."""
    with np.errstate(all="ignore"):
        y = t64 * ref.bf16_to_f64(wbits) * moe_ref.rms(t64, float(np.float32(eps)))[:, None]
        return f64(torch.from_numpy(y.astype(np.float32)).to(torch.bfloat16))


def form(mx, fmt, R, C):
    t = mx.MxTensor.empty(fmt, R, C)
    t.codes.fill_(0xA5)
    t.scales.fill_(0xA5)
    return t


SIZES = [(1, 1), (1, 8), (3, 33), (1, 2048), (31, 256), (33, 257), (130, 1000), (5, 1024), (129, 1025), (64, 2048), (7, 2049),
         (300, 4096), (3, 4097), (40, 8192), (5, 8191), (2, 16384), (3, 16383)]


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("residual,y,row,col", [(True, True, "e2m1", "e4m3"), (False, True, None, None), (True, False, "e4m3", None),
                                                (False, False, None, "e5m2"), (True, False, "e2m1", "e4m3")])
def test_norm(mx, R, C, residual, y, row, col):
    rng = np.random.default_rng(R * 31 + C)
    xb, wb = random_bits(rng, R, C, 1.0), weight_bits(rng, C)
    rb = random_bits(rng, R, C, 1.0) if residual else None
    eps = 1e-5
    out = torch.full((R, C), 7.0, dtype=torch.bfloat16, device="cuda") if y else None
    r, c = form(mx, row, R, C) if row else None, form(mx, col, C, R) if col else None
    x = to_dev(xb)
    res = to_dev(rb) if residual else None
    total, rstd = mx.rms_norm(x, to_dev(wb), eps, residual=res, out=out, row=r, col=c)
    t64 = ref.bf16_to_f64(xb)
    if residual:
        t64 = ref.round_bf16(t64 + ref.bf16_to_f64(rb))
        same(total, t64)
    else:
        assert total is x and np.array_equal(bits_of(x), xb)
    want = moe_ref.rms(t64, float(np.float32(eps)))
    assert (np.abs(rstd.cpu().numpy().astype(np.float64) - want) <= (2.0 ** -24 + 2.0 ** -40) * want).all()
    y64 = expected_y(t64, eps, wb)
    if y:
        same(out, y64)
    if row:
        same(mx.dequantize(r), check_form(r, y64, row))
    if col:
        same(mx.dequantize(c), check_form(c, y64.T, col))


@pytest.mark.parametrize("R,C,ld,shift", [(70, 256, 264, 0), (70, 250, 256, 0), (37, 1000, 1003, 1), (65, 2048, 2050, 3), (9, 8192, 8200, 8),
                                          (33, 4096, 4097, 5)])
def test_strides_and_alignment(mx, R, C, ld, shift):
    """Every matrix with its own stride and offset; what lies between the rows stays."""
    rng = np.random.default_rng(C)
    xb, rb, wb = random_bits(rng, R, C, 1.0), random_bits(rng, R, C, 1.0), weight_bits(rng, C)
    r, c = form(mx, "e2m1", R, C), form(mx, "e5m2", C, R)
    outs = [torch.full((R, ld + 2 * i), 7.0, dtype=torch.bfloat16, device="cuda") for i in range(2)]
    w = wide(wb[None], C, shift)[0]
    total, rstd = mx.rms_norm(wide(xb, ld, shift), w, 0.0, residual=wide(rb, ld + 1, 0), total=outs[0][:, :C], out=outs[1][:, :C], row=r,
                              col=c)
    t64 = ref.round_bf16(ref.bf16_to_f64(xb) + ref.bf16_to_f64(rb))
    same(total, t64)
    y64 = expected_y(t64, 0.0, wb)
    same(outs[1][:, :C], y64)
    check_form(r, y64, "e2m1")
    check_form(c, y64.T, "e5m2")
    assert all(bool((o[:, C:] == 7.0).all()) for o in outs)


@pytest.mark.parametrize("C", [512, 515, 8192])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_total_in_place(mx, C, which):
    rng = np.random.default_rng(C)
    R = 77
    x, res, w = to_dev(random_bits(rng, R, C)), to_dev(random_bits(rng, R, C)), to_dev(weight_bits(rng, C))
    y, y2 = (torch.empty(R, C, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    c, c2 = form(mx, "e4m3", C, R), form(mx, "e4m3", C, R)
    total, rstd = mx.rms_norm(x, w, residual=res, out=y, col=c)
    mine = {"x": x, "residual": res}[which]
    got, rstd2 = mx.rms_norm(x, w, residual=res, total=mine, out=y2, col=c2)
    assert got is mine and torch.equal(mine, total) and torch.equal(rstd, rstd2) and torch.equal(y, y2)
    assert torch.equal(c.codes, c2.codes) and torch.equal(c.scales, c2.scales)


@pytest.mark.parametrize("R,C", [(33, 512), (33, 515), (9, 8191), (40, 8192)])
@pytest.mark.parametrize("which", ["x", "residual", "x, alone"])
def test_result_in_place(mx, R, C, which):
    """y over x or the residual, at rows on and off 16 bytes (515 and 8191: a granule holds parts of two rows)."""
    rng = np.random.default_rng(C)
    xb, rb, wb = random_bits(rng, R, C, 1.0), random_bits(rng, R, C, 1.0), weight_bits(rng, C)
    x, r = to_dev(xb), to_dev(rb)
    row = form(mx, "e2m1", R, C)
    if which == "x, alone":
        t64 = ref.bf16_to_f64(xb)
        mx.rms_norm(x, to_dev(wb), out=x, row=row)
        col = form(mx, "e4m3", C, R)
        with pytest.raises(RuntimeError, match="ez_mx_rms_norm"):
            mx.rms_norm(x, to_dev(wb), out=x, col=col)
    else:
        t64 = ref.round_bf16(ref.bf16_to_f64(xb) + ref.bf16_to_f64(rb))
        col = form(mx, "e4m3", C, R)
        total, _ = mx.rms_norm(x, to_dev(wb), residual=r, out=x if which == "x" else r, row=row, col=col)
        same(total, t64)
        check_form(col, expected_y(t64, 1e-6, wb).T, "e4m3")
    y64 = expected_y(t64, 1e-6, wb)
    same(r if which == "residual" else x, y64)
    check_form(row, y64, "e2m1")


def test_zero_rows_infinities_and_nan(mx):
    """A row of zeros: y is zero (with eps = 0 NaN, 0 / 0).  A row with an infinity has rstd
    0: zeros, and NaN at the infinity; a row with a NaN is NaN.  The others are as without
    them, but for the blocks of the column form that they share."""
    rng = np.random.default_rng(0)
    R, C = 64, 320
    b, w = random_bits(rng, R, C, 1.0), weight_bits(rng, C)
    b[3] = 0
    b[5, 7], b[6, 9], b[40, 0] = 0x7F80, 0x7FC1, 0xFF80
    for eps in (1e-6, 0.0):
        out, r, c = torch.empty(R, C, dtype=torch.bfloat16, device="cuda"), form(mx, "e2m1", R, C), form(mx, "e4m3", C, R)
        total, rstd = mx.rms_norm(to_dev(b), to_dev(w), eps, out=out, row=r, col=c)
        y64 = expected_y(ref.bf16_to_f64(b), eps, w)
        same(out, y64)
        good = [i for i in range(R) if i not in (3, 5, 6, 40)]
        check_form(r, y64, "e2m1")
        check_form(c, y64.T, "e4m3")
        assert bool((out[3] == 0).all()) if eps else bool(torch.isnan(out[3]).all())
        for row, at in ((5, 7), (40, 0)):
            assert rstd[row] == 0 and bool(torch.isnan(out[row, at])) and int(torch.isnan(out[row]).sum()) == 1
        assert bool(torch.isnan(out[6]).all()) and bool(torch.isfinite(out[good]).all())


def test_large_and_small_values(mx):
    """Squares whose sum leaves FP32 make rstd 0; the smallest BF16 values have zero squares."""
    R, C = 2, 64
    b = np.full((R, C), 0x7F00, np.uint16)
    b[1] = 0x0001
    out = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    w = to_dev(np.full((1, C), 0x3F80, np.uint16))[0]
    _, rstd = mx.rms_norm(to_dev(b), w, 1e-6, out=out)
    assert rstd[0] == 0 and bool((out[0] == 0).all())
    assert abs(float(rstd[1]) - 1000) < 1e-2


def test_no_rows(mx):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    total, rstd = mx.rms_norm(x, w, out=torch.empty_like(x))
    assert rstd.shape == (0,)
    dw, add = torch.full((64,), 3.0, device="cuda"), torch.arange(64.0, device="cuda")
    mx.rms_norm_backward(x, x, rstd, w, dweight=dw)
    assert bool((dw == 0).all())
    mx.rms_norm_backward(x, x, rstd, w, dweight=dw, add=add)
    assert torch.equal(dw, add)


def bounds(d64, t64, r64, w64, g64):
    """How far dx (before its rounding) and dweight may be off."""
    r = r64[:, None]
    n, g = t64 * r, d64 * w64
    c, cmag = (g * n).mean(axis=1, keepdims=True), np.abs(g * n).mean(axis=1, keepdims=True)
    off = 4 * U24 * (r * (np.abs(g) + np.abs(n * c)) + np.abs(g64)) + r * np.abs(n) * 46 * U24 * cmag
    return off, (-(-len(d64) // 304) + 76 + 32 + 3) * U24 * np.abs(d64 * n).sum(axis=0)


@pytest.mark.parametrize("R,C", SIZES + [(3000, 96), (700, 2048), (900, 1000), (1001, 2731)])
@pytest.mark.parametrize("dtotal,add", [(True, True), (False, False), (True, None)])
def test_backward(mx, R, C, dtotal, add):
    rng = np.random.default_rng(R + 17 * C)
    tb, db, gb, wb = random_bits(rng, R, C, 1.0), random_bits(rng, R, C, 1.0), random_bits(rng, R, C, 1.0), weight_bits(rng, C)
    t64, d64, g64, w64 = (ref.bf16_to_f64(v) for v in (tb, db, gb, wb))
    rstd32 = moe_ref.rms(t64, 1e-6).astype(np.float32)
    rstd = torch.from_numpy(rstd32).cuda()
    dw = None if add is None else torch.full((C,), 5.0, device="cuda")
    more = torch.from_numpy(rng.standard_normal(C).astype(np.float32)).cuda() if add else None
    dx = mx.rms_norm_backward(to_dev(db), to_dev(tb), rstd, to_dev(wb), dtotal=to_dev(gb) if dtotal else None, dweight=dw, add=more)
    r64 = rstd32.astype(np.float64)
    want, wantw = moe_ref.rms_backward(d64, t64, r64, w64, g64 if dtotal else None)
    n, g = t64 * r64[:, None], d64 * w64
    c, cmag = (g * n).mean(axis=1, keepdims=True), np.abs(g * n).mean(axis=1, keepdims=True)
    r = r64[:, None]
    off = 4 * U24 * (r * (np.abs(g) + np.abs(n * c)) + (np.abs(g64) if dtotal else 0)) + r * np.abs(n) * 46 * U24 * cmag
    assert near(dx, want, off)
    if dw is not None:
        m64 = more.cpu().numpy().astype(np.float64) if add else 0.0
        off = (-(-R // 304) + 76 + 32 + 3) * U24 * (np.abs(d64 * n).sum(axis=0) + np.abs(m64))
        assert (np.abs(dw.cpu().numpy() - (wantw + m64)) <= off).all()
        if add:       # into the addend itself
            mx.rms_norm_backward(to_dev(db), to_dev(tb), rstd, to_dev(wb), dweight=more, add=more)
            assert torch.equal(more, dw)


@pytest.mark.parametrize("R,C,ld,shift", [(70, 256, 264, 0), (37, 1000, 1003, 1), (65, 2048, 2050, 3), (33, 4096, 4097, 5)])
def test_backward_strides(mx, R, C, ld, shift):
    rng = np.random.default_rng(C)
    bits = [random_bits(rng, R, C, 1.0) for _ in range(3)]
    wb = weight_bits(rng, C)
    rstd = torch.rand(R, device="cuda") + 0.5
    dw, dw2 = torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    w = to_dev(wb)
    want = mx.rms_norm_backward(*(to_dev(b) for b in bits[:2]), rstd, w, dtotal=to_dev(bits[2]), dweight=dw)
    out = torch.full((R, ld + 2), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.rms_norm_backward(wide(bits[0], ld, shift), wide(bits[1], ld + 1), rstd, w, dtotal=wide(bits[2], ld + 3, 2), out=out[:, :C], dweight=dw2)
    assert bool((out[:, C:] == 7.0).all())
    # the rows' places decide which threads add what: the bounds of test_backward
    d64, t64, g64 = (ref.bf16_to_f64(bits[i]) for i in (0, 1, 2))
    r64, w64 = f64(rstd), ref.bf16_to_f64(wb)
    exact, exactw = moe_ref.rms_backward(d64, t64, r64, w64, g64)
    off, offw = bounds(d64, t64, r64, w64, g64)
    assert near(want, exact, off) and near(out[:, :C], exact, off)
    assert (np.abs(f64(dw) - exactw) <= offw).all() and (np.abs(f64(dw2) - exactw) <= offw).all()
    same_place = mx.rms_norm_backward(*(wide(b, ld, shift) for b in bits[:2]), rstd, w, dtotal=wide(bits[2], ld, shift),
                                      out=wide(bits[0], ld, shift))
    assert near(same_place, exact, off)
    for i in (0, 2):     # in place of dy, of dtotal
        m = [wide(b, ld, shift) for b in bits]
        got = mx.rms_norm_backward(m[0], m[1], rstd, w, dtotal=m[2], out=m[i])
        assert got is m[i] and torch.equal(got, same_place)


def test_backward_against_differences(mx):
    """The loss sum(dy y) in 64 bits along the gradients: central differences of a step
    whose square is far below the bound, and gradients off by 2^-8 of each component."""
    rng = np.random.default_rng(11)
    R, C = 6, 96
    tb, db, wb = random_bits(rng, R, C, 0.2), random_bits(rng, R, C, 0.2), weight_bits(rng, C)
    t64, d64, w64 = (ref.bf16_to_f64(v) for v in (tb, db, wb))
    rstd = torch.from_numpy(moe_ref.rms(t64, 0.0).astype(np.float32)).cuda()
    dw = torch.empty(C, device="cuda")
    dx = f64(mx.rms_norm_backward(to_dev(db), to_dev(tb), rstd, to_dev(wb), dweight=dw))

    def loss(t, w):
        return (d64 * t * moe_ref.rms(t, 0.0)[:, None] * w).sum()

    for d, at in ((dx, lambda e: (t64 + e, w64)), (f64(dw), lambda e: (t64, w64 + e))):
        e = 1e-5 / np.abs(d).max()
        slope = (loss(*at(e * d)) - loss(*at(-e * d))) / (2 * e)
        assert abs(slope / (d * d).sum() - 1) <= 2.0 ** -7


def test_equal_inputs_give_equal_bits(mx):
    rng = np.random.default_rng(2)
    R, C = 1000, 2731
    t, d, w = to_dev(random_bits(rng, R, C)), to_dev(random_bits(rng, R, C)), to_dev(weight_bits(rng, C))
    rstd = torch.rand(R, device="cuda")
    first = None
    for _ in range(4):
        dw = torch.empty(C, device="cuda")
        dx = mx.rms_norm_backward(d, t, rstd, w, dweight=dw)
        if first is not None:
            assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
        first = dx, dw
