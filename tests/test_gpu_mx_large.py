"""Microscaled operators at sizes of training: the kernels' instances for many
tiles (from two, and from four, tiles of 128 x 128 per SM on), lined and at odd
alignments."""
import numpy as np
import pytest
import torch

import mx_ref as ref
from test_gpu_mx import U16, bits_of, check_form, mx, random_bits, same, to_dev  # noqa: F401

pytestmark = pytest.mark.gpu

TWO = [(2100, 2403), (2111, 2400)]           # 323 tiles on 152 SMs
FOUR = [(3100, 3299), (3200, 3296)]          # 650


@pytest.mark.parametrize("R,C", TWO + FOUR)
@pytest.mark.parametrize("row,col", [("e2m1", "e4m3"), ("e5m2", "e2m1")])
def test_quantize_and_back(mx, R, C, row, col):
    bits = random_bits(np.random.default_rng(R + C), R, C)
    x, x64 = to_dev(bits), ref.bf16_to_f64(bits)
    r, c = mx.MxTensor.empty(row, R, C), mx.MxTensor.empty(col, C, R)
    for t in (r, c):
        t.codes.fill_(0xA5)
        t.scales.fill_(0xA5)
    mx.quantize(x, row=r, col=c)
    for t, v, fmt in ((r, x64, row), (c, x64.T, col)):
        value = check_form(t, v, fmt)
        same(mx.dequantize(t), value)
        # rows that begin anywhere, with room between them
        ld = t.cols + 3
        buf = torch.full((5 + t.rows * ld,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[5:].as_strided((t.rows, t.cols), (ld, 1))
        same(mx.dequantize(t, out=out), value)
        out.fill_(7.0)
        assert bool((buf == 7.0).all())
    # one form alone is the same
    for t in (mx.MxTensor.empty(row, R, C), mx.MxTensor.empty(col, C, R)):
        both = r if t.rows == R else c
        mx.quantize(x, row=t if both is r else None, col=t if both is c else None)
        assert torch.equal(t.codes, both.codes) and torch.equal(t.scales, both.scales)


@pytest.mark.parametrize("R,C", TWO[:1] + FOUR)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_swiglu_and_backward(mx, fmt, R, C):
    """Each result has to be the rounding of a number within 2^-16 of the 64-bit
    value, as at small sizes (|g| < 60)."""
    rng = np.random.default_rng(R + C)
    gb, ub, db = (random_bits(rng, R, C, 0.7) for _ in range(3))
    gb = bits_of(torch.from_numpy(np.clip(ref.bf16_to_f64(gb), -60, 60)).to(torch.bfloat16))
    if C % 8:           # two halves of one matrix
        gu = torch.cat((to_dev(gb), to_dev(ub)), dim=1)
        gate, up = gu[:, :C], gu[:, C:]
    else:
        gate, up = to_dev(gb), to_dev(ub)
    g8, u8 = mx.MxTensor.empty(fmt, R, C), mx.MxTensor.empty(fmt, R, C)
    h = mx.swiglu(gate, up, g8, u8)
    for t, bits in ((g8, gb), (u8, ub)):
        check_form(t, ref.bf16_to_f64(bits), fmt)

    def near(got, want, off):
        """As in mx_ref, on the GPU."""
        def rounded(v):
            q = torch.exp2((torch.frexp(v)[1].double() - 8).clamp(min=-133))
            return torch.round(v / q) * q
        return bool(((rounded(want - off) <= got.double()) & (got.double() <= rounded(want + off))).all())

    def parts(g):
        s = 1 / (1 + torch.exp(-g))
        return s, g * s

    want = parts(gate.double())[1] * up.double()
    assert near(h, want, U16 * want.abs())
    d = to_dev(db)
    wide = torch.full((R, 2 * C + 3), 5.0, dtype=torch.bfloat16, device="cuda")
    dg, du = (wide[:, :C], wide[:, C:2 * C]) if C % 8 else (torch.empty_like(d), torch.empty_like(d))
    h2 = torch.empty_like(d)
    mx.swiglu_backward(g8, u8, d, dg, du, h=h2)
    vg, vu, d64 = mx.dequantize(g8).double(), mx.dequantize(u8).double(), d.double()
    s, a = parts(vg)
    assert near(h2, a * vu, U16 * (a * vu).abs())
    assert near(du, d64 * a, U16 * (d64 * a).abs())
    assert near(dg, d64 * vu * s * (1 + vg * (1 - s)), U16 * (d64 * vu).abs() * s * (1 + vg.abs() * (1 - s)))
    assert bool((wide[:, 2 * C:] == 5.0).all())
    dg2, du2 = torch.empty_like(d), torch.empty_like(d)
    mx.swiglu_backward(g8, u8, d, dg2, du2)
    assert torch.equal(dg2, dg) and torch.equal(du2, du)


@pytest.mark.parametrize("out,add", [("bf16", None), ("f32", None), ("f32", "apart"), ("f32", "in place")])
@pytest.mark.parametrize("fmt,K", [("e4m3", 2500), ("e4m3", 7000), ("e2m1", 14000)])
@pytest.mark.parametrize("M,N", [(2500, 3808), (2500, 3804), (2500, 3801)])
def test_product_of_several_wide_tiles_to_a_pair(mx, M, N, fmt, K, out, add):
    """Two tiles of 256 columns to a pair of CTAs and up to three segments to a sum:
    the two sums in tensor memory take turns and overlap.  C from the lanes, by TMA
    and across the lanes.  Products of -1, 0 and 1 add up to integers below 2^24, in
    any order exactly."""
    g = torch.Generator(device="cuda")
    g.manual_seed(K + N)
    x, y = (torch.randint(-1, 2, (r, K), generator=g, device="cuda", dtype=torch.int8) for r in (M, N))
    a, b = mx.MxTensor.empty(fmt, M, K), mx.MxTensor.empty(fmt, N, K)
    mx.quantize(x.to(torch.bfloat16), row=a)
    mx.quantize(y.to(torch.bfloat16), row=b)
    want = x.float() @ y.float().t()
    more = None
    if add:
        more = torch.randint(-2 ** 22, 2 ** 22, (M, N), generator=g, device="cuda").float()
        want = want + more
    kind = torch.bfloat16 if out == "bf16" else torch.float32
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = mx.matmul(a, b, dtype=kind, out=more if add == "in place" else None, add=more, status=status)
    assert int(status.item()) == 0 and torch.equal(c, want.to(kind))
