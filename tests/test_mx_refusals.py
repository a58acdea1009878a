"""What the microscaled entry points refuse, without a GPU: every refusal
happens on the host before any CUDA call (addresses here are never
dereferenced), and the Python layer's checks of shapes and types."""
import numpy as np
import pytest
import torch

import mx_ref as ref

GOOD = 1 << 20


@pytest.fixture(scope="module")
def B():
    from lossless_bf16_exponent_codec_gb300 import build
    build.build()
    from lossless_bf16_exponent_codec_gb300 import binding
    return binding


def rc(B, fn, *a):
    try:
        fn(*a)
    except B.EzError as e:
        return e.status
    return B.EZ_OK


def change(base, **kw):
    d = dict(base)
    d.update(kw)
    return list(d.values())


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3", "e5m2"])
@pytest.mark.parametrize("R,C", [(0, 0), (1, 1), (1, 32), (127, 33), (128, 128), (129, 129), (1000, 4100)])
def test_sizes_match_the_layout(B, fmt, R, C):
    from lossless_bf16_exponent_codec_gb300 import mx
    codes, scales, _ = ref.quantize(np.zeros((R, C)), fmt) if R and C else (np.zeros((R, 0)), np.zeros(0), None)
    assert B.ez_mx_sizes(mx.FORMATS[fmt], R, C) == (codes.size, scales.size)
    if R and C:   # every scale has a byte of its own inside the tiles
        at = ref.scale_index(R, -(-C // 32))
        assert len(np.unique(at)) == at.size and at.max() < scales.size


def test_sizes_refuse(B):
    for f, r, c in ((0, 1, 1), (4, 1, 1), (1, 1 << 32, 1), (1, 1, 1 << 32), (1, 1 << 21, 1 << 20)):
        assert rc(B, B.ez_mx_sizes, f, r, c) == B.EZ_ERR_ARG


def test_quantize_refuses(B):
    base = dict(x=GOOD, rows=4, cols=64, ldx=64, rf=1, rc=GOOD, rs=GOOD, cf=2, cc=GOOD, cs=GOOD, s=0)
    for bad in (dict(x=None), dict(x=GOOD + 1), dict(ldx=63), dict(rf=4), dict(cf=9), dict(rf=0, cf=0), dict(rc=None),
                dict(rs=None), dict(rc=GOOD + 8), dict(cs=GOOD + 4), dict(cc=None), dict(rows=1 << 40),
                dict(cols=1 << 33, ldx=1 << 33)):
        assert rc(B, B.ez_mx_quantize, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    for none in (dict(rows=0, x=None), dict(cols=0, rc=None)):
        assert rc(B, B.ez_mx_quantize, *change(base, **none)) == B.EZ_OK


def test_dequantize_refuses(B):
    base = dict(f=1, c=GOOD, sc=GOOD, rows=4, cols=64, out=GOOD, ldo=64, s=0)
    for bad in (dict(f=0), dict(f=7), dict(c=None), dict(sc=GOOD + 1), dict(out=None), dict(out=GOOD + 1), dict(ldo=10)):
        assert rc(B, B.ez_mx_dequantize, *change(base, **bad)) == B.EZ_ERR_ARG, bad


def test_matmul_refuses(B):
    base = dict(fa=1, ac=GOOD, asc=GOOD, M=4, fb=1, bc=GOOD, bs=GOOD, N=8, K=64, add=None, c=GOOD, ldc=8, f32=0,
                st=GOOD, s=0)
    for bad in (dict(fa=0), dict(fb=4), dict(ac=None), dict(asc=GOOD + 8), dict(bc=GOOD + 1), dict(bs=None),
                dict(c=None), dict(c=GOOD + 1), dict(ldc=7), dict(st=None), dict(st=GOOD + 2), dict(add=GOOD),
                dict(add=GOOD + 2, f32=1), dict(c=GOOD + 2, f32=1), dict(M=1 << 32), dict(K=1 << 39)):
        assert rc(B, B.ez_mx_matmul, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    for pair in (dict(fa=1, fb=2), dict(fa=3, fb=1)):
        assert rc(B, B.ez_mx_matmul, *change(base, **pair)) == B.EZ_ERR_UNSUPPORTED
    assert rc(B, B.ez_mx_matmul, *change(base, M=0, c=None)) == B.EZ_OK


def test_swiglu_refuses(B):
    base = dict(f=2, g=GOOD, ldg=64, u=GOOD, ldu=64, rows=4, cols=64, gc=GOOD, gs=GOOD, uc=GOOD, us=GOOD, h=GOOD,
                ldh=64, s=0)
    for bad in (dict(f=0), dict(g=None), dict(u=GOOD + 1), dict(ldg=1), dict(ldu=63), dict(gc=None), dict(us=GOOD + 2),
                dict(h=None), dict(ldh=5)):
        assert rc(B, B.ez_mx_swiglu, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    assert rc(B, B.ez_mx_swiglu, *change(base, f=1)) == B.EZ_ERR_UNSUPPORTED
    base = dict(f=2, gc=GOOD, gs=GOOD, uc=GOOD, us=GOOD, rows=4, cols=64, d=GOOD, ldd=64, dg=GOOD, ldg=64, du=GOOD,
                ldu=64, h=None, ldh=0, s=0)
    for bad in (dict(f=5), dict(gc=GOOD + 1), dict(us=None), dict(d=None), dict(ldd=1), dict(dg=None), dict(du=GOOD + 1),
                dict(ldu=3), dict(h=GOOD, ldh=3), dict(h=GOOD + 1, ldh=64)):
        assert rc(B, B.ez_mx_swiglu_backward, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    assert rc(B, B.ez_mx_swiglu_backward, *change(base, f=1)) == B.EZ_ERR_UNSUPPORTED


def test_python_layer_refuses(B):
    from lossless_bf16_exponent_codec_gb300 import mx
    a = mx.MxTensor.empty("e2m1", 4, 64, device="cpu")
    b = mx.MxTensor.empty("e2m1", 8, 96, device="cpu")
    e = mx.MxTensor.empty("e4m3", 8, 64, device="cpu")
    with pytest.raises(ValueError, match="inner sizes"):
        mx.matmul(a, b)
    with pytest.raises(ValueError, match="do not multiply"):
        mx.matmul(a, e)
    with pytest.raises(ValueError, match="unknown microscaled format"):
        mx.MxTensor.empty("e3m2", 4, 64, device="cpu")
    with pytest.raises(ValueError, match="do not hold"):
        mx.dequantize(mx.MxTensor("e2m1", 4, 64, a.codes[:3], a.scales))
    with pytest.raises(ValueError, match="neither"):
        mx.quantize(torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA matrix"):
        mx.quantize(torch.zeros(4, 64, dtype=torch.bfloat16), row=a)
    a.codes = a.codes[:3]          # a form is checked again when a tensor of it is replaced
    with pytest.raises(ValueError, match="do not hold"):
        mx.matmul(a, a)
    a = mx.MxTensor.empty("e2m1", 4, 64, device="cpu")
    with pytest.raises(ValueError, match="e4m3 or e5m2"):
        mx.swiglu_backward(a, a, None, None, None)


def test_wait_limit_refuses(B):
    for bad in (-1, 1 << 32):
        with pytest.raises(ValueError, match="polls"):
            B.ez_mx_wait_limit(bad)
    B.ez_mx_wait_limit(0)
    B.ez_mx_wait_limit()


@pytest.mark.parametrize("part", ["codes", "scales"])
def test_a_form_is_checked_in_every_call(B, part):
    """Also when one of its tensors changes under the same object."""
    from lossless_bf16_exponent_codec_gb300 import mx
    a = mx.MxTensor.empty("e2m1", 200, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA matrix"):
        mx.dequantize(a)
    t = getattr(a, part)
    t.data = t[:len(t) // 2].clone()
    with pytest.raises(ValueError, match="do not hold"):
        mx.dequantize(a)
    a.rows = 100                    # nor do the tensors of a form say how large it is
    with pytest.raises(ValueError, match="do not hold"):
        mx.dequantize(a)
