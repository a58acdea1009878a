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
    assert rc(B, B.ez_mx_wait_limit, (1 << 24) + 1) == B.EZ_ERR_ARG
    for good in (0, 1 << 24):
        B.ez_mx_wait_limit(good)
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


class OnGpu:
    """A CPU tensor that says it is on a GPU (nothing here reads its memory there)."""
    is_cuda = True

    def __init__(self, t, device):
        self.t, self.at = t, device

    def get_device(self):
        return self.at

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.mark.parametrize("current,far", [(1, None), (0, 0), (0, 1), (0, 2), (0, 3), (0, 4)])
def test_other_devices_are_refused(B, monkeypatch, current, far):
    """Every tensor has to be on the current device: all on another one, or the one
    numbered `far`."""
    from lossless_bf16_exponent_codec_gb300 import mx
    monkeypatch.setattr(B, "_current", lambda: (lambda: current, lambda d: 0))

    class Launched(Exception):
        pass

    class Lib:
        def __getattr__(self, name):
            def launch(*a):
                raise Launched(name)
            return launch

    monkeypatch.setattr(B, "lib", lambda: Lib())
    R, C = 32, 64
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731

    def tensors(*kinds):
        """The call's tensors, the one numbered `far` on device 1."""
        out, n = [], 0
        for kind in kinds:
            at = lambda: 1 if n == far else 0  # noqa: E731
            if kind == "form":
                out.append(mx.MxTensor("e4m3", R, C, OnGpu(u8(R, C), at()), OnGpu(u8(512), at())))
            elif kind == "col":
                out.append(mx.MxTensor("e4m3", C, R, OnGpu(u8(C, R), at()), OnGpu(u8(512), at())))
            else:
                out.append(OnGpu(kind, at()))
            n += 1
        return out

    word = torch.zeros(1, dtype=torch.int32)
    calls = [
        (3, lambda x, r, c: mx.quantize(x, row=r, col=c), (bf(R, C), "form", "col")),
        (2, lambda t, o: mx.dequantize(t, out=o), ("form", bf(R, C))),
        (5, lambda a, b, o, d, s: mx.matmul(a, b, out=o, add=d, status=s),
         ("form", "form", torch.zeros(R, R), torch.zeros(R, R), word)),
        (5, lambda g, u, g8, u8_, o: mx.swiglu(g, u, g8, u8_, out=o), (bf(R, C), bf(R, C), "form", "form", bf(R, C))),
        (5, lambda g8, u8_, d, dg, du: mx.swiglu_backward(g8, u8_, d, dg, du),
         ("form", "form", bf(R, C), bf(R, C), bf(R, C))),
    ]
    for n, call, kinds in calls:
        wrong = far is None or far < n
        with pytest.raises(ValueError if wrong else Launched, match="current device" if wrong else "ez_mx"):
            call(*tensors(*kinds))
    # a form in two halves
    t = mx.MxTensor("e4m3", R, C, OnGpu(u8(R, C), 0), OnGpu(u8(512), 1))
    with pytest.raises(ValueError, match="same one"):
        mx.dequantize(t, out=OnGpu(bf(R, C), 0))


def test_matrices_that_require_grad_are_refused(B, monkeypatch):
    """While gradients are recorded: their history would be lost without a word."""
    from lossless_bf16_exponent_codec_gb300 import mlp, mx
    monkeypatch.setattr(B, "_current", lambda: (lambda: 0, lambda d: 0))
    done = []
    monkeypatch.setattr(B, "lib", lambda: type("L", (), {"__getattr__": lambda s, name: lambda *a: done.append(name)})())
    R, C = 32, 64
    leaf = lambda kind, *s: OnGpu(torch.zeros(*s, dtype=kind, requires_grad=True), 0)  # noqa: E731
    plain = lambda kind, *s: OnGpu(torch.zeros(*s, dtype=kind), 0)  # noqa: E731
    bf, f32 = torch.bfloat16, torch.float32
    form = lambda: mx.MxTensor("e4m3", R, C, plain(torch.uint8, R, C), plain(torch.uint8, 512))  # noqa: E731
    calls = [lambda: mx.swiglu(leaf(bf, R, C), plain(bf, R, C), form(), form(), out=plain(bf, R, C)),
             lambda: mx.swiglu(plain(bf, R, C), leaf(bf, R, C), form(), form(), out=plain(bf, R, C)),
             lambda: mx.swiglu_backward(form(), form(), leaf(bf, R, C), plain(bf, R, C), plain(bf, R, C)),
             lambda: mx.matmul(form(), form(), out=plain(f32, R, R), add=leaf(f32, R, R), status=plain(torch.int32, 1))]
    for call in calls:
        with pytest.raises(ValueError, match="requires grad"):
            call()
        assert not done
        with torch.no_grad():
            call()
        assert len(done) == 1
        done.clear()
    # weights are parameters of some optimiser: their forms hold no history
    mx.quantize(leaf(bf, R, C), row=form())
    assert done == ["ez_mx_quantize"]
    with pytest.raises(ValueError, match="requires grad"):
        mlp.GatedMLP.forward(None, torch.zeros(2, 8, dtype=bf, requires_grad=True))
