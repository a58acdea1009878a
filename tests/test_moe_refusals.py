"""What the norm's and the experts' entry points refuse, without a GPU: every
refusal happens on the host before any CUDA call (addresses here are never
dereferenced), the Python layer's checks, and the sizes that the host computes."""
import pytest
import torch

import moe_ref
from test_mx_refusals import B, GOOD, change, rc  # noqa: F401  (B: the fixture)

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def moe(B):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import moe
    return moe


def test_norm_refuses(B):  # noqa: F811
    base = dict(x=GOOD, ldx=64, r=GOOD, ldr=64, rows=4, cols=64, w=GOOD, eps=1e-6, t=GOOD, ldt=64, rstd=GOOD, low=GOOD, y=GOOD + 8192, ldy=64, rf=1,
                rc=GOOD, rs=GOOD, cf=2, cc=GOOD, cs=GOOD, s=0)
    for bad in (dict(x=None), dict(x=GOOD + 1), dict(ldx=63), dict(r=GOOD + 1), dict(ldr=5), dict(w=None), dict(w=GOOD + 1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(t=None), dict(t=GOOD + 1), dict(ldt=3), dict(rstd=None),
                dict(rstd=GOOD + 2), dict(low=None), dict(low=GOOD + 1), dict(y=GOOD + 1), dict(ldy=63), dict(rf=4), dict(rc=None), dict(rs=GOOD + 8),
                dict(cf=9), dict(cc=None), dict(y=GOOD, ldy=72), dict(t=GOOD + 8192), dict(r=None, t=None, y=GOOD), dict(cs=GOOD + 4), dict(rows=1 << 40), dict(cols=0), dict(y=None, rf=0, cf=0), dict(ldt=72),
                dict(ldt=72, t=GOOD + 4096, r=GOOD + 4096)):
        assert rc(B, B.ez_mx_rms_norm, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    assert rc(B, B.ez_mx_rms_norm, *change(base, cols=16385, ldx=20000, ldr=20000, ldt=20000, ldy=20000)) == B.EZ_ERR_UNSUPPORTED
    assert rc(B, B.ez_mx_rms_norm, *change(base, rows=0, x=None, y=None)) == B.EZ_OK


def test_norm_backward_refuses(B):  # noqa: F811
    ws = B.ez_mx_rms_norm_ws(4, 64)
    assert ws >= 64 * 4
    base = dict(dy=GOOD, ldd=64, t=GOOD + 4096, ldt=64, rstd=GOOD, w=GOOD, g=GOOD + 8192, ldg=64, rows=4, cols=64, dx=GOOD + 16384, ldx=64,
                add=GOOD, dw=GOOD, ws=GOOD, n=ws, s=0)
    for bad in (dict(dy=None), dict(ldd=63), dict(t=None), dict(t=GOOD + 1), dict(ldt=1), dict(rstd=None), dict(rstd=GOOD + 1), dict(w=None),
                dict(g=GOOD + 1), dict(ldg=63), dict(dx=None), dict(ldx=2), dict(add=GOOD + 2), dict(dw=None), dict(dw=GOOD + 1), dict(ws=None),
                dict(ws=GOOD + 8), dict(cols=0), dict(rows=1 << 40), dict(dx=GOOD, ldx=72), dict(dx=GOOD + 8192, ldx=72)):
        assert rc(B, B.ez_mx_rms_norm_backward, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    assert rc(B, B.ez_mx_rms_norm_backward, *change(base, n=ws - 1)) == B.EZ_ERR_CAPACITY
    assert rc(B, B.ez_mx_rms_norm_backward, *change(base, cols=16385, ldd=20000, ldt=20000, ldg=20000, ldx=20000)) == B.EZ_ERR_UNSUPPORTED
    assert rc(B, B.ez_mx_rms_norm_backward, *change(base, rows=0, dw=None, add=None, dy=None)) == B.EZ_OK
    for r, c in ((1, 0), (1 << 33, 1)):
        assert rc(B, B.ez_mx_rms_norm_ws, r, c) == B.EZ_ERR_ARG
    assert rc(B, B.ez_mx_rms_norm_ws, 1, 16385) == B.EZ_ERR_UNSUPPORTED


@pytest.mark.parametrize("T,k,E", [(0, 4, 3), (1, 1, 1), (1, 8, 64), (5, 3, 7), (200, 6, 66), (1000, 8, 1024), (16384, 8, 64)])
def test_rows_of_a_routing(B, moe, T, k, E):  # noqa: F811
    rows = B.ez_moe_rows(T, k, E)
    assert rows == moe._rows(T, k, E) and rows % 128 == 0
    pairs = T * k
    # the worst choice: as many experts as possible with one pair more than whole tiles
    for spread in {1, min(E, max(pairs, 1)), max(1, min(E, pairs // 129))}:
        counts = [1] * spread if pairs >= spread else []
        if counts:
            counts[0] += (pairs - spread) // 128 * 128
            assert sum(-(-c // 128) * 128 for c in counts) <= rows
    if pairs <= 2000:
        import numpy as np
        ids = np.arange(pairs).reshape(T, k) % E if pairs else np.zeros((0, k), int)
        assert moe_ref.routing(ids, E)[1][-1] <= rows


def test_routing_refuses(B):  # noqa: F811
    assert rc(B, B.ez_moe_rows, 4, 2, 0) == B.EZ_ERR_ARG
    assert rc(B, B.ez_moe_rows, 1 << 31, 1 << 31, 4) == B.EZ_ERR_ARG
    assert rc(B, B.ez_moe_rows, 1 << 31, 1, 4) == B.EZ_ERR_ARG
    assert rc(B, B.ez_moe_rows, 4, 2, 1025) == B.EZ_ERR_UNSUPPORTED
    assert B.ez_moe_sort_ws(4, 2, 8) == 0
    n = B.ez_moe_sort_ws(5000, 2, 8)
    assert n > 0
    base = dict(ids=GOOD, b=4, ld=2, T=5000, k=2, E=8, c=GOOD, o=GOOD, sl=GOOD, so=GOOD, ws=GOOD, n=n, s=0)
    for bad in (dict(ids=None), dict(ids=GOOD + 2), dict(b=2), dict(ld=1), dict(E=0), dict(c=None), dict(o=GOOD + 1), dict(sl=None),
                dict(so=GOOD + 2), dict(ws=None), dict(ws=GOOD + 1), dict(b=8, ids=GOOD + 4)):
        assert rc(B, B.ez_moe_sort, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    assert rc(B, B.ez_moe_sort, *change(base, n=n - 1)) == B.EZ_ERR_CAPACITY
    assert rc(B, B.ez_moe_sort, *change(base, E=1025)) == B.EZ_ERR_UNSUPPORTED


def test_dispatch_and_combine_refuse(B):  # noqa: F811
    base = dict(x=GOOD, ldx=64, T=4, cols=64, o=GOOD, so=GOOD, sl=GOOD, k=2, E=8, w=None, rf=1, rc=GOOD, rs=GOOD, cf=2, cc=GOOD, cs=GOOD, s=0)
    for bad in (dict(x=None), dict(x=GOOD + 1), dict(ldx=63), dict(o=None), dict(so=GOOD + 2), dict(sl=None), dict(sl=GOOD + 1), dict(w=GOOD + 1), dict(rf=0, cf=0), dict(rf=7),
                dict(rc=None), dict(cs=GOOD + 8), dict(E=0), dict(cols=1 << 33)):
        assert rc(B, B.ez_moe_dispatch, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    assert rc(B, B.ez_moe_dispatch, *change(base, E=2000)) == B.EZ_ERR_UNSUPPORTED
    for none in (dict(T=0, x=None), dict(cols=0, rc=None)):
        assert rc(B, B.ez_moe_dispatch, *change(base, **none)) == B.EZ_OK
    base = dict(i=GOOD, ld=64, rows=256, cols=64, sl=GOOD, w=None, T=4, k=2, y=GOOD + 4096, ldy=64, s=0)
    for bad in (dict(i=None), dict(i=GOOD + 1), dict(ld=63), dict(sl=None), dict(sl=GOOD + 1), dict(w=GOOD + 2), dict(y=None), dict(ldy=1), dict(y=GOOD),
                dict(T=1 << 40), dict(rows=1 << 31), dict(T=1 << 20, k=1 << 20)):
        assert rc(B, B.ez_moe_combine, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    assert rc(B, B.ez_moe_combine, *change(base, T=0, y=None)) == B.EZ_OK
    base = dict(d=GOOD, ldd=64, i=GOOD, ld=64, rows=256, cols=64, sl=GOOD, T=4, k=2, dw=GOOD, s=0)
    for bad in (dict(d=None), dict(ldd=1), dict(i=None), dict(ld=63), dict(sl=None), dict(dw=None), dict(dw=GOOD + 2), dict(rows=1 << 31)):
        assert rc(B, B.ez_moe_weight_gradient, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    assert rc(B, B.ez_moe_weight_gradient, *change(base, k=0, dw=None)) == B.EZ_OK


def test_products_refuse(B):  # noqa: F811
    base = dict(fa=2, ac=GOOD, asc=GOOD, rows=256, fb=2, bc=GOOD, bs=GOOD, E=4, N=64, K=64, c=GOOD, o=GOOD, p=10, out=GOOD, ldc=64, f32=0,
                st=GOOD, s=0)
    for bad in (dict(fa=0), dict(fb=4), dict(ac=None), dict(asc=GOOD + 8), dict(bc=GOOD + 1), dict(bs=None), dict(rows=200), dict(K=0), dict(E=0),
                dict(c=None), dict(o=GOOD + 1), dict(out=None), dict(out=GOOD + 1), dict(out=GOOD + 2, f32=1), dict(ldc=63),
                dict(st=None), dict(st=GOOD + 2), dict(N=1 << 32), dict(rows=1 << 31), dict(N=1 << 31, K=1 << 20)):
        assert rc(B, B.ez_moe_matmul, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    for bad in (dict(fa=1), dict(fb=1), dict(E=1025)):
        assert rc(B, B.ez_moe_matmul, *change(base, **bad)) == B.EZ_ERR_UNSUPPORTED, bad
    for none in (dict(rows=0, out=None), dict(N=0, ldc=0), dict(p=0, out=None)):
        assert rc(B, B.ez_moe_matmul, *change(base, **none)) == B.EZ_OK, none
    base = dict(fa=2, ac=GOOD, asc=GOOD, N=64, fb=3, bc=GOOD, bs=GOOD, K=64, rows=256, E=4, o=GOOD, add=None, c=GOOD, ldc=64, st=GOOD, s=0)
    for bad in (dict(fa=0), dict(fb=4), dict(ac=None), dict(bs=GOOD + 8), dict(rows=100), dict(E=0), dict(o=None), dict(add=GOOD + 2),
                dict(c=None), dict(c=GOOD + 2), dict(ldc=63), dict(st=None), dict(N=1 << 32), dict(rows=1 << 31)):
        assert rc(B, B.ez_moe_gradient, *change(base, **bad)) == B.EZ_ERR_ARG, bad
    for bad in (dict(fa=1), dict(fb=1, fa=1), dict(E=1025)):
        assert rc(B, B.ez_moe_gradient, *change(base, **bad)) == B.EZ_ERR_UNSUPPORTED, bad
    assert rc(B, B.ez_moe_gradient, *change(base, N=0, c=None)) == B.EZ_OK


def host_routing(moe, T=4, k=2, E=3):
    rows = moe._rows(T, k, E)
    return moe.Routing(T, k, E, torch.zeros(E, dtype=I32), torch.zeros(E + 1, dtype=I32), torch.zeros(T, k, dtype=I32),
                       torch.zeros(rows, dtype=I32))


def test_python_layer_refuses(B, moe):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import mx
    x = torch.zeros(4, 64, dtype=BF16)
    r = host_routing(moe)
    a, b = mx.MxTensor.empty("e4m3", r.rows, 64, device="cpu"), mx.MxStack.empty("e4m3", 3, 32, 64, device="cpu")
    cases = [
        ("neither", lambda: mx.rms_norm(x, x[0])),
        ("CUDA matrix", lambda: mx.rms_norm(x, x[0], out=x)),
        ("CUDA matrix", lambda: mx.rms_norm_backward(x, x, x[0], x[0])),
        ("int32 or int64", lambda: moe.sort(x, 4)),
        ("int32 or int64", lambda: moe.sort(torch.zeros(4, 2, dtype=I32), 4)),
        ("neither", lambda: moe.dispatch(x, r)),
        ("CUDA matrix", lambda: moe.dispatch(x, r, row=a)),
        ("CUDA matrix", lambda: moe.combine(x, r)),
        ("CUDA matrix", lambda: moe.weight_gradient(x, x, r)),
        ("inner sizes", lambda: moe.expert_matmul(a, mx.MxStack.empty("e4m3", 3, 32, 96, device="cpu"), r)),
        ("do not multiply", lambda: moe.expert_matmul(a, mx.MxStack.empty("e2m1", 3, 32, 64, device="cpu"), r)),
        ("for a routing", lambda: moe.expert_matmul(a, mx.MxStack.empty("e4m3", 4, 32, 64, device="cpu"), r)),
        ("for a routing", lambda: moe.expert_matmul(mx.MxTensor.empty("e4m3", 128, 64, device="cpu"), b, r)),
        ("BF16 or FP32", lambda: moe.expert_matmul(a, b, r, out=torch.zeros(r.rows, 32, dtype=torch.float16))),
        ("CUDA matrix", lambda: moe.expert_matmul(a, b, r, out=torch.zeros(r.rows, 32, dtype=BF16))),
        ("e4m3 or e5m2", lambda: moe.expert_gradient(*(mx.MxTensor.empty("e2m1", 8, r.rows, device="cpu") for _ in range(2)), r)),
        ("for a routing", lambda: moe.expert_gradient(*(mx.MxTensor.empty("e4m3", 8, 128, device="cpu") for _ in range(2)), r)),
        ("CUDA matrices", lambda: moe.expert_gradient(*(mx.MxTensor.empty("e4m3", 8, r.rows, device="cpu") for _ in range(2)), r,
                                                      out=torch.zeros(3, 8, 8))),
        ("unknown microscaled", lambda: mx.MxStack.empty("e3m2", 3, 32, 64, device="cpu")),
    ]
    for match, call in cases:
        with pytest.raises(ValueError, match=match):
            call()
    b.codes = b.codes[:5]
    with pytest.raises(ValueError, match="do not hold"):
        moe.expert_matmul(a, b, r)
    with pytest.raises(IndexError):
        b[3]


def test_stack_holds_its_forms(B):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import mx
    s = mx.MxStack.empty("e2m1", 5, 130, 70, device="cpu")
    assert len(s) == 5 and s.codes.shape == (650, 48)
    codes, scales = B.ez_mx_sizes(B.EZ_MX_E2M1, 130, 70)
    assert s.scales.numel() == 5 * scales and s.codes.numel() == 5 * codes
    f = s[2]
    assert (f.rows, f.cols, f.format) == (130, 70, "e2m1")
    assert f.codes.data_ptr() == s.codes.data_ptr() + 2 * codes and f.scales.data_ptr() == s.scales.data_ptr() + 2 * scales
    mx._form(f, "f")
