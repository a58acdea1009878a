"""Tokens sorted by expert and back, and the experts' products, on the GPU
against 64-bit arithmetic.

Orders and forms are compared exactly.  combine: k FP32 multiply-adds of exact
inputs, each off by 2^-24 of a partial sum: k 2^-24 sum|w v| before the one
rounding.  The weights' gradient: a lane adds at most 8 ceil(C / 256) terms and
the tree 5 sums.  Products as those of two matrices: (K + 2) 2^-23 sum|a b|."""
import numpy as np
import pytest
import torch

import moe_ref
import mx_ref as ref
from test_gpu_mx import U23, mx, near, random_bits, to_dev  # noqa: F401  (mx: the fixture)

pytestmark = pytest.mark.gpu
U24 = 2.0 ** -24


@pytest.fixture(scope="module")
def moe(mx):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import moe
    return moe


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def choices(rng, T, k, E, kind="some"):
    """ids [T, k]: a few experts far more popular than the others; "dropped": of the last
    tokens none, and some out of range; "one": all the same expert; "twice": an expert
    chosen twice by a token."""
    like = 2.0 * rng.standard_normal(E)
    ids = np.argsort(-(like + rng.gumbel(size=(T, E))), axis=1)[:, :k].astype(np.int32)
    if kind == "dropped":
        ids[T - T // 3:] = -1
        ids[0, 0] = E
        ids[T // 2, k - 1] = 1 << 30
    elif kind == "one":
        ids[:] = E - 1
    elif kind == "twice":
        ids[:, k - 1] = ids[:, 0]
    elif kind == "none":
        ids[:] = -5
    return ids


def route(moe, ids, E, dtype=torch.int32):
    return moe.sort(torch.from_numpy(ids).to(dtype).cuda(), E)


# ------------------------------------------------------------------- sort

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (7, 1, 200), (200, 6, 66), (513, 8, 64), (128, 1, 1), (129, 1, 2),
                                   (700, 3, 1024), (9000, 2, 33), (5000, 8, 160)])
@pytest.mark.parametrize("kind", ["some", "dropped", "one", "twice", "none"])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(moe, T, k, E, kind, dtype):
    ids = choices(np.random.default_rng(T + E), T, k, E, kind)
    r = route(moe, ids, E, dtype)
    counts, offsets, slots, sources = moe_ref.routing(ids, E)
    assert r.rows == len(sources) and r.tokens == T and r.choices == k and r.experts == E
    for got, want in ((r.counts, counts), (r.offsets, offsets), (r.slots, slots), (r.sources, sources)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_sort_of_no_tokens_and_of_strided_ids(moe):
    r = moe.sort(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 7)
    assert r.rows == 0 and r.counts.tolist() == [0] * 7 and r.offsets.tolist() == [0] * 8
    ids = choices(np.random.default_rng(1), 300, 4, 9)
    wide = torch.full((300, 11), 3, dtype=torch.int64, device="cuda")
    wide[:, :4] = torch.from_numpy(ids).cuda()
    r = moe.sort(wide[:, :4], 9)
    assert np.array_equal(r.slots.cpu().numpy(), moe_ref.routing(ids, 9)[2])
    big = torch.full((2, 2), 1 << 33, dtype=torch.int64, device="cuda")     # no expert in its low half either
    assert moe.sort(big, 4).slots.tolist() == [[-1, -1], [-1, -1]]


# --------------------------------------------------------------- dispatch

def check_rows(t, want64, fmt, used, col):
    """A form filled up to `used` rows (columns of the column form), 0xA5 behind."""
    code, scale, value = ref.quantize(want64, fmt)
    codes, scales = t.codes.cpu().numpy(), t.scales.cpu().numpy()
    rows, cols = want64.shape
    nb = -(-cols // 32)
    at = ref.scale_index(-(-rows // 128) * 128, -(-nb // 4) * 4)     # every byte of the tiles
    if col:
        n = used * (4 if fmt == "e2m1" else 8) // 8
        assert np.array_equal(codes[:, :n], code[:, :n]) and (codes[:, n:] == 0xA5).all()
        assert np.array_equal(scales[at[:, :used // 32]], scale[at[:, :used // 32]]) and (scales[at[:, used // 32:]] == 0xA5).all()
    else:
        assert np.array_equal(codes[:used], code[:used]) and (codes[used:] == 0xA5).all()
        assert np.array_equal(scales[at[:used]], scale[at[:used]]) and (scales[at[used:]] == 0xA5).all()


def blank(mx, fmt, R, C):  # noqa: F811
    t = mx.MxTensor.empty(fmt, R, C)
    t.codes.fill_(0xA5)
    t.scales.fill_(0xA5)
    return t


@pytest.mark.parametrize("T,k,E,C", [(1, 1, 1, 1), (1, 8, 64, 2048), (5, 2, 3, 33), (130, 2, 4, 128), (200, 6, 20, 257), (64, 4, 8, 1000),
                                     (700, 8, 16, 1100), (1200, 8, 8, 2056)])
@pytest.mark.parametrize("row,col", [("e2m1", None), ("e4m3", None), ("e2m1", "e4m3"), (None, "e2m1"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("kind,weighted", [("some", False), ("dropped", True), ("dropped", False), ("twice", False)])
def test_dispatch(mx, moe, T, k, E, C, row, col, kind, weighted):  # noqa: F811
    rng = np.random.default_rng(T * 7 + C)
    ids = choices(rng, T, k, E, kind)
    _, offsets, _, sources = moe_ref.routing(ids, E)
    r = route(moe, ids, E)
    bits = random_bits(rng, T, C)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda() if weighted else None
    forms = [blank(mx, fmt, a, b) if fmt else None for fmt, a, b in ((row, r.rows, C), (col, C, r.rows))]
    moe.dispatch(to_dev(bits), r, row=forms[0], col=forms[1], weights=w)
    x64 = ref.bf16_to_f64(bits)
    if weighted:     # an FP32 product, then BF16
        w32 = w.cpu().numpy()
        g = np.zeros((r.rows, C), np.float32)
        at = np.nonzero(sources >= 0)[0]
        g[at] = x64.astype(np.float32)[sources[at] // k] * w32.reshape(-1)[sources[at], None]
        g = torch.from_numpy(g).to(torch.bfloat16).double().numpy()
    else:
        g = moe_ref.ordered(x64, sources, k)
    for t, v, fmt, is_col in ((forms[0], g, row, False), (forms[1], g.T, col, True)):
        if t is not None:
            check_rows(t, v, fmt, int(offsets[-1]), is_col)


def test_dispatch_of_strided_tokens_with_infinities(mx, moe):  # noqa: F811
    """Odd strides, and values that poison their blocks: of the tokens they are in, and of
    the columns' blocks, only."""
    rng = np.random.default_rng(8)
    T, k, E, C = 90, 3, 6, 201
    ids = choices(rng, T, k, E)
    _, offsets, _, sources = moe_ref.routing(ids, E)
    bits = random_bits(rng, T, C)
    bits[4, 40], bits[60, 200] = 0x7F80, 0xFFC0
    mem = torch.zeros(T, C + 12, dtype=torch.bfloat16, device="cuda")
    x = mem[:, 5:5 + C]
    x.copy_(to_dev(bits))
    r = route(moe, ids, E)
    row, col = blank(mx, "e4m3", r.rows, C), blank(mx, "e5m2", C, r.rows)
    moe.dispatch(x, r, row=row, col=col)
    g = moe_ref.ordered(ref.bf16_to_f64(bits), sources, k)
    check_rows(row, g, "e4m3", int(offsets[-1]), False)
    alone = blank(mx, "e4m3", r.rows, C)
    moe.dispatch(x, r, row=alone)
    assert torch.equal(alone.codes, row.codes) and torch.equal(alone.scales, row.scales)
    check_rows(col, g.T, "e5m2", int(offsets[-1]), True)


# ---------------------------------------------------------------- combine

@pytest.mark.parametrize("T,k,E,C", [(1, 1, 1, 1), (1, 8, 64, 2048), (5, 2, 3, 33), (130, 2, 4, 256), (200, 6, 20, 257), (64, 9, 12, 1000),
                                     (33, 17, 20, 1025), (20, 4, 8, 5001), (40, 8, 16, 4096)])
@pytest.mark.parametrize("kind,weighted", [("some", True), ("dropped", False), ("dropped", True), ("twice", True), ("none", True)])
def test_combine(moe, T, k, E, C, kind, weighted):
    rng = np.random.default_rng(T * 3 + C)
    ids = choices(rng, T, k, E, kind)
    _, _, slots, sources = moe_ref.routing(ids, E)
    r = route(moe, ids, E)
    bits = random_bits(rng, r.rows, C)
    bits[sources < 0] = 0x7FC0           # what no pair names is not read
    rows = to_dev(bits)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda() if weighted else None
    y = moe.combine(rows, r, weights=w)
    v = ref.bf16_to_f64(bits)
    want, mag = moe_ref.combine(v, slots, None if w is None else w.cpu().numpy().astype(np.float64))
    assert near(y, want, k * U24 * mag)
    # the weights' gradient
    dyb = random_bits(rng, T, C, 0.5)
    dw = moe.weight_gradient(to_dev(dyb), rows, r).cpu().numpy()
    # odd strides
    mem = torch.full((T, C + 3), 7.0, dtype=torch.bfloat16, device="cuda")
    wide = torch.zeros(r.rows, C + 5, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:C + 1] = rows
    moe.combine(wide[:, 1:C + 1], r, weights=w, out=mem[:, :C])
    assert torch.equal(mem[:, :C], y) and bool((mem[:, C:] == 7.0).all())
    dy = torch.zeros(T, C + 9, dtype=torch.bfloat16, device="cuda")
    dy[:, 3:C + 3] = to_dev(dyb)
    dw2 = moe.weight_gradient(dy[:, 3:C + 3], wide[:, 1:C + 1], r).cpu().numpy()
    d64 = ref.bf16_to_f64(dyb)
    for got in (dw, dw2):
        for j in range(k):
            some = slots[:, j] >= 0
            terms = d64[some] * v[slots[some, j]]
            assert (np.abs(got[some, j] - terms.sum(axis=1)) <= (8 * -(-C // 256) + 5) * U24 * np.abs(terms).sum(axis=1)).all()
            assert (got[~some, j] == 0).all()


def test_gradient_of_the_way_there_and_back_against_differences(mx, moe):  # noqa: F811
    """combine is linear in the rows and in the weights: its value against dy is <w, dweights>
    and <rows, gradient of the rows>."""
    rng = np.random.default_rng(4)
    T, k, E, C = 50, 3, 5, 96
    ids = choices(rng, T, k, E, "dropped")
    _, offsets, slots, sources = moe_ref.routing(ids, E)
    r = route(moe, ids, E)
    bits, dyb = random_bits(rng, r.rows, C, 0.2), random_bits(rng, T, C, 0.2)
    w = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32)).cuda()
    v, d64, w64 = ref.bf16_to_f64(bits), ref.bf16_to_f64(dyb), w.cpu().numpy().astype(np.float64)
    value = (moe_ref.combine(v, slots, w64)[0] * d64).sum()
    mag = (moe_ref.combine(v, slots, w64)[1] * np.abs(d64)).sum()
    dw = moe.weight_gradient(to_dev(dyb), to_dev(bits), r).cpu().numpy().astype(np.float64)
    assert abs((dw * w64).sum() - value) <= 64 * U24 * mag
    g = mx.MxTensor.empty("e4m3", r.rows, C)
    moe.dispatch(to_dev(dyb), r, row=g, weights=w)
    used = int(offsets[-1])
    g64 = f64(mx.dequantize(g))[:used]
    # E4M3: half a step is 2^-4 of a value, and under 2^-9 of the block's largest for the small ones
    blocks = np.abs(g64).reshape(used, C // 32, 32).max(axis=2).repeat(32, axis=1) * 2.0 ** -8
    off = ((2.0 ** -4 + 2.0 ** -8) * np.abs(moe_ref.ordered(d64, sources, k, w64)[:used]) + blocks) * np.abs(v[:used]) * (sources[:used, None] >= 0)
    assert abs((g64 * v[:used]).sum() - value) <= off.sum()


# ---------------------------------------------------------------- products

def stack_of(mx, fmt, mats):  # noqa: F811
    """A stack of the row forms of BF16 matrices [E, N, K] (bits)."""
    E, N, K = mats.shape
    s = mx.MxStack.empty(fmt, E, N, K)
    s.codes.fill_(0xA5)
    s.scales.fill_(0xA5)
    for e in range(E):
        mx.quantize(to_dev(mats[e]), row=s[e])
    return s


def tokens_of(mx, fmt, bits, sources, col=False):  # noqa: F811
    """The form of a matrix [rows, C] in the experts' order, zero in the padding, and its
    values."""
    z = bits.copy()
    z[sources < 0] = 0
    x = z.T.copy() if col else z
    t = mx.MxTensor.empty(fmt, *x.shape)
    mx.quantize(to_dev(x), row=t)
    return t, ref.quantize(ref.bf16_to_f64(x), fmt)[2]


PRODUCTS = [("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e5m2", "e4m3")]


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 1, 1), (1, 2, 8, 256, 128), (4, 8, 64, 192, 257), (130, 2, 4, 129, 300), (300, 4, 6, 320, 96),
                                       (200, 6, 33, 513, 640), (1000, 2, 3, 700, 1100), (2100, 1, 2, 264, 512), (600, 3, 5, 2000, 160)])
@pytest.mark.parametrize("fa,fb", PRODUCTS)
@pytest.mark.parametrize("kind,dtype", [("some", torch.bfloat16), ("dropped", torch.float32)])
def test_expert_matmul(mx, moe, T, k, E, N, K, fa, fb, kind, dtype):  # noqa: F811
    rng = np.random.default_rng(T + N + K)
    ids = choices(rng, T, k, E, kind)
    counts, offsets, _, sources = moe_ref.routing(ids, E)
    r = route(moe, ids, E)
    a, va = tokens_of(mx, fa, random_bits(rng, r.rows, K, 1.0), sources)
    mats = np.stack([random_bits(rng, N, K, 0.5) for _ in range(E)])
    b = stack_of(mx, fb, mats)
    out = torch.full((r.rows, N), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = moe.expert_matmul(a, b, r, out=out, status=status)
    assert got is out and int(status.item()) == 0
    mem = torch.full((r.rows, N + 7), 5.0, dtype=dtype, device="cuda")      # rows at any alignment
    wide = mem[:, 3:N + 3]
    wide.fill_(7.0)
    moe.expert_matmul(a, b, r, out=wide, status=status)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi == lo:
            continue
        vb = ref.quantize(ref.bf16_to_f64(mats[e]), fb)[2]
        want, off = va[lo:hi] @ vb.T, (K + 2) * U23 * (np.abs(va[lo:hi]) @ np.abs(vb).T)
        for c in (out, wide):
            if dtype is torch.bfloat16:
                assert near(c[lo:hi], want, off)
            else:
                assert (np.abs(f64(c[lo:hi]) - want) <= off).all()
            assert bool((c[lo + counts[e]:hi] == 0).all())
    for c in (out, wide):
        assert bool((c[int(offsets[-1]):] == 7.0).all())
    assert bool((mem[:, :3] == 5.0).all()) and bool((mem[:, N + 3:] == 5.0).all()) and int(status.item()) == 0


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 1, 1), (1, 2, 8, 256, 128), (130, 2, 4, 129, 300), (300, 4, 6, 320, 96), (200, 6, 33, 130, 140),
                                       (2100, 1, 2, 264, 512), (4000, 2, 2, 96, 130), (600, 3, 5, 160, 2000)])
@pytest.mark.parametrize("fa,fb", [("e5m2", "e4m3"), ("e4m3", "e4m3")])
@pytest.mark.parametrize("kind", ["some", "dropped", "none"])
def test_expert_gradient(mx, moe, T, k, E, N, K, fa, fb, kind):  # noqa: F811
    rng = np.random.default_rng(T + 2 * N + K)
    ids = choices(rng, T, k, E, kind)
    counts, offsets, _, sources = moe_ref.routing(ids, E)
    r = route(moe, ids, E)
    a, va = tokens_of(mx, fa, random_bits(rng, r.rows, N, 0.5), sources, col=True)
    b, vb = tokens_of(mx, fb, random_bits(rng, r.rows, K, 0.5), sources, col=True)
    # what lies behind the last expert is not looked at: the scale of a NaN
    used = int(offsets[-1])
    for t in (a, b):
        at = ref.scale_index(-(-t.rows // 128) * 128, t.cols // 32)
        s = t.scales.cpu().numpy()
        s[at[:, used // 32:]] = 255
        t.scales.copy_(torch.from_numpy(s))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = np.stack([va[:, lo:hi] @ vb[:, lo:hi].T for lo, hi in zip(offsets, offsets[1:])])
    mag = np.stack([np.abs(va[:, lo:hi]) @ np.abs(vb[:, lo:hi]).T for lo, hi in zip(offsets, offsets[1:])])
    n = (counts[:, None, None].astype(np.float64) + 2) * U23
    out = torch.full((E, N, K), 7.0, device="cuda")
    assert moe.expert_gradient(a, b, r, out=out, status=status) is out
    assert (np.abs(f64(out) - want) <= n * mag).all()
    more = torch.from_numpy(rng.standard_normal((E, N, K)).astype(np.float32)).cuda()
    m64 = f64(more)
    got = moe.expert_gradient(a, b, r, add=more, status=status)
    off = n * mag + U24 * np.abs(want + m64) + U24 * n * mag
    assert (np.abs(f64(got) - (want + m64)) <= off).all()
    mem = torch.full((E, N, K + 3), 5.0, device="cuda")
    wide = mem[:, :, :K]
    wide.copy_(more)
    moe.expert_gradient(a, b, r, out=wide, add=wide, status=status)
    assert (np.abs(f64(wide) - (want + m64)) <= off).all()
    assert bool((mem[:, :, K:] == 5.0).all()) and int(status.item()) == 0


def test_gradient_of_no_rows(mx, moe):  # noqa: F811
    r = moe.sort(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3)
    a, b = mx.MxTensor.empty("e4m3", 40, 0), mx.MxTensor.empty("e4m3", 50, 0)
    assert bool((moe.expert_gradient(a, b, r) == 0).all())
    add = torch.randn(3, 40, 50, device="cuda")
    assert torch.equal(moe.expert_gradient(a, b, r, add=add), add)


def test_time_outs_are_told(mx, moe):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import binding as B
    rng = np.random.default_rng(6)
    ids = choices(rng, 500, 2, 4)
    r = route(moe, ids, 4)
    _, _, _, sources = moe_ref.routing(ids, 4)
    a, _ = tokens_of(mx, "e4m3", random_bits(rng, r.rows, 512, 0.5), sources)
    b = stack_of(mx, "e4m3", np.stack([random_bits(rng, 300, 512, 0.5) for _ in range(4)]))
    c, _ = tokens_of(mx, "e4m3", random_bits(rng, r.rows, 300, 0.5), sources, col=True)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    used = int(r.offsets[-1].item())
    calls = [lambda: moe.expert_matmul(a, b, r, status=status)[:used], lambda: moe.expert_gradient(c, c, r, status=status)]
    for call in calls:
        good = call()
        assert int(status.item()) == 0
        try:
            B.ez_mx_wait_limit(0)
            call()
        finally:
            B.ez_mx_wait_limit()
        assert int(status.item()) == 8
        status.zero_()
        assert torch.equal(call(), good) and int(status.item()) == 0
