"""How the norm's and the experts' operators are called: streams, memory of
results, gradients that are not recorded, routings whose contents make no sense."""
import numpy as np
import pytest
import torch

import moe_ref
from test_gpu_moe import blank, choices, moe, route, stack_of, tokens_of  # noqa: F401  (moe: the fixture)
from test_gpu_mx import mx, random_bits, to_dev  # noqa: F401  (mx: the fixture)

pytestmark = pytest.mark.gpu
BUSY = 60_000_000      # cycles that keep a stream occupied: some 30 ms


def calls(mx, moe):  # noqa: F811
    """Calls that allocate what they return, as functions of a stream, to lists of tensors."""
    rng = np.random.default_rng(2)
    T, k, E, C, N = 2000, 2, 4, 1024, 512
    ids = choices(rng, T, k, E)
    _, offsets, _, sources = moe_ref.routing(ids, E)
    used = int(offsets[-1])
    dev = torch.from_numpy(ids).cuda()
    r = moe.sort(dev, E)
    x, res, w = to_dev(random_bits(rng, T, C)), to_dev(random_bits(rng, T, C)), to_dev(random_bits(rng, 1, C, 0.0))[0]
    rows = to_dev(random_bits(rng, r.rows, C))
    y = torch.empty_like(x)
    rstd = torch.rand(T, device="cuda")
    dw = torch.empty(C, device="cuda")
    a, _ = tokens_of(mx, "e4m3", random_bits(rng, r.rows, C, 0.5), sources)
    b = stack_of(mx, "e4m3", np.stack([random_bits(rng, N, C, 0.5) for _ in range(E)]))
    c, _ = tokens_of(mx, "e4m3", random_bits(rng, r.rows, N, 0.5), sources, col=True)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    return {
        "norm": lambda s: list(mx.rms_norm(x, w, residual=res, out=y, stream=s)),
        "norm_back": lambda s: [mx.rms_norm_backward(x, res, rstd, w, dweight=dw, stream=s), dw],
        "sort": lambda s: [getattr(q, n) for q in [moe.sort(dev, E, stream=s)] for n in ("counts", "offsets", "slots", "sources")],
        "combine": lambda s: [moe.combine(rows, r, stream=s)],
        "weights": lambda s: [moe.weight_gradient(x, rows, r, stream=s)],
        "matmul": lambda s: [moe.expert_matmul(a, b, r, status=st, stream=s)[:used]],
        "gradient": lambda s: [moe.expert_gradient(c, c, r, status=st, stream=s)],
    }


@pytest.mark.parametrize("name", ["norm", "norm_back", "sort", "combine", "weights", "matmul", "gradient"])
@pytest.mark.parametrize("as_int", [False, True])
def test_results_are_memory_of_their_stream(mx, moe, name, as_int):  # noqa: F811
    call = calls(mx, moe)[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    # results that are dropped while their stream has yet to write them
    gone = [(t.data_ptr(), t.nbytes) for t in call(stream)]
    held = [torch.full((n,), 5, dtype=torch.uint8, device="cuda") for _, n in gone for _ in range(3)]
    got = call(stream)
    torch.cuda.synchronize()
    assert all(bool((h == 5).all()) for h in held)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_what_requires_grad_is_refused(mx, moe):  # noqa: F811
    rng = np.random.default_rng(3)
    x = to_dev(random_bits(rng, 40, 64))
    w = x[0].clone()
    r = route(moe, choices(rng, 40, 2, 3), 3)
    rows = torch.zeros(r.rows, 64, dtype=torch.bfloat16, device="cuda")
    wt = torch.ones(40, 2, device="cuda")
    form = blank(mx, "e4m3", r.rows, 64)
    t = [x.clone().requires_grad_(), w.clone().requires_grad_(), rows.clone().requires_grad_(), wt.clone().requires_grad_()]
    rstd, vec = torch.ones(40, device="cuda"), torch.zeros(64, device="cuda")
    for call in (lambda: mx.rms_norm(t[0], w, out=x), lambda: mx.rms_norm(x, t[1], out=x), lambda: mx.rms_norm(x, w, residual=t[0], out=x),
                 lambda: mx.rms_norm_backward(t[0], x, rstd, w), lambda: mx.rms_norm_backward(x, x, rstd, w, dtotal=t[0]),
                 lambda: mx.rms_norm_backward(x, x, rstd, w, dweight=vec, add=vec.clone().requires_grad_()),
                 lambda: moe.dispatch(t[0], r, row=form), lambda: moe.dispatch(x, r, row=form, weights=t[3]),
                 lambda: moe.combine(t[2], r), lambda: moe.combine(rows, r, weights=t[3]), lambda: moe.weight_gradient(t[0], rows, r),
                 lambda: moe.weight_gradient(x, t[2], r)):
        with pytest.raises(ValueError, match="requires grad"):
            call()
        with torch.no_grad():
            call()


def test_other_shapes_and_types_are_refused(mx, moe):  # noqa: F811
    rng = np.random.default_rng(3)
    x = to_dev(random_bits(rng, 40, 64))
    r = route(moe, choices(rng, 40, 2, 3), 3)
    rows = torch.zeros(r.rows, 64, dtype=torch.bfloat16, device="cuda")
    form, col = blank(mx, "e4m3", r.rows, 64), blank(mx, "e4m3", 64, r.rows)
    w, rstd = x[0].clone(), torch.ones(40, device="cuda")
    stack = stack_of(mx, "e4m3", np.stack([random_bits(rng, 32, 64) for _ in range(3)]))
    bad = moe.Routing(40, 2, 3, r.counts.long(), r.offsets[:3], r.slots[:39], r.sources[:100])
    for call in (lambda: mx.rms_norm(x, w[:60], out=x), lambda: mx.rms_norm(x, w.float(), out=x), lambda: mx.rms_norm(x, w, residual=x[:30], out=x),
                 lambda: mx.rms_norm(x, w, total=x[:, :60], out=x), lambda: mx.rms_norm(x, w, out=x.float()),
                 lambda: mx.rms_norm(x, w, rstd=rstd[:5], out=x), lambda: mx.rms_norm(x, w, row=form), lambda: mx.rms_norm(x, w, col=form),
                 lambda: mx.rms_norm(x.t(), w[:40].clone(), out=x), lambda: mx.rms_norm_backward(x, x[:9], rstd, w),
                 lambda: mx.rms_norm_backward(x, x, rstd.double(), w), lambda: mx.rms_norm_backward(x, x, rstd, w, add=rstd),
                 lambda: mx.rms_norm_backward(x, x, rstd, w, dweight=rstd), lambda: moe.dispatch(x[:30], r, row=form),
                 lambda: moe.dispatch(x, r, row=col), lambda: moe.dispatch(x, r, row=form, weights=rstd),
                 lambda: moe.dispatch(x, bad, row=form), lambda: moe.combine(rows[:100], r), lambda: moe.combine(rows, bad),
                 lambda: moe.combine(rows, r, out=x[:20]), lambda: moe.weight_gradient(x, rows[:, :60], r),
                 lambda: moe.weight_gradient(x, rows, bad), lambda: moe.expert_matmul(form, stack, bad),
                 lambda: moe.expert_gradient(col, col, bad), lambda: moe.expert_gradient(col, col, r, out=torch.zeros(3, 64, 60, device="cuda")),
                 lambda: moe.expert_gradient(col, col, r, out=torch.zeros(3, 64, 64, device="cuda"), add=torch.zeros(3, 64, 70, device="cuda")[:, :, :64]),
                 lambda: moe.expert_gradient(col, col, r, out=torch.zeros(3, 64, 64, device="cuda").transpose(1, 2)),
                 lambda: moe.expert_matmul(form, stack, r, status=rstd), lambda: moe.sort(torch.zeros(4, 2, device="cuda"), 3)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("seed", range(6))
def test_no_content_of_a_routing_leads_outside(mx, moe, seed):  # noqa: F811
    """Counts, offsets, slots and sources of any values (each is cut to its range, in the kernels)
    make results unspecified, but only those: what lies around every result stays."""
    rng = np.random.default_rng(seed)
    T, k, E, C, N = 300, 3, 5, 264, 140
    rows = moe._rows(T, k, E)

    def any_int(*shape):
        v = rng.integers(-2 ** 31, 2 ** 31, size=shape)
        near = rng.integers(-300, rows + 300, size=shape)
        return torch.from_numpy(np.where(rng.random(shape) < 0.5, v, near).astype(np.int32)).cuda()

    r = moe.Routing(T, k, E, any_int(E), any_int(E + 1), any_int(T, k), any_int(rows))
    around = 4096

    def guarded(n, dtype):
        mem = torch.full((n * torch.empty(0, dtype=dtype).element_size() + 2 * around,), 0xA5, dtype=torch.uint8, device="cuda")
        return mem, mem[around:-around].view(dtype)

    mems = []

    def form(fmt, a, b):
        t = mx.MxTensor.empty(fmt, a, b)
        for n in ("codes", "scales"):
            mem, inner = guarded(getattr(t, n).numel(), torch.uint8)
            mems.append(mem)
            inner.zero_()
            setattr(t, n, inner.view(getattr(t, n).shape))
        return t

    def matrix(dtype, *shape):
        mem, inner = guarded(int(np.prod(shape)), dtype)
        mems.append(mem)
        return inner.view(shape)

    x, dy = to_dev(random_bits(rng, T, C)), to_dev(random_bits(rng, T, C))
    row, col = form("e4m3", rows, C), form("e4m3", C, rows)
    moe.dispatch(x, r, row=row, col=col, weights=torch.ones(T, k, device="cuda"))
    for fmt in ("e2m1", "e5m2"):
        moe.dispatch(x, r, row=form(fmt, rows, C))
    values = to_dev(random_bits(rng, rows, C))
    moe.combine(values, r, out=matrix(torch.bfloat16, T, C))
    moe.weight_gradient(dy, values, r, out=matrix(torch.float32, T, k))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (N, 700):       # tiles by tokens and by weights
        b = stack_of(mx, "e4m3", np.stack([random_bits(rng, n, C) for _ in range(E)]))
        moe.expert_matmul(row, b, r, out=matrix(torch.bfloat16, rows, n), status=status)
        moe.expert_matmul(row, b, r, out=matrix(torch.float32, rows, n), status=status)
    moe.expert_gradient(col, col, r, out=matrix(torch.float32, E, C, C), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for mem in mems:
        assert bool((mem[:around] == 0xA5).all()) and bool((mem[-around:] == 0xA5).all())


def test_offsets_past_32_bits(mx, moe):  # noqa: F811
    """Matrices of more than 2^32 bytes: their last rows are those of the same calls on these rows alone."""
    T, C, E, n = 270_000, 8192, 3, 200
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(T, C, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen)
    w = (1 + 0.1 * torch.randn(C, device="cuda", generator=gen)).to(torch.bfloat16)
    tail = x[-n:].clone()
    ids = torch.randint(0, E, (T, 1), device="cuda", generator=gen)
    r = moe.sort(ids, E)
    assert r.rows * C > 1 << 31
    small = mx.MxTensor.empty("e4m3", n, C)
    mx.quantize(tail, row=small)
    want = mx.dequantize(small)
    row, col = mx.MxTensor.empty("e4m3", r.rows, C), mx.MxTensor.empty("e5m2", C, r.rows)
    moe.dispatch(x, r, row=row)
    alone = row.codes.clone()
    moe.dispatch(x, r, row=row, col=col)
    used = int(r.offsets[-1])
    assert torch.equal(alone[:used], row.codes[:used])
    del alone
    rows = mx.dequantize(row)
    back = moe.combine(rows, r)
    assert torch.equal(back[-n:], want)
    dw = moe.weight_gradient(back, rows, r)
    exact = want.double().square().sum(1)          # C terms: 256 to a lane, a chain of 128 for each half, then 6 sums
    assert (dw[-n:, 0].double() - exact).abs().le((128 + 6) * 2.0 ** -24 * exact).all()
    del rows, back, row, col
    out, tiny = torch.empty_like(x), torch.empty_like(tail)
    form, less = mx.MxTensor.empty("e4m3", T, C), mx.MxTensor.empty("e4m3", n, C)
    total, rstd = mx.rms_norm(x, w, residual=x, out=out, row=form)
    total_n, rstd_n = mx.rms_norm(tail, w, residual=tail, out=tiny, row=less)
    assert torch.equal(total[-n:], total_n) and torch.equal(rstd[-n:], rstd_n) and torch.equal(out[-n:], tiny)
    assert torch.equal(form.codes[-n:], less.codes)
    dx = mx.rms_norm_backward(x, total, rstd, w, dtotal=out)
    assert torch.equal(dx[-n:], mx.rms_norm_backward(tail, total_n, rstd_n, w, dtotal=tiny))
