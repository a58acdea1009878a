"""Shapes of what goes with a routing, without a GPU: the library is a fake that
notes its calls, and the tensors say that they are on the GPU."""
import pytest
import torch

from test_moe_refusals import moe  # noqa: F401  (the fixture)
from test_mx_refusals import B  # noqa: F401  (the fixture)

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
T, k, E, C = 4, 2, 3, 64


class OnGpu(torch.Tensor):
    """A CPU tensor that answers as one on device 0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def on(t):
    return t.as_subclass(OnGpu)


@pytest.fixture
def calls(B, moe, form, monkeypatch):  # noqa: F811
    done = []
    monkeypatch.setattr(B, "_current", lambda: (lambda: 0, lambda d: 0))
    monkeypatch.setattr(B, "_raw", None)
    monkeypatch.setattr(B, "lib", lambda: type("L", (), {"__getattr__": lambda s, name: lambda *a: done.append(name)})())
    return done


@pytest.fixture
def form(B, moe):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import mx
    t = mx.MxTensor.empty("e4m3", moe._rows(T, k, E), C, device="cpu")
    t.codes, t.scales = on(t.codes), on(t.scales)
    return t


def routing(moe, slots):  # noqa: F811
    rows = moe._rows(T, k, E)
    return moe.Routing(T, k, E, on(torch.zeros(E, dtype=I32)), on(torch.zeros(E + 1, dtype=I32)), on(slots),
                       on(torch.zeros(rows, dtype=I32)))


def good_and_bad(dtype):
    """[T, k], the same in one row, and what would be indexed in another order."""
    v = torch.zeros(T, k, dtype=dtype)
    return (v, v.flatten()), (torch.zeros(k, T, dtype=dtype), torch.zeros(2 * T, k // 2, dtype=dtype), torch.zeros(1, T * k, dtype=dtype),
                              torch.zeros(T, 1, k, dtype=dtype), torch.zeros(T * k + 1, dtype=dtype), torch.zeros(T, k + 1, dtype=dtype)[:, :k])


def test_weights_and_slots_in_another_order_are_refused(moe, calls, form):  # noqa: F811
    good, bad = good_and_bad(F32)
    good_slots, bad_slots = good_and_bad(I32)
    x, r = on(torch.zeros(T, C, dtype=BF16)), routing(moe, good_slots[0])
    rows = on(torch.zeros(r.rows, C, dtype=BF16))
    by_weights = {"dispatch": lambda w: moe.dispatch(x, r, row=form, weights=on(w)),
                  "combine": lambda w: moe.combine(rows, r, weights=on(w), out=x),
                  "weight_gradient": lambda w: moe.weight_gradient(x, rows, r, out=on(w))}
    by_slots = {"dispatch": lambda r: moe.dispatch(x, r, row=form), "combine": lambda r: moe.combine(rows, r, out=x),
                "weight_gradient": lambda r: moe.weight_gradient(x, rows, r, out=on(good[0]))}
    for name in by_weights:
        for w in good:
            by_weights[name](w)
        for s in good_slots:
            by_slots[name](routing(moe, s))
        assert calls == ["ez_moe_" + name] * 4
        for w in bad:
            with pytest.raises(ValueError, match="out" if name == "weight_gradient" else "weights"):
                by_weights[name](w)
        for s in bad_slots:
            with pytest.raises(ValueError, match="slots"):
                by_slots[name](routing(moe, s))
        assert len(calls) == 4, name
        calls.clear()
