"""The norm's backward pass takes no part in autograd and says so, without a GPU: the
library is a fake that notes its calls, and the tensors say that they are on the GPU."""
import pytest
import torch

from test_moe_shapes import on
from test_mx_refusals import B  # noqa: F401  (the fixture)

BF16, F32 = torch.bfloat16, torch.float32


def test_everything_that_dx_would_be_differentiable_in(B, monkeypatch):  # noqa: F811
    from lossless_bf16_exponent_codec_gb300 import mx
    done = []
    monkeypatch.setattr(B, "_current", lambda: (lambda: 0, lambda d: 0))
    monkeypatch.setattr(B, "_raw", None)
    monkeypatch.setattr(B, "lib", lambda: type("L", (), {"__getattr__": lambda s, name: lambda *a: done.append(name)})())
    given = {"dy": torch.zeros(4, 64, dtype=BF16), "total": torch.zeros(4, 64, dtype=BF16), "rstd": torch.zeros(4), "weight": torch.zeros(64, dtype=BF16),
             "dtotal": torch.zeros(4, 64, dtype=BF16)}
    out = on(torch.zeros(4, 64, dtype=BF16))
    for name in given:
        args = {n: on(t.clone().requires_grad_(n == name)) for n, t in given.items()}
        with pytest.raises(ValueError, match=f"{name}.*requires grad"):
            mx.rms_norm_backward(**args, out=out)
        assert done == []
        with torch.no_grad():
            mx.rms_norm_backward(**args, out=out)
        assert done.pop() == "ez_mx_rms_norm_backward"
    mx.rms_norm_backward(**{n: on(t) for n, t in given.items()}, out=out)
    assert done.pop() == "ez_mx_rms_norm_backward"
