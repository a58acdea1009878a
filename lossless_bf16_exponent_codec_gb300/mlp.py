"""A gated MLP on microscaled operands: what a rank computes with weights that
came out of the compressed all-gather.

    h = silu(x Wg^T) * (x Wu^T),   y = h Wd^T

Forward products run in 4 bits.  What the backward pass needs is kept in 8: the
column form of x (the operand of the weight gradient) and the gate and up
values.  Backward, the output gradients are quantised once into the operand of
the data gradient and the one of the weight gradient, which is summed in FP32.

``python -m lossless_bf16_exponent_codec_gb300.mlp`` gathers random weights
through the 3-bit exponent code and runs training steps and a decoding step.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import mx
from .mx import MxTensor


def _form(x: torch.Tensor, fmt: str, col: bool = False) -> MxTensor:
    R, C = x.shape
    t = MxTensor.empty(fmt, C, R, x.device) if col else MxTensor.empty(fmt, R, C, x.device)
    mx.quantize(x, row=None if col else t, col=t if col else None)
    return t


def _forms(x: torch.Tensor, row: str, col: str):
    R, C = x.shape
    r, c = MxTensor.empty(row, R, C, x.device), MxTensor.empty(col, C, R, x.device)
    mx.quantize(x, row=r, col=c)
    return r, c


@dataclass
class Kept:
    """What a forward pass keeps for its backward pass: 8 bits a value."""
    x: MxTensor       # column form of x
    gate: MxTensor
    up: MxTensor


class GatedMLP:
    """``gate_up`` [2 F, K] (gate rows first) and ``down`` [K, F] in BF16, as
    gathered.  ``grad`` is the format of the gradients' operands and ``kept``
    that of the checkpoint ("e4m3" or "e5m2").

    The products run without the host looking at them.  Their time-outs are collected
    in ``status``: while ``status_word()`` is not 0, what ``forward`` and ``backward``
    returned since it was cleared, and the gradient sums, must not be used."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, grad: str = "e5m2", kept: str = "e4m3"):
        self.F, self.K = gate_up.shape[0] // 2, gate_up.shape[1]
        if tuple(gate_up.shape) != (2 * self.F, self.K) or tuple(down.shape) != (self.K, self.F):
            raise ValueError(f"gate_up {tuple(gate_up.shape)} and down {tuple(down.shape)} do not make a gated MLP")
        self.grad, self.kept = grad, kept
        self.status = torch.zeros(1, dtype=torch.int32, device=gate_up.device)
        self.load(gate_up, down)
        self.d_gate_up = torch.zeros(2 * self.F, self.K, dtype=torch.float32, device=gate_up.device)
        self.d_down = torch.zeros(self.K, self.F, dtype=torch.float32, device=gate_up.device)

    def load(self, gate_up: torch.Tensor, down: torch.Tensor) -> None:
        """Quantise newly gathered weights: 4 bits for the forward products, the
        transpose in 8 for the data gradients."""
        self.w1, self.w1t = _forms(gate_up, "e2m1", "e4m3")
        self.w2, self.w2t = _forms(down, "e2m1", "e4m3")

    def status_word(self) -> int:
        """EZ_DSTAT_* bits of all products since the last ``clear_status`` (waits for
        them)."""
        return int(self.status.item())

    def clear_status(self) -> None:
        self.status.zero_()

    def forward(self, x: torch.Tensor, keep: bool = True):
        """y [T, K] of x [T, K], and what ``backward`` needs (None unless ``keep``).
        Autograd sees none of it: ``backward`` gives dx."""
        if x.requires_grad:
            mx._no_history("x")
        T = x.shape[0]
        if keep:
            x4, x8 = _forms(x, "e2m1", self.kept)
        else:
            x4, x8 = _form(x, "e2m1"), None
        gu = mx.matmul(x4, self.w1, status=self.status)
        gate8, up8 = (MxTensor.empty(self.kept, T, self.F, x.device) for _ in range(2))
        h = mx.swiglu(gu[:, :self.F], gu[:, self.F:], gate8, up8)
        y = mx.matmul(_form(h, "e2m1"), self.w2, status=self.status)
        return y, Kept(x8, gate8, up8) if keep else None

    def backward(self, dy: torch.Tensor, kept: Kept) -> torch.Tensor:
        """dx [T, K]; the weight gradients are added to ``d_gate_up`` and ``d_down``."""
        T, F = dy.shape[0], self.F
        dy_row, dy_col = _forms(dy, self.grad, self.grad)
        dh = mx.matmul(dy_row, self.w2t, status=self.status)
        dgu = torch.empty(T, 2 * F, dtype=torch.bfloat16, device=dy.device)
        h = torch.empty(T, F, dtype=torch.bfloat16, device=dy.device)
        mx.swiglu_backward(kept.gate, kept.up, dh, dgu[:, :F], dgu[:, F:], h=h)
        mx.matmul(dy_col, _form(h, self.kept, col=True), out=self.d_down, add=self.d_down, status=self.status)
        dgu_row, dgu_col = _forms(dgu, self.grad, self.grad)
        mx.matmul(dgu_col, kept.x, out=self.d_gate_up, add=self.d_gate_up, status=self.status)
        return mx.matmul(dgu_row, self.w1t, status=self.status)


def gathered(flat: torch.Tensor, K: int, F: int):
    """gate_up [2 F, K] and down [K, F] as views of a gathered flat parameter
    (``Codec.gather_decode``'s result: raw BF16 patterns)."""
    w = flat.view(torch.bfloat16)
    return w[:2 * F * K].view(2 * F, K), w[2 * F * K:3 * F * K].view(K, F)


def descend(flat: torch.Tensor, K: int, F: int, mlp: GatedMLP, rate: float = 20.0):
    """A plain gradient step on the gathered weights, which clears the sums."""
    gate_up, down = gathered(flat, K, F)
    for w, d in ((gate_up, mlp.d_gate_up), (down, mlp.d_down)):
        w.copy_(w.float() - rate * d)
        d.zero_()
    return gate_up, down


def main(K: int = 1024, F: int = 4096, T: int = 2048, W: int = 8, steps: int = 3) -> None:
    from .codec import Codec
    torch.manual_seed(0)
    n = 3 * F * K
    shards = torch.randn(n, device="cuda").mul_(0.02).to(torch.bfloat16)
    codec = Codec(n, W)
    codec.stats(shards)
    codec.encode_code3(shards)
    recv, offsets = codec.exchange()
    flat = codec.gather_decode(recv, offsets)
    assert codec.status_word() == 0 and torch.equal(flat[:n].view(torch.bfloat16), shards)
    mlp = GatedMLP(*gathered(flat, K, F))
    x, target = (torch.randn(T, K, device="cuda").to(torch.bfloat16) for _ in range(2))
    for step in range(steps):
        y, kept = mlp.forward(x)
        dy = (y.float() - target.float()).div_(T * K).to(torch.bfloat16)
        mlp.backward(dy, kept)
        if mlp.status_word():
            raise RuntimeError(f"step {step}: a product timed out, status {mlp.status_word()}")
        loss = (y.float() - target.float()).square().mean().item() / 2
        print(f"step {step}: loss {loss:.6f}, |d gate_up| {mlp.d_gate_up.norm().item():.4e}, "
              f"|d down| {mlp.d_down.norm().item():.4e}")
        mlp.load(*descend(flat, K, F, mlp))
    y, _ = mlp.forward(x[:1], keep=False)
    print(f"one token: {tuple(y.shape)}, status {mlp.status_word()}, payload {recv.numel() / (2 * n):.3f} of BF16")


if __name__ == "__main__":
    main()
