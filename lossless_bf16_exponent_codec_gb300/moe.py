"""Experts on microscaled operands: tokens sorted by expert and back, the
experts' products, and a layer of gated experts made of them.

A thin layer over the ``ez_moe_*`` entry points of include/expzip.h, by the rules
of ``mx`` (checks, streams, memory of results, no autograd).  The host never
looks at how many tokens an expert has: everything works on as many rows as any
choice can need, and ends where the device says that the experts' rows end.

    routing = sort(ids, experts)                  # ids [T, k]: the experts each token chose
    dispatch(x, routing, row=x4, col=x8)          # forms of the tokens' rows in the experts' order
    y = expert_matmul(x4, w4, routing)            # each expert's rows times its own matrix
    out = combine(y, routing, weights)            # back to the tokens, weighted

and the gradients: ``dispatch`` with the weights (of ``combine``'s input),
``weight_gradient`` (of the weights), ``combine`` without weights (of
``dispatch``'s input), ``expert_matmul`` with the transposed matrices and
``expert_gradient`` (of the matrices).

``python -m lossless_bf16_exponent_codec_gb300.moe`` gathers random weights through
the 3-bit exponent code and runs training steps and a decoding step.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import binding as B
from . import mx
from .mlp import load_norm, new_norm
from .mx import MxStack, MxTensor, _apart, _filled, _form, _matrix, _new, _no_history, _off_gpu, _on, _stack, _vector

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


class Routing:
    """Who goes where: ``tokens`` tokens with ``choices`` choices each among
    ``experts`` experts, in ``rows`` rows.  int32 tensors on the device: ``counts``
    [experts], ``offsets`` [experts + 1] (multiples of 128), ``slots`` [tokens,
    choices] (the row of each choice, -1 if its id named no expert) and ``sources``
    [rows] (the choice, token * choices + j, of each row, -1 in the padding).  Those
    of ``sort`` lie one behind the other in one tensor, of which views are made when
    they are asked for: making four tensors took the host longer than the launch."""
    __slots__ = ("tokens", "choices", "experts", "rows", "_parts", "_memory")

    def __init__(self, tokens: int, choices: int, experts: int, counts: torch.Tensor, offsets: torch.Tensor,
                 slots: torch.Tensor, sources: torch.Tensor):
        self.tokens, self.choices, self.experts = tokens, choices, experts
        self.rows = _rows(tokens, choices, experts)
        self._parts, self._memory = [counts, offsets, slots, sources], None

    @classmethod
    def _of(cls, tokens: int, choices: int, experts: int, rows: int, memory: torch.Tensor) -> "Routing":
        r = cls.__new__(cls)
        r.tokens, r.choices, r.experts, r.rows, r._parts, r._memory = tokens, choices, experts, rows, [None] * 4, memory
        return r

    def _part(self, i: int) -> torch.Tensor:
        t = self._parts[i]
        if t is None:
            E, T, k = self.experts, self.tokens, self.choices
            size, step, at = ((E,), (1,), 0) if i == 0 else ((E + 1,), (1,), E) if i == 1 else \
                ((T, k), (k, 1), 2 * E + 1) if i == 2 else ((self.rows,), (1,), 2 * E + 1 + T * k)
            t = self._parts[i] = self._memory.as_strided(size, step, at)
        return t

    counts = property(lambda self: self._part(0))
    offsets = property(lambda self: self._part(1))
    slots = property(lambda self: self._part(2))
    sources = property(lambda self: self._part(3))

    def _at(self, i: int, device: int) -> int:
        """Address of counts, offsets, slots or sources, after its checks."""
        E, n = self.experts, self.tokens * self.choices
        if self._memory is None:
            if i == 2:
                return _per_choice(self._parts[2], "routing.slots", device, self, _I32)
            return _vector(self._parts[i], "routing." + ("counts", "offsets", "slots", "sources")[i], device,
                           (E, E + 1, n, self.rows)[i], _I32)
        if self._memory.get_device() != device:
            raise _apart()
        return self._memory.data_ptr() + 4 * (0, E, 2 * E + 1, 2 * E + 1 + n)[i]

    def __repr__(self) -> str:
        return f"Routing({self.tokens} tokens x {self.choices} of {self.experts} experts, {self.rows} rows)"


def _per_choice(t: torch.Tensor, what: str, device: int, r: Routing, dtype: torch.dtype) -> int:
    """Address of a value for each choice, [tokens, choices] or all in one row, after its
    checks: any other shape would be read in another order than its own."""
    at = _vector(t, what, device, r.tokens * r.choices, dtype)
    if t.dim() != 1 and t.shape != (r.tokens, r.choices):
        raise ValueError(f"{what}: shape {tuple(t.shape)} instead of {(r.tokens, r.choices)}")
    return at


def _rows(tokens: int, choices: int, experts: int) -> int:
    """As ez_moe_rows, in fewer steps of the host."""
    pairs = tokens * choices
    return (pairs + 127 * min(experts, pairs)) // 128 * 128


def sort(ids: torch.Tensor, experts: int, stream=None) -> Routing:
    """The routing of ``ids`` [T, k] (int32 or int64): choices of one expert in
    ascending order of (token, choice).  Ids outside [0, experts) name no expert."""
    kind = ids.dtype
    if (kind is not _I32 and kind is not torch.int64) or ids.dim() != 2 or not ids.is_cuda:
        raise ValueError(f"ids: a CUDA matrix of int32 or int64 is needed, got {kind} of {ids.dim()} dimensions")
    device = ids.get_device()
    ld = _matrix(ids, "ids", device, None, kind)
    T, k = ids.shape
    rows, need = _rows(T, k, experts), B.ez_moe_sort_ws(T, k, experts) if T * k > 1024 else 0
    if stream is None:
        memory = torch.empty(2 * experts + 1 + T * k + rows, dtype=_I32, device=ids.device)
        ws = torch.empty(need // 4, dtype=_I32, device=ids.device) if need else None
    else:
        memory = _new((2 * experts + 1 + T * k + rows,), _I32, ids.device, stream)
        ws = _new((need // 4,), _I32, ids.device, stream) if need else None
    at = memory.data_ptr()
    slots = at + 8 * experts + 4
    rc = B.lib().ez_moe_sort(ids.data_ptr(), ids.element_size(), ld, T, k, experts, at, at + 4 * experts, slots,
                             slots + 4 * T * k, None if ws is None else ws.data_ptr(), need, _on(stream, device, device))
    if rc:
        raise B.EzError("ez_moe_sort", rc)
    return Routing._of(T, k, experts, rows, memory)


def dispatch(x: torch.Tensor, routing: Routing, row: Optional[MxTensor] = None, col: Optional[MxTensor] = None,
             weights: Optional[torch.Tensor] = None, stream=None) -> None:
    """Fill ``row`` [rows, C] with the row form and ``col`` [C, rows] with the column
    form of the tokens' rows of ``x`` [T, C] in the experts' order, zeros in the
    padding; with ``weights`` [T, k] FP32 of each row times its choice's weight,
    rounded to BF16.  What lies behind the last expert is left as it was."""
    if row is None and col is None:
        raise ValueError("dispatch: neither a row form nor a column form to fill")
    device = x.get_device()
    ld = _matrix(x, "x", device)
    T, C = x.shape
    r = routing
    if T != r.tokens:
        raise ValueError(f"x: {T} rows for a routing of {r.tokens} tokens")
    if x.requires_grad or (weights is not None and weights.requires_grad):
        _no_history("x" if x.requires_grad else "weights")
    wp = None if weights is None else _per_choice(weights, "weights", device, r, _F32)
    rf, rc, rs = _filled(row, "row", r.rows, C, device)
    cf, cc, cs = _filled(col, "col", C, r.rows, device)
    status = B.lib().ez_moe_dispatch(x.data_ptr(), ld, T, C, r._at(1, device), r._at(3, device), r._at(2, device),
                                     r.choices, r.experts, wp, rf, rc, rs, cf, cc, cs, _on(stream, device, device))
    if status:
        raise B.EzError("ez_moe_dispatch", status)


def combine(rows: torch.Tensor, routing: Routing, weights: Optional[torch.Tensor] = None,
            out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """BF16 [T, C]: for each token the sum over its choices of the weight (1 without
    ``weights`` [T, k] FP32) times the choice's row of ``rows`` [rows, C]."""
    device = rows.get_device()
    ld = _matrix(rows, "rows", device)
    r = routing
    n, C = rows.shape
    if n != r.rows:
        raise ValueError(f"rows: {n} rows for a routing of {r.rows}")
    if rows.requires_grad or (weights is not None and weights.requires_grad):
        _no_history("rows" if rows.requires_grad else "weights")
    wp = None if weights is None else _per_choice(weights, "weights", device, r, _F32)
    if out is None:
        out = _new((r.tokens, C), _BF16, rows.device, stream)
    ldo = _matrix(out, "out", device, (r.tokens, C))
    rc = B.lib().ez_moe_combine(rows.data_ptr(), ld, n, C, r._at(2, device), wp, r.tokens, r.choices,
                                out.data_ptr(), ldo, _on(stream, device, device))
    if rc:
        raise B.EzError("ez_moe_combine", rc)
    return out


def weight_gradient(dy: torch.Tensor, rows: torch.Tensor, routing: Routing, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """FP32 [T, k]: the gradient of ``combine``'s weights, each token's ``dy`` [T, C]
    times its choices' rows (0 for choices without one)."""
    device = dy.get_device()
    ldd = _matrix(dy, "dy", device)
    r = routing
    T, C = dy.shape
    ld = _matrix(rows, "rows", device, (r.rows, C))
    if T != r.tokens:
        raise ValueError(f"dy: {T} rows for a routing of {r.tokens} tokens")
    if dy.requires_grad or rows.requires_grad:
        _no_history("dy" if dy.requires_grad else "rows")
    if out is None:
        out = _new((T, r.choices), _F32, dy.device, stream)
    rc = B.lib().ez_moe_weight_gradient(dy.data_ptr(), ldd, rows.data_ptr(), ld, r.rows, C, r._at(2, device), T,
                                        r.choices, _per_choice(out, "out", device, r, _F32), _on(stream, device, device))
    if rc:
        raise B.EzError("ez_moe_weight_gradient", rc)
    return out


def _status(status: Optional[torch.Tensor], device: torch.device) -> torch.Tensor:
    if status is None:
        return mx.status_word(device)
    if status.dtype is not _I32 or not status.is_cuda:
        raise ValueError("status is an int32 word on the GPU")
    return status


def expert_matmul(a: MxTensor, b: MxStack, routing: Routing, out: Optional[torch.Tensor] = None,
                  dtype: torch.dtype = torch.bfloat16, status: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """[rows, N] in ``dtype`` or ``out``'s (BF16 or FP32): each expert's rows of ``a``
    [rows, K] times the transpose of its matrix of ``b`` (experts x [N, K]).  Padding
    gives zeros (``dispatch`` leaves it zero) but for matrices with infinities or NaN;
    what lies behind the last expert is left as it was.  ``status`` as in ``mx.matmul``."""
    fa, R, K, da, ac, asc = _form(a, "a")
    fb, E, N, Kb, db, bc, bsc = _stack(b, "b")
    r = routing
    if K != Kb:
        raise ValueError(f"expert_matmul: inner sizes {K} and {Kb} differ")
    if fa != fb and (fa == B.EZ_MX_E2M1 or fb == B.EZ_MX_E2M1):
        raise ValueError(f"expert_matmul: {a.format} and {b.format} do not multiply (both e2m1, or both 8-bit formats)")
    if R != r.rows or E != r.experts:
        raise ValueError(f"expert_matmul: {R} rows and {E} matrices for a routing of {r.rows} and {r.experts}")
    if out is None:
        out = _new((R, N), dtype, a.codes.device, stream)
    kind = out.dtype
    if kind is not _BF16 and kind is not _F32:
        raise ValueError(f"expert_matmul: out is BF16 or FP32, got {kind}")
    device = out.get_device()
    ld = _matrix(out, "out", device, (R, N), kind)
    status = _status(status, out.device)
    if ac is None or bc is None:
        raise _off_gpu()
    if not device == da == db:
        raise _apart()
    rc = B.lib().ez_moe_matmul(fa, ac, asc, R, fb, bc, bsc, E, N, K, r._at(0, device), r._at(1, device),
                               r.tokens * r.choices, out.data_ptr(), ld, 1 if kind is _F32 else 0, status.data_ptr(),
                               _on(stream, device, status.get_device()))
    if rc:
        raise B.EzError("ez_moe_matmul", rc)
    return out


def expert_gradient(a: MxTensor, b: MxTensor, routing: Routing, out: Optional[torch.Tensor] = None,
                    add: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """FP32 [experts, N, K]: for each expert the sum over its rows of a column of
    ``a`` [N, rows] times a column of ``b`` [K, rows] (8-bit forms, zero in the
    padding), with ``add`` of the same strides (or ``out`` itself) added."""
    fa, N, R, da, ac, asc = _form(a, "a")
    fb, K, Rb, db, bc, bsc = _form(b, "b")
    r = routing
    if fa == B.EZ_MX_E2M1 or fb == B.EZ_MX_E2M1:
        raise ValueError(f"expert_gradient: operands are e4m3 or e5m2, got {a.format} and {b.format}")
    if R != r.rows or Rb != R:
        raise ValueError(f"expert_gradient: {R} and {Rb} columns for a routing of {r.rows} rows")
    shape = (r.experts, N, K)
    if out is None:
        out = _new(shape, _F32, a.codes.device, stream)
    device = out.get_device()
    ld = _matrices(out, "out", device, shape)
    ap = None
    if add is not None:
        if _matrices(add, "add", device, shape) != ld:
            raise ValueError("expert_gradient: add and out have different strides")
        if add.requires_grad:
            _no_history("add")
        ap = add.data_ptr()
    status = _status(status, out.device)
    if ac is None or bc is None:
        raise _off_gpu()
    if not device == da == db:
        raise _apart()
    rc = B.lib().ez_moe_gradient(fa, ac, asc, N, fb, bc, bsc, K, R, r.experts,
                                 r._at(1, device), ap, out.data_ptr(), ld, status.data_ptr(), _on(stream, device, status.get_device()))
    if rc:
        raise B.EzError("ez_moe_gradient", rc)
    return out


def _matrices(t: torch.Tensor, what: str, device: int, shape: Tuple[int, int, int]) -> int:
    """Row stride of FP32 matrices that lie one behind the other, after their checks."""
    if t.dtype is not _F32 or tuple(t.shape) != shape or not t.is_cuda:
        raise ValueError(f"{what}: CUDA matrices of FP32 {shape} are needed, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != device:
        raise _apart()
    E, N, K = shape
    apart, ld, one = t.stride()
    ld = ld if N > 1 else apart if E > 1 else K
    if (K > 1 and one != 1) or ld < K or (E > 1 and apart != N * ld):
        raise ValueError(f"{what}: rows have to be contiguous and the matrices one behind the other (strides {t.stride()})")
    return ld


# ------------------------------------------------------------------- a layer

def _quantize_each(w: torch.Tensor, row: MxStack, col: MxStack) -> None:
    """The forms of the matrices w [E, N, K] in BF16 and of their transposes."""
    for e in range(w.shape[0]):
        mx.quantize(w[e], row=row[e], col=col[e])


@dataclass
class Kept:
    """What a forward pass keeps for its backward pass: 8 bits a value, the experts'
    results (for the weights' gradient) and what the norm needs in BF16."""
    routing: Routing
    weights: torch.Tensor
    x: MxTensor                         # column form of the dispatched rows
    gate: MxTensor
    up: MxTensor
    rows: torch.Tensor                  # the experts' results
    total: Optional[torch.Tensor]       # with a norm: x + residual
    rstd: Optional[torch.Tensor]


class ExpertMLP:
    """Gated experts: ``gate_up`` [E, 2 F, K] (gate rows first) and ``down`` [E, K, F]
    in BF16, as gathered, on tokens that have chosen among them; with ``norm`` [K]
    in BF16 a root-mean-square norm of the residual stream stands in front.  ``grad``
    and ``kept`` as in ``mlp.GatedMLP``, and so are ``status`` and what it means."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, norm: Optional[torch.Tensor] = None,
                 grad: str = "e5m2", kept: str = "e4m3", eps: float = 1e-6):
        self.E, self.F, self.K = gate_up.shape[0], gate_up.shape[1] // 2, gate_up.shape[2]
        self._fits(gate_up, down)
        self.grad, self.kept, self.eps = grad, kept, eps
        device = gate_up.device
        self.status = torch.zeros(1, dtype=_I32, device=device)
        self.norm = new_norm(norm, self.K, device)
        E, F2, F, K = self.E, 2 * self.F, self.F, self.K
        self.w1, self.w1t = (MxStack.empty(*stack, device) for stack in (("e2m1", E, F2, K), ("e4m3", E, K, F2)))
        self.w2, self.w2t = (MxStack.empty(*stack, device) for stack in (("e2m1", E, K, F), ("e4m3", E, F, K)))
        self.load(gate_up, down, norm)
        self.d_gate_up = torch.zeros(self.E, 2 * self.F, self.K, dtype=_F32, device=device)
        self.d_down = torch.zeros(self.E, self.K, self.F, dtype=_F32, device=device)
        self.d_norm = None if norm is None else torch.zeros(self.K, dtype=_F32, device=device)

    def _fits(self, gate_up: torch.Tensor, down: torch.Tensor) -> None:
        if tuple(gate_up.shape) != (self.E, 2 * self.F, self.K) or tuple(down.shape) != (self.E, self.K, self.F):
            raise ValueError(f"gate_up {tuple(gate_up.shape)} and down {tuple(down.shape)} do not make gated experts, "
                             f"{self.E} of {self.K} and {self.F}")

    def load(self, gate_up: torch.Tensor, down: torch.Tensor, norm: Optional[torch.Tensor] = None) -> None:
        """Quantise newly gathered weights: 4 bits for the forward products, the
        transposes in 8 for the data gradients.  The norm's weight is copied: nothing that
        is given here is looked at later.  A layer made with a norm needs one here too.

        Everything goes, on the current stream, into the memory that the layer has had from
        the start: passes captured before run with what was loaded last, and passes on other
        streams have to be over."""
        self._fits(gate_up, down)
        load_norm(self.norm, norm)
        _quantize_each(gate_up, self.w1, self.w1t)
        _quantize_each(down, self.w2, self.w2t)

    def status_word(self) -> int:
        """EZ_DSTAT_* bits of all products since the last ``clear_status`` (waits for
        them)."""
        return int(self.status.item())

    def clear_status(self) -> None:
        self.status.zero_()

    def forward(self, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, keep: bool = True,
                residual: Optional[torch.Tensor] = None, total: Optional[torch.Tensor] = None):
        """y [T, K] = sum over the choices ``ids`` [T, k] of ``weights`` [T, k] (FP32)
        times the expert's result on x [T, K] (with a norm: on the norm of x +
        residual, which goes to ``total`` if it is given), and what ``backward``
        needs (None unless ``keep``).  That holds ``weights`` and, with a norm, ``total`` as
        given, or x where there is neither it nor a residual: what is written into these
        tensors before ``backward`` makes the gradients wrong."""
        if x.requires_grad:
            _no_history("x")
        rstd = None
        if self.norm is None:
            if residual is not None or total is not None:
                raise ValueError("a residual and its total go with a norm")
        else:
            h = torch.empty(x.shape, dtype=_BF16, device=x.device)
            total, rstd = mx.rms_norm(x, self.norm, self.eps, residual=residual, total=total, out=h)
            x = h
        F, K = self.F, self.K
        routing = sort(ids, self.E)
        R = routing.rows
        x4 = MxTensor.empty("e2m1", R, K, x.device)
        x8 = MxTensor.empty(self.kept, K, R, x.device) if keep else None
        dispatch(x, routing, row=x4, col=x8)
        gu = expert_matmul(x4, self.w1, routing, status=self.status)
        gate8, up8 = (MxTensor.empty(self.kept, R, F, x.device) for _ in range(2))
        h = mx.swiglu(gu[:, :F], gu[:, F:], gate8, up8)
        h4 = MxTensor.empty("e2m1", R, F, x.device)
        mx.quantize(h, row=h4)
        rows = expert_matmul(h4, self.w2, routing, status=self.status)
        y = combine(rows, routing, weights)
        return y, Kept(routing, weights, x8, gate8, up8, rows, total, rstd) if keep else None

    def backward(self, dy: torch.Tensor, kept: Kept, dtotal: Optional[torch.Tensor] = None):
        """(dx [T, K], dweights [T, k]); the gradients of the experts' matrices and of
        the norm are added to ``d_gate_up``, ``d_down`` and ``d_norm``.  With a norm dx
        is the gradient of x and of the residual, ``dtotal`` what reaches their sum on
        other ways."""
        if dtotal is not None and self.norm is None:
            raise ValueError("dtotal goes with a norm")
        r, F, K = kept.routing, self.F, self.K
        R, new = r.rows, lambda *shape: torch.empty(*shape, dtype=_BF16, device=dy.device)
        dweights = weight_gradient(dy, kept.rows, r)
        row, col = MxTensor.empty(self.grad, R, K, dy.device), MxTensor.empty(self.grad, K, R, dy.device)
        dispatch(dy, r, row=row, col=col, weights=kept.weights)
        dh = expert_matmul(row, self.w2t, r, status=self.status)
        dgu, h = new(R, 2 * F), new(R, F)
        mx.swiglu_backward(kept.gate, kept.up, dh, dgu[:, :F], dgu[:, F:], h=h)
        h8 = MxTensor.empty(self.kept, F, R, dy.device)
        mx.quantize(h, col=h8)
        expert_gradient(col, h8, r, out=self.d_down, add=self.d_down, status=self.status)
        row, col = MxTensor.empty(self.grad, R, 2 * F, dy.device), MxTensor.empty(self.grad, 2 * F, R, dy.device)
        mx.quantize(dgu, row=row, col=col)
        expert_gradient(col, kept.x, r, out=self.d_gate_up, add=self.d_gate_up, status=self.status)
        dx = combine(expert_matmul(row, self.w1t, r, status=self.status), r)
        if self.norm is not None:
            dx = mx.rms_norm_backward(dx, kept.total, kept.rstd, self.norm, dtotal=dtotal, out=dx, dweight=self.d_norm,
                                      add=self.d_norm)
        return dx, dweights


def gathered(flat: torch.Tensor, E: int, K: int, F: int):
    """gate_up [E, 2 F, K], down [E, K, F] and norm [K] as views of a gathered flat
    parameter (``Codec.gather_decode``'s result: raw BF16 patterns)."""
    w = flat.view(_BF16)
    n = 2 * E * F * K
    return w[:n].view(E, 2 * F, K), w[n:n + n // 2].view(E, K, F), w[n + n // 2:n + n // 2 + K]


def main(E: int = 16, k: int = 2, K: int = 512, F: int = 1024, T: int = 2048, W: int = 8, steps: int = 3,
         rate: float = 20.0) -> None:
    from .codec import Codec
    torch.manual_seed(0)
    n = 3 * E * F * K + K
    shards = torch.randn(n, device="cuda").mul_(0.02)
    shards[-K:] = 1.0
    shards = shards.to(_BF16)
    codec = Codec(n, W)
    codec.stats(shards)
    codec.encode_code3(shards)
    flat = codec.gather_decode()
    assert codec.status_word() == 0 and torch.equal(flat[:n].view(_BF16), shards)
    layer = ExpertMLP(*gathered(flat, E, K, F))
    x, target = (torch.randn(T, K, device="cuda").to(_BF16) for _ in range(2))
    router = torch.randn(K, E, device="cuda").mul_(K ** -0.5).to(_BF16)
    for step in range(steps):
        top = torch.topk((x @ router).float(), k, dim=1)
        weights = torch.softmax(top.values, dim=1)
        y, kept = layer.forward(x, top.indices, weights)
        dy = (y.float() - target.float()).div_(T * K).to(_BF16)
        _, dweights = layer.backward(dy, kept)
        if layer.status_word():
            raise RuntimeError(f"step {step}: a product timed out, status {layer.status_word()}")
        loss = (y.float() - target.float()).square().mean().item() / 2
        print(f"step {step}: loss {loss:.6f}, |d gate_up| {layer.d_gate_up.norm().item():.4e}, |d down| "
              f"{layer.d_down.norm().item():.4e}, |d norm| {layer.d_norm.norm().item():.4e}, |d weights| "
              f"{dweights.norm().item():.4e}, tokens per expert {kept.routing.counts.tolist()}")
        parts = gathered(flat, E, K, F)
        for w, d in zip(parts, (layer.d_gate_up, layer.d_down, layer.d_norm)):
            w.copy_(w.float() - rate * d)
            d.zero_()
        layer.load(*parts)
    y, _ = layer.forward(x[:1], top.indices[:1], weights[:1], keep=False)
    print(f"one token: {tuple(y.shape)}, status {layer.status_word()}")


if __name__ == "__main__":
    main()
