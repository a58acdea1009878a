"""Microscaled (MX) tensors: 4- and 8-bit forms of BF16 matrices, their
products, and a gated unit that keeps its inputs in 8 bits.

A thin layer over the ``ez_mx_*`` entry points of include/expzip.h, which
define the formats and the layout: it checks shapes, types and strides, takes
or allocates the caller's buffers with torch and forwards each call on the
current stream.

    x4, x8 = MxTensor.empty("e2m1", T, K), MxTensor.empty("e4m3", K, T)
    quantize(x, row=x4, col=x8)          # forward operand, 8-bit checkpoint
    y = matmul(x4, w4)                   # [T, N] BF16, w4 an MxTensor [N, K]
    dw = matmul(dy8, x8, add=dw)         # [N, K] FP32, dy8 the column form of dy

A call given a ``stream`` runs there, after what the caller has ordered before it.
A result that it allocates is that stream's memory, as if made under
``torch.cuda.stream(stream)``: to use it on another one, wait for ``stream``, and
keep it, or ``record_stream`` it, until that use is over.

No call takes part in autograd: gradients come from ``swiglu_backward`` and from
products with the other forms.  A matrix that a result would be differentiable in
is therefore refused while gradients are recorded, if it requires them.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import binding as B

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
FORMATS = {"e2m1": B.EZ_MX_E2M1, "e4m3": B.EZ_MX_E4M3, "e5m2": B.EZ_MX_E5M2}


class MxTensor:
    """One form [rows, cols] of a microscaled matrix: ``codes`` (uint8, ``rows``
    rows of 16 or 32 bytes a block of 32 values) and ``scales`` (uint8, 512-byte
    tiles of 128 rows by 4 blocks).  Both are looked at in every call: they may be
    replaced, and their memory released and taken again, between calls."""
    __slots__ = ("format", "rows", "cols", "codes", "scales")

    def __init__(self, format: str, rows: int, cols: int, codes: torch.Tensor, scales: torch.Tensor):
        self.format, self.rows, self.cols, self.codes, self.scales = format, rows, cols, codes, scales

    def __repr__(self) -> str:
        return f"MxTensor({self.format!r}, {self.rows}, {self.cols}, on {self.codes.device})"

    @classmethod
    def empty(cls, format: str, rows: int, cols: int, device="cuda") -> "MxTensor":
        c, s = B.ez_mx_sizes(_format(format), rows, cols)
        return cls(format, rows, cols, torch.empty(rows, c // max(rows, 1), dtype=torch.uint8, device=device),
                   torch.empty(s, dtype=torch.uint8, device=device))


def _format(name: str) -> int:
    if name not in FORMATS:
        raise ValueError(f"unknown microscaled format {name!r}: one of {sorted(FORMATS)}")
    return FORMATS[name]


def _form(t: MxTensor, what: str):
    """(format, rows, cols, device, codes, scales) of a form whose tensors hold it;
    the addresses are None if they are not on one GPU."""
    rows, cols, codes, scales = t.rows, t.cols, t.codes, t.scales
    f, nb = FORMATS.get(t.format) or _format(t.format), (cols + 31) // 32
    if codes.nbytes != rows * nb * (16 if f == B.EZ_MX_E2M1 else 32) \
            or scales.nbytes != (rows + 127) // 128 * ((nb + 3) // 4) * 512 \
            or not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError(f"{what}: codes and scales do not hold a {t.format} form [{rows}, {cols}]")
    device = codes.get_device()
    if device < 0 or scales.get_device() != device:
        return f, rows, cols, device, None, None
    return f, rows, cols, device, codes.data_ptr(), scales.data_ptr()


def _apart():
    return ValueError(f"all tensors have to be on the current device, cuda:{B._current()[0]()}")


def _off_gpu():
    return ValueError("codes and scales have to be on the GPU, on the same one")


def _matrix(t: torch.Tensor, what: str, device: int, shape: Optional[Tuple[int, int]] = None,
            dtype: torch.dtype = _BF16) -> int:
    """Row stride of a row-major matrix on a device, after its checks."""
    size = t.shape
    if t.dtype is not dtype or len(size) != 2 or t.get_device() != device or device < 0:
        if t.dtype is not dtype or len(size) != 2 or not t.is_cuda:
            raise ValueError(f"{what}: a CUDA matrix of {dtype} is needed, got {t.dtype} of {len(size)} dimensions")
        raise _off_gpu() if device < 0 else _apart()
    if shape is not None and size != shape:
        raise ValueError(f"{what}: shape {tuple(size)} instead of {shape}")
    rows, cols = size
    ld, one = t.stride()
    if cols > 1 and one != 1 or rows > 1 and ld < cols:
        raise ValueError(f"{what}: rows have to be contiguous and apart (strides {t.stride()})")
    return ld if rows > 1 else cols


def _no_history(what: str) -> None:
    """For a matrix that requires grad."""
    if torch.is_grad_enabled():
        raise ValueError(f"{what} requires grad, which this call does not record: detach it, or call under no_grad")


# The C entry points are called without the wrappers of `binding`: these calls
# are often shorter than a general wrapper's steps.

def _on(stream, device: int, also: int) -> Optional[int]:
    """The stream to launch on.  The kernels run on the current device, so what they
    are given has to be there."""
    current = B._raw or B._current()
    if not device == also == current[0]():
        raise _apart()
    return current[1](device) if stream is None else B._stream(stream)


def _new(shape, dtype: torch.dtype, device, stream) -> torch.Tensor:
    """Memory for a result that is written on ``stream``: the allocator hands out
    and takes back blocks in the order of one stream, so it has to be that one."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(B._stream(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def quantize(x: torch.Tensor, row: Optional[MxTensor] = None, col: Optional[MxTensor] = None,
             stream=None) -> None:
    """Fill ``row`` with the row form of ``x`` [R, C] and ``col`` with its
    column form (the transpose, [C, R]), in one pass over ``x``."""
    if row is None and col is None:
        raise ValueError("quantize: neither a row form nor a column form to fill")
    device = cd = x.get_device()
    ld = _matrix(x, "x", device)
    R, C = x.shape
    rf = cf = 0
    rc = rs = cc = cs = None
    if row is not None:
        rf, r, c, rd, rc, rs = _form(row, "row")
        if r != R or c != C:
            raise ValueError(f"row: form [{r}, {c}] of a matrix [{R}, {C}]")
        if rc is None:
            raise _off_gpu()
        if rd != device:
            raise _apart()
    if col is not None:
        cf, r, c, cd, cc, cs = _form(col, "col")
        if r != C or c != R:
            raise ValueError(f"col: form [{r}, {c}] of a matrix [{R}, {C}]")
        if cc is None:
            raise _off_gpu()
    status = B.lib().ez_mx_quantize(x.data_ptr(), R, C, ld, rf, rc, rs, cf, cc, cs, _on(stream, device, cd))
    if status:
        raise B.EzError("ez_mx_quantize", status)


def dequantize(t: MxTensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The values of ``t`` as BF16 [rows, cols] (exact)."""
    f, rows, cols, device, codes, scales = _form(t, "t")
    if out is None:
        out = _new((rows, cols), _BF16, t.codes.device, stream)
    ld = _matrix(out, "out", device, (rows, cols))
    if codes is None:
        raise _off_gpu()
    rc = B.lib().ez_mx_dequantize(f, codes, scales, rows, cols, out.data_ptr(), ld, _on(stream, device, device))
    if rc:
        raise B.EzError("ez_mx_dequantize", rc)
    return out


_status = {}


def status_word(device) -> torch.Tensor:
    """The int32 word of a device that collects the EZ_DSTAT_* bits of products
    called without a word of their own (made at the first of them, which therefore
    has to come before a stream capture)."""
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError(f"status_word: a CUDA device is needed, got {device}")
    n = torch.cuda.current_device() if device.index is None else device.index
    if n not in _status:
        # from the host, so that it is there for every stream
        _status[n] = torch.tensor([0], dtype=torch.int32, device=torch.device("cuda", n))
    return _status[n]


def matmul(a: MxTensor, b: MxTensor, out: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
           add: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
           stream=None) -> torch.Tensor:
    """``a`` [M, K] times the transpose of ``b`` [N, K]: [M, N] in ``dtype`` or
    ``out``'s (BF16 or FP32).  ``add``: an FP32 matrix to add to an FP32 result,
    of the result's strides (or ``out`` itself).  ``status``: an int32 word that
    receives EZ_DSTAT_TIMEOUT, without one ``status_word``'s: as nothing else tells of
    it, read the word before a result counts (``int(word.item())`` waits for the
    product; it stays set until it is cleared)."""
    fa, M, K, da, ac, asc = _form(a, "a")
    fb, N, Kb, db, bc, bsc = _form(b, "b")
    if K != Kb:
        raise ValueError(f"matmul: inner sizes {K} and {Kb} differ")
    if fa != fb and (fa == B.EZ_MX_E2M1 or fb == B.EZ_MX_E2M1):
        raise ValueError(f"matmul: {a.format} and {b.format} do not multiply (both e2m1, or both 8-bit formats)")
    shape = (M, N)
    if out is None:
        out = _new(shape, _F32 if add is not None else dtype, a.codes.device, stream)
    kind = out.dtype
    if kind is not _BF16 and kind is not _F32:
        raise ValueError(f"matmul: out is BF16 or FP32, got {kind}")
    f32 = 1 if kind is _F32 else 0
    device = out.get_device()
    ld = _matrix(out, "out", device, shape, kind)
    more = None
    if add is not None:
        if not f32:
            raise ValueError("matmul: add needs an FP32 result")
        if _matrix(add, "add", device, shape, _F32) != ld:
            raise ValueError("matmul: add and out have different row strides")
        if add.requires_grad:
            _no_history("add")
        more = add.data_ptr()
    if status is None:
        status = status_word(out.device)
    elif status.dtype is not _I32 or not status.is_cuda:
        raise ValueError("matmul: status is an int32 word on the GPU")
    if ac is None or bc is None:
        raise _off_gpu()
    if not device == da == db:
        raise _apart()
    rc = B.lib().ez_mx_matmul(fa, ac, asc, M, fb, bc, bsc, N, K, more, out.data_ptr(), ld, f32, status.data_ptr(),
                              _on(stream, device, status.get_device()))
    if rc:
        raise B.EzError("ez_mx_matmul", rc)
    return out


def swiglu(gate: torch.Tensor, up: torch.Tensor, gate8: MxTensor, up8: MxTensor,
           out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """silu(gate) * up as BF16, filling ``gate8`` and ``up8`` (e4m3 or e5m2) with
    the 8-bit row forms of the inputs for ``swiglu_backward``."""
    shape = tuple(gate.shape)
    device = gate.get_device()
    ldg, ldu = _matrix(gate, "gate", device), _matrix(up, "up", device, shape)
    if gate.requires_grad or up.requires_grad:
        _no_history("gate" if gate.requires_grad else "up")
    f, kept, gc, gs, uc, us = _gated_forms(gate8, up8, shape)
    if out is None:
        out = _new(shape, _BF16, gate.device, stream)
    ldh = _matrix(out, "out", device, shape)
    rc = B.lib().ez_mx_swiglu(f, gate.data_ptr(), ldg, up.data_ptr(), ldu, shape[0], shape[1], gc, gs, uc, us,
                              out.data_ptr(), ldh, _on(stream, device, kept))
    if rc:
        raise B.EzError("ez_mx_swiglu", rc)
    return out


def swiglu_backward(gate8: MxTensor, up8: MxTensor, dh: torch.Tensor, dgate: torch.Tensor, dup: torch.Tensor,
                    h: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write the gradients of gate and up, and h again if it is given, from the
    8-bit checkpoint of ``swiglu`` and the gradient ``dh`` of its result."""
    shape = (gate8.rows, gate8.cols)
    f, device, gc, gs, uc, us = _gated_forms(gate8, up8, shape)
    ldd, ldg, ldu = (_matrix(dh, "dh", device, shape), _matrix(dgate, "dgate", device, shape),
                     _matrix(dup, "dup", device, shape))
    hp, ldh = (None, 0) if h is None else (h.data_ptr(), _matrix(h, "h", device, shape))
    if dh.requires_grad:
        _no_history("dh")
    rc = B.lib().ez_mx_swiglu_backward(f, gc, gs, uc, us, shape[0], shape[1], dh.data_ptr(), ldd, dgate.data_ptr(), ldg,
                                       dup.data_ptr(), ldu, hp, ldh, _on(stream, device, device))
    if rc:
        raise B.EzError("ez_mx_swiglu_backward", rc)


def _gated_forms(gate8: MxTensor, up8: MxTensor, shape):
    f, rows, cols, dg, gc, gs = _form(gate8, "gate8")
    fu, rows_u, cols_u, du, uc, us = _form(up8, "up8")
    if f != fu or f == B.EZ_MX_E2M1:
        raise ValueError(f"swiglu: the checkpoint is e4m3 or e5m2, got {gate8.format} and {up8.format}")
    if (rows, cols) != shape or (rows_u, cols_u) != shape:
        raise ValueError(f"swiglu: checkpoint forms do not have the shape {shape}")
    if gc is None or uc is None:
        raise _off_gpu()
    if dg != du:
        raise _apart()
    return f, dg, gc, gs, uc, us
