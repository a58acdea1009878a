"""The cases that the microscaled (MX) operators are measured on, with their plain forms.

A microscaled tensor [rows, cols] holds E2M1 (4 bits), E4M3 or E5M2 (8 bits) codes in blocks of 32 values along a row,
with one scale byte k + 127 for each block; a value is code * 2^k.  ``plain`` below are those operators in elementary
torch operations in 32 bits; with ``own`` set, ``run`` calls the library's.

  quant   BF16 [R, C] to the row form and/or the column form (the transpose, blocks along a column), and back
  matmul  C[M, N] = A[M, K] B[N, K]^T of two microscaled tensors, BF16 or FP32 out, with or without an FP32 addend
  gated   h = silu(g) u, g and u kept in 8 bits; and the gradients of g and u from what was kept, with h again
"""
import math

import torch

own = False

BLOCK = 32
# largest magnitude, its frexp mantissa and exponent, mantissa bits, smallest normal exponent, range of k
FORMATS = {
    "e2m1": (6.0, 0.75, 3, 1, 0, -127, 125),
    "e4m3": (448.0, 0.875, 9, 3, -6, -124, 119),
    "e5m2": (57344.0, 0.875, 16, 2, -14, -117, 112),
}
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token's activations on their way into a 4-bit product: latency
        {"name": "quant_token", "op": "quant", "R": 1, "C": 5120, "row": "e2m1", "col": ""},
        # a weight matrix of odd sizes: both 4-bit forms, for the forward product and the data gradient
        {"name": "quant_weight_odd", "op": "quant", "R": 2001, "C": 4109, "row": "e2m1", "col": "e2m1"},
        # a training batch's activations: the 4-bit operand of the forward product and the 8-bit checkpoint in one call
        {"name": "quant_save_large", "op": "quant", "R": 16384, "C": 8192, "row": "e2m1", "col": "e4m3"},
        # a decoding step of one token: the weights are read once, everything else is latency
        {"name": "matmul4_token", "op": "matmul", "M": 1, "N": 8192, "K": 8192, "a": "e2m1", "b": "e2m1", "out": "bf16", "add": False},
        # a decoding step of a batch of sequences
        {"name": "matmul4_batch", "op": "matmul", "M": 48, "N": 10240, "K": 5120, "a": "e2m1", "b": "e2m1", "out": "bf16", "add": False},
        # a prompt of odd length against a weight of odd sizes
        {"name": "matmul4_ragged", "op": "matmul", "M": 1111, "N": 2049, "K": 4100, "a": "e2m1", "b": "e2m1", "out": "bf16", "add": False},
        # a training batch's forward product
        {"name": "matmul4_large", "op": "matmul", "M": 8192, "N": 8192, "K": 8192, "a": "e2m1", "b": "e2m1", "out": "bf16", "add": False},
        # a weight gradient: 8-bit output gradients times the 8-bit activation checkpoint, added to the FP32 gradient so far
        {"name": "matmul8_wgrad", "op": "matmul", "M": 8192, "N": 4096, "K": 16384, "a": "e5m2", "b": "e4m3", "out": "f32", "add": True},
        # the gated unit of a short sequence, odd width
        {"name": "gated_short", "op": "gated", "R": 129, "C": 2731, "fmt": "e4m3"},
        # the gated unit of a training batch
        {"name": "gated_large", "op": "gated", "R": 8192, "C": 14336, "fmt": "e4m3"},
        # its backward pass from the 8-bit checkpoint, odd sizes
        {"name": "gated_back_odd", "op": "gated_back", "R": 777, "C": 2730, "fmt": "e5m2"},
        # the same for a training batch
        {"name": "gated_back_large", "op": "gated_back", "R": 8192, "C": 14336, "fmt": "e4m3"},
    ]


def _size(rng, lo, hi, odd=0.5):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd:
        step = 32 if n >= 64 else 1
        n = max(step, n // step * step)
    return max(lo, min(hi, n)) if n != 3072 else 3040


def draw(rng):
    op = rng.choice(["quant", "quant", "matmul", "matmul", "matmul", "gated", "gated_back"])
    if op == "quant":
        row, col = rng.choice([("e2m1", ""), ("e2m1", "e2m1"), ("e2m1", "e4m3"), ("", "e5m2"), ("e4m3", ""), ("e4m3", "e4m3"), ("", "e2m1")])
        return {"op": op, "R": _size(rng, 1, 16384), "C": _size(rng, 32, 8192), "row": row, "col": col}
    if op == "matmul":
        if rng.random() < 0.5:
            a = b = "e2m1"
        else:
            a, b = rng.choice(["e4m3", "e5m2"]), rng.choice(["e4m3", "e5m2"])
        out = rng.choice(["bf16", "f32"])
        return {"op": op, "M": _size(rng, 1, 8192), "N": _size(rng, 64, 8192), "K": _size(rng, 32, 8192), "a": a, "b": b,
                "out": out, "add": out == "f32" and rng.random() < 0.5}
    return {"op": op, "R": _size(rng, 1, 8192), "C": _size(rng, 32, 14336), "fmt": rng.choice(["e4m3", "e5m2"])}


# ------------------------------------------------- the format in torch, 32 bits

def _cdiv(a, b):
    return -(-a // b)


def _pow2(k):
    """2^k in FP32 for integers -149 < k <= 127, as a product of two normal powers."""
    a = torch.div(k, 2, rounding_mode="floor")
    two = lambda e: ((e + 127) << 23).view(torch.float32)  # noqa: E731
    return two(a) * two(k - a)


def _quantize(x, fmt):
    """x [rows, cols] (any float type) -> values as FP32 [rows, cols] before scaling, and k [rows, blocks]; k = 128 marks a block
    with an infinity or NaN."""
    top, fm, fe, mbits, emin, kmin, kmax = FORMATS[fmt]
    rows, cols = x.shape
    nb = _cdiv(cols, BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - cols)).view(rows, nb, BLOCK)
    amax = v.abs().amax(dim=2)
    bad = ~torch.isfinite(amax)
    m, e = torch.frexp(torch.where(bad, 0.0, amax))
    k = torch.where(amax > 0, e - fe + (m > fm).int(), kmin).clamp(kmin, kmax).int()
    k = torch.where(bad, 128, k)
    v = torch.where(bad[..., None], 0.0, v) * _pow2(-k.clamp(max=127))[..., None]
    a = v.abs()
    ea = ((a.view(torch.int32) >> 23) - 127).clamp(emin, 127)
    q = _pow2(ea - mbits)
    r = torch.clamp(torch.round(a / q) * q, max=top)
    return torch.copysign(r, v).view(rows, nb * BLOCK)[:, :cols], k


def _values(r, k):
    """Codes' values r [rows, cols] times 2^k: FP32."""
    rows, cols = r.shape
    s = torch.where(k == 128, math.nan, _pow2(k.clamp(max=127)))
    return r * s.repeat_interleave(BLOCK, dim=1)[:, :cols]


def _pack(r, fmt):
    """Code bytes [rows, pitch]: 16 (E2M1, low half first) or 32 bytes a block, zeros past cols."""
    rows, cols = r.shape
    r = torch.nn.functional.pad(r, (0, _cdiv(cols, BLOCK) * BLOCK - cols))
    if fmt != "e2m1":
        return r.to(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).view(torch.uint8)
    table = torch.tensor(E2M1_VALUES, device=r.device)
    c = torch.searchsorted(table, r.abs().contiguous()).to(torch.uint8) | (torch.signbit(r).to(torch.uint8) << 3)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous()


def _unpack(codes, fmt, cols):
    if fmt != "e2m1":
        return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2).float()[:, :cols]
    table = torch.tensor(E2M1_VALUES + tuple(-v for v in E2M1_VALUES), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=2).view(codes.shape[0], -1)
    return table[c.int()][:, :cols]


def _tile_scales(k):
    """Scale bytes in their layout: 512-byte tiles of 128 rows by 4 blocks, byte (r % 32) * 16 + (r / 32) * 4 + block."""
    rows, nb = k.shape
    rt, kt = _cdiv(rows, 128), _cdiv(nb, 4)
    s = torch.nn.functional.pad((k + 127).to(torch.uint8), (0, kt * 4 - nb, 0, rt * 128 - rows))
    return s.view(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(s, rows, cols):
    nb = _cdiv(cols, BLOCK)
    rt, kt = _cdiv(rows, 128), _cdiv(nb, 4)
    return s.view(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :nb].int() - 127


def _decode(t):
    """FP32 values of a microscaled tensor as the library lays it out."""
    return _values(_unpack(t["codes"], t["fmt"], t["cols"]), _untile_scales(t["scales"], t["rows"], t["cols"]))


def _encode(x, fmt):
    r, k = _quantize(x, fmt)
    return {"fmt": fmt, "rows": x.shape[0], "cols": x.shape[1], "codes": _pack(r, fmt), "scales": _tile_scales(k)}


# -------------------------------------------------------------------- inputs

def _activations(g, rows, cols):
    """Activations: normal, a few channels much larger, tokens of different norm."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(torch.bfloat16)


def _weights(g, rows, cols):
    return (0.02 * torch.randn(rows, cols, generator=g, device="cuda")).to(torch.bfloat16)


def _gradients(g, rows, cols):
    """Gradients: small, heavy-tailed."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return (1e-4 * x * torch.exp(torch.randn(rows, cols, generator=g, device="cuda"))).to(torch.bfloat16)


def _operands(case, g):
    weight_grad = case["add"] or case["a"] == "e5m2"
    a = _gradients(g, case["M"], case["K"]) if weight_grad else _activations(g, case["M"], case["K"])
    b = _activations(g, case["N"], case["K"]) if weight_grad else _weights(g, case["N"], case["K"])
    return _encode(a, case["a"]), _encode(b, case["b"])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    state = {"case": case}
    if case["op"] == "quant":
        R, C = case["R"], case["C"]
        state["x"] = _activations(g, R, C)
        shapes = {"row": (R, C), "col": (C, R)}
        for side, (r, c) in shapes.items():
            if case[side]:
                state[side] = _buffers(case[side], r, c)
                state[side + "_values"] = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "matmul":
        state["a"], state["b"] = _operands(case, g)
        shape, kind = (case["M"], case["N"]), torch.bfloat16 if case["out"] == "bf16" else torch.float32
        state["add"] = 1e-3 * torch.randn(shape, generator=g, device="cuda") if case["add"] else None
        state["c"] = torch.empty(shape, dtype=kind, device="cuda")
        state["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        R, C = case["R"], case["C"]
        gu = torch.randn(R, 2 * C, generator=g, device="cuda").to(torch.bfloat16)
        state["gate"], state["up"] = gu[:, :C], gu[:, C:]
        new = lambda: torch.empty(R, C, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        state["h"] = new()
        if case["op"] == "gated":
            state["gate8"], state["up8"] = _buffers(case["fmt"], R, C), _buffers(case["fmt"], R, C)
            state["gate_values"], state["up_values"] = new(), new()
        else:
            state["gate8"], state["up8"] = _encode(state["gate"], case["fmt"]), _encode(state["up"], case["fmt"])
            state["gate"] = state["up"] = None
            state["dh"] = _gradients(g, R, C)
            state["dgate"], state["dup"] = new(), new()
    return state


def _buffers(fmt, rows, cols):
    nb = _cdiv(cols, BLOCK)
    return {"fmt": fmt, "rows": rows, "cols": cols,
            "codes": torch.empty(rows, nb * (16 if fmt == "e2m1" else 32), dtype=torch.uint8, device="cuda"),
            "scales": torch.empty(_cdiv(rows, 128) * _cdiv(nb, 4) * 512, dtype=torch.uint8, device="cuda")}


# ---------------------------------------------------------------------- run

def run(state):
    return _own(state) if own else _plain(state)


def _mx(t):
    from lossless_bf16_exponent_codec_gb300 import mx
    return None if t is None else mx.MxTensor(t["fmt"], t["rows"], t["cols"], t["codes"], t["scales"])


def _own(s):
    from lossless_bf16_exponent_codec_gb300 import mx
    op = s["case"]["op"]
    if op == "quant":
        row, col = _mx(s.get("row")), _mx(s.get("col"))
        mx.quantize(s["x"], row=row, col=col)
        return {side: mx.dequantize(t, out=s[side + "_values"]) for side, t in (("row", row), ("col", col)) if t is not None}
    if op == "matmul":
        return mx.matmul(_mx(s["a"]), _mx(s["b"]), out=s["c"], add=s["add"], status=s["status"])
    gate8, up8 = _mx(s["gate8"]), _mx(s["up8"])
    if op == "gated":
        h = mx.swiglu(s["gate"], s["up"], gate8, up8, out=s["h"])
        return {"h": h, "gate": mx.dequantize(gate8, out=s["gate_values"]), "up": mx.dequantize(up8, out=s["up_values"])}
    mx.swiglu_backward(gate8, up8, s["dh"], s["dgate"], s["dup"], h=s["h"])
    return {"dgate": s["dgate"], "dup": s["dup"], "h": s["h"]}


def _plain(s):
    case = s["case"]
    if case["op"] == "quant":
        x = s["x"]
        return {side: _values(*_quantize(v, case[side])).to(torch.bfloat16) for side, v in (("row", x), ("col", x.t())) if case[side]}
    if case["op"] == "matmul":
        c = _decode(s["a"]) @ _decode(s["b"]).t()
        c = c if s["add"] is None else c + s["add"]
        return c.to(torch.bfloat16) if case["out"] == "bf16" else c
    if case["op"] == "gated":
        g, u = s["gate"].float(), s["up"].float()
        keep = lambda v: _values(*_quantize(v, case["fmt"])).to(torch.bfloat16)  # noqa: E731
        return {"h": (g / (1 + torch.exp(-g)) * u).to(torch.bfloat16), "gate": keep(g), "up": keep(u)}
    g, u, dh = _decode(s["gate8"]), _decode(s["up8"]), s["dh"].float()
    p = 1 / (1 + torch.exp(-g))
    out = {"dgate": dh * u * p * (1 + g * (1 - p)), "dup": dh * g * p, "h": g * p * u}
    return {n: v.to(torch.bfloat16) for n, v in out.items()}


# --------------------------------------------------------------------- work

def _held(fmt, rows, cols):
    return rows * _cdiv(cols, BLOCK) * ((16 if fmt == "e2m1" else 32) + 1) if fmt else 0


def work(case):
    if case["op"] == "quant":
        R, C = case["R"], case["C"]
        forms = bool(case["row"]) + bool(case["col"])
        return {"bytes": 2 * R * C * (1 + forms) + _held(case["row"], R, C) + _held(case["col"], C, R), "flops": 4 * R * C * forms}
    if case["op"] == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        out = M * N * ((2 if case["out"] == "bf16" else 4) + (4 if case["add"] else 0))
        return {"bytes": _held(case["a"], M, K) + _held(case["b"], N, K) + out, "flops": 2 * M * N * K}
    R, C = case["R"], case["C"]
    kept = 2 * _held(case["fmt"], R, C)
    if case["op"] == "gated":  # g, u in; h, the checkpoint and its values out
        return {"bytes": 2 * R * C * 5 + kept, "flops": 20 * R * C}
    return {"bytes": 2 * R * C * 4 + kept, "flops": 20 * R * C}


# -------------------------------------------------------------------- exact

def _exact_values(x, fmt):
    """The value nearest to each x among code * 2^k, in 64 bits: every magnitude of the format in a table, the nearest by the table's
    midpoints, the even code on a midpoint."""
    top, _, _, mbits, emin, kmin, kmax = FORMATS[fmt]
    mags, e = [m * 2.0 ** (emin - mbits) for m in range(2 ** mbits)], emin
    while mags[-1] < top:
        mags += [(1 + m / 2 ** mbits) * 2.0 ** e for m in range(2 ** mbits)]
        e += 1
    mags = [m for m in mags if m <= top]
    mids = torch.tensor([(p + q) / 2 for p, q in zip(mags, mags[1:])], dtype=torch.float64, device=x.device)
    mags = torch.tensor(mags, dtype=torch.float64, device=x.device)
    rows, cols = x.shape
    done = []
    for part in x.split(2048):
        out = torch.empty(part.shape, dtype=torch.float64, device=x.device)
        for c0 in range(0, cols, BLOCK * 64):
            c1 = min(cols, c0 + BLOCK * 64)
            v = part[:, c0:c1].double()
            blocks = _cdiv(c1 - c0, BLOCK)
            spread = torch.zeros(v.shape[0], blocks * BLOCK, dtype=torch.float64, device=x.device)
            spread[:, :c1 - c0] = v.abs()
            amax = spread.view(v.shape[0], blocks, BLOCK).max(dim=2).values
            k = torch.ceil(torch.log2(amax / top))
            k = torch.where(amax <= top * torch.exp2(k - 1), k - 1, k)
            k = torch.where(amax > top * torch.exp2(k), k + 1, k)
            scale = torch.exp2(k.clamp(kmin, kmax))[..., None].expand(-1, -1, BLOCK).reshape(v.shape[0], -1)[:, :c1 - c0]
            y = v.abs() / scale
            lo = torch.searchsorted(mids, y)
            tie = (lo < len(mids)) & (mids[lo.clamp(max=len(mids) - 1)] == y) & (lo % 2 == 1)
            out[:, c0:c1] = mags[lo + tie.long()] * scale * torch.sign(v)
        done.append(out)
    return torch.cat(done)


def _exact_tensor(t):
    """A microscaled tensor's values in 64 bits, from the bits of its codes and its scale bytes."""
    rows, cols, fmt = t["rows"], t["cols"], t["fmt"]
    mbits, emin = FORMATS[fmt][3:5]
    i = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(cols, device="cuda")[None, :] // BLOCK
    tiles = _cdiv(_cdiv(cols, BLOCK), 4)
    scale = t["scales"][(i // 128 * tiles + b // 4) * 512 + i % 32 * 16 + i % 128 // 32 * 4 + b % 4].double() - 127
    j = torch.arange(cols, device="cuda")
    code = t["codes"].int()[:, j // 2] >> (4 * (j % 2)).int() & 15 if fmt == "e2m1" else t["codes"].int()[:, j]
    bits = 4 if fmt == "e2m1" else 8
    mag = code & ((1 << (bits - 1)) - 1)
    e, m = mag >> mbits, (mag & ((1 << mbits) - 1)).double() / 2 ** mbits
    value = torch.where(e > 0, (1 + m) * torch.exp2((e - 1 + emin).double()), m * 2.0 ** emin)
    return torch.where(code >> (bits - 1) > 0, -value, value) * torch.exp2(scale)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["x"]
        return {side: _exact_values(v, case[side]) for side, v in (("row", x), ("col", x.t().contiguous())) if case[side]}
    if case["op"] == "matmul":
        c = torch.matmul(_exact_tensor(s["a"]), _exact_tensor(s["b"]).t())
        return c if s["add"] is None else c + s["add"].double()
    if case["op"] == "gated":
        g, u = s["gate"].double(), s["up"].double()
        return {"h": g * torch.sigmoid(g) * u, "gate": _exact_values(s["gate"].contiguous(), case["fmt"]),
                "up": _exact_values(s["up"].contiguous(), case["fmt"])}
    g, u, dh = _exact_tensor(s["gate8"]), _exact_tensor(s["up8"]), s["dh"].double()
    p = torch.sigmoid(g)
    return {"dgate": dh * u * (p + g * p * (1 - p)), "dup": dh * g * p, "h": g * p * u}
