"""The cases that the operators around experts and residual streams are measured on, with their plain forms.

They work next to the microscaled (MX) tensors: [rows, cols] in E2M1 (4 bits), E4M3 or E5M2 (8 bits) codes in blocks of 32
values along a row, with one scale byte k + 127 for each block; a value is code * 2^k.  ``plain`` below are the operators in
elementary torch operations in 32 bits; with ``own`` set, ``run`` calls the library's.

  norm       total = x + residual, y = total * rstd * weight with rstd = 1 / sqrt(mean(total^2) + eps): y in BF16 and/or in
             microscaled row and column forms; and its gradients
  dispatch   (token, choice) pairs sorted by expert, each expert's rows from a multiple of 128 on; the tokens' values in that
             order, in microscaled row and column forms
  combine    y[t] = sum over choices of weight * row; its gradients: weight * dy in the experts' order and forms, and the
             weights' gradients
  experts    each expert's rows times its own matrix, of microscaled operands
  gradient   each expert's matrix of sums over its rows (the weight gradient), added to an FP32 one
"""
import math

import torch

own = False

BLOCK, ALIGN, EPS = 32, 128, 1e-6
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
        # one token between two layers: the residual's addition and the norm in front of a 4-bit product; latency
        {"name": "norm_token", "op": "norm", "T": 1, "C": 2048, "residual": True, "y": True, "row": "e2m1", "col": ""},
        # a training batch: the 4-bit operand of the forward product and the 8-bit checkpoint for the weight gradient
        {"name": "norm_large", "op": "norm", "T": 16384, "C": 8192, "residual": True, "y": False, "row": "e2m1", "col": "e4m3"},
        # the backward pass of a short batch of odd sizes
        {"name": "norm_back_odd", "op": "norm_back", "T": 1001, "C": 2731, "residual": True},
        # the same for a training batch, with the gradient that comes along the residual stream
        {"name": "norm_back_large", "op": "norm_back", "T": 16384, "C": 8192, "residual": True},
        # a decoding step of one token: its choices sorted, its row quantised for each expert; latency
        {"name": "dispatch_token", "op": "dispatch", "T": 1, "k": 8, "E": 64, "C": 2048, "row": "e2m1", "col": "", "dropped": False},
        # a training batch to 64 experts: 4-bit operand and 8-bit checkpoint
        {"name": "dispatch_large", "op": "dispatch", "T": 16384, "k": 8, "E": 64, "C": 2048, "row": "e2m1", "col": "e4m3", "dropped": False},
        # a padded batch of odd sizes on its way back from the experts (choices of the padding are dropped)
        {"name": "combine_odd", "op": "combine", "T": 1543, "k": 6, "E": 66, "C": 2731, "weighted": True, "dropped": True},
        # a training batch's gradients on their way to the experts, and the gradients of the weights
        {"name": "combine_back_large", "op": "combine_back", "T": 16384, "k": 6, "E": 64, "C": 2048, "row": "e5m2", "col": "e5m2", "dropped": False},
        # a decoding step of four sequences: the chosen experts' matrices are read once
        {"name": "experts_token", "op": "experts", "T": 4, "k": 8, "E": 64, "N": 2048, "K": 2048, "a": "e2m1", "b": "e2m1", "dropped": False},
        # a prompt of odd length through 8-bit matrices, most experts with a part of a tile
        {"name": "experts_ragged", "op": "experts", "T": 1111, "k": 6, "E": 64, "N": 2816, "K": 2048, "a": "e4m3", "b": "e4m3", "dropped": False},
        # a training batch's forward product
        {"name": "experts_large", "op": "experts", "T": 16384, "k": 8, "E": 64, "N": 2048, "K": 2048, "a": "e2m1", "b": "e2m1", "dropped": False},
        # a training batch's weight gradients, added to the FP32 gradients so far
        {"name": "gradient_large", "op": "gradient", "T": 16384, "k": 8, "E": 64, "N": 2048, "K": 2048, "a": "e5m2", "b": "e4m3", "add": True, "dropped": False},
    ]


def _size(rng, lo, hi, odd=0.5):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() >= odd:
        step = 32 if n >= 64 else 1
        n = max(step, n // step * step)
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_back", "dispatch", "dispatch", "combine", "combine_back", "experts", "experts", "gradient"])
    if op == "norm":
        row, col = rng.choice([("e2m1", ""), ("e2m1", "e4m3"), ("e4m3", "e4m3"), ("", "e5m2"), ("", "")])
        return {"op": op, "T": _size(rng, 1, 16384), "C": _size(rng, 32, 8192), "residual": rng.random() < 0.7,
                "y": not (row or col) or rng.random() < 0.4, "row": row, "col": col}
    if op == "norm_back":
        return {"op": op, "T": _size(rng, 1, 16384), "C": _size(rng, 32, 8192), "residual": rng.random() < 0.7}
    T, k, E = _size(rng, 1, 16384), rng.randint(1, 8), _size(rng, 8, 128)
    case = {"op": op, "T": T, "k": k, "E": E, "dropped": rng.random() < 0.3}
    if op in ("experts", "gradient"):
        # padding: up to 127 rows an expert
        most = 2048 * 2048
        N, K = _size(rng, 32, 2816), _size(rng, 64, 2816)
        case["E"] = E = min(E, 64)
        case["N"], case["K"] = min(N, most // K), K
        if op == "experts":
            case["a"], case["b"] = rng.choice([("e2m1", "e2m1"), ("e2m1", "e2m1"), ("e4m3", "e4m3"), ("e5m2", "e4m3")])
        else:
            case["a"], case["b"], case["add"] = rng.choice(["e4m3", "e5m2"]), "e4m3", rng.random() < 0.7
        return case
    case["C"] = _size(rng, 32, 8192 if T * k <= 32768 else 2048)
    if op == "dispatch":
        case["row"], case["col"] = rng.choice([("e2m1", ""), ("e2m1", "e4m3"), ("e4m3", "e4m3"), ("", "e5m2")])
    elif op == "combine":
        case["weighted"] = rng.random() < 0.6
    else:
        case["row"], case["col"] = rng.choice([("e5m2", "e5m2"), ("e4m3", "e4m3")])
    return case


def _cdiv(a, b):
    return -(-a // b)


def _rows(case):
    """Rows that hold any choice of experts: each expert's are filled up to a multiple of 128."""
    pairs = case["T"] * case["k"]
    return (pairs + (ALIGN - 1) * min(case["E"], pairs)) // ALIGN * ALIGN


# ------------------------------------------------- the format in torch, 32 bits

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
    ea = ((v.abs().view(torch.int32) >> 23) - 127).clamp(emin, 127)
    q = _pow2(ea - mbits)
    r = torch.clamp(torch.round(v.abs() / q) * q, max=top)
    return torch.copysign(r, v).view(rows, nb * BLOCK)[:, :cols], k


def _values(r, k):
    """Codes' values r [rows, cols] times 2^k: FP32."""
    rows, cols = r.shape
    s = torch.where(k == 128, math.nan, _pow2(k.clamp(max=127)))
    return r * s.repeat_interleave(BLOCK, dim=1)[:, :cols]


def _kept(x, fmt):
    """The values that a form of x stands for, in BF16 (which holds them)."""
    return torch.cat([_values(*_quantize(p, fmt)).to(torch.bfloat16) for p in x.split(max(1, 2 ** 27 // x.shape[1]))])


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


def _zeros(fmt, rows, cols):
    """A form's memory; all zero bytes stand for zeros."""
    nb = _cdiv(cols, BLOCK)
    return {"fmt": fmt, "rows": rows, "cols": cols,
            "codes": torch.zeros(rows, nb * (16 if fmt == "e2m1" else 32), dtype=torch.uint8, device="cuda"),
            "scales": torch.zeros(_cdiv(rows, 128) * _cdiv(nb, 4) * 512, dtype=torch.uint8, device="cuda")}


# --------------------------------------------------- experts' order in torch

def _sort(ids, E, rows):
    """counts [E], offsets [E + 1], slots [T, k] and sources [rows] (-1: no choice there)."""
    flat = ids.reshape(-1).long()
    hit = flat[:, None] == torch.arange(E, device=ids.device)[None, :]
    before = torch.cumsum(hit, dim=0, dtype=torch.int32)
    counts = before[-1]
    ends = torch.cumsum((counts + ALIGN - 1) // ALIGN * ALIGN, dim=0, dtype=torch.int32)
    offsets = torch.cat((torch.zeros_like(ends[:1]), ends))
    kept = (flat >= 0) & (flat < E)
    e = flat.clamp(0, E - 1)
    slots = torch.where(kept, offsets[e] + before.gather(1, e[:, None])[:, 0] - 1, -1).to(torch.int32)
    sources = torch.full((rows + 1,), -1, dtype=torch.int32, device=ids.device)
    sources[torch.where(kept, slots, rows).long()] = torch.arange(flat.numel(), dtype=torch.int32, device=ids.device)
    return {"counts": counts, "offsets": offsets, "slots": slots.view(ids.shape), "sources": sources[:rows]}


def _ids(case, g):
    """Choices of different experts, some far more popular than others; choices of a padded batch's last tokens are dropped."""
    T, k, E = case["T"], case["k"], case["E"]
    liking = torch.randn(E, generator=g, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp(1e-6, 1 - 1e-6)))
    ids = torch.topk(liking + noise, k, dim=1).indices.to(torch.int32)
    if case["dropped"]:
        ids[T - T // 4:] = -1
    return ids


# -------------------------------------------------------------------- inputs

def _activations(g, rows, cols):
    """Activations: normal, a few channels much larger, tokens of different norm."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(torch.bfloat16)


def _gradients(g, rows, cols):
    """Gradients: small, heavy-tailed."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    return (1e-4 * x * torch.exp(torch.randn(rows, cols, generator=g, device="cuda"))).to(torch.bfloat16)


def _choice_weights(g, T, k):
    return torch.softmax(torch.randn(T, k, generator=g, device="cuda"), dim=1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    state, op = {"case": case}, case["op"]
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op in ("norm", "norm_back"):
        T, C = case["T"], case["C"]
        state["w"] = (1 + 0.1 * torch.randn(C, generator=g, device="cuda")).to(torch.bfloat16)
        if op == "norm":
            state["x"] = _activations(g, T, C)
            state["residual"] = _activations(g, T, C) if case["residual"] else None
            state["total"] = new(T, C) if case["residual"] else None
            state["rstd"] = new(T, dtype=torch.float32)
            state["y"] = new(T, C) if case["y"] else None
            _form_buffers(state, case, T, C)
            return state
        state["total"] = _activations(g, T, C)
        state["rstd"] = 1 / torch.sqrt(state["total"].float().square().mean(dim=1) + EPS)
        state["dy"] = _gradients(g, T, C)
        state["dtotal"] = _gradients(g, T, C) if case["residual"] else None
        state["dx"], state["dw"] = new(T, C), new(C, dtype=torch.float32)
        state["add"] = 1e-3 * torch.randn(C, generator=g, device="cuda")
        return state
    T, k, E, R = case["T"], case["k"], case["E"], _rows(case)
    ids = _ids(case, g)
    if op == "dispatch":
        state["ids"] = ids
        state["x"] = _activations(g, T, case["C"])
        _form_buffers(state, case, R, case["C"])
        return state
    plan = state["plan"] = _sort(ids, E, R)
    if op in ("combine", "combine_back"):
        C = case["C"]
        state["out"] = _activations(g, R, C) * (plan["sources"] >= 0)[:, None]
        if op == "combine":
            state["weights"] = _choice_weights(g, T, k) if case["weighted"] else None
            state["y"] = new(T, C)
        else:
            state["weights"] = _choice_weights(g, T, k)
            state["dy"] = _gradients(g, T, C)
            state["dweights"] = new(T, k, dtype=torch.float32)
            _form_buffers(state, case, R, C)
        return state
    # the ends of the experts' rows on the host: only the plain forms look at them
    state["ends"] = plan["offsets"].tolist()
    N, K = case["N"], case["K"]
    held = (plan["sources"] >= 0)[:, None]
    state["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op == "experts":
        make = _gradients if case["a"] == "e5m2" else _activations
        state["a"] = _encode(make(g, R, K) * held, case["a"])
        parts = [_encode((0.02 * torch.randn(N, K, generator=g, device="cuda")).to(torch.bfloat16), case["b"]) for _ in range(E)]
        state["b"] = {"fmt": case["b"], "count": E, "rows": N, "cols": K, "codes": torch.cat([p["codes"] for p in parts]),
                      "scales": torch.cat([p["scales"] for p in parts])}
        state["c"] = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    else:
        make = _gradients if case["a"] == "e5m2" else _activations
        state["a"] = _encode((make(g, R, N) * held).t().contiguous(), case["a"])
        state["b"] = _encode((_activations(g, R, K) * held).t().contiguous(), case["b"])
        state["add"] = 1e-3 * torch.randn(E, N, K, generator=g, device="cuda") if case["add"] else None
        state["c"] = new(E, N, K, dtype=torch.float32)
    return state


def _form_buffers(state, case, rows, cols):
    for side, (r, c) in {"row": (rows, cols), "col": (cols, rows)}.items():
        if case[side]:
            state[side] = _zeros(case[side], r, c)
            state[side + "_values"] = torch.empty(r, c, dtype=torch.bfloat16, device="cuda")


# ---------------------------------------------------------------------- run

def run(state):
    return _own(state) if own else _plain(state)


def _mx(t):
    from lossless_bf16_exponent_codec_gb300 import mx
    if t is None:
        return None
    if "count" in t:
        return mx.MxStack(t["fmt"], t["count"], t["rows"], t["cols"], t["codes"], t["scales"])
    return mx.MxTensor(t["fmt"], t["rows"], t["cols"], t["codes"], t["scales"])


def _own(s):
    from lossless_bf16_exponent_codec_gb300 import moe, mx
    case, op = s["case"], s["case"]["op"]
    row, col = _mx(s.get("row")), _mx(s.get("col"))

    def forms(out):
        for side, t in (("row", row), ("col", col)):
            if t is not None:
                out[side] = mx.dequantize(t, out=s[side + "_values"])
        return out

    if op == "norm":
        total, rstd = mx.rms_norm(s["x"], s["w"], eps=EPS, residual=s["residual"], total=s["total"], rstd=s["rstd"],
                                  out=s["y"], row=row, col=col)
        return forms({"total": total, "rstd": rstd, "y": s["y"]})
    if op == "norm_back":
        dx = mx.rms_norm_backward(s["dy"], s["total"], s["rstd"], s["w"], dtotal=s["dtotal"], out=s["dx"], dweight=s["dw"],
                                  add=s["add"])
        return {"dx": dx, "dw": s["dw"]}
    if op == "dispatch":
        routing = moe.sort(s["ids"], case["E"])
        moe.dispatch(s["x"], routing, row=row, col=col)
        return forms({"counts": routing.counts, "offsets": routing.offsets, "slots": routing.slots})
    p = s["plan"]
    routing = moe.Routing(case["T"], case["k"], case["E"], p["counts"], p["offsets"], p["slots"], p["sources"])
    if op == "combine":
        return moe.combine(s["out"], routing, weights=s["weights"], out=s["y"])
    if op == "combine_back":
        moe.dispatch(s["dy"], routing, weights=s["weights"], row=row, col=col)
        return forms({"dweights": moe.weight_gradient(s["dy"], s["out"], routing, out=s["dweights"])})
    if op == "experts":
        return moe.expert_matmul(_mx(s["a"]), _mx(s["b"]), routing, out=s["c"], status=s["status"])
    return moe.expert_gradient(_mx(s["a"]), _mx(s["b"]), routing, out=s["c"], add=s["add"], status=s["status"])


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "norm":
        x = s["x"]
        total = x if s["residual"] is None else (x.float() + s["residual"].float()).to(torch.bfloat16)
        t = total.float()
        rstd = 1 / torch.sqrt(t.square().mean(dim=1) + EPS)
        y = (t * rstd[:, None] * s["w"].float()).to(torch.bfloat16)
        out = {"total": total, "rstd": rstd, "y": y if case["y"] else None}
        return _plain_forms(out, case, y)
    if op == "norm_back":
        t, dy, w, rstd = s["total"].float(), s["dy"].float(), s["w"].float(), s["rstd"][:, None]
        n = t * rstd
        dn = dy * w
        dx = rstd * (dn - n * (dn * n).mean(dim=1, keepdim=True))
        if s["dtotal"] is not None:
            dx = dx + s["dtotal"].float()
        return {"dx": dx.to(torch.bfloat16), "dw": (dy * n).sum(dim=0) + s["add"]}
    if op == "dispatch":
        plan = _sort(s["ids"], case["E"], _rows(case))
        out = {n: plan[n] for n in ("counts", "offsets", "slots")}
        return _plain_forms(out, case, _ordered(s["x"], plan, case["k"]))
    plan, k = s["plan"], case["k"]
    if op in ("combine", "combine_back"):
        there = (plan["slots"] >= 0)[..., None]
        rows = lambda j: s["out"][plan["slots"][:, j].clamp(min=0).long()].float() * there[:, j]  # noqa: E731
        if op == "combine":
            y = torch.zeros(case["T"], case["C"], device="cuda")
            for j in range(k):
                y += rows(j) if s["weights"] is None else rows(j) * s["weights"][:, j:j + 1]
            return y.to(torch.bfloat16)
        dy = s["dy"].float()
        dweights = torch.stack([(dy * rows(j)).sum(dim=1) for j in range(k)], dim=1)
        return _plain_forms({"dweights": dweights}, case, _ordered(s["dy"], plan, k, s["weights"]))
    ends = s["ends"]
    a = _decode(s["a"])
    if op == "experts":
        b = s["b"]
        c = torch.zeros(s["c"].shape, dtype=torch.bfloat16, device="cuda")
        codes, scales = b["codes"].view(b["count"], b["rows"], -1), b["scales"].view(b["count"], -1)
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi > lo:
                w = _decode({**b, "codes": codes[e], "scales": scales[e]})
                c[lo:hi] = (a[lo:hi] @ w.t()).to(torch.bfloat16)
        return c
    b = _decode(s["b"])
    c = torch.stack([a[:, lo:hi] @ b[:, lo:hi].t() for lo, hi in zip(ends, ends[1:])])
    return c if s["add"] is None else c + s["add"]


def _ordered(x, plan, k, weights=None):
    """Rows of x in the experts' order, in BF16: zeros where there is no choice."""
    src = plan["sources"].long()
    at = src.clamp(min=0)
    rows = x[at // k]
    if weights is not None:
        rows = (rows.float() * weights.reshape(-1)[at][:, None]).to(torch.bfloat16)
    return torch.where((src >= 0)[:, None], rows, 0.0)


def _plain_forms(out, case, x):
    for side in ("row", "col"):
        if case[side]:
            out[side] = _kept(x if side == "row" else x.t(), case[side])
    return out


# --------------------------------------------------------------------- work

def _held(fmt, rows, cols):
    return rows * _cdiv(cols, BLOCK) * ((16 if fmt == "e2m1" else 32) + 1) if fmt else 0


def _form_bytes(case, rows, cols):
    """The forms, and their values in BF16."""
    return sum(_held(case[s], r, c) + 2 * r * c for s, r, c in (("row", rows, cols), ("col", cols, rows)) if case[s])


def work(case):
    op = case["op"]
    if op in ("norm", "norm_back"):
        T, C = case["T"], case["C"]
        if op == "norm":
            read = 2 * T * C * (1 + case["residual"]) + 2 * C
            return {"bytes": read + 2 * T * C * (case["residual"] + case["y"]) + 4 * T + _form_bytes(case, T, C), "flops": 8 * T * C}
        return {"bytes": 2 * T * C * (3 + case["residual"]) + 4 * T + 10 * C, "flops": 10 * T * C}
    T, k, E = case["T"], case["k"], case["E"]
    pairs = (T - (T // 4 if case["dropped"] else 0)) * k
    if op == "dispatch":
        C = case["C"]
        return {"bytes": 2 * T * C + 8 * T * k + 8 * E + _form_bytes(case, pairs, C), "flops": 4 * pairs * C}
    if op == "combine":
        C = case["C"]
        return {"bytes": 2 * pairs * C + 2 * T * C + T * k * (4 + 4 * case["weighted"]), "flops": 2 * pairs * C}
    if op == "combine_back":
        C = case["C"]
        return {"bytes": 2 * T * C + 2 * pairs * C + 12 * T * k + _form_bytes(case, pairs, C), "flops": 6 * pairs * C}
    N, K = case["N"], case["K"]
    if op == "experts":
        chosen = min(E, pairs)
        return {"bytes": _held(case["a"], pairs, K) + chosen * _held(case["b"], N, K) + 2 * pairs * N, "flops": 2 * pairs * N * K}
    return {"bytes": _held(case["a"], N, pairs) + _held(case["b"], K, pairs) + 4 * E * N * K * (1 + case["add"]), "flops": 2 * pairs * N * K}


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


def _exact_tensor(fmt, rows, cols, codes, scales):
    """A microscaled tensor's values in 64 bits, from the bits of its codes and its scale bytes."""
    mbits, emin = FORMATS[fmt][3:5]
    i = torch.arange(rows, device="cuda")[:, None]
    b = torch.arange(cols, device="cuda")[None, :] // BLOCK
    tiles = _cdiv(_cdiv(cols, BLOCK), 4)
    scale = scales[(i // 128 * tiles + b // 4) * 512 + i % 32 * 16 + i % 128 // 32 * 4 + b % 4].double() - 127
    j = torch.arange(cols, device="cuda")
    code = codes.int()[:, j // 2] >> (4 * (j % 2)).int() & 15 if fmt == "e2m1" else codes.int()[:, j]
    bits = 4 if fmt == "e2m1" else 8
    mag = code & ((1 << (bits - 1)) - 1)
    e, m = mag >> mbits, (mag & ((1 << mbits) - 1)).double() / 2 ** mbits
    value = torch.where(e > 0, (1 + m) * torch.exp2((e - 1 + emin).double()), m * 2.0 ** emin)
    return torch.where(code >> (bits - 1) > 0, -value, value) * torch.exp2(scale)


def _exact_order(ids, E):
    """counts, offsets and slots by a stable sort, expert by expert."""
    flat = ids.reshape(-1).cpu()
    order = torch.argsort(flat, stable=True).tolist()
    flat = flat.tolist()
    lists = [[] for _ in range(E)]
    for i in order:
        if 0 <= flat[i] < E:
            lists[flat[i]].append(i)
    offsets, slots = [0], [-1] * len(flat)
    for members in lists:
        for n, i in enumerate(members):
            slots[i] = offsets[-1] + n
        offsets.append(offsets[-1] + _cdiv(len(members), ALIGN) * ALIGN)
    new = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return new([len(m) for m in lists]), new(offsets), new(slots).view(ids.shape)


def _exact_forms(out, case, slots, rows, value):
    """Forms of the matrix whose row slots[t, j] is value(j)[t] and which is zero elsewhere (values that BF16 holds)."""
    x = torch.zeros(rows, case["C"], dtype=torch.bfloat16, device="cuda")
    for j in range(case["k"]):
        t = torch.nonzero(slots[:, j] >= 0)[:, 0]
        x[slots[t, j].long()] = value(j)[t].to(torch.bfloat16)
    for side in ("row", "col"):
        if case[side]:
            out[side] = _exact_values(x if side == "row" else x.t().contiguous(), case[side])
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        total = s["x"].double()
        if s["residual"] is not None:
            total = (total + s["residual"].double()).to(torch.bfloat16).double()
        rstd = torch.rsqrt((total * total).sum(dim=1) / case["C"] + EPS)
        y = total.mul_(rstd[:, None]).mul_(s["w"].double())
        out = {"total": s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double(), "rstd": rstd,
               "y": y if case["y"] else None}
        for side in ("row", "col"):
            if case[side]:
                v = y.to(torch.bfloat16)
                out[side] = _exact_values(v if side == "row" else v.t().contiguous(), case[side])
        return out
    if op == "norm_back":
        # through d(total / rms): rms^2 = 1 / rstd^2
        t, dy, rstd = s["total"].double(), s["dy"].double(), s["rstd"].double()
        g = dy * s["w"].double()
        along = torch.einsum("tc,tc->t", g, t) / case["C"]
        dx = rstd[:, None] * g - (rstd ** 3 * along)[:, None] * t
        if s["dtotal"] is not None:
            dx += s["dtotal"].double()
        return {"dx": dx, "dw": torch.einsum("tc,tc,t->c", dy, t, rstd) + s["add"].double()}
    if op == "dispatch":
        counts, offsets, slots = _exact_order(s["ids"], case["E"])
        return _exact_forms({"counts": counts, "offsets": offsets, "slots": slots}, case, slots, _rows(case), lambda j: s["x"])
    slots = s["plan"]["slots"]
    if op in ("combine", "combine_back"):
        out = torch.cat((s["out"], torch.zeros_like(s["out"][:1])))     # row -1
        if op == "combine":
            w = s["weights"].double() if s["weights"] is not None else torch.ones(slots.shape, dtype=torch.float64, device="cuda")
            return sum(out[slots[:, j].long()].double() * w[:, j, None] for j in range(case["k"]))
        dy = s["dy"].double()
        dweights = torch.stack([torch.einsum("tc,tc->t", dy, out[slots[:, j].long()].double()) for j in range(case["k"])], dim=1)
        return _exact_forms({"dweights": dweights}, case, slots, _rows(case), lambda j: dy * s["weights"][:, j, None].double())
    ends, N, K = s["plan"]["offsets"].tolist(), case["N"], case["K"]
    a, b = s["a"], s["b"]
    av = _exact_tensor(case["a"], a["rows"], a["cols"], a["codes"], a["scales"])
    if op == "experts":
        c = torch.zeros(a["rows"], N, dtype=torch.float64, device="cuda")
        size, tiles = b["codes"].shape[0] // case["E"], b["scales"].numel() // case["E"]
        for e in range(case["E"]):
            if ends[e + 1] > ends[e]:
                w = _exact_tensor(case["b"], N, K, b["codes"][e * size:(e + 1) * size], b["scales"][e * tiles:(e + 1) * tiles])
                torch.matmul(av[ends[e]:ends[e + 1]], w.t(), out=c[ends[e]:ends[e + 1]])
        return c
    bv = _exact_tensor(case["b"], b["rows"], b["cols"], b["codes"], b["scales"])
    c = torch.zeros(case["E"], N, K, dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
    for e in range(case["E"]):
        c[e] += av[:, ends[e]:ends[e + 1]] @ bv[:, ends[e]:ends[e + 1]].t()
    return c
