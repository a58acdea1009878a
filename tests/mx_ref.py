"""Plain 64-bit implementation of the microscaled operators on the host
(numpy), written from their definitions: tables of element values, nearest
element by comparison of distances, scale tiles by index."""
import numpy as np

# element magnitudes in code order, largest first argument F, range of k
MAGS = {
    "e2m1": np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]),
    "e4m3": np.array([m * 2.0 ** -9 for m in range(8)]
                     + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]),
    "e5m2": np.array([m * 2.0 ** -16 for m in range(4)]
                     + [(1 + m / 4) * 2.0 ** (e - 15) for e in range(1, 31) for m in range(4)]),
}
K_RANGE = {"e2m1": (-127, 125), "e4m3": (-124, 119), "e5m2": (-117, 112)}


def bf16_to_f64(u16: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        return (u16.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def scale_index(rows: int, nb: int) -> np.ndarray:
    """Byte of scale (row, block) in the scale tiles."""
    r, b = np.arange(rows)[:, None], np.arange(nb)[None, :]
    return (r // 128 * -(-nb // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4


def quantize(x: np.ndarray, fmt: str):
    """x [rows, cols] in 64 bits -> (code bytes [rows, pitch], scale bytes,
    values [rows, cols])."""
    rows, cols = x.shape
    mags, (kmin, kmax) = MAGS[fmt], K_RANGE[fmt]
    F, nb = mags[-1], -(-cols // 32)
    pad = np.zeros((rows, nb * 32))
    pad[:, :cols] = x
    blk = pad.reshape(rows, nb, 32)
    bad = ~np.isfinite(blk).all(axis=2)
    amax = np.abs(np.where(bad[..., None], 0.0, blk)).max(axis=2)
    with np.errstate(divide="ignore"):
        k = np.where(amax > 0, np.ceil(np.log2(np.where(amax > 0, amax, 1) / F)), kmin)
    k = np.where((amax > 0) & (amax > F * 2.0 ** k), k + 1, k)
    k = np.where((amax > 0) & (amax <= F * 2.0 ** (k - 1)), k - 1, k)
    k = np.clip(k, kmin, kmax)
    y = np.where(bad[..., None], 0.0, blk) / (2.0 ** k)[..., None]
    a = np.minimum(np.abs(y), F)
    hi = np.searchsorted(mags, a).clip(1, len(mags) - 1)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    value = np.copysign(mags[code], y) * (2.0 ** k)[..., None]
    value = np.where(bad[..., None], np.nan, value).reshape(rows, nb * 32)[:, :cols]
    sign = np.signbit(y)
    code = (code + np.where(sign, 8 if fmt == "e2m1" else 128, 0)).astype(np.uint8).reshape(rows, nb * 32)
    if fmt == "e2m1":
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    scales = np.zeros(-(-rows // 128) * -(-nb // 4) * 512, np.uint8)
    scales[scale_index(rows, nb)] = np.where(bad, 255, k + 127).astype(np.uint8)
    return code, scales, value


def silu_parts(g):
    s = 1 / (1 + np.exp(-g))
    return s, g * s


def round_bf16(x: np.ndarray) -> np.ndarray:
    """The BF16 value nearest to each x, ties to even (8 significant bits, steps
    of at least 2^-133)."""
    _, e = np.frexp(x)
    q = np.exp2(np.maximum(e - 8, -133).astype(np.float64))
    return np.round(x / q) * q


def is_rounding_near(got, want, off) -> bool:
    """Whether each BF16 value got is the rounding of some number within off of
    want (rounding is monotonic, so the interval's ends are enough)."""
    got = np.asarray(got, np.float64)
    return bool(((round_bf16(want - off) <= got) & (got <= round_bf16(want + off))).all())
