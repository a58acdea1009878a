"""Plain 64-bit implementations (numpy) of the norm and of the way of tokens to
their experts and back, written from their definitions."""
import numpy as np


def rms(x64, eps):
    """rstd of each row."""
    return 1 / np.sqrt((x64 ** 2).mean(axis=1) + eps)


def rms_backward(dy, total, rstd, w, dtotal=None):
    """(dx, dweight) by differentiating total / rms."""
    C = total.shape[1]
    g = dy * w
    dx = rstd[:, None] * g - rstd[:, None] ** 3 * total * (g * total).sum(axis=1, keepdims=True) / C
    return dx if dtotal is None else dx + dtotal, (dy * total * rstd[:, None]).sum(axis=0)


def routing(ids, experts):
    """counts, offsets, slots and sources of ids [T, k], one pair after the other."""
    T, k = ids.shape
    lists = [[] for _ in range(experts)]
    for i, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < experts:
            lists[e].append(i)
    pairs = T * k
    rows = (pairs + 127 * min(experts, pairs)) // 128 * 128
    slots, sources, offsets = np.full(pairs, -1, np.int32), np.full(rows, -1, np.int32), [0]
    for members in lists:
        for n, i in enumerate(members):
            slots[i] = offsets[-1] + n
            sources[offsets[-1] + n] = i
        offsets.append(offsets[-1] + -(-len(members) // 128) * 128)
    return np.array([len(m) for m in lists], np.int32), np.array(offsets, np.int32), slots.reshape(T, k), sources


def ordered(x, sources, choices, weights=None):
    """Rows of x in the experts' order, zeros where there is no pair; weighted
    values unrounded."""
    out = np.zeros((len(sources), x.shape[1]))
    r = np.nonzero(sources >= 0)[0]
    out[r] = x[sources[r] // choices]
    if weights is not None:
        out[r] *= weights.reshape(-1)[sources[r], None]
    return out


def combine(rows, slots, weights=None):
    """(y, sum of magnitudes)."""
    T, k = slots.shape
    y, mag = np.zeros((T, rows.shape[1])), np.zeros((T, rows.shape[1]))
    for t in range(T):
        for j in range(k):
            if slots[t, j] >= 0:
                v = rows[slots[t, j]] * (1.0 if weights is None else weights[t, j])
                y[t] += v
                mag[t] += np.abs(v)
    return y, mag
