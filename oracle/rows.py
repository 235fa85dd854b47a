"""Float64 oracle of the norm and rotation of rows (include/qli.h: qli_rotate,
qli_prepare_q, qli_append_kv) and of the positions a drafted token sees."""
import numpy as np


def frequencies(dim, base=10000.0, factor=1.0, trained=None, ramp=(1.0, 32.0)):
    """Radians per position of each pair; between the turns of the ramp the part that stays
    is linear in the turns."""
    f = np.asarray(base, dtype=np.float64) ** (-np.arange(0, dim, 2) / dim)
    keep = np.zeros(dim // 2)
    if trained is not None:
        keep = np.clip((trained * f / (2 * np.pi) - ramp[0]) / (ramp[1] - ramp[0]), 0, 1)
    return f if factor == 1.0 else f * keep + f / factor * (1 - keep)


def rotate(x, positions, f, offset, half, magnitude=1.0, inverse=False):
    """x [T, .., D] by positions [T]; the angles in long double, reduced there."""
    n = len(f)
    turn = np.asarray(positions, dtype=np.longdouble)[:, None] * (np.asarray(f, dtype=np.longdouble) / (2 * np.pi))
    angle = 2 * np.pi * (turn - np.rint(turn)).astype(np.float64)
    angle = angle.reshape(angle.shape[:1] + (1,) * (x.ndim - 2) + (n,))
    first = offset + (np.arange(n) if half else 2 * np.arange(n))
    second = first + (n if half else 1)
    a, b, y = x[..., first], x[..., second], x.copy()
    c, s, m = np.cos(angle), np.sin(angle), magnitude
    if inverse:
        s, m = -s, 1 / magnitude
    y[..., first], y[..., second] = m * (a * c - b * s), m * (b * c + a * s)
    return y


def normalise(x, norm, weight=None, bias=None, eps=1e-6):
    if norm is None:
        return x
    if norm == "layer":
        x = x - x.mean(axis=-1, keepdims=True)
    y = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    y = y if weight is None else y * weight
    return y if bias is None else y + bias


def tree_positions(k_len, n, mask, window=0):
    """Positions that a token with the mask (a Python int) sees of k_len, the last n
    of which are its request's nodes."""
    if k_len < n:
        return np.zeros(0, dtype=np.int64)
    nodes = [k_len - n + i for i in range(n) if mask >> i & 1]
    seen = np.concatenate([np.arange(k_len - n), np.asarray(nodes, dtype=np.int64)])
    return seen[max(0, len(seen) - window):] if window else seen
