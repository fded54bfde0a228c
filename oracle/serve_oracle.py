"""Plain float64 forms of the serving operators (head norm and rotation, the
paged 8-bit cache, attention of a few new tokens over it), numpy on the CPU.
Test infrastructure; shares nothing with the CUDA path."""
import math

import numpy as np


def norm_rope(x, pos, inv_freq=None, weight=None, eps=1e-6, interleaved=False):
    """x [N, d] -> the normed and turned rows."""
    y = np.array(x, np.float64)
    d = y.shape[1]
    if weight is not None:
        y = y / np.sqrt((y * y).mean(axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if inv_freq is not None:
        half = len(inv_freq)
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            assert b < d
            t = np.asarray(pos, np.float64) * inv_freq[i]
            ya, yb = y[:, a].copy(), y[:, b].copy()
            y[:, a] = ya * np.cos(t) - yb * np.sin(t)
            y[:, b] = ya * np.sin(t) + yb * np.cos(t)
    return y


def e4m3_value(byte):
    """The number an e4m3 byte stands for (bias 7, no infinity, NaN at 0x7f)."""
    s, e, m = byte >> 7, byte >> 3 & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if s else v


def e4m3_round(x):
    """Nearest e4m3 number, ties to the even mantissa; |x| <= 448."""
    x = np.asarray(x, np.float64)
    _, ex = np.frexp(np.where(x == 0, 1.0, np.abs(x)))        # |x| = m 2^ex, m in [1/2, 1)
    step = np.exp2(np.maximum(ex - 1, -6) - 3.0)
    return np.rint(x / step) * step                            # rint: ties to even


def row_exponent(row):
    """Smallest e >= -80 with max |x| <= 448 * 2^e; 0 for a row of zeros; None for one with a NaN or infinity."""
    top = np.abs(np.asarray(row, np.float64)).max()
    if not np.isfinite(top):
        return None
    if top == 0:
        return 0
    e = -80
    while top > 448.0 * 2.0 ** e:
        e += 1
    return e


def quantise(row):
    """(values in units of 2^e, stored exponent byte)."""
    e = row_exponent(row)
    if e is None:
        return np.full(len(row), math.nan), 255
    return e4m3_round(np.asarray(row, np.float64) / 2.0 ** e), e + 127


def tree_attention(q, k, v, ctx, see, scale):
    """q [T, d]; k, v [ctx + n, d]; see [T, n] truth values: (O [T, d], LSE [T], sum of p |v| [T, d])."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    T = q.shape[0]
    O, A, lse = np.zeros((T, v.shape[1])), np.zeros((T, v.shape[1])), np.full(T, -math.inf)
    for t in range(T):
        keys = np.concatenate([np.arange(ctx), ctx + np.flatnonzero(see[t])])
        if len(keys) == 0:
            continue
        s = k[keys] @ q[t] * scale
        m = s.max()
        w = np.exp(s - m)
        lse[t] = m + math.log(w.sum())
        O[t] = w @ v[keys] / w.sum()
        A[t] = w @ np.abs(v[keys]) / w.sum()
    return O, lse, A
