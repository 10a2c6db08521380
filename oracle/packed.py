"""Packed sequences in plain NumPy: attention with grouped heads, its gradients, rotary positions with several axes.

Attention is float64, one sequence and head at a time (``oracle.general``): rows [cu[b], cu[b + 1]) of q, k and v are
sequence b, query head h reads key head h / G. Rows outside the sequences stay NaN. ``rope`` rounds each product and
sum to float32, as its definition says, so that results can be compared bit for bit; ``dtype=numpy.float64`` gives the
unrounded rotation.

Pins (``tests/test_oracle_packed.py``): one sequence with a head of its own equals ``oracle.general``; the gradients of
shared heads against central finite differences; the rotation against complex multiplication, ``oracle.paged.rotate``
and its own inverse.
"""

import numpy as np

from . import general


def _sequences(cu):
    return [(int(a), int(b)) for a, b in zip(cu[:-1], cu[1:]) if b > a]


def forward(q, k, v, cu, causal, scale, window=0):
    """q [T, Hq, d], k and v [T, Hkv, d]; O [T, Hq, d] and LSE [T, Hq]."""
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    o, lse = np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    for a, b in _sequences(cu):
        for h in range(Hq):
            o[a:b, h], lse[a:b, h] = general.forward_head(q[a:b, h], k[a:b, h // G], v[a:b, h // G], causal, scale, window)
    return o, lse


def backward(q, k, v, o, lse, do, cu, causal, scale, window=0):
    """dQ, dK, dV of L = sum(O * dO); a key head's gradients are the sums over the query heads that read it."""
    G = q.shape[1] // k.shape[1]
    dq, dk, dv = (np.full(x.shape, np.nan) for x in (q, k, v))
    for a, b in _sequences(cu):
        dk[a:b], dv[a:b] = 0, 0
        for h in range(q.shape[1]):
            dq[a:b, h], x, y = general.backward_head(q[a:b, h], k[a:b, h // G], v[a:b, h // G], o[a:b, h], lse[a:b, h],
                                                     do[a:b, h], causal, scale, window)
            dk[a:b, h // G] += x
            dv[a:b, h // G] += y
    return dq, dk, dv


def rope(x, positions, axis_of, cos, sin, interleaved, inverse=False, dtype=np.float32):
    """x [T, H, d] turned: pair i by the angle of positions[axis_of[i]][t], column i of cos and sin [max_pos, rot / 2]."""
    y = np.array(x, dtype=dtype)
    n = len(axis_of)
    for i in range(n):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        p = np.asarray(positions)[axis_of[i]]
        c, s = np.asarray(cos, dtype=dtype)[p, i][:, None], np.asarray(sin, dtype=dtype)[p, i][:, None]
        if inverse:
            s = -s
        a, b = y[..., ia].copy(), y[..., ib].copy()
        with np.errstate(invalid="ignore", over="ignore"):
            y[..., ia] = a * c - b * s
            y[..., ib] = b * c + a * s
    return y
