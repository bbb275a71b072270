"""Two sharper limits on the 4-bit attention than kv4_cases.attend_bounds, which
bounds each element by the worst case of every rounding: one on the rms of the
error, one on the weight that each tile of keys gets."""
from __future__ import annotations

import math

import numpy as np

from oracle import kv4 as okv
from tests import kv4_cases as kc


def rms_limit(q, k, v, queries, dtype):
    """(O, rms limit) of one sequence.  Roundings are independent and even, so
    their squares add up.  O's own: at most half a step, EPS |o|.  P s_v's, one for
    each key: at most 2^-11 of p v, so 2^-11 sqrt(sum (p v)^2).  The scores' sums
    in fp32: 8 steps of 2^-22 of sqrt(sum (q k)^2), felt as that share of |p v| with the
    keys' scores all apart: sqrt(sum (p v)^2) again, and of the sum p: |o| times
    sqrt(sum p^2).  Each is bounded by its largest size; even ones have 0.58 of it, so
    nothing is added for chance."""
    n, hq, d = q.shape
    L, hk, _ = k.shape
    o, square = np.zeros((n, hq, d)), 0.0
    for i in range(n):
        m = L - queries + i + 1
        for h in range(hq):
            kk, vv = k[:m, h // (hq // hk)], v[:m, h // (hq // hk)]
            x = kk @ q[i, h] / math.sqrt(d)
            p = np.exp(x - x.max())
            p /= p.sum()
            o[i, h] = p @ vv
            spread = np.sqrt((p[:, None] ** 2 * vv ** 2).sum(axis=0))
            ds = 8 * 2.0 ** -22 * math.sqrt(((kk * q[i, h]) ** 2).sum(axis=1).max() / d)
            square += ((kc.EPS[dtype] * o[i, h]) ** 2 + (2.0 ** -11 * spread) ** 2 + (ds * spread) ** 2 +
                       (ds * o[i, h]) ** 2 * (p ** 2).sum()).sum()
    return o, math.sqrt(square / o.size)


def rms(x):
    return math.sqrt((x ** 2).mean())


TILE, LANES = 32, 64  # keys of a tile of the schedule; tiles t and t + LANES share a channel


def markers(n, d):
    """V rows [n, 1, d] that mark their tile: one in channel t % LANES."""
    v = np.zeros((n, 1, d))
    at = np.arange(n)
    v[at, 0, at // TILE % LANES] = 1.0
    return v


def marked_weights(n, dtype, value):
    """What O holds in the first LANES channels if every key has weight 1 / n, and
    how far it may be off: P s_v and O are rounded once each, and sums of positive
    terms lose at most 2^-21 of themselves in each of their n / 16 steps (what
    partial states add is within that)."""
    tile = np.arange(n) // TILE % LANES
    want = np.bincount(tile, minlength=LANES) / n * value
    return want, want * (kc.EPS[dtype] + 2.0 ** -11 + n / 16 * 2.0 ** -21) + 2.0 ** -25


def marked_value(group, dtype):
    """The value that a row's marker is held as."""
    x = np.zeros((1, 64 if group < 128 else 128))
    x[0, 0] = 1.0
    return float(okv.values(*okv.quantise(x, group, dtype), group)[0, 0])
