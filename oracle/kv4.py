"""Oracle of the paged 4-bit K/V cache: codes, page plan and attention.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A row's channels are coded in groups: a = max |x|, s = a / 7 rounded to the
16-bit type, code = clamp(round_half_even(x / s), -7, 7), value = code * s;
a == 0 gives s = 0 and codes 0, a group with an infinity or a NaN s = NaN and
codes 0.  All arithmetic in fp64, one channel order (natural); ``pack`` restates
the pool's byte order one nibble at a time.  The page plan is a loop over host
lists.
"""
from __future__ import annotations

import math

import numpy as np

# significand bits and smallest exponent of a normal value
FORMATS = {"fp16": (11, -14, 65504.0), "bf16": (8, -126, (2.0 - 2.0 ** -7) * 2.0 ** 127)}


def round_to(x, dtype):
    """fp64 values rounded to the nearest of the 16-bit type (ties to even),
    overflow to infinity."""
    bits, emin, top = FORMATS[dtype]
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        _, e = np.frexp(np.where(np.isfinite(x), x, 0.0))
        step = np.ldexp(1.0, np.maximum(e - 1, emin) - (bits - 1))
        y = np.rint(x / step) * step
        y = np.where(np.abs(y) > top, np.copysign(np.inf, x), y)
    return np.where(np.isfinite(x), y, x)


def quantise(x, group, dtype):
    """x fp64 [..., d] (exact values of the type) -> (codes int8 [..., d],
    scales fp64 [..., d / group])."""
    y = x.reshape(x.shape[:-1] + (x.shape[-1] // group, group))
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        a = np.abs(y).max(axis=-1)  # NaN if one is there
        s = round_to(a / 7.0, dtype)
        c = np.clip(np.rint(y / s[..., None]), -7, 7)
    bad = ~np.isfinite(a)
    s = np.where(bad, np.nan, s)
    c = np.where((bad | (s == 0))[..., None], 0.0, c)
    return c.reshape(x.shape).astype(np.int8), s


def values(codes, scales, group):
    """fp64 values the codes stand for."""
    with np.errstate(invalid="ignore"):
        return codes.astype(np.float64) * np.repeat(scales, group, axis=-1)


def nibble_of(which, d):
    """(byte, high) of each channel's nibble in a packed row."""
    t = d // 32
    byte, high = np.zeros(d, dtype=np.int64), np.zeros(d, dtype=np.int64)
    for c in range(d):
        if which == "k":
            word, at = c // 8, c % 8
            byte[c] = 4 * ((word % 4) * t + word // 4) + at // 2
        else:
            half, at = c // 4, c % 4
            byte[c] = 2 * ((half % 8) * t + half // 8) + at // 2
        high[c] = at % 2
    return byte, high


def pack(codes, which):
    """Packed bytes [..., d / 2] of codes [..., d]."""
    d = codes.shape[-1]
    byte, high = nibble_of(which, d)
    out = np.zeros(codes.shape[:-1] + (d // 2,), dtype=np.uint8)
    for c in range(d):
        out[..., byte[c]] |= ((codes[..., c] + 8) << (4 * high[c])).astype(np.uint8)
    return out


def unpack(packed, which):
    d = packed.shape[-1] * 2
    byte, high = nibble_of(which, d)
    return (((packed[..., byte] >> (4 * high)) & 15).astype(np.int8) - 8).astype(np.int8)


class Pages:
    """The page plan's state and one step of it, on host lists."""

    def __init__(self, num_pages, page_size, max_seqs, max_pages):
        self.num_pages, self.page, self.max_pages = num_pages, page_size, max_pages
        self.table = [[-1] * max_pages for _ in range(max_seqs)]
        self.len = [0] * max_seqs
        self.stack = list(range(num_pages - 1, -1, -1))
        self.free = num_pages

    def plan(self, new_len, max_tokens):
        """(token_start, slots, granted) of one step; the state moves on."""
        P, n = self.page, len(new_len)
        pages = lambda t: -(-t // P)
        drop = [min(-x, self.len[s]) if x < 0 else 0 for s, x in enumerate(new_len)]
        back = []
        for s in range(n):
            for j in range(pages(self.len[s] - drop[s]), pages(self.len[s])):
                back.append(self.table[s][j])
                self.table[s][j] = -1
        have = self.free + len(back)
        for k, page in enumerate(back):
            self.stack[have - 1 - k] = page
        start, slots, granted = [0], [-1] * max_tokens, []
        needed = taken = 0
        for s in range(n):
            grow = max(0, new_len[s])
            a, b = pages(self.len[s]), pages(self.len[s] + grow)
            end = start[-1] + grow
            fits = end <= max_tokens and b <= self.max_pages
            if fits:
                needed += b - a
            ok = grow == 0 or (fits and (a == b or needed <= have))
            if ok:
                for j in range(a, b):
                    self.table[s][j] = self.stack[have - 1 - taken]
                    taken += 1
                for i in range(grow):
                    p = self.len[s] + i
                    slots[start[-1] + i] = self.table[s][p // P] * P + p % P
                self.len[s] += grow
            self.len[s] -= drop[s]
            granted.append(int(ok))
            start.append(end)
        self.free = have - taken
        return start, slots, granted


def attend(q, k, v, queries, scale=None):
    """One sequence: q [n, hq, d], k and v [L, hk, d], all fp64; query i sees
    keys 0 .. L - n + i.  Returns O, LSE [n, hq], sum p |v| (normalised), and the
    largest scale * sum_c |q_c| times a key's largest magnitude per query."""
    n, hq, d = q.shape
    L, hk, _ = k.shape
    scale = 1.0 / math.sqrt(d) if not scale else scale
    o = np.zeros((n, hq, d))
    mag = np.zeros((n, hq, d))
    lse = np.full((n, hq), -np.inf)
    reach = np.zeros((n, hq))
    for i in range(n):
        m = L - queries + i + 1
        if m <= 0:
            continue
        for h in range(hq):
            kk, vv = k[:m, h // (hq // hk)], v[:m, h // (hq // hk)]
            with np.errstate(invalid="ignore"):
                x = scale * (kk @ q[i, h])
                top = x.max()
                p = np.exp(x - top)
                z = p.sum()
                o[i, h] = p @ vv / z
                mag[i, h] = p @ np.abs(vv) / z
                lse[i, h] = top + math.log(z) if z == z else np.nan
                reach[i, h] = scale * np.abs(q[i, h]).sum() * np.abs(kk).max()
    return o, lse, mag, reach
