"""Shared machinery of the paged 4-bit cache's tests: numpy <-> torch in both
16-bit types, pools filled by the oracle, and the attention's error bound."""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv4 as okv

TORCH = {"fp16": torch.float16, "bf16": torch.bfloat16}
EPS = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step, relative


def draw(rng, shape, dtype, scale=1.0):
    """fp64 array of N(0, scale^2) values of the type."""
    return okv.round_to(rng.standard_normal(shape) * scale, dtype)


def to_device(x, dtype, device="cuda"):
    """fp64 values of the type -> tensor (the conversion is exact)."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(TORCH[dtype]).to(device)


def to_numpy(t):
    return t.detach().to("cpu", torch.float64).numpy()


def same(got, want):
    """Equal values, NaN where NaN."""
    return np.array_equal(np.isnan(got), np.isnan(want)) and \
        np.array_equal(got[~np.isnan(want)], want[~np.isnan(want)])


class Pool:
    """A pool of random codes and scales, with the tables of sequences of the
    given lengths over shuffled pages."""

    def __init__(self, rng, lengths, hk, d, group, page, dtype, spare=3, max_pages=None):
        self.hk, self.d, self.group, self.page, self.dtype = hk, d, group, page, dtype
        self.lengths = list(lengths)
        used = [-(-n // page) for n in lengths]
        self.num_pages = sum(used) + spare
        self.max_pages = max(used + [1]) if max_pages is None else max_pages
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lengths), self.max_pages), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(used):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.free = order[at:].astype(np.int32)
        shape = (self.num_pages, hk, page, d)
        self.codes, self.scales = {}, {}
        for w in "kv":
            x = draw(rng, shape, dtype)
            if w == "k":
                x[..., :: 37] *= 8.0  # a few strong channels, as keys have
                x = okv.round_to(x, dtype)
            self.codes[w], self.scales[w] = okv.quantise(x, group, dtype)

    def row(self, which, s):
        """Sequence s's values, fp64 [len, hk, d]."""
        n = self.lengths[s]
        pages = self.table[s, :-(-n // self.page)]
        c, sc = self.codes[which][pages], self.scales[which][pages]
        x = okv.values(c, sc, self.group)                       # [pages, hk, page, d]
        return x.transpose(0, 2, 1, 3).reshape(-1, self.hk, self.d)[:n]

    def tensors(self, device="cuda"):
        out = []
        for w in "kv":
            out.append(torch.from_numpy(okv.pack(self.codes[w], w)).to(device))
            out.append(to_device(self.scales[w], self.dtype, device))
        return out

    def cache(self, device="cuda", lengths=None):
        import tile_routed_mixed_b200 as tm
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(device)
        stack = np.full(self.num_pages, -1, dtype=np.int32)
        stack[:len(self.free)] = self.free
        tables = (i32(self.table), i32(self.lengths if lengths is None else lengths), i32(stack),
                  i32([len(self.free)]))
        return tm.TileMixKV4Cache(self.num_pages, self.page, self.hk, self.d, len(self.lengths),
                                  self.max_pages, group=self.group, dtype=TORCH[self.dtype],
                                  device=device, pool=self.tensors(device), tables=tables)


def attend_bounds(o, lse, mag, reach, dtype, vmax, keys):
    """Largest |error| of O and of the LSE that the arithmetic allows.

    Scores: at most 8 accumulating products per group, each within 2^-22 of the
    sum of magnitudes (fp32 sums of the products, which may be truncated), which
    the largest |k| over its code bounds by 3 reach (a subnormal scale may leave
    a smaller largest code), so 8 * 2^-22 * 3 reach; as much again covers q's
    rounding to its scaled fp16, the sum over groups and the two products by
    scales.  A probability is off by that factor (in numerator and sum: twice),
    by ex2's 2^-22 and by its rounding times the scale to 11 bits, 2^-11; below
    fp16's normal range by 2^-25 of a unit of sigma / 32 each, seven times for
    the code.  The products with V take the codes as they are, |code| <= 7 with
    vmax the largest scale: each of the keys / 16 accumulating steps, and two
    where partial states are joined, is within 2^-21 of the sums' magnitude, at
    most 7 sum(P s_v), 8 with P s_v's rounding.  O's own rounding is half a step;
    subnormal results half a unit of 2^-24 (fp16)."""
    ds = 16 * 2.0 ** -22 * 3 * reach
    rel = 2.0 ** -11 + 2 * ds + 2.0 ** -18
    tiny = keys * 7 * 2.0 ** -30 * vmax + (keys / 16 + 2) * 2.0 ** -21 * 8 * vmax
    tiny += 2.0 ** -25 if dtype == "fp16" else 0.0
    do = EPS[dtype] * np.abs(o) + (1 + EPS[dtype]) * rel[..., None] * mag + tiny
    dl = ds + 2.0 ** -18 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))
    return do, dl


def check_attend(got_o, got_lse, q, pool, lengths, token_start, hq, scale=None, kv=None):
    """Every sequence's queries against the oracle.  kv(s) gives K and V (fp64)
    of a sequence; by default the pool's rows."""
    worst = 0.0
    for s, n in enumerate(lengths):
        a, b = token_start[s], token_start[s + 1]
        if a == b:
            continue
        k, v = kv(s) if kv else (pool.row("k", s), pool.row("v", s))
        o, lse, mag, reach = okv.attend(q[a:b], k, v, b - a, scale)
        do, dl = attend_bounds(o, lse, mag, reach, pool.dtype, np.abs(v).max() / 7 if n else 0.0, n)
        err = np.abs(got_o[a:b] - o)
        assert np.isfinite(got_o[a:b]).all(), s
        assert (err <= do).all(), (s, float((err / do).max()))
        worst = max(worst, float((err / np.maximum(do, 1e-300)).max()))
        if got_lse is not None:
            gl = got_lse[:, a:b].T
            dead = ~np.isfinite(lse)
            assert np.array_equal(gl[dead], lse[dead])
            assert (np.abs(gl[~dead] - lse[~dead]) <= dl[~dead]).all()
    return worst
