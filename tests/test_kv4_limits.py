"""The limits of kv4_limits tell mistakes apart that the element-wise bound lets
through: they are planted in the oracle here."""
import numpy as np
import pytest

from oracle import kv4 as okv

pytest.importorskip("torch")
from tests import kv4_cases as kc  # noqa: E402
from tests import kv4_limits as kl  # noqa: E402


def _rounded(x, bits):
    """x to `bits` bits, to nearest."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 2.0 ** bits), e - bits)


@pytest.mark.parametrize("q_scale", [1.0, 8.0])
def test_the_rms_limit_rejects_small_mistakes(q_scale):
    rng = np.random.default_rng(1)
    n, queries, d = 300, 2, 128
    pool = kc.Pool(rng, [n], 2, d, 32, 16, "fp16")
    k, v = pool.row("k", 0), pool.row("v", 0)
    q = kc.draw(rng, (queries, 4, d), "fp16", q_scale)
    o, limit = kl.rms_limit(q, k, v, queries, "fp16")
    assert np.allclose(o, okv.attend(q, k, v, queries)[0], rtol=1e-9, atol=1e-12)
    attend = lambda q, k, v: okv.attend(q, k, v, queries)[0]

    def with_p(bits):
        """The definition with P v rounded to `bits` bits, key by key."""
        out = np.zeros_like(o)
        for i in range(queries):
            m = n - queries + i + 1
            for h in range(4):
                x = k[:m, h // 2] @ q[i, h] / np.sqrt(d)
                p = np.exp(x - x.max())
                out[i, h] = _rounded(p[:, None] * v[:m, h // 2], bits).sum(axis=0) / p.sum()
        return out

    good = okv.round_to(with_p(11), "fp16")
    assert kl.rms(good - o) <= limit
    wrong = [("v off by 0.3%", attend(q, k, v * 1.003)), ("o off by 2%", o * 1.02),
             ("q to 7 bits", attend(_rounded(q, 7), k, v)), ("P v to 7 bits", with_p(7))]
    if q_scale == 1.0:  # (else most keys have next to no weight)
        wrong.append(("a key lost", attend(q, np.delete(k, 50, 0), np.delete(v, 50, 0))))
    for name, bad in wrong:
        assert kl.rms(okv.round_to(bad, "fp16") - o) > limit, name


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("n", [700, 20000])
def test_marked_tiles_show_one_that_is_lost_or_doubled(dtype, n):
    """At every place of the schedule, with O and with the LSE."""
    value = kl.marked_value(32, dtype)
    want, slack = kl.marked_weights(n, dtype, value)
    tiles = -(-n // kl.TILE)
    keys = np.bincount(np.arange(n) // kl.TILE)
    for t in range(0, tiles, max(1, tiles // 40)):
        for factor in (0, 2):
            w = np.ones(n)
            w[np.arange(n) // kl.TILE == t] = factor
            got = np.bincount(np.arange(n) // kl.TILE % kl.LANES, weights=w, minlength=kl.LANES) / w.sum() * value
            assert (np.abs(got - want) > slack).any()
            assert abs(np.log(n + (factor - 1) * keys[t]) - np.log(n)) > 2.0 ** -18 + 2.0 ** -22 * np.log(n)
