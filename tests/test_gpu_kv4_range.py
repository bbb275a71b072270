"""GPU parity of the 4-bit attention over the whole range of the cache's types:
V scales, K scales and scores of every magnitude that append can write."""
import numpy as np
import pytest

from oracle import kv4 as okv

torch = pytest.importorskip("torch")
from tests import kv4_cases as kc  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(autouse=True)
def _status():
    yield
    import tile_routed_mixed_b200 as tm
    assert tm.tilemix_get_error() == tm.OK


def _fill(pool, which, scale_of):
    """Rows of `which` with magnitudes scale_of(position) (an array per sequence)."""
    rng = np.random.default_rng(97)
    for s, n in enumerate(pool.lengths):
        x = np.clip(rng.standard_normal((n, pool.hk, pool.d)), -3.9, 3.9)
        x = okv.round_to(x * np.asarray(scale_of(np.arange(n), n), dtype=np.float64)[:, None, None], pool.dtype)
        c, sc = okv.quantise(x, pool.group, pool.dtype)
        pages, rows = pool.table[s, np.arange(n) // pool.page], np.arange(n) % pool.page
        pool.codes[which][pages, :, rows] = c
        pool.scales[which][pages, :, rows] = sc


def _largest(pool, s, queries):
    """The largest V scale that each query meets, [queries, 1, 1]."""
    n = pool.lengths[s]
    pages, rows = pool.table[s, np.arange(n) // pool.page], np.arange(n) % pool.page
    top = pool.scales["v"][pages, :, rows].max(axis=(1, 2))
    return np.array([top[:max(0, n - queries + i + 1)].max(initial=0.0) for i in range(queries)])[:, None, None]


def _check(pool, queries, hq, q_scale=1.0, scale=0.0, seed=5):
    """Attention of the last queries[s] tokens against the oracle, within the
    bound of kv4_cases with each query's own largest V scale (and half a step of
    a subnormal bf16 output)."""
    rng = np.random.default_rng(seed)
    start = np.concatenate([[0], np.cumsum(queries)])
    q = kc.draw(rng, (int(start[-1]), hq, pool.d), pool.dtype, q_scale)
    start_d = torch.tensor(start.tolist(), dtype=torch.int32, device="cuda")
    o, lse = pool.cache().attend(kc.to_device(q, pool.dtype), max(pool.lengths), token_start=start_d,
                                 max_new=max(queries), softmax_scale=scale, lse=True)
    o, lse = kc.to_numpy(o), kc.to_numpy(lse).T
    for s, n in enumerate(pool.lengths):
        a, b = start[s], start[s + 1]
        want, wlse, mag, reach = okv.attend(q[a:b], pool.row("k", s), pool.row("v", s), b - a, scale or None)
        do, dl = kc.attend_bounds(want, wlse, mag, reach, pool.dtype, _largest(pool, s, b - a), n)
        do = do + 2.0 ** -134
        assert np.isfinite(o[a:b]).all() and np.isfinite(lse[a:b]).all(), s
        assert (np.abs(o[a:b] - want) <= do).all(), (s, float((np.abs(o[a:b] - want) / do).max()))
        assert (np.abs(lse[a:b] - wlse) <= dl).all(), s


SHAPES = [(128, 32, 1, [1, 1]), (128, 128, 2, [3, 1]), (64, 32, 2, [7, 2]), (128, 64, 5, [5, 3])]


@pytest.mark.parametrize("d,group,rep,queries", SHAPES)
@pytest.mark.parametrize("power", [-126, -110, -95, -88, -70, -60, 60, 93, 97, 104, 115, 125])
def test_values_of_one_magnitude(d, group, rep, queries, power):
    """All of V near one power of two, from the smallest normal bf16 to the largest."""
    rng = np.random.default_rng(1)
    pool = kc.Pool(rng, [40, 1500], 2, d, group, 32, "bf16")
    _fill(pool, "v", lambda at, n: np.full(n, 2.0 ** power))
    _check(pool, queries, 2 * rep)


@pytest.mark.parametrize("d,group,rep,queries", SHAPES)
@pytest.mark.parametrize("turn", ["grow", "fall", "zeros_first", "zeros_last"])
def test_values_of_all_magnitudes(d, group, rep, queries, turn):
    """V from 2^-120 to 2^120 along a sequence, either way, and rows of zeros
    before or behind tiny and huge ones: partial results of very different units
    are joined."""
    rng = np.random.default_rng(2)
    pool = kc.Pool(rng, [200, 2500], 2, d, group, 16, "bf16")

    def scale_of(at, n):
        if turn == "grow":
            return 2.0 ** (at * 240 // n - 120.0)
        if turn == "fall":
            return 2.0 ** (120.0 - at * 240 // n)
        half = (at < n // 2) == (turn == "zeros_first")
        return np.where(half, 0.0, 2.0 ** np.where(at % 2 == 0, 110.0, -110.0) if n > 1000 else 2.0 ** -115)

    _fill(pool, "v", scale_of)
    _check(pool, queries, 2 * rep)


@pytest.mark.parametrize("dtype,group,rep,new,low,high", [("bf16", 32, 1, 1, -53, 110), ("bf16", 64, 4, 3, 0, 122),
                                                          ("fp16", 64, 4, 3, -9, 14)])
def test_values_that_jump(dtype, group, rep, new, low, high):
    """One huge row behind many small ones, where a warp has several tiles: what
    it had before keeps its share of the sum."""
    lengths = [4000, 3970, 4100, 3900, 4050]
    pool = kc.Pool(np.random.default_rng(6), lengths, 8, 64, group, 64, dtype)
    _fill(pool, "v", lambda at, n: np.where(at == n // 3, 2.0 ** high, 2.0 ** low))
    _check(pool, [new] * 5, 8 * rep)


@pytest.mark.parametrize("dtype,own,later", [("bf16", 0, 40), ("bf16", 0, 62), ("bf16", 0, 98), ("bf16", 0, 125),
                                             ("bf16", -50, 124), ("bf16", -100, 0), ("bf16", 100, 125),
                                             ("fp16", -9, 13), ("fp16", -14, 0)])
@pytest.mark.parametrize("d,group,rep,queries", [(128, 32, 1, 3), (128, 64, 4, 5), (64, 64, 2, 21), (64, 32, 1, 40)])
@pytest.mark.parametrize("length", [45, 1300])
def test_a_later_tokens_values_cost_earlier_queries_nothing(dtype, own, later, d, group, rep, queries, length):
    """V rows that only the last queries see, far larger than the others: the
    queries in front of them are as exact as without."""
    rng = np.random.default_rng(3)
    pool = kc.Pool(rng, [length], 2, d, group, 16, dtype)
    _fill(pool, "v", lambda at, n: np.where(at < n - (queries + 1) // 2, 2.0 ** own, 2.0 ** later))
    _check(pool, [queries], 2 * rep)


def test_zeros_before_a_later_tokens_values():
    """Queries that see rows of zeros only, and one that sees a huge row: as
    outputs, and as partial results of several CTAs."""
    for length in (50, 4000):
        pool = kc.Pool(np.random.default_rng(4), [length], 1, 128, 32, 16, "bf16")
        _fill(pool, "v", lambda at, n: np.where((at < n - 1) & (at > 40), 0.0, 2.0 ** 120))
        _check(pool, [3], 2)
        _fill(pool, "v", lambda at, n: np.where(at < n - 1, 0.0, 1.0))
        _check(pool, [3], 2)


def _put(pool, which, s, x):
    """Rows x [n, hk, d] as sequence s's K or V."""
    n = pool.lengths[s]
    c, sc = okv.quantise(okv.round_to(x, pool.dtype), pool.group, pool.dtype)
    pages, rows = pool.table[s, np.arange(n) // pool.page], np.arange(n) % pool.page
    pool.codes[which][pages, :, rows] = c
    pool.scales[which][pages, :, rows] = sc


SCORES = [("fp16", p) for p in (18, 22, 25, 26, 27, 28, 29, 31, 34)] + \
         [("bf16", p) for p in (22, 26, 28, 30, 40, 70, 110)]


@pytest.mark.parametrize("dtype,power", SCORES)
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("value", [2.0 ** -13, 1.0, 2.0 ** 12])
def test_equal_scores_of_any_size(dtype, power, sign, value):
    """Keys that are all the same, with scores (in powers of two) up to 2^power:
    O is the mean of V, whatever the size of the scores (their rounding is the
    same for all keys), the LSE the score itself to a rounding or two."""
    d, rep, queries = 128, 2, [2, 1]
    pool = kc.Pool(np.random.default_rng(7), [700, 33], 2, d, 32, 16, dtype)
    _fill(pool, "v", lambda at, n: np.full(n, value))
    size = 2.0 ** ((power - 4) / 2)            # d size^2 / sqrt(d) * log2(e) = 2^(4.03 + 2 log2(size))
    for s, n in enumerate(pool.lengths):
        _put(pool, "k", s, np.full((n, 2, d), size))
    q = okv.round_to(np.full((3, 2 * rep, d), sign * size), dtype)
    start = [0, 2, 3]
    o, lse = pool.cache().attend(kc.to_device(q, dtype), 700, max_new=2, lse=True,
                                 token_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    o, lse = kc.to_numpy(o), kc.to_numpy(lse).T
    for s, n in enumerate(pool.lengths):
        a, b = start[s], start[s + 1]
        want, wlse, mag, _ = okv.attend(q[a:b], pool.row("k", s), pool.row("v", s), b - a)
        do, _ = kc.attend_bounds(want, wlse, mag, np.zeros(wlse.shape), dtype, _largest(pool, s, b - a), n)
        assert np.isfinite(o[a:b]).all()
        assert (np.abs(o[a:b] - want) <= do).all(), float((np.abs(o[a:b] - want) / do).max())
        assert (np.abs(lse[a:b] - wlse) <= 2.0 ** -18 + 2.0 ** -20 * np.abs(wlse)).all()


# (channel 0 alone makes the score here: fp16 ends at 65504^2 / sqrt(128) * log2(e), 2^29)
@pytest.mark.parametrize("dtype,power", [x for x in SCORES if x[0] == "bf16" or x[1] < 29])
@pytest.mark.parametrize("rising", [False, True])
def test_scores_that_differ_by_their_last_bits(dtype, power, rising):
    """A large common score and small differences, at random or rising along the
    sequence.  Rounded to fp32 many differences are gone, so all that can be asked
    is a finite mean of V's rows with weights between zero and one, whose sum is one."""
    d = 128
    rng = np.random.default_rng(8)
    pool = kc.Pool(rng, [1500, 64], 1, d, 32, 32, dtype)
    size = 2.0 ** ((power + 3) / 2)
    q = np.zeros((3, 2, d))
    q[..., 0], q[..., 40] = size, 1.0
    q = okv.round_to(q, dtype)
    for s, n in enumerate(pool.lengths):
        x = np.zeros((n, 1, d))
        x[..., 0] = size
        x[:, 0, 40] = np.linspace(-2000, 2000, n) if rising else rng.uniform(-2000, 2000, n)
        _put(pool, "k", s, x)
        v = np.clip(rng.standard_normal((n, 1, d)), -3, 3) * 2.0 ** -13
        v[..., 100:] = 2.0 ** -13              # the same in all rows: the sum of the weights
        _put(pool, "v", s, v)
    start = [0, 2, 3]
    o = pool.cache().attend(kc.to_device(q, dtype), 1500, max_new=2,
                            token_start=torch.tensor(start, dtype=torch.int32, device="cuda"))
    o = kc.to_numpy(o)
    assert np.isfinite(o).all()
    for s, n in enumerate(pool.lengths):
        for i in range(start[s], start[s + 1]):
            v = pool.row("v", s)[:n - (start[s + 1] - i) + 1, 0]
            slack = 2.0 ** -6 * np.abs(v).max()    # bf16's rounding, P s_v's and the sums'
            assert (o[i] >= v.min(axis=0) - slack).all() and (o[i] <= v.max(axis=0) + slack).all()


@pytest.mark.parametrize("d,group,rep,queries", SHAPES)
@pytest.mark.parametrize("power", [-126, -110, -70, 70, 100, 104, 112, 120, 125])
def test_keys_of_one_magnitude(d, group, rep, queries, power):
    """All of K near one power of two, with queries that bring the scores back to
    ordinary ones."""
    pool = kc.Pool(np.random.default_rng(9), [40, 1500], 2, d, group, 32, "bf16")
    _fill(pool, "k", lambda at, n: np.full(n, 2.0 ** power))
    _check(pool, queries, 2 * rep, q_scale=2.0 ** -min(max(power, -124), 124))


@pytest.mark.parametrize("d,group,rep,queries", SHAPES)
def test_keys_of_many_magnitudes(d, group, rep, queries):
    """K from 2^-100 to 2^100 along a sequence."""
    pool = kc.Pool(np.random.default_rng(10), [200, 1900], 2, d, group, 32, "bf16")
    _fill(pool, "k", lambda at, n: 2.0 ** (at * 200 // n - 100.0))
    _check(pool, queries, 2 * rep, q_scale=2.0 ** -99)


@pytest.mark.parametrize("d,group,rep,queries", SHAPES)
@pytest.mark.parametrize("power", [90, 104, 116, 122])
def test_one_key_takes_all(d, group, rep, queries, power):
    """Keys so large that the largest score takes all: O is its row of V, wherever
    the next score is further away than the scores' rounding."""
    rng = np.random.default_rng(11)
    pool = kc.Pool(rng, [33, 700], 2, d, group, 32, "bf16")
    _fill(pool, "k", lambda at, n: np.full(n, 2.0 ** power))
    start = np.concatenate([[0], np.cumsum(queries)])
    q = kc.draw(rng, (int(start[-1]), 2 * rep, d), "bf16")
    o = pool.cache().attend(kc.to_device(q, "bf16"), 700, max_new=max(queries),
                            token_start=torch.tensor(start.tolist(), dtype=torch.int32, device="cuda"))
    o = kc.to_numpy(o)
    assert np.isfinite(o).all()
    sure = 0
    for s, n in enumerate(pool.lengths):
        k, v = pool.row("k", s), pool.row("v", s)
        for i in range(start[s], start[s + 1]):
            m = n - (start[s + 1] - i) + 1
            for h in range(2 * rep):
                x = k[:m, h // rep] @ q[i, h]
                first, second = np.argsort(x)[::-1][:2]
                reach = np.abs(q[i, h]).sum() * np.abs(k[:m, h // rep]).max()
                if x[first] - x[second] > 2.0 ** -16 * reach:
                    sure += 1
                    # the value itself, rounded; P s_v to 11 bits
                    assert (np.abs(o[i, h] - v[first, h // rep]) <=
                            (kc.EPS["bf16"] + 2.0 ** -10) * np.abs(v[first, h // rep])).all()
    assert sure > 0


@pytest.mark.parametrize("own,later", [(-118, -76), (-89, 118), (-110, 77), (-120, 120), (-60, 122), (-40, 125)])
@pytest.mark.parametrize("d,group,rep,queries", [(128, 64, 1, 9), (128, 64, 4, 4), (64, 32, 2, 21)])
@pytest.mark.parametrize("length", [23, 1100])
def test_a_later_tokens_values_far_above_tiny_ones(own, later, d, group, rep, queries, length):
    """One huge row among the newest tokens over rows of tiny ones: neither end of
    the type may cost the other's queries their bits."""
    pool = kc.Pool(np.random.default_rng(12), [length], 2, d, group, 16, "bf16")
    _fill(pool, "v", lambda at, n: np.where(at == n - (queries + 1) // 2, 2.0 ** later, 2.0 ** own))
    _check(pool, [queries], 2 * rep)
