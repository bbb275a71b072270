"""Append and gather at the sizes from which a thread takes four tokens, on both
sides of the rule, bit for bit."""
import numpy as np
import pytest

from oracle import kv4 as okv

torch = pytest.importorskip("torch")
from tests import kv4_cases as kc  # noqa: E402

pytestmark = pytest.mark.gpu

FORMATS = [("fp16", 128, 32), ("bf16", 128, 32), ("fp16", 128, 64), ("bf16", 128, 64),
           ("fp16", 128, 128), ("bf16", 128, 128), ("fp16", 64, 32), ("bf16", 64, 32),
           ("fp16", 64, 64), ("bf16", 64, 64)]
HK = 8
WIDE = 148 * 2048 * 2  # chunks of eight channels from which on a thread takes four tokens


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.fixture(autouse=True)
def _status():
    yield
    import tile_routed_mixed_b200 as tm
    assert tm.tilemix_get_error() == tm.OK


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _rows(rng, n, d, dtype):
    """Ordinary rows, with zeros, infinities, NaN and tiny values among them."""
    x = kc.draw(rng, (n, HK, d), dtype, 2.0)
    x[::97] = 0.0
    x[5::211, 1, 3] = np.inf
    x[7::301, -1, -1] = np.nan
    x[11::53] *= 2.0 ** -12
    return okv.round_to(x, dtype)


@pytest.mark.parametrize("dtype,d,group", FORMATS)
@pytest.mark.parametrize("more", [-1, 0, 13])
def test_append_around_four_tokens_a_thread(dtype, d, group, more):
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(60)
    n, page = WIDE // (HK * d // 8) + more, 64
    num_pages = n // page + 2
    k, v = (_rows(rng, n, d, dtype) for _ in range(2))
    slots = rng.permutation(num_pages * page)[:n].astype(np.int64)
    slots[[0, 17, 18, 19, n - 1]] = -1
    slots[[3, 40, n - 2]] = [num_pages * page, -7, 2 ** 31 - 1]
    cache = tm.TileMixKV4Cache(num_pages, page, HK, d, 1, 1, group=group, dtype=kc.TORCH[dtype])
    for x in (cache.k_codes, cache.v_codes):
        x.fill_(0x5A)
    for x in (cache.k_scale, cache.v_scale):
        x.fill_(3.0)
    cache.append(kc.to_device(k, dtype), kc.to_device(v, dtype), _i32(slots))
    assert tm.tilemix_get_error() == tm.ERR_INVALID_ARG
    real = np.nonzero((slots >= 0) & (slots < num_pages * page))[0]
    p, r = slots[real] // page, slots[real] % page
    for w, x, codes, scale in (("k", k, cache.k_codes, cache.k_scale), ("v", v, cache.v_codes, cache.v_scale)):
        c, s = okv.quantise(x, group, dtype)
        want_c = np.full((num_pages, HK, page, d // 2), 0x5A, dtype=np.uint8)
        want_s = np.full((num_pages, HK, page, d // group), 3.0)
        want_c[p, :, r] = okv.pack(c, w)[real]
        want_s[p, :, r] = s[real]
        assert np.array_equal(codes.cpu().numpy(), want_c), w
        assert kc.same(kc.to_numpy(scale), want_s), w


@pytest.mark.parametrize("dtype,d,group", FORMATS)
@pytest.mark.parametrize("more,clipped", [(-1, False), (0, False), (13, True)])
def test_gather_around_four_tokens_a_thread(dtype, d, group, more, clipped):
    """One sequence far longer than the average (several sweeps of its CTAs), short
    and empty ones beside it; rows that lie outside the output at both ends."""
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(61)
    rows, page = WIDE // (HK * d // 8) + more, 32
    lengths = [0, 1, 37, rows - 1400, 0, 500, 16, 64, 3]
    pool = kc.Pool(rng, lengths, HK, d, group, page, dtype)
    pool.scales["v"][pool.table[3, 2], 1, 3] = np.nan
    # sequence 1 before the output, the last rows of sequence 5 behind it
    starts = [0, -1, 0, 40, 5, rows - 450, rows - 500, rows - 600, rows - 700] if clipped else \
        [0, 0, 1, 40, 5, rows - 500, rows - 1000, rows - 900, rows - 800]
    cache = pool.cache()
    out = [torch.full((rows, HK, d), 9.0, dtype=kc.TORCH[dtype], device="cuda") for _ in range(2)]
    cache.gather(_i32(starts), rows, out=out)
    if clipped:
        assert tm.tilemix_get_error() == tm.ERR_INVALID_ARG
    for w, t in zip("kv", out):
        want = np.full((rows, HK, d), 9.0)
        for s, n in enumerate(lengths):
            a, b = max(0, starts[s]), min(rows, starts[s] + n)
            want[a:b] = okv.round_to(pool.row(w, s), dtype)[a - starts[s]:max(0, b - starts[s])]
        assert kc.same(kc.to_numpy(t), want)
