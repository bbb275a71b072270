"""The 4-bit attention against the sharper limits of kv4_limits, and with more
queries than a few column blocks hold."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from tests import kv4_cases as kc  # noqa: E402
from tests import kv4_limits as kl  # noqa: E402

pytestmark = pytest.mark.gpu

FORMATS = [("fp16", 128, 32), ("bf16", 128, 32), ("fp16", 128, 64), ("bf16", 128, 64),
           ("fp16", 128, 128), ("bf16", 128, 128), ("fp16", 64, 32), ("bf16", 64, 32),
           ("fp16", 64, 64), ("bf16", 64, 64)]


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


@pytest.mark.parametrize("dtype,d,group", FORMATS)
@pytest.mark.parametrize("lengths,queries,rep,q_scale", [([900, 40, 333], [1, 1, 1], 3, 1.0),
                                                         ([700, 65, 130], [5, 2, 20], 4, 1.0),
                                                         ([800, 64], [1, 3], 2, 8.0)])
def test_rms_of_the_error(dtype, d, group, lengths, queries, rep, q_scale):
    rng = np.random.default_rng(50)
    pool = kc.Pool(rng, lengths, 2, d, group, 32, dtype)
    start = np.concatenate([[0], np.cumsum(queries)])
    q = kc.draw(rng, (int(start[-1]), 2 * rep, d), dtype, q_scale)
    o = kc.to_numpy(pool.cache().attend(kc.to_device(q, dtype), max(lengths), token_start=_i32(start),
                                        max_new=max(queries)))
    for s in range(len(lengths)):
        a, b = start[s], start[s + 1]
        want, limit = kl.rms_limit(q[a:b], pool.row("k", s), pool.row("v", s), b - a, dtype)
        assert kl.rms(o[a:b] - want) <= limit, (s, kl.rms(o[a:b] - want) / limit)


@pytest.mark.parametrize("dtype,d,group", FORMATS)
@pytest.mark.parametrize("lengths,hk,new,page", [([20000], 1, 1, 128), ([9000, 9000], 2, 4, 16),
                                                 ([700, 5000, 33, 0, 12000, 64, 1, 2500], 3, 1, 64),
                                                 ([4096] * 8, 4, 2, 32)])
def test_each_tile_counts_once(dtype, d, group, lengths, hk, new, page):
    """K is zero, so all keys that a query sees have the same weight, and V marks the
    tile: a tile that the split over warps and CTAs leaves out or takes twice shows in
    O and in the LSE."""
    rng = np.random.default_rng(51)
    import tile_routed_mixed_b200 as tm
    value = kl.marked_value(group, dtype)
    used = [-(-n // page) for n in lengths]
    order = torch.randperm(sum(used) + 1, generator=torch.Generator().manual_seed(3)).tolist()
    cache = tm.TileMixKV4Cache(sum(used) + 1, page, hk, d, len(lengths), max(used), group=group,
                               dtype=kc.TORCH[dtype])
    table, at = np.full((len(lengths), max(used)), -1, dtype=np.int32), 0
    slots, rows = [], []
    for s, n in enumerate(lengths):
        table[s, :used[s]] = order[at:at + used[s]]
        at += used[s]
        pos = np.arange(n)
        slots.append(table[s, pos // page] * page + pos % page)
        rows.append(kl.markers(n, d))
    cache.block_table.copy_(torch.from_numpy(table))
    cache.seq_len.copy_(torch.tensor(lengths, dtype=torch.int32))
    v = torch.from_numpy(np.concatenate(rows)).to(kc.TORCH[dtype]).cuda().expand(-1, hk, -1).contiguous()
    cache.append(torch.zeros_like(v), v, _i32(np.concatenate(slots)))
    start = [new * s for s in range(len(lengths) + 1)]
    q = kc.draw(rng, (start[-1], 2 * hk, d), dtype)
    o, lse = cache.attend(kc.to_device(q, dtype), max(lengths), token_start=_i32(start), max_new=new, lse=True)
    o, lse = kc.to_numpy(o), kc.to_numpy(lse)
    for s, n in enumerate(lengths):
        for i in range(new):
            m = n - new + i + 1
            got = o[start[s] + i]
            if m <= 0:
                assert not got.any() and np.isneginf(lse[:, start[s] + i]).all()
                continue
            want, slack = kl.marked_weights(m, dtype, value)
            assert (np.abs(got[:, :kl.LANES] - want) <= slack).all(), (s, i)
            assert not got[:, kl.LANES:].any()
            assert (np.abs(lse[:, start[s] + i] - np.log(m)) <= 2.0 ** -18 + 2.0 ** -22 * np.log(m)).all()


@pytest.mark.parametrize("dtype,d,group,rep,lengths,queries", [
    ("fp16", 128, 32, 4, [600, 300], [300, 300]), ("bf16", 64, 64, 1, [1030, 257, 20], [257, 130, 20]),
    ("bf16", 128, 128, 7, [200, 100], [90, 33])])
def test_a_chunk_of_a_prompt(dtype, d, group, rep, lengths, queries):
    """Tens of column blocks: a chunk of a prompt over what is cached before it, a
    whole prompt among them (its first query sees one key)."""
    rng = np.random.default_rng(52)
    pool = kc.Pool(rng, lengths, 2, d, group, 16, dtype)
    start = np.concatenate([[0], np.cumsum(queries)])
    q = kc.draw(rng, (int(start[-1]), 2 * rep, d), dtype)
    o, lse = pool.cache().attend(kc.to_device(q, dtype), max(lengths), token_start=_i32(start),
                                 max_new=max(queries), lse=True)
    kc.check_attend(kc.to_numpy(o), kc.to_numpy(lse), q, pool, lengths, start, 2 * rep)
    for s in range(len(lengths)):
        a, b = start[s], start[s + 1]
        want, limit = kl.rms_limit(q[a:b], pool.row("k", s), pool.row("v", s), b - a, dtype)
        assert kl.rms(kc.to_numpy(o)[a:b] - want) <= limit
