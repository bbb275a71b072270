"""GPU tests of how the 4-bit cache's calls go together: refused tokens, tables,
streams and sizes, each against the oracle."""
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


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


# -------------------------------------------------------- refused tokens ---

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("graph", [False, True])
def test_a_step_that_is_refused(dtype, graph):
    """Steps through plan, append and attend in a pool that runs out and with rows
    that are full: the queries of refused sequences get zeros and an LSE of
    -infinity, all others what the oracle says; a later step goes on from there."""
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(40)
    hq, hk, d, page, group = 6, 2, 64, 16, 32
    cache = tm.TileMixKV4Cache(9, page, hk, d, 4, 3, group=group, dtype=kc.TORCH[dtype])
    want = okv.Pages(9, page, 4, 3)
    coded = lambda x: okv.values(*okv.quantise(x, group, dtype), group)
    hist = [[np.zeros((0, hk, d))] * 2 for _ in range(4)]
    # pages of 16, three a row, nine in all: 2 + 1 + 3 + 2; sequence 2 is full, one page
    # is left for two that need one; then sequence 2 ends and all fit
    steps = [[30, 16, 48, 20], [1, 1, 1, 13], [17, 2, 0, 1], [1, 16, -48, 1], [2, 17, 33, 0]]
    top = max(sum(max(x, 0) for x in st) for st in steps)
    new, out = _i32([0] * 4), cache.new_plan(top)
    q, k, v = (torch.zeros((top, h, d), dtype=kc.TORCH[dtype], device="cuda") for h in (hq, hk, hk))
    o, lse = torch.zeros_like(q), torch.zeros((hq, top), device="cuda")

    def step():
        cache.plan(new, out=out)
        cache.append(k, v, out.slots)
        cache.attend(q, 48, token_start=out.token_start, max_new=48, out=o, lse=lse, granted=out.granted)

    run = step
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        run = g.replay
    refused = 0
    for st in steps:
        qh, kh, vh = (kc.draw(rng, (top, h, d), dtype) for h in (hq, hk, hk))
        for t, x in ((q, qh), (k, kh), (v, vh)):
            t.copy_(kc.to_device(x, dtype))
        new.copy_(_i32(st))
        o.fill_(7.0)
        lse.fill_(7.0)
        run()
        start, _, granted = want.plan(st, top)
        assert out.granted.tolist() == granted and out.token_start.tolist() == start
        got, gl = kc.to_numpy(o), kc.to_numpy(lse)
        for s, m in enumerate(st):
            a, b = start[s], start[s + 1]
            if not granted[s]:
                refused += 1
                assert not got[a:b].any() and np.isneginf(gl[:, a:b]).all()
                continue
            hist[s] = [x[:max(0, len(x) + m)] for x in hist[s]] if m < 0 else \
                [np.concatenate([x, coded(y[a:b])]) for x, y in zip(hist[s], (kh, vh))]
        pool = type("P", (), {"dtype": dtype})
        live = [s for s in range(4) if granted[s]]
        for s in live:
            kc.check_attend(got[start[s]:start[s + 1]], gl[:, start[s]:start[s + 1]], qh[start[s]:start[s + 1]], pool,
                            [len(hist[s][0])], [0, start[s + 1] - start[s]], hq, kv=lambda _: hist[s])
        assert (got[start[-1]:] == 7.0).all() and (gl[:, start[-1]:] == 7.0).all()
        assert cache.seq_len.tolist() == [len(x[0]) for x in hist]
    assert refused >= 3
    bad = _i32([1] * 3)
    with pytest.raises(ValueError):
        cache.attend(q[:4], 48, granted=bad)


def test_refused_among_many_and_long():
    """Granted or not over units that several CTAs share, one query per sequence."""
    rng = np.random.default_rng(41)
    lengths = [int(x) for x in rng.integers(1, 3000, 24)]
    pool = kc.Pool(rng, lengths, 2, 64, 64, 64, "bf16")
    q = kc.draw(rng, (24, 4, 64), "bf16")
    granted = [int(x) for x in rng.integers(0, 2, 24)]
    o, lse = pool.cache().attend(kc.to_device(q, "bf16"), 3000, lse=True, granted=_i32(granted))
    o, lse = kc.to_numpy(o), kc.to_numpy(lse)
    for s in range(24):
        if granted[s]:
            one = type("P", (), {"dtype": "bf16"})
            kc.check_attend(o[s:s + 1], lse[:, s:s + 1], q[s:s + 1], one, [lengths[s]], [0, 1], 4,
                            kv=lambda _: (pool.row("k", s), pool.row("v", s)))
        else:
            assert not o[s].any() and np.isneginf(lse[:, s]).all()


# --------------------------------------------------------------- streams ---

def test_tensors_dropped_after_a_call_on_another_stream():
    """q, token_start and the appended rows are dropped and their sizes allocated and
    filled again while the side stream has not begun: results are those of the
    first contents."""
    rng = np.random.default_rng(42)
    pool = kc.Pool(rng, [500, 90], 2, 128, 32, 16, "fp16")
    cache = pool.cache()
    side = torch.cuda.Stream()
    out = torch.empty((3, 4, 128), dtype=torch.float16, device="cuda")
    k2, v2 = (torch.empty((590, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2))
    q, k, v = (kc.draw(rng, (3, h, 128), "fp16") for h in (4, 2, 2))
    slots = [int(pool.table[0, 499 // 16]) * 16 + 499 % 16] + [int(pool.table[1, p // 16]) * 16 + p % 16 for p in (88, 89)]
    tensors = [kc.to_device(x, "fp16") for x in (q, k, v)] + [_i32(slots), _i32([0, 1, 3]), _i32([0, 500])]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # a tenth of a second
    cache.append(tensors[1], tensors[2], tensors[3], stream=side)
    cache.attend(tensors[0], 500, token_start=tensors[4], max_new=2, out=out, stream=side)
    cache.gather(tensors[5], 590, out=(k2, v2), stream=side)
    shapes = [(x.shape, x.dtype) for x in tensors]
    del tensors
    for _ in range(4):  # (garbage that is legal as slots, offsets and values)
        junk = [torch.zeros(s, dtype=t, device="cuda") for s, t in shapes]
    torch.cuda.synchronize()
    del junk
    coded = lambda x: okv.values(*okv.quantise(x, 32, "fp16"), 32)
    hist = []
    for s, (a, b) in enumerate(((0, 1), (1, 3))):
        hist.append([np.concatenate([pool.row(w, s)[:-(b - a)], coded(x[a:b])]) for w, x in (("k", k), ("v", v))])
    kc.check_attend(kc.to_numpy(out), None, q, pool, [500, 90], [0, 1, 3], 4, kv=lambda s: hist[s])
    for t, i in ((k2, 0), (v2, 1)):
        assert np.array_equal(kc.to_numpy(t), okv.round_to(np.concatenate([h[i] for h in hist]), "fp16"))


# ---------------------------------------------------------- shared pages ---

def test_a_shared_prefix_ends_as_documented():
    """Two requests share two full pages: one drops to them and is cleared by hand,
    the other goes on reading them, and no later request is given them before it
    has ended as well."""
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(43)
    hq, hk, d, page, group = 4, 2, 64, 16, 32
    cache = tm.TileMixKV4Cache(8, page, hk, d, 3, 6, group=group)
    coded = lambda x: okv.values(*okv.quantise(x, group, "fp16"), group)
    pool = type("P", (), {"dtype": "fp16"})

    def step(new):
        n = sum(max(x, 0) for x in new)
        q, k, v = (kc.draw(rng, (n, h, d), "fp16") for h in (hq, hk, hk))
        plan = cache.plan(_i32(new), max_tokens=n)
        assert plan.granted.tolist() == [1] * 3
        if n:
            cache.append(kc.to_device(k, "fp16"), kc.to_device(v, "fp16"), plan.slots)
        at = 0
        for s, m in enumerate(new):
            if m > 0:
                hist[s] = [np.concatenate([x, coded(y[at:at + m])]) for x, y in zip(hist[s], (k, v))]
                at += m
            elif m:
                hist[s] = [x[:len(x) + m] for x in hist[s]]
        if n:
            o, lse = cache.attend(kc.to_device(q, "fp16"), 96, token_start=plan.token_start, max_new=max(new),
                                  lse=True, granted=plan.granted)
            kc.check_attend(kc.to_numpy(o), kc.to_numpy(lse), q, pool, [len(h[0]) for h in hist],
                            plan.token_start.tolist(), hq, kv=lambda s: hist[s])

    empty = [np.zeros((0, hk, d))] * 2
    hist = [empty, empty, empty]
    step([32, 0, 0])
    shared = cache.block_table[0, :2].tolist()
    cache.block_table[1, :2] = cache.block_table[0, :2]
    cache.seq_len[1] = 32
    hist[1] = hist[0]
    step([3, 20, 0])              # both grow into pages of their own
    step([1, -20, 0])             # the second ends: back to the shared tokens
    cache.block_table[1] = -1
    cache.seq_len[1] = 0
    hist[1] = empty
    step([1, 0, 70])              # five pages, none of them shared
    held = cache.block_table[2, :5].tolist()
    assert len(set(held + shared)) == 7
    step([1, 0, 1])
    step([-38, 0, 1])             # the first ends and returns them
    assert set(shared) <= set(cache.free_list[:int(cache.free_count)].tolist())
    step([16, 0, 1])


# ------------------------------------------------------------------ size ---

def test_a_pool_beyond_four_gigabytes():
    """Rows on both sides of the byte offset 2^32 in a pool of 4.7 GB for each of K and
    V: appended, attended to and read back."""
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(44)
    hq, hk, d, page, group, n = 8, 8, 128, 1024, 32, 2300
    cache = tm.TileMixKV4Cache(9000, page, hk, d, 2, 4, group=group, dtype=torch.bfloat16)
    edge = 2 ** 32 // (page * hk * d // 2)             # the page that starts at 2^32
    table = [[edge, 8999, edge - 1, -1], [1, edge + 1, -1, -1]]
    lengths = [n, 1100]
    cache.block_table.copy_(torch.tensor(table, dtype=torch.int32))
    cache.seq_len.copy_(torch.tensor(lengths, dtype=torch.int32))
    slots = np.concatenate([np.array(table[s])[np.arange(m) // page] * page + np.arange(m) % page
                            for s, m in enumerate(lengths)])
    k, v = (kc.draw(rng, (sum(lengths), hk, d), "bf16") for _ in range(2))
    cache.append(kc.to_device(k, "bf16"), kc.to_device(v, "bf16"), _i32(slots))
    coded = [okv.values(*okv.quantise(x, group, "bf16"), group) for x in (k, v)]
    got = cache.gather(_i32([0, n]), sum(lengths))
    for t, x in zip(got, coded):
        assert np.array_equal(kc.to_numpy(t), okv.round_to(x, "bf16"))
    q = kc.draw(rng, (3, hq, d), "bf16")
    o, lse = cache.attend(kc.to_device(q, "bf16"), n, token_start=_i32([0, 2, 3]), max_new=2, lse=True)
    pool = type("P", (), {"dtype": "bf16"})
    kc.check_attend(kc.to_numpy(o), kc.to_numpy(lse), q, pool, lengths, [0, 2, 3], hq,
                    kv=lambda s: [x[n * s:n * s + lengths[s]] for x in coded])
