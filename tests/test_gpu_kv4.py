"""GPU parity of the paged 4-bit cache: plan, append, gather and attention
against the oracle."""
import ctypes

import numpy as np
import pytest

from oracle import kv4 as okv

torch = pytest.importorskip("torch")
from tests import kv4_cases as kc  # noqa: E402

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


def _i32(x, device="cuda"):
    return torch.tensor(list(x), dtype=torch.int32, device=device)


# ------------------------------------------------------------------- plan ---

def _same_tables(cache, want):
    got = cache.block_table.tolist()
    assert got == want.table
    assert cache.seq_len.tolist() == want.len
    assert int(cache.free_count) == want.free
    assert cache.free_list.tolist()[:want.free] == want.stack[:want.free]


def _same_plan(plan, want):
    assert plan.token_start.tolist() == want[0]
    assert plan.slots.tolist() == want[1]
    assert plan.granted.tolist() == want[2]


@pytest.mark.parametrize("nseq,page,num_pages,max_pages,max_tokens,top", [
    (1, 16, 9, 8, 64, 40),
    (7, 16, 40, 6, 200, 60),        # rows, the pool and the slots all run out now and then
    (33, 32, 60, 12, 700, 90),
    (300, 64, 400, 4, 5000, 150),   # several CTAs
    (1500, 16, 3000, 3, 3001, 20),  # several sequences per thread
])
def test_plan_steps(nseq, page, num_pages, max_pages, max_tokens, top):
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(nseq)
    cache = tm.TileMixKV4Cache(num_pages, page, 1, 64, nseq, max_pages, group=64)
    want = okv.Pages(num_pages, page, nseq, max_pages)
    refused = 0
    for step in range(24):
        new = rng.integers(-top, top + 1, nseq)
        new[rng.random(nseq) < 0.2] = 0
        if step % 5 == 4:
            new = np.minimum(new, 0)
        if step == 7:
            new[:] = -2 ** 31       # every request ends
        if step == 9:
            new[nseq // 2] = 2 ** 31 - 1
        new = [int(x) for x in new]
        plan = cache.plan(_i32(new), max_tokens=max_tokens)
        w = want.plan(new, max_tokens)
        w = ([min(x, 2 ** 31 - 1) for x in w[0]], w[1], w[2])
        _same_plan(plan, w)
        _same_tables(cache, want)
        refused += w[2].count(0)
    assert refused > 0  # the limits were met


def test_plan_long_prompts_and_their_rollback():
    """Prompts over many pages and CTAs; dropping them again leaves the tables
    and the stack as they were."""
    import tile_routed_mixed_b200 as tm
    nseq, page = 37, 16
    rng = np.random.default_rng(0)
    first = [int(x) for x in rng.integers(0, 200, nseq)]
    new = [int(x) for x in rng.integers(1, 3000, nseq)]
    num_pages = sum(-(-(a + b) // page) for a, b in zip(first, new)) + 5
    cache = tm.TileMixKV4Cache(num_pages, page, 1, 64, nseq, 256, group=64)
    want = okv.Pages(num_pages, page, nseq, 256)
    cache.plan(_i32(first), max_tokens=sum(first))
    want.plan(first, sum(first))
    before = [x.clone() for x in (cache.block_table, cache.seq_len, cache.free_list, cache.free_count)]
    plan = cache.plan(_i32(new), max_tokens=sum(new) + 3)
    _same_plan(plan, want.plan(new, sum(new) + 3))
    _same_tables(cache, want)
    out = cache.plan(_i32([-x for x in new]), max_tokens=0)
    assert out.granted.tolist() == [1] * nseq and out.token_start.tolist() == [0] * (nseq + 1)
    after = (cache.block_table, cache.seq_len, cache.free_list, cache.free_count)
    assert all(torch.equal(a, b) for a, b in zip(before, after))


def test_plan_most_and_no_sequences():
    import tile_routed_mixed_b200 as tm
    nseq = tm.PAGE_PLAN_MAX_SEQS
    cache = tm.TileMixKV4Cache(nseq, 16, 1, 64, nseq, 2, group=64)
    want = okv.Pages(nseq, 16, nseq, 2)
    for new in ([1] * nseq, [16] * nseq, [-1, 3] * (nseq // 2)):
        _same_plan(cache.plan(_i32(new), max_tokens=20000), want.plan(new, 20000))
        _same_tables(cache, want)
    out = cache.plan(torch.empty(0, dtype=torch.int32, device="cuda"), max_tokens=5)
    assert out.token_start.tolist() == [0] and out.slots.tolist() == [-1] * 5
    _same_tables(cache, want)


def test_plan_of_the_first_rows_leaves_the_others():
    import tile_routed_mixed_b200 as tm
    cache = tm.TileMixKV4Cache(20, 16, 1, 64, 6, 3, group=64)
    want = okv.Pages(20, 16, 6, 3)
    _same_plan(cache.plan(_i32([17] * 6), max_tokens=102), want.plan([17] * 6, 102))
    out = cache.new_plan(9, nseq=2)
    buf = torch.full((12,), 77, dtype=torch.int32, device="cuda")
    out = out._replace(slots=buf[1:10])  # slots off the 16-byte grid
    w = want.plan([5, -4], 9)
    _same_plan(cache.plan(_i32([5, -4]), out=out), w)
    assert buf[0] == 77 and buf[10] == 77
    _same_tables(cache, want)


def test_plan_reports_tables_that_contradict_themselves():
    import tile_routed_mixed_b200 as tm
    cache = tm.TileMixKV4Cache(8, 16, 1, 64, 3, 2, group=64)
    for spoil in ("len", "count", "stack", "entry"):
        cache.seq_len.copy_(_i32([16, 0, 0]))
        cache.block_table.copy_(torch.tensor([[7, -1], [-1, -1], [-1, -1]], dtype=torch.int32))
        cache.free_list.copy_(_i32(range(8)))
        cache.free_count.fill_(7)
        new = [1, 1, 1]
        if spoil == "len":
            cache.seq_len[1] = 33
        elif spoil == "count":
            cache.free_count.fill_(9)
        elif spoil == "stack":
            cache.free_list[6] = 8
        else:
            cache.block_table[0, 0] = -5
            new = [-16, 1, 1]
        cache.plan(_i32(new), max_tokens=4)
        assert tm.tilemix_get_error() == tm.ERR_INVALID_ARG, spoil
        assert tm.tilemix_get_error() == tm.OK


# ----------------------------------------------------------------- append ---

def _edge_rows(rng, n, hk, d, group, dtype):
    """Random rows with, among them: zeros, ties, subnormals, the largest values,
    infinities and NaNs in single groups."""
    x = kc.draw(rng, (n, hk, d), dtype, 3.0)
    tiny = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -133
    top = okv.FORMATS[dtype][2]
    x[0] = 0.0
    x[1] = tiny * rng.integers(-12, 13, (hk, d))
    x[2] = tiny * rng.integers(-3, 4, (hk, d))
    # s = 1/4 exactly, and every half step of it: ties
    x[3] = 0.25 * (rng.integers(-7, 7, (hk, d)) + 0.5)
    x[3, :, ::group] = 1.75
    x[4] = np.where(rng.random((hk, d)) < 0.5, top, -top)
    x[5] = okv.round_to(top * rng.uniform(-1, 1, (hk, d)), dtype)
    x[6, 0, 3] = np.inf
    x[6, -1, d - 1] = -np.inf
    x[7, 0, group - 1] = np.nan
    x[8] = okv.round_to(x[8] * (2.0 ** -14 if dtype == "fp16" else 2.0 ** -120), dtype)
    # magnitudes a / 7 apart by single steps: scales next to their midpoints
    x[9] = okv.round_to(1.0 + 2.0 ** -10 * rng.integers(0, 1024, (hk, d)), dtype)
    return x


@pytest.mark.parametrize("dtype,d,group", FORMATS)
def test_append_codes_bit_for_bit(dtype, d, group):
    rng = np.random.default_rng(d + group)
    n, hk, page = 150, 3, 16
    pool = kc.Pool(rng, [page * 14], hk, d, group, page, dtype, spare=1)
    cache = pool.cache()
    k, v = (_edge_rows(rng, n, hk, d, group, dtype) for _ in range(2))
    slots = rng.permutation(pool.num_pages * page)[:n].astype(np.int32)
    slots[[11, 40]] = -1
    cache.append(kc.to_device(k, dtype), kc.to_device(v, dtype), _i32(slots))
    torch.cuda.synchronize()
    for w, x, codes, scale in (("k", k, cache.k_codes, cache.k_scale), ("v", v, cache.v_codes, cache.v_scale)):
        c, s = okv.quantise(x, group, dtype)
        want_c, want_s = okv.pack(pool.codes[w], w), pool.scales[w].copy()
        for t in range(n):
            if slots[t] >= 0:
                want_c[slots[t] // page, :, slots[t] % page] = okv.pack(c[t], w)
                want_s[slots[t] // page, :, slots[t] % page] = s[t]
        assert np.array_equal(codes.cpu().numpy(), want_c), w
        assert kc.same(kc.to_numpy(scale), want_s), w


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_every_quotient_of_a_scale(dtype):
    """Each finite positive value of the type's 2^10 (2^7) significands against
    scales of many significands: the quotients next to and on the half steps."""
    rng = np.random.default_rng(5)
    bits = okv.FORMATS[dtype][0]
    n, d, page = 512, 128, 64
    sig = rng.integers(2 ** (bits - 1), 2 ** bits, (n, 1)) * 2.0 ** -(bits - 1)
    s = okv.round_to(7 * sig, dtype)                      # the group's largest
    k = okv.round_to(s * rng.uniform(-1, 1, (n, d)), dtype)
    half = okv.round_to(okv.round_to(s / 7, dtype) * (rng.integers(-7, 7, (n, d)) + 0.5), dtype)
    k = np.where(rng.random((n, d)) < 0.7, half, k)       # half steps, rounded to the type
    k[:, 0] = s[:, 0]
    k = np.clip(k, -s, s)[:, None, :]
    pool = kc.Pool(rng, [n], 1, d, d, page, dtype, spare=0)
    cache = pool.cache()
    cache.append(kc.to_device(k, dtype), kc.to_device(-k, dtype), _i32(range(n)))
    for w, x, codes in (("k", k, cache.k_codes), ("v", -k, cache.v_codes)):
        c, _ = okv.quantise(x, d, dtype)
        got = okv.unpack(codes.cpu().numpy(), w).reshape(n, 1, d)
        assert np.array_equal(got, c)


def test_append_strided_rows_and_bad_slots():
    """K and V as parts of one wider tensor; slots outside the pool are skipped
    and reported; slots -1 are skipped."""
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(2)
    hk, d, n, page = 2, 64, 9, 32
    pool = kc.Pool(rng, [page], hk, d, 32, page, "bf16", spare=1)
    cache = pool.cache()
    wide = kc.draw(rng, (n, 5 * hk, d), "bf16")
    t = kc.to_device(wide, "bf16")
    slots = [0, 5, -1, 63, 64, -7, 2 ** 31 - 1, 10, 33]
    cache.append(t[:, hk:2 * hk], t[:, 3 * hk:4 * hk], _i32(slots))
    assert tm.tilemix_get_error() == tm.ERR_INVALID_ARG
    cache.append(t[:0, :hk], t[:0, :hk], _i32([]))
    for w, a, codes in (("k", hk, cache.k_codes), ("v", 3 * hk, cache.v_codes)):
        c, _ = okv.quantise(wide[:, a:a + hk], 32, "bf16")
        want = okv.pack(pool.codes[w], w)
        for i, x in enumerate(slots):
            if 0 <= x < 64:
                want[x // page, :, x % page] = okv.pack(c[i], w)
        assert np.array_equal(codes.cpu().numpy(), want)


# ----------------------------------------------------------------- gather ---

@pytest.mark.parametrize("dtype,d,group", FORMATS)
def test_gather(dtype, d, group):
    rng = np.random.default_rng(d + group + 1)
    lengths, page, hk = [0, 1, 70, 16, 33], 32, 2
    pool = kc.Pool(rng, lengths, hk, d, group, page, dtype)
    pool.scales["v"][pool.table[2, 0], 1, 3] = np.nan  # a group that was not finite
    cache = pool.cache()
    starts, rows = [5, 200, 10, 100, 140], 210
    out = [torch.full((rows, hk, d), 9.0, dtype=kc.TORCH[dtype], device="cuda") for _ in range(2)]
    got = cache.gather(_i32(starts), rows, out=out)
    for w, t in zip("kv", got):
        want = np.full((rows, hk, d), 9.0)
        for s, n in enumerate(lengths):
            want[starts[s]:starts[s] + n] = okv.round_to(pool.row(w, s), dtype)
        assert kc.same(kc.to_numpy(t), want)


def test_gather_reports_rows_and_pages_outside():
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(3)
    pool = kc.Pool(rng, [40, 20], 1, 64, 64, 16, "fp16")
    for what in ("rows", "page", "start"):
        cache = pool.cache()
        starts, rows = [0, 40], 60
        if what == "rows":
            rows = 50
        elif what == "start":
            starts = [-3, 40]
        else:
            cache.block_table[0, 1] = pool.num_pages
        k, _ = cache.gather(_i32(starts), rows, out=[torch.zeros((rows, 1, 64), dtype=torch.float16, device="cuda")
                                                    for _ in range(2)])
        assert tm.tilemix_get_error() == tm.ERR_INVALID_ARG, what
        want = np.zeros((rows, 1, 64))
        for s, n in enumerate([40, 20]):
            for p, x in enumerate(okv.round_to(pool.row("k", s), "fp16")):
                if 0 <= starts[s] + p < rows and not (what == "page" and s == 0 and p // 16 == 1):
                    want[starts[s] + p] = x
        assert np.array_equal(kc.to_numpy(k), want), what


# ----------------------------------------------------------------- attend ---

def _attend(pool, queries, hq, seed=0, q_scale=1.0, scale=0.0, max_new=None, cache=None):
    rng = np.random.default_rng(seed)
    start = np.concatenate([[0], np.cumsum(queries)])
    n = int(start[-1])
    q = kc.draw(rng, (n + 2, hq, pool.d), pool.dtype, q_scale)
    cache = cache or pool.cache()
    qd = kc.to_device(q, pool.dtype)
    out = torch.full_like(qd, 7.0)
    lse = torch.full((hq, n + 2), 7.0, dtype=torch.float32, device="cuda")
    cache.attend(qd, max(pool.lengths + [1]), token_start=_i32(start),
                 max_new=max_new or max(max(queries), 1), softmax_scale=scale, out=out, lse=lse)
    o, l = kc.to_numpy(out), kc.to_numpy(lse)
    assert (o[n:] == 7.0).all() and (l[:, n:] == 7.0).all()  # rows behind the last sequence
    worst = kc.check_attend(o, l, q, pool, pool.lengths, start, hq, scale or None)
    for space in cache._spaces.values():
        assert not space[1].any()
    return out, lse, worst


LENGTHS = [1, 0, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 129, 300]


@pytest.mark.parametrize("dtype,d,group", FORMATS)
def test_attend_single_tokens(dtype, d, group):
    rng = np.random.default_rng(1)
    pool = kc.Pool(rng, LENGTHS, 2, d, group, 16, dtype)
    _attend(pool, [1] * len(LENGTHS), 6)


@pytest.mark.parametrize("dtype,d,group", FORMATS)
def test_attend_several_tokens(dtype, d, group):
    """Up to 40 queries, more of them than a column block holds; sequences with
    none; queries before the first key (nothing to attend to)."""
    rng = np.random.default_rng(2)
    lengths = [40, 5, 64, 200, 3, 33, 0, 90]
    pool = kc.Pool(rng, lengths, 2, d, group, 32, dtype)
    _attend(pool, [7, 1, 0, 40, 5, 2, 2, 16], 6)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 512, 1024])
def test_attend_page_sizes(page):
    rng = np.random.default_rng(page)
    pool = kc.Pool(rng, [page - 1, page, page + 1, 3 * page + 7, 1], 1, 128, 64, page, "fp16")
    _attend(pool, [1, 2, 3, 2, 1], 4)


@pytest.mark.parametrize("hq,hk,new", [(1, 1, 1), (8, 1, 1), (9, 1, 1), (16, 1, 1), (17, 1, 3), (5, 5, 1),
                                       (28, 4, 1), (24, 8, 3), (3, 1, 5), (64, 2, 2)])
def test_attend_head_layouts(hq, hk, new):
    rng = np.random.default_rng(hq)
    lengths = [130, 31, 77]
    pool = kc.Pool(rng, lengths, hk, 64, 32, 16, "bf16")
    _attend(pool, [new] * 3, hq)
    _attend(pool, [new] * 3, hq, max_new=1)  # a bound that is too small costs only time


@pytest.mark.parametrize("hk,length,new", [(1, 20000, 1), (2, 9000, 4), (8, 5000, 1)])
def test_attend_long_sequence_over_many_ctas(hk, length, new):
    rng = np.random.default_rng(length)
    pool = kc.Pool(rng, [length], hk, 128, 128, 128, "fp16")
    cache = pool.cache()
    first = _attend(pool, [new], 4 * hk, cache=cache)
    again = _attend(pool, [new], 4 * hk, cache=cache)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_attend_ragged_batch_over_many_ctas():
    rng = np.random.default_rng(9)
    lengths = [int(x) for x in rng.integers(0, 700, 90)]
    pool = kc.Pool(rng, lengths, 2, 64, 64, 64, "bf16")
    _attend(pool, [int(x) for x in rng.integers(0, 4, 90)], 4)


def test_attend_many_short_sequences():
    rng = np.random.default_rng(10)
    pool = kc.Pool(rng, [int(x) for x in rng.integers(0, 20, 700)], 1, 64, 32, 16, "fp16")
    _attend(pool, [1] * 700, 2)


@pytest.mark.parametrize("q_scale", [2.0 ** -12, 30.0])
def test_attend_flat_and_peaked_scores(q_scale):
    """Nearly uniform probabilities, and scores so far apart that most are zero
    and the running maximum moves often."""
    rng = np.random.default_rng(11)
    pool = kc.Pool(rng, [500, 65], 2, 128, 32, 16, "fp16")
    _attend(pool, [2, 1], 4, q_scale=q_scale)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_attend_scales_of_many_magnitudes(dtype):
    """V scales over nine powers of two, growing along the sequence (the output's
    power of two moves), with zero groups and a zero query among them."""
    rng = np.random.default_rng(12)
    pool = kc.Pool(rng, [400], 1, 128, 32, 16, dtype)
    pages = pool.table[0, :25]
    for i, page in enumerate(pages):
        pool.scales["v"][page] *= 2.0 ** (i % 9 - 4)
        pool.scales["k"][page, :, ::5] = 0.0
        pool.scales["v"][page, :, 1::4] = 0.0
    _attend(pool, [3], 2)
    _attend(pool, [1], 2, q_scale=0.0)


def test_attend_softmax_scale_and_one_row_per_sequence():
    rng = np.random.default_rng(13)
    lengths = [77, 0, 40]
    pool = kc.Pool(rng, lengths, 2, 128, 64, 32, "fp16")
    cache = pool.cache()
    q = kc.draw(rng, (3, 4, 128), "fp16")
    o, lse = cache.attend(kc.to_device(q, "fp16"), 77, softmax_scale=0.031, lse=True)
    kc.check_attend(kc.to_numpy(o), kc.to_numpy(lse), q, pool, lengths, [0, 1, 2, 3], 4, 0.031)
    assert not kc.to_numpy(o)[1].any() and np.isneginf(kc.to_numpy(lse)[:, 1]).all()


def test_attend_only_reads_the_rows_it_should():
    """Rows past a sequence's length, other pages and free pages may hold
    anything: NaN scales there change no result."""
    rng = np.random.default_rng(14)
    lengths = [19, 40, 33]
    pool = kc.Pool(rng, lengths, 1, 128, 128, 16, "bf16")
    clean = _attend(pool, [1, 3, 2], 2)
    for w in "kv":
        live = np.zeros(pool.scales[w].shape[:3], dtype=bool)
        for s, n in enumerate(lengths):
            for p in range(n):
                live[pool.table[s, p // 16], :, p % 16] = True
        pool.scales[w][~live] = np.nan
    dirty = _attend(pool, [1, 3, 2], 2)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


def test_attend_a_group_that_is_not_finite():
    """A NaN scale of V reaches its group's channels only; one of K the queries
    that see its key."""
    rng = np.random.default_rng(15)
    pool = kc.Pool(rng, [60], 2, 128, 32, 16, "fp16")
    pool.scales["v"][pool.table[0, 1], 0, 4, 2] = np.nan        # key 20, KV head 0, channels 64 .. 95
    pool.scales["k"][pool.table[0, 3], 1, 10, 0] = np.nan       # key 58, KV head 1
    q = kc.draw(rng, (2, 2, 128), "fp16")
    o = kc.to_numpy(pool.cache().attend(kc.to_device(q, "fp16"), 60, token_start=_i32([0, 2]), max_new=2))
    want = np.zeros((2, 2, 128), dtype=bool)
    want[:, 0, 64:96] = True                                     # both queries see key 20
    want[:, 1] = True                                            # queries 58 and 59 see key 58
    assert np.array_equal(np.isnan(o), want)


def test_attend_pages_outside_the_pool_are_reported():
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(16)
    for page in (-1, 10 ** 6):
        pool = kc.Pool(rng, [50, 64], 1, 64, 64, 16, "fp16")
        cache = pool.cache()
        cache.block_table[1, 2] = page
        q = kc.draw(rng, (2, 2, 64), "fp16")
        o = kc.to_numpy(cache.attend(kc.to_device(q, "fp16"), 64))
        assert tm.tilemix_get_error() == tm.ERR_INVALID_ARG
        kc.check_attend(o, None, q, pool, [50], [0, 1], 2)      # the other sequence is right


# ------------------------------------------------------- used as a server ---

def test_steps_from_prefill_on():
    """A batch prefilled with the routed kernel, its K and V put in the cache, and
    decode steps with growing lengths: plan, append, attend, with a request
    ending and one starting; then a sequence gathered again."""
    import oracle
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(20)
    dtype, hq, hk, d, page, group = "fp16", 6, 2, 128, 16, 64
    lengths = [70, 33, 128]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    masks, _, _ = oracle.build_routing("sptrans", 75, 0, lengths, hk, [1] * 3, True)
    pre = tm.TileMixPrefill(lengths, hq, hk, d, masks, [1] * 3)
    q, k, v = (kc.draw(rng, (int(cu[-1]), h, d), dtype) for h in (hq, hk, hk))
    qd, kd, vd = (kc.to_device(x, dtype) for x in (q, k, v))
    pre(qd, kd, vd)
    cache = tm.TileMixKV4Cache(40, page, hk, d, 4, 12, group=group)
    plan = cache.plan(_i32(lengths + [0]), max_tokens=240)
    assert plan.token_start.tolist() == list(cu) + [int(cu[-1])]
    cache.append(kd, vd, plan.slots[:int(cu[-1])])
    coded = lambda x: okv.values(*okv.quantise(x, group, dtype), group)
    hist = [[coded(x[cu[s]:cu[s + 1]]) for x in (k, v)] for s in range(3)] + [[np.zeros((0, hk, d))] * 2]
    for step, new in enumerate([[1, 1, 1, 0], [3, 0, 1, 20], [-2 ** 31, 2, 17, 1], [5, 1, 1, -3]]):
        n = sum(x for x in new if x > 0)
        plan = cache.plan(_i32(new), max_tokens=n)
        assert plan.granted.tolist() == [1] * 4
        q, k, v = (kc.draw(rng, (n, h, d), dtype) for h in (hq, hk, hk))
        cache.append(kc.to_device(k, dtype), kc.to_device(v, dtype), plan.slots)
        o, lse = cache.attend(kc.to_device(q, dtype), 192, token_start=plan.token_start,
                              max_new=max(new), lse=True)
        at = 0
        for s, m in enumerate(new):
            if m < 0:
                hist[s] = [x[:max(0, len(x) + m)] for x in hist[s]]
            elif m:
                hist[s] = [np.concatenate([x, coded(y[at:at + m])]) for x, y in zip(hist[s], (k, v))]
                at += m
        lens = [len(h[0]) for h in hist]
        assert cache.seq_len.tolist() == lens
        pool = type("P", (), {"dtype": dtype})
        kc.check_attend(kc.to_numpy(o), kc.to_numpy(lse), q, pool, lens, plan.token_start.tolist(), hq,
                        kv=lambda s: hist[s])
    kg, vg = cache.gather(_i32(np.concatenate([[0], np.cumsum(lens)[:-1]])), sum(lens))
    for t, i in ((kg, 0), (vg, 1)):
        assert np.array_equal(kc.to_numpy(t), okv.round_to(np.concatenate([h[i] for h in hist]), dtype))


def test_step_captured_into_a_graph_and_replayed():
    """plan + append + attend captured once and replayed with other inputs, with
    eager calls of the same cache in between."""
    rng = np.random.default_rng(21)
    pool = kc.Pool(rng, [60, 17, 100], 2, 64, 32, 16, "bf16", spare=12, max_pages=10)
    cache = pool.cache()
    n, hq = 3, 4
    new = _i32([1, 1, 1])
    qd, kd, vd = (torch.zeros((n, h, 64), dtype=torch.bfloat16, device="cuda") for h in (hq, 2, 2))
    out, lse = torch.zeros_like(qd), torch.zeros((hq, n), device="cuda")
    plan = cache.new_plan(n)

    def step():
        cache.plan(new, out=plan)
        cache.append(kd, vd, plan.slots)
        cache.attend(qd, 160, token_start=plan.token_start, out=out, lse=lse)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hist = [[pool.row("k", s), pool.row("v", s)] for s in range(3)]
    coded = lambda x: okv.values(*okv.quantise(x, 32, "bf16"), 32)
    for i in range(6):
        q, k, v = (kc.draw(rng, (n, h, 64), "bf16") for h in (hq, 2, 2))
        for t, x in ((qd, q), (kd, k), (vd, v)):
            t.copy_(kc.to_device(x, "bf16"))
        if i == 3:
            step()  # the same call outside the graph
        else:
            graph.replay()
        for s in range(n):
            hist[s] = [np.concatenate([x, coded(y[s:s + 1])]) for x, y in zip(hist[s], (k, v))]
        kc.check_attend(kc.to_numpy(out), kc.to_numpy(lse), q, pool, [len(h[0]) for h in hist],
                        [0, 1, 2, 3], hq, kv=lambda s: hist[s])


def test_two_streams_at_once():
    """Attention of one cache on two streams, many times over: each stream has a
    workspace of its own."""
    rng = np.random.default_rng(22)
    pool = kc.Pool(rng, [3000, 2000], 2, 128, 64, 64, "fp16")
    cache = pool.cache()
    q = [kc.draw(rng, (2, 4, 128), "fp16") for _ in range(2)]
    qd = [kc.to_device(x, "fp16") for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(x) for x in qd]
    torch.cuda.synchronize()
    for _ in range(50):
        for i, s in enumerate(streams):
            cache.attend(qd[i], 3000, out=outs[i], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        kc.check_attend(kc.to_numpy(outs[i]), None, q[i], pool, [3000, 2000], [0, 1, 2], 4)


def test_workspace_size_is_checked():
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(23)
    pool = kc.Pool(rng, [40], 1, 64, 64, 16, "fp16")
    cache = pool.cache()
    q = kc.to_device(kc.draw(rng, (1, 2, 64), "fp16"), "fp16")
    cache.attend(q, 40)
    a = cache._attn
    need = tm.tilemix_kv4_attn_workspace_size(a)
    assert a.workspace_bytes == need
    for change in (dict(workspace_bytes=need - 1), dict(workspace=None), dict(workspace=a.workspace + 16)):
        b = tm.KV4AttnArgs.from_buffer_copy(a)
        for x, y in change.items():
            setattr(b, x, y)
        with pytest.raises(tm.TileMixError) as e:
            tm.tilemix_kv4_attn(b)
        assert e.value.status == tm.ERR_WORKSPACE
    assert ctypes.sizeof(a) > 0


def test_call_site_refusals():
    """Wrong types, shapes, layouts and counts are refused before anything is
    enqueued, and leave the cache usable."""
    import tile_routed_mixed_b200 as tm
    rng = np.random.default_rng(24)
    pool = kc.Pool(rng, [40, 3], 2, 64, 32, 16, "fp16")
    cache = pool.cache()
    h = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")
    bad = [
        lambda: cache.plan(_i32([1, 1, 1]), max_tokens=3),                          # more than max_seqs
        lambda: cache.plan(_i32([1, 1])),                                           # no slots given
        lambda: cache.plan(_i32([1, 1]).long(), max_tokens=2),
        lambda: cache.plan(_i32([1, 1], "cpu"), max_tokens=2),
        lambda: cache.plan(_i32([1, 0, 1, 0])[::2], max_tokens=2),
        lambda: cache.plan(_i32([1, 1]), max_tokens=3, out=cache.new_plan(2)),
        lambda: cache.plan(_i32([1]), out=cache.new_plan(2)),
        lambda: cache.append(h(2, 2, 64), h(2, 2, 64).bfloat16(), _i32([0, 1])),
        lambda: cache.append(h(1, 2, 64), h(2, 2, 64), _i32([0, 1])),               # fewer rows than slots
        lambda: cache.append(h(2, 2, 128)[..., ::2], h(2, 2, 64), _i32([0, 1])),
        lambda: cache.append(h(2, 64, 2).transpose(1, 2), h(2, 2, 64), _i32([0, 1])),
        lambda: cache.append(h(2, 2, 64), h(2, 2, 64), _i32([0, 1]).long()),
        lambda: cache.gather(_i32([0, 0, 0]), 5),
        lambda: cache.gather(_i32([0, 40]), 43, out=(h(43, 2, 64), h(42, 2, 64))),
        lambda: cache.attend(h(2, 3, 64), 40),                                      # 3 heads over 2
        lambda: cache.attend(h(2, 4, 32), 40),
        lambda: cache.attend(h(3, 4, 64), 40),                                      # more rows than sequences
        lambda: cache.attend(h(2, 4, 64).float(), 40),
        lambda: cache.attend(h(2, 4, 64), 40, out=h(2, 4, 64).bfloat16()),
        lambda: cache.attend(h(2, 4, 64), 40, lse=torch.zeros((2, 4), device="cuda")),
        lambda: cache.attend(h(2, 4, 64), 40, token_start=_i32([0, 1, 2, 2])),
        lambda: tm.TileMixKV4Cache(4, 16, 1, 64, 2, 2, group=128),
        lambda: tm.TileMixKV4Cache(4, 16, 1, 64, 2, 2, dtype=torch.float32),
        lambda: tm.TileMixKV4Cache(4, 16, 1, 64, 2, 2, device="cpu"),
        lambda: tm.TileMixKV4Cache(0, 16, 1, 64, 2, 2),
        lambda: tm.TileMixKV4Cache(4, 16, 1, 64, 2, 2, pool=pool.tensors()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("case %d was taken" % i)
    for f in (lambda: cache.attend(h(2, 4, 64), 40, softmax_scale=float("nan")),
              lambda: cache.attend(h(2, 4, 64), 40, max_new=0),
              lambda: cache.attend(h(2, 4, 64), 0)):
        with pytest.raises(tm.TileMixError):
            f()
    _attend(pool, [1, 2], 4, cache=cache)


def test_two_threads_on_one_cache():
    """Two host threads with a stream each, calling one object."""
    import threading
    rng = np.random.default_rng(25)
    pool = kc.Pool(rng, [900, 70], 2, 64, 64, 32, "bf16")
    cache = pool.cache()
    q = [kc.draw(rng, (2, 4 * (i + 1), 64), "bf16") for i in range(2)]
    qd = [kc.to_device(x, "bf16") for x in q]
    outs = [None, None]
    torch.cuda.synchronize()

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(200):
            outs[i] = cache.attend(qd[i], 900, stream=s)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        kc.check_attend(kc.to_numpy(outs[i]), None, q[i], pool, [900, 70], [0, 1, 2], 4 * (i + 1))


def test_bounds_that_are_too_small_cost_only_time():
    rng = np.random.default_rng(26)
    pool = kc.Pool(rng, [700, 300], 2, 64, 32, 16, "fp16")
    cache = pool.cache()
    q = kc.draw(rng, (5, 6, 64), "fp16")
    o = cache.attend(kc.to_device(q, "fp16"), 1, token_start=_i32([0, 3, 5]), max_new=1)
    kc.check_attend(kc.to_numpy(o), None, q, pool, [700, 300], [0, 3, 5], 6)


def test_rows_of_one_page_in_many_sequences():
    """Sequences that share their first pages (a common prefix) read the same rows."""
    rng = np.random.default_rng(27)
    pool = kc.Pool(rng, [64, 50, 33], 1, 128, 64, 16, "bf16")
    pool.table[1, :2] = pool.table[0, :2]
    pool.table[2, :2] = pool.table[0, :2]
    _attend(pool, [1, 1, 2], 2)


def test_plans_of_very_different_sizes_from_two_threads():
    """What one call asks of the kernel does not depend on another's size."""
    import threading
    import tile_routed_mixed_b200 as tm
    sizes = [1, tm.PAGE_PLAN_MAX_SEQS]
    caches = [tm.TileMixKV4Cache(n, 16, 1, 64, n, 1) for n in sizes]
    news = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in sizes]
    outs = [c.new_plan(16) for c in caches]
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5000):
                    caches[i].plan(news[i], out=outs[i])
        except RuntimeError as e:
            failed.append((sizes[i], e))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert tm.tilemix_get_error() == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("d,group,rep", [(128, 32, 1), (128, 64, 2), (128, 128, 5), (64, 32, 5), (64, 64, 1)])
@pytest.mark.parametrize("length", [3, 33, 60, 700])
def test_attend_not_finite_rows_of_later_tokens(dtype, d, group, rep, length):
    """A new token's row that is not finite reaches its own query and later ones,
    not those in front of it."""
    rng = np.random.default_rng(31)
    new = 3
    pool = kc.Pool(rng, [length], 2, d, group, 16, dtype)
    for back, w, head, i in ((1, "v", 0, 0), (2, "v", 1, d // group - 1), (1, "k", 1, 0)):
        pos = length - back
        pool.scales[w][pool.table[0, pos // 16], head, pos % 16, i] = np.nan
    q = kc.draw(rng, (new, 2 * rep, d), dtype)
    o, lse = pool.cache().attend(kc.to_device(q, dtype), length, token_start=_i32([0, new]), max_new=new, lse=True)
    o, lse = kc.to_numpy(o), kc.to_numpy(lse).T
    k, v = pool.row("k", 0), pool.row("v", 0)
    want, wlse, mag, reach = okv.attend(q, k, v, new)
    assert np.array_equal(np.isnan(o), np.isnan(want))
    assert np.array_equal(np.isnan(lse), np.isnan(wlse))
    do, dl = kc.attend_bounds(want, wlse, mag, reach, dtype, np.nanmax(np.abs(v)) / 7, length)
    seen, fin = ~np.isnan(want), ~np.isnan(wlse)
    assert (np.abs(o - want)[seen] <= do[seen]).all()
    assert (np.abs(lse - wlse)[fin] <= dl[fin]).all()
