"""The paged 4-bit cache without a GPU: the oracle's pins and the library's
synchronous argument checks."""
import ctypes

import numpy as np
import pytest

from oracle import kv4 as okv

torch = pytest.importorskip("torch")
from tests import kv4_cases as kc  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tile_routed_mixed_b200 import build
    build.build()


# ---------------------------------------------------------------- oracle ---

def test_round_to_matches_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(4000) * 10.0 ** rng.integers(-9, 6, 4000),
                        rng.integers(-40, 40, 500) * 2.0 ** -25, [0.0, 65504.0, 65519.0, 65520.0, 7e4]])
    for dtype in ("fp16", "bf16"):
        want = torch.from_numpy(x).to(torch.float32).to(kc.TORCH[dtype]).double().numpy()
        got = okv.round_to(x.astype(np.float32).astype(np.float64), dtype)
        assert np.array_equal(got, want)


def test_hand_quantised_group():
    # a = 3.5, s = 0.5: quotients 7, -7, 1, 0.5 (tie to 0), 1.5 (tie to 2), -0.5, -2.5, 0
    x = np.zeros((1, 32))
    x[0, :8] = [3.5, -3.5, 0.5, 0.25, 0.75, -0.25, -1.25, 0.0]
    c, s = okv.quantise(x, 32, "fp16")
    assert s.tolist() == [[0.5]]
    assert c[0, :8].tolist() == [7, -7, 1, 0, 2, 0, -2, 0]
    c, s = okv.quantise(np.zeros((1, 32)), 32, "bf16")
    assert not c.any() and not s.any()
    x[0, 9] = np.inf
    c, s = okv.quantise(x, 32, "fp16")
    assert not c.any() and np.isnan(s).all()


@pytest.mark.parametrize("d", [64, 128])
def test_pack_places(d):
    """The header's places: K's 32-bit words and V's halfwords, low nibble first."""
    rng = np.random.default_rng(d)
    c = rng.integers(-7, 8, (3, d)).astype(np.int8)
    u = (c + 8).astype(np.uint64)
    words = okv.pack(c, "k").view("<u4")
    halves = okv.pack(c, "v").view("<u2")
    for w in range(d // 8):
        want = sum(u[:, 8 * w + i] << np.uint64(4 * i) for i in range(8))
        assert np.array_equal(words[:, (w % 4) * (d // 32) + w // 4], want)
    for h in range(d // 4):
        want = sum(u[:, 4 * h + i] << np.uint64(4 * i) for i in range(4))
        assert np.array_equal(halves[:, (h % 8) * (d // 32) + h // 8], want)
    for w in "kv":
        assert np.array_equal(okv.unpack(okv.pack(c, w), w), c)


def test_hand_plan():
    p = okv.Pages(num_pages=4, page_size=16, max_seqs=3, max_pages=2)  # stack 3 2 1 0, top 0
    assert p.plan([17, 1, 0], 20) == ([0, 17, 18, 18], [*range(0, 16), 16, 32, -1, -1], [1, 1, 1])
    assert p.table[0] == [0, 1] and p.table[1] == [2, -1] and p.free == 1
    # sequence 0 has no third entry, sequence 1 needs none, sequence 2 gets page 3
    assert p.plan([16, 1, 1], 20) == ([0, 16, 17, 18], [-1] * 16 + [33, 48, -1, -1], [0, 1, 1])
    # sequence 0 ends: pages 0 and 1 go back, 0 on top; sequence 2 takes it
    assert p.plan([-99, 0, 16], 16) == ([0, 0, 0, 16], [*range(49, 64), 0], [1, 1, 1])
    assert p.stack[:p.free] == [1]
    # one page left for two that need one: the first gets it
    assert p.plan([1, 30, 0], 40)[2] == [1, 0, 1]


def test_attend_equals_softmax_of_the_whole_matrix():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o, lse, _, _ = okv.attend(q, k, v, 3)
    for i in range(3):
        for h in range(4):
            e = np.exp(k[:7 + i, h // 2] @ q[i, h] / np.sqrt(8))
            assert np.allclose(o[i, h], (e[:, None] * v[:7 + i, h // 2]).sum(0) / e.sum(), rtol=1e-12)
            assert np.isclose(lse[i, h], np.log(e.sum()), rtol=1e-12)
    o, lse, _, _ = okv.attend(q, k[:2], v[:2], 3)  # query 0 sits before the first key
    assert not o[0].any() and np.isneginf(lse[0]).all() and np.isfinite(lse[1:]).all()


def test_a_planted_mistake_is_outside_the_bound():
    """The bound the kernel is held to tells a wrong key, scale or mask apart."""
    rng = np.random.default_rng(2)
    pool = kc.Pool(rng, [100], 1, 64, 32, 16, "fp16")
    k, v = pool.row("k", 0), pool.row("v", 0)
    q = kc.draw(rng, (1, 2, 64), "fp16")
    o, lse, mag, reach = okv.attend(q, k, v, 1)
    do, dl = kc.attend_bounds(o, lse, mag, reach, "fp16", np.abs(v).max() / 7, 100)
    swapped = k.copy()
    swapped[[3, 4]] = swapped[[4, 3]]
    for bad in (okv.attend(q, swapped, v, 1), okv.attend(q, k[:99], v[:99], 1), okv.attend(q, k, v * 1.01, 1)):
        assert (np.abs(bad[0] - o) > do).any()
    assert (np.abs(okv.attend(q, k[:99], v[:99], 1)[1] - lse) > dl).any()


# -------------------------------------------------------------- refusals ---

P = 1 << 20  # an aligned address that is never read


def _cache(tm, **over):
    c = tm.KV4Cache(k_codes=P, k_scale=P, v_codes=P, v_scale=P, num_pages=8, page_size=16, hk=2, d=128,
                    group=32, dtype=0)
    for k, v in over.items():
        setattr(c, k, v)
    return c


CACHE_FAULTS = [(dict(d=96), "UNSUPPORTED"), (dict(d=64, group=128), "UNSUPPORTED"),
                (dict(group=16), "UNSUPPORTED"), (dict(dtype=2), "UNSUPPORTED"),
                (dict(page_size=24), "UNSUPPORTED"), (dict(page_size=8), "UNSUPPORTED"),
                (dict(page_size=2048), "UNSUPPORTED"), (dict(num_pages=0), "INVALID_ARG"),
                (dict(num_pages=1 << 27), "INVALID_ARG"), (dict(hk=0), "INVALID_ARG"),
                (dict(k_codes=None), "INVALID_ARG"), (dict(v_scale=P + 8), "INVALID_ARG")]


def _refuse(tm, fn, args, status):
    with pytest.raises(tm.TileMixError) as e:
        tm._check(fn(ctypes.byref(args), None), "call")
    assert e.value.status == getattr(tm, "ERR_" + status)


@pytest.mark.parametrize("over,status", CACHE_FAULTS + [
    (dict(k=None), "INVALID_ARG"), (dict(v=P + 2), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"),
    (dict(n=-1), "INVALID_ARG"), (dict(n=1 << 27), "INVALID_ARG"), (dict(k_stride=248), "INVALID_ARG"),
    (dict(v_stride=260), "INVALID_ARG")], ids=str)
def test_append_refusals(over, status):
    import tile_routed_mixed_b200 as tm
    over = dict(over)
    keys = [f[0] for f in tm.KV4Cache._fields_]
    c = _cache(tm, **{k: over.pop(k) for k in list(over) if k in keys})
    a = tm.KV4AppendArgs(cache=c, k=P, v=P, k_stride=256, v_stride=256, slots=P, n=4)
    for k, v in over.items():
        setattr(a, k, v)
    _refuse(tm, tm.lib().tilemix_kv4_append, a, status)


@pytest.mark.parametrize("over,status", CACHE_FAULTS + [
    (dict(block_table=None), "INVALID_ARG"), (dict(seq_len=None), "INVALID_ARG"),
    (dict(out_start=None), "INVALID_ARG"), (dict(k=None), "INVALID_ARG"), (dict(v=P + 4), "INVALID_ARG"),
    (dict(nseq=-1), "INVALID_ARG"), (dict(nseq=65536), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"),
    (dict(rows=-1), "INVALID_ARG")], ids=str)
def test_gather_refusals(over, status):
    import tile_routed_mixed_b200 as tm
    over = dict(over)
    keys = [f[0] for f in tm.KV4Cache._fields_]
    c = _cache(tm, **{k: over.pop(k) for k in list(over) if k in keys})
    a = tm.KV4GatherArgs(cache=c, block_table=P, seq_len=P, out_start=P, k=P, v=P, nseq=2, max_pages=4, rows=9)
    for k, v in over.items():
        setattr(a, k, v)
    _refuse(tm, tm.lib().tilemix_kv4_gather, a, status)


@pytest.mark.parametrize("over,status", CACHE_FAULTS + [
    (dict(q=None), "INVALID_ARG"), (dict(o=P + 8), "INVALID_ARG"), (dict(seq_len=None), "INVALID_ARG"),
    (dict(block_table=None), "INVALID_ARG"), (dict(sync=None), "INVALID_ARG"), (dict(hq=5), "INVALID_ARG"),
    (dict(hq=0), "INVALID_ARG"), (dict(nseq=-1), "INVALID_ARG"), (dict(total_q=-1), "INVALID_ARG"),
    (dict(max_new=0), "INVALID_ARG"), (dict(max_seqlen=0), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"),
    (dict(total_q=1, token_start=None), "INVALID_ARG"), (dict(total_q=1 << 30), "INVALID_ARG"),
    (dict(nseq=1 << 20, max_pages=1 << 12), "INVALID_ARG"),
    (dict(softmax_scale=-1.0), "INVALID_ARG"), (dict(softmax_scale=float("nan")), "INVALID_ARG"),
    (dict(softmax_scale=float("inf")), "INVALID_ARG"), (dict(workspace=None), "WORKSPACE"),
    (dict(workspace_bytes=1000), "WORKSPACE"), (dict(workspace=P + 16), "WORKSPACE")], ids=str)
def test_attention_refusals(over, status):
    import tile_routed_mixed_b200 as tm
    over = dict(over)
    keys = [f[0] for f in tm.KV4Cache._fields_]
    c = _cache(tm, **{k: over.pop(k) for k in list(over) if k in keys})
    a = tm.KV4AttnArgs(cache=c, q=P, o=P, token_start=P, seq_len=P, block_table=P, nseq=2, total_q=3, max_new=2,
                       max_seqlen=64, max_pages=4, hq=4, workspace=P, workspace_bytes=1 << 28, sync=P)
    for k, v in over.items():
        setattr(a, k, v)
    _refuse(tm, tm.lib().tilemix_kv4_attn, a, status)


@pytest.mark.parametrize("over,status", [
    (dict(new_len=None), "INVALID_ARG"), (dict(seq_len=None), "INVALID_ARG"),
    (dict(block_table=None), "INVALID_ARG"), (dict(free_list=None), "INVALID_ARG"),
    (dict(free_count=None), "INVALID_ARG"), (dict(token_start=None), "INVALID_ARG"),
    (dict(slots=None), "INVALID_ARG"), (dict(granted=None), "INVALID_ARG"), (dict(nseq=-1), "INVALID_ARG"),
    (dict(nseq=8193), "UNSUPPORTED"), (dict(max_pages=0), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(page_size=48), "UNSUPPORTED"), (dict(max_tokens=-1), "INVALID_ARG"),
    (dict(num_pages=1 << 27), "INVALID_ARG")], ids=str)
def test_plan_refusals(over, status):
    import tile_routed_mixed_b200 as tm
    a = tm.PagePlanArgs(new_len=P, seq_len=P, block_table=P, free_list=P, free_count=P, token_start=P, slots=P,
                        granted=P, nseq=2, max_pages=4, num_pages=8, page_size=16, max_tokens=4)
    for k, v in over.items():
        setattr(a, k, v)
    _refuse(tm, tm.lib().tilemix_page_plan, a, status)


def test_null_arguments_and_empty_calls():
    import tile_routed_mixed_b200 as tm
    L = tm.lib()
    n = ctypes.c_size_t(0)
    for fn in (L.tilemix_page_plan, L.tilemix_kv4_append, L.tilemix_kv4_gather, L.tilemix_kv4_attn):
        assert fn(None, None) == tm.ERR_INVALID_ARG
    assert L.tilemix_kv4_attn_workspace_size(None, ctypes.byref(n)) == tm.ERR_INVALID_ARG
    # nothing to do: nothing is launched, so no pointer is needed
    c = _cache(tm, k_codes=None)
    assert L.tilemix_kv4_append(ctypes.byref(tm.KV4AppendArgs(cache=c)), None) == tm.OK
    assert L.tilemix_kv4_gather(ctypes.byref(tm.KV4GatherArgs(cache=c, max_pages=1)), None) == tm.OK
    a = tm.KV4AttnArgs(cache=c, hq=2, max_new=1, max_seqlen=1, max_pages=1)
    assert L.tilemix_kv4_attn(ctypes.byref(a), None) == tm.OK
    # the workspace does not grow with the batch
    assert L.tilemix_kv4_attn_workspace_size(ctypes.byref(a), ctypes.byref(n)) == tm.OK
    small = n.value
    a.nseq, a.total_q, a.max_seqlen, a.max_pages = 4096, 4096, 1 << 20, 1 << 16
    assert L.tilemix_kv4_attn_workspace_size(ctypes.byref(a), ctypes.byref(n)) == tm.OK
    assert n.value == small
