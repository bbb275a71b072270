"""The paged 4-bit cache's call site without a GPU: what it refuses and what it
keeps, on objects that are not constructed (a cache needs a device)."""
import pytest

torch = pytest.importorskip("torch")

NAMES = ["k_codes", "k_scale", "v_codes", "v_scale", "block_table", "seq_len", "free_list", "free_count"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from tile_routed_mixed_b200 import build
    build.build()


def _bare(**fields):
    """A cache without its device side."""
    import tile_routed_mixed_b200 as tm
    c = object.__new__(tm.TileMixKV4Cache)
    c.__dict__.update(fields)
    return c


@pytest.mark.parametrize("name", NAMES)
def test_the_tensors_cannot_be_rebound(name):
    """The kernels read and write at the addresses taken when the object was made: a
    tensor put in the place of one would never be read, and the old one's memory,
    freed, would be written."""
    x = torch.zeros(3)
    c = _bare(_tensors={name: x})
    with pytest.raises(AttributeError):
        setattr(c, name, torch.ones(3))
    assert getattr(c, name) is x


class _Tensor:
    """Stands for a tensor on a device: notes the streams that hold its memory."""
    is_cuda = True

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


class _Stream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device = handle, device


def test_a_call_on_another_stream_holds_its_tensors(monkeypatch):
    """A tensor that the caller drops right after a call on another stream must not
    be handed out again while that stream still reads it; the same for the
    cache's own when the cache goes."""
    import contextlib

    import tile_routed_mixed_b200.kv4 as kv4
    entered = []

    @contextlib.contextmanager
    def on(stream):
        entered.append(stream)
        yield

    monkeypatch.setattr(kv4.torch.cuda, "stream", on)
    own, dev = [_Tensor() for _ in NAMES], torch.device("cuda", 0)
    c = _bare(_tensors=dict(zip(NAMES, own)), _held_on=set(), device=dev, _index=0)
    q, plan, host = _Tensor(), kv4.PagePlan(_Tensor(), _Tensor(), _Tensor()), torch.zeros(2)
    streams = [_Stream(11, dev), _Stream(12, dev)]
    for s in (streams[0], streams[1], streams[0]):
        assert c._elsewhere(s, lambda *a: a, q, None, 7, plan, host, True) == (q, None, 7, plan, host, True)
    assert entered == [streams[0], streams[1], streams[0]]
    for x in (q, *plan):
        assert x.streams == [streams[0], streams[1], streams[0]]
    for x in own:
        assert x.streams == streams
    with pytest.raises(ValueError):
        c._elsewhere(_Stream(13, torch.device("cuda", 1)), lambda *a: a, q)
    assert len(q.streams) == 3


@pytest.mark.parametrize("over", [
    dict(page_size=24), dict(page_size=8), dict(page_size=2048), dict(page_size=0), dict(num_pages=1 << 27),
    dict(num_pages=0), dict(hk=0), dict(hk=1 << 15), dict(max_seqs=1 << 20, max_pages=1 << 12), dict(max_pages=0),
    dict(d=96), dict(group=16), dict(d=64, group=128), dict(dtype=torch.float32)], ids=str)
def test_the_constructor_refuses_what_the_calls_would(over):
    """Before anything is allocated."""
    import tile_routed_mixed_b200 as tm
    args = dict(num_pages=8, page_size=16, hk=2, d=128, max_seqs=2, max_pages=4, group=32, dtype=torch.float16)
    args.update(over)
    with pytest.raises(ValueError):
        tm.TileMixKV4Cache(**args)


# ------------------------------------------- outputs that share memory ---

BASE = 1 << 30  # addresses that are never read


def _refused(fn, args):
    import ctypes

    import tile_routed_mixed_b200 as tm
    assert fn(ctypes.byref(args), None) == tm.ERR_INVALID_ARG


def test_attention_refuses_outputs_over_its_inputs():
    """Every warp of a unit reads its rows of q, at its own time, and the first that
    is done writes its rows of o: in place, or with o over part of q, later
    readers would get outputs for queries."""
    import tile_routed_mixed_b200 as tm
    c = tm.KV4Cache(k_codes=BASE, k_scale=BASE, v_codes=BASE, v_scale=BASE, num_pages=8, page_size=16, hk=2, d=128,
                    group=32, dtype=0)
    size = 5 * 4 * 128 * 2  # bytes of q
    for o, lse in ((0, None), (size - 16, None), (-size + 16, None), (size, 0), (size, size), (size, -4), (size, 2 * size - 4)):
        a = tm.KV4AttnArgs(cache=c, q=BASE, o=BASE + o, token_start=BASE, seq_len=BASE, block_table=BASE, nseq=2,
                           total_q=5, max_new=3, max_seqlen=64, max_pages=4, hq=4, workspace=BASE,
                           workspace_bytes=1 << 28, sync=BASE, lse=None if lse is None else BASE + lse)
        _refused(tm.lib().tilemix_kv4_attn, a)


def test_gather_refuses_k_and_v_in_one_place():
    import tile_routed_mixed_b200 as tm
    c = tm.KV4Cache(k_codes=BASE, k_scale=BASE, v_codes=BASE, v_scale=BASE, num_pages=8, page_size=16, hk=2, d=128,
                    group=32, dtype=0)
    size = 9 * 2 * 128 * 2
    for v in (0, size - 16, 16 - size):
        _refused(tm.lib().tilemix_kv4_gather,
                 tm.KV4GatherArgs(cache=c, block_table=BASE, seq_len=BASE, out_start=BASE, k=BASE, v=BASE + v, nseq=2,
                                  max_pages=4, rows=9))


def test_plan_refuses_arrays_that_share_memory():
    """Some CTAs still read new_len when another writes granted, and so on."""
    import itertools

    import tile_routed_mixed_b200 as tm
    names = ["token_start", "slots", "granted", "new_len", "seq_len", "block_table", "free_list", "free_count"]
    words = dict(token_start=4, slots=4, granted=3, new_len=3, seq_len=3, block_table=12, free_list=8, free_count=1)
    apart = {n: BASE + 256 * i for i, n in enumerate(names)}
    for x, y in itertools.combinations(names, 2):
        for at in (0, words[x] * 4 - 4, 4 - words[y] * 4):
            a = tm.PagePlanArgs(nseq=3, max_pages=4, num_pages=8, page_size=16, max_tokens=4, **apart)
            setattr(a, y, apart[x] + at)
            _refused(tm.lib().tilemix_page_plan, a)


def test_the_package_imports_with_a_torch_that_has_no_cuda():
    """The host-side entry points (routing, tile offsets, status strings) need none."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = ("import torch\n"
            "for x in ('_cuda_getCurrentRawStream', '_cuda_getDevice', '_cuda_isCurrentStreamCapturing'):\n"
            "    delattr(torch._C, x)\n"
            "import tile_routed_mixed_b200 as tm\n"
            "print(tm.tilemix_tile_offsets([0, 100, 300])[0][-1], tm.TileMixKV4Cache.__name__)\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == ["3", "TileMixKV4Cache"]
