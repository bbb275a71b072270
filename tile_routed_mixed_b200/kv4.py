"""Paged 4-bit K/V cache: the call site of ``tilemix_page_plan``,
``tilemix_kv4_append``, ``tilemix_kv4_gather`` and ``tilemix_kv4_attn``.

One object holds a pool of pages, the batch's block table, lengths and free
stack (all on the device), and the attention's workspaces.  A step is

    plan = cache.plan(new_len, max_tokens=n)      # pages and slots
    cache.append(k, v, plan.slots)                # rows in, 4 bits
    o = cache.attend(q, max_seqlen, token_start=plan.token_start, max_new=m,
                     granted=plan.granted)

and none of it reads anything back to the host.  A sequence that the plan refuses
(plan.granted 0: no pages, or no room in its row) stays as it was, and its queries
get O = 0 and an LSE of -infinity.
"""
from __future__ import annotations

import ctypes
import threading
from typing import NamedTuple

import torch

from . import (KV_DTYPES, KV4_SYNC_WORDS, KV4AppendArgs, KV4AttnArgs, KV4Cache, KV4GatherArgs,
               PagePlanArgs, _check, lib, tilemix_kv4_attn_workspace_size)


class PagePlan(NamedTuple):
    """Outputs of a plan, int32 on the device: token_start [nseq + 1] (the first
    of each sequence's new tokens), slots [max_tokens], granted [nseq]."""
    token_start: torch.Tensor
    slots: torch.Tensor
    granted: torch.Tensor


# (a torch without CUDA has none of these, and can make no cache)
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the current stream's handle, by device index
_device_now = getattr(torch._C, "_cuda_getDevice", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)
_i32 = torch.int32


def _held(name):
    """A tensor of the object, to be written in place: the calls' argument blocks hold
    its address, so another one cannot take its place."""
    return property(lambda self: self._tensors[name])


def _dtype_id(dtype):
    names = {torch.float16: "fp16", torch.bfloat16: "bf16"}
    if dtype not in names:
        raise ValueError("dtype must be torch.float16 or torch.bfloat16")
    return KV_DTYPES[names[dtype]]


class TileMixKV4Cache:
    """max_seqs sequences with up to max_pages pages each, over num_pages pages
    of page_size tokens; hk KV heads of d channels, one scale per `group`
    channels.  Sequences are rows 0 .. max_seqs - 1 of the tables and start
    empty; the calls take the first nseq of them.

    pool     (k_codes, k_scale, v_codes, v_scale) to use instead of new ones
    tables   (block_table [max_seqs, max_pages], seq_len [max_seqs],
             free_list [num_pages], free_count [1]), int32, likewise

    plan() takes the pages that it frees for the sequence's own.  Rows of block_table
    that name the same pages (a common prefix, full pages that all only read) are
    right for append, gather and attend; such a sequence drops no further than to
    the shared tokens, and at its end its row and its length are cleared in place.

    The tensors (k_codes, k_scale, v_codes, v_scale, block_table, seq_len,
    free_list, free_count) are the object's for good: write them in place.

    The object belongs to one device, whichever is current; `stream` picks the
    stream of a call (default: the current one of that device).  A call with
    `stream` holds the memory of its tensors until that stream is done with them
    (they may be dropped after the call); new tensors that it returns belong to that
    stream, which another has to wait for.  Two calls that
    change the same tables or rows, or read what another writes, must be ordered
    by the caller, as for any tensor.  attend() keeps a workspace per stream, so
    calls on different streams may run at the same time; a call that is being
    captured into a CUDA graph takes one from the graph's own memory."""

    _names = ("k_codes", "k_scale", "v_codes", "v_scale", "block_table", "seq_len", "free_list", "free_count")
    (k_codes, k_scale, v_codes, v_scale, block_table, seq_len, free_list, free_count) = map(_held, _names)

    def __init__(self, num_pages, page_size, hk, d, max_seqs, max_pages, group=32,
                 dtype=torch.float16, device="cuda", pool=None, tables=None):
        L = lib()
        self.num_pages, self.page_size = int(num_pages), int(page_size)
        self.hk, self.d, self.group = int(hk), int(d), int(group)
        self.max_seqs, self.max_pages = int(max_seqs), int(max_pages)
        self.dtype = dtype
        dt = _dtype_id(dtype)
        self.device = torch.device(device)
        if self.device.type != "cuda":
            raise ValueError("the cache lives on a CUDA device")
        if self.d not in (64, 128) or self.group not in (32, 64, 128) or self.group > self.d:
            raise ValueError("d is 64 or 128, group 32, 64 or 128 and at most d")
        if min(self.num_pages, self.page_size, self.hk, self.max_seqs, self.max_pages) < 1:
            raise ValueError("sizes start at 1")
        if self.page_size not in (16, 32, 64, 128, 256, 512, 1024):
            raise ValueError("page_size is a power of two, 16 to 1024")
        if self.num_pages * self.page_size >= 1 << 31 or self.max_seqs * self.max_pages >= 1 << 31 or \
                self.hk > 32767:
            raise ValueError("num_pages * page_size and max_seqs * max_pages stay below 2^31, hk below 2^15")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        dev = self.device
        rows = (self.num_pages, self.hk, self.page_size)
        shapes = [(rows + (self.d // 2,), torch.uint8), (rows + (self.d // self.group,), dtype)] * 2
        if pool is None:
            pool = [torch.zeros(s, dtype=t, device=dev) for s, t in shapes]
        for x, (s, t) in zip(pool, shapes, strict=True):
            self._expect(x, t, s, "pool")
        shapes = [((self.max_seqs, self.max_pages), _i32), ((self.max_seqs,), _i32),
                  ((self.num_pages,), _i32), ((1,), _i32)]
        if tables is None:
            tables = (torch.full(shapes[0][0], -1, dtype=_i32, device=dev),
                      torch.zeros(self.max_seqs, dtype=_i32, device=dev),
                      torch.arange(self.num_pages - 1, -1, -1, dtype=_i32, device=dev),
                      torch.full((1,), self.num_pages, dtype=_i32, device=dev))
        for x, (s, t) in zip(tables, shapes, strict=True):
            self._expect(x, t, s, "tables")
        self._tensors = dict(zip(self._names, (*pool, *tables)))
        c = KV4Cache()
        c.k_codes, c.k_scale = self.k_codes.data_ptr(), self.k_scale.data_ptr()
        c.v_codes, c.v_scale = self.v_codes.data_ptr(), self.v_scale.data_ptr()
        c.num_pages, c.page_size, c.hk, c.d = self.num_pages, self.page_size, self.hk, self.d
        c.group, c.dtype = self.group, dt
        self._plan = PagePlanArgs()
        self._plan.seq_len, self._plan.block_table = self.seq_len.data_ptr(), self.block_table.data_ptr()
        self._plan.free_list, self._plan.free_count = self.free_list.data_ptr(), self.free_count.data_ptr()
        self._plan.max_pages, self._plan.num_pages = self.max_pages, self.num_pages
        self._plan.page_size = self.page_size
        self._append = KV4AppendArgs(cache=c)
        self._gather = KV4GatherArgs(cache=c, max_pages=self.max_pages)
        self._gather.block_table, self._gather.seq_len = self.block_table.data_ptr(), self.seq_len.data_ptr()
        self._attn = KV4AttnArgs(cache=c, max_pages=self.max_pages)
        self._attn.block_table, self._attn.seq_len = self.block_table.data_ptr(), self.seq_len.data_ptr()
        # a step's calls are a few microseconds of host time each: the argument
        # blocks and the functions are kept
        self._calls = {
            "tilemix_page_plan": (L.tilemix_page_plan, ctypes.byref(self._plan)),
            "tilemix_kv4_append": (L.tilemix_kv4_append, ctypes.byref(self._append)),
            "tilemix_kv4_gather": (L.tilemix_kv4_gather, ctypes.byref(self._gather)),
            "tilemix_kv4_attn": (L.tilemix_kv4_attn, ctypes.byref(self._attn)),
        }
        self._lock = threading.Lock()  # on the blocks: a call fills one and enqueues it
        self._spaces = {}
        self._held_on = set()  # streams, by handle, that _tensors are recorded on
        self._f32 = torch.empty(0, dtype=torch.float32, device=dev)

    # ---------------------------------------------------------------- checks

    def _refuse(self, what, x, dtype, shape):
        raise ValueError("%s: expected a contiguous %s tensor of shape %s on %s, got %s %s on %s"
                         % (what, dtype, tuple(shape), self.device, x.dtype, tuple(x.shape), x.device))

    def _expect(self, x, dtype, shape, what):
        """x is a contiguous tensor of this device, of that type and shape."""
        if not (x.dtype is dtype and x.get_device() == self._index and x.shape == shape
                and x.is_contiguous()):
            self._refuse(what, x, dtype, shape)

    def _vector(self, x, what, extra=0):
        """Entries of an int32 vector with one for each sequence (and `extra`)."""
        shape = x.shape
        if not (x.dtype is _i32 and x.get_device() == self._index and len(shape) == 1
                and x.is_contiguous()):
            self._refuse(what, x, _i32, ("nseq",))
        n = shape[0] - extra
        if not 0 <= n <= self.max_seqs:
            raise ValueError("%s: the cache holds %d sequences" % (what, self.max_seqs))
        return n

    def _elsewhere(self, stream, fn, *args):
        """fn(*args) with this object's device, and `stream`, current."""
        if stream is None:
            with torch.cuda.device(self._index):
                return fn(*args)
        if stream.device != self.device:
            raise ValueError("the stream belongs to %s, the cache to %s" % (stream.device, self.device))
        self._hold(stream, args)
        if stream.cuda_stream not in self._held_on:  # (for as long as they live)
            self._hold(stream, self._tensors.values())
            self._held_on.add(stream.cuda_stream)
        with torch.cuda.stream(stream):
            return fn(*args)

    def _hold(self, stream, args):
        """Tensors among args, dropped by the caller after the call, are not handed out
        again before `stream` is done with them."""
        for x in args:
            if isinstance(x, (tuple, list)):
                self._hold(stream, x)
            elif getattr(x, "is_cuda", False):
                x.record_stream(stream)

    def _call(self, name):
        fn, args = self._calls[name]
        rc = fn(args, _stream_of(self._index))
        if rc:
            _check(rc, name)

    # ----------------------------------------------------------------- calls

    def new_plan(self, max_tokens, nseq=None):
        """Buffers of a plan, for plan(out=...)."""
        n = self.max_seqs if nseq is None else int(nseq)
        new = lambda m: torch.empty(m, dtype=_i32, device=self.device)
        return PagePlan(new(n + 1), new(int(max_tokens)), new(n))

    def plan(self, new_len, max_tokens=None, out=None, stream=None):
        """Pages and slots for new_len[s] more tokens (fewer, if negative) of each
        sequence (see tilemix_page_plan).  new_len: int32 [nseq] on the device;
        max_tokens: the number of slots, or `out` from new_plan()."""
        if stream is not None or _device_now() != self._index:
            return self._elsewhere(stream, self.plan, new_len, max_tokens, out)
        n = self._vector(new_len, "new_len")
        if out is None:
            if max_tokens is None:
                raise ValueError("max_tokens or out")
            out = self.new_plan(max_tokens, n)
        token_start, slots, granted = out
        tokens = slots.shape[0]
        self._expect(token_start, _i32, (n + 1,), "token_start")
        self._expect(slots, _i32, (tokens,), "slots")
        self._expect(granted, _i32, (n,), "granted")
        if max_tokens is not None and max_tokens != tokens:
            raise ValueError("max_tokens is %d, out has %d slots" % (max_tokens, tokens))
        a = self._plan
        with self._lock:
            a.token_start = token_start.data_ptr()
            # (an empty tensor has no address)
            a.new_len = new_len.data_ptr() if n else a.token_start
            a.granted = granted.data_ptr() if n else a.token_start
            a.slots = slots.data_ptr()
            a.nseq, a.max_tokens = n, tokens
            self._call("tilemix_page_plan")
        return out

    def append(self, k, v, slots, stream=None):
        """Rows of k and v [n, hk, d] (the heads of a token contiguous, tokens at
        any stride) to slots [n] (int32; -1: skipped)."""
        if stream is not None or _device_now() != self._index:
            return self._elsewhere(stream, self.append, k, v, slots)
        n = slots.shape[0]
        self._expect(slots, _i32, (n,), "slots")
        k_stride, v_stride = self._rows(k, n, "k"), self._rows(v, n, "v")
        if n == 0:
            return
        a = self._append
        with self._lock:
            a.k, a.v, a.slots, a.n = k.data_ptr(), v.data_ptr(), slots.data_ptr(), n
            a.k_stride, a.v_stride = k_stride, v_stride
            self._call("tilemix_kv4_append")

    def _rows(self, x, n, what):
        """The stride of x's tokens."""
        shape = x.shape
        if not (x.dtype is self.dtype and x.get_device() == self._index and len(shape) == 3
                and shape[0] >= n and shape[1] == self.hk and shape[2] == self.d):
            self._refuse(what, x, self.dtype, ("%d or more" % n, self.hk, self.d))
        token, head, channel = x.stride()
        if channel != 1 or (self.hk > 1 and head != self.d):
            raise ValueError("%s: a token's heads must be contiguous" % what)
        return token if shape[0] > 1 else self.hk * self.d

    def gather(self, out_start, rows, out=None, stream=None):
        """K and V of the sequences' tokens as 16-bit values: position p of
        sequence s at row out_start[s] + p (int32 [nseq]) of two [rows, hk, d]
        tensors (`out`, or new ones, whose other rows hold nothing meaningful)."""
        if stream is not None or _device_now() != self._index:
            return self._elsewhere(stream, self.gather, out_start, rows, out)
        n = self._vector(out_start, "out_start")
        rows = int(rows)
        if out is None:
            new = self.k_scale.new_empty
            out = new(rows, self.hk, self.d), new(rows, self.hk, self.d)
        else:
            for x in out:
                self._expect(x, self.dtype, (rows, self.hk, self.d), "out")
        a = self._gather
        with self._lock:
            a.out_start, a.nseq, a.rows = out_start.data_ptr(), n, rows
            a.k, a.v = out[0].data_ptr(), out[1].data_ptr()
            self._call("tilemix_kv4_gather")
        return tuple(out)

    def attend(self, q, max_seqlen, token_start=None, max_new=1, softmax_scale=0.0, out=None,
               lse=False, stream=None, granted=None):
        """Attention of the newest tokens over the cache (see tilemix_kv4_attn).
        q [rows, hq, d]: sequence s's queries are rows token_start[s] ..
        token_start[s + 1] - 1 (int32 [nseq + 1]), or row s if token_start is
        None.  max_seqlen and max_new bound the lengths and the queries per
        sequence.  granted: the plan's (int32 [nseq]); a step whose plan may refuse
        tokens has to pass it, as a refused sequence's queries stand for tokens that
        are not in the cache.  Returns o like q, or (o, LSE [hq, rows]) if lse; `out` and a
        tensor as `lse` are written in place.  Rows that no sequence covers are
        not written (in a new tensor they hold nothing meaningful)."""
        if stream is not None or _device_now() != self._index:
            return self._elsewhere(stream, self.attend, q, max_seqlen, token_start, max_new,
                                   softmax_scale, out, lse, None, granted)
        shape = q.shape
        if not (q.dtype is self.dtype and q.get_device() == self._index and len(shape) == 3
                and shape[2] == self.d and q.is_contiguous()):
            self._refuse("q", q, self.dtype, ("rows", "hq", self.d))
        rows, hq, _ = shape
        if hq < 1 or hq % self.hk != 0:
            raise ValueError("q has %d heads, the cache %d" % (hq, self.hk))
        if token_start is None:
            n, start = rows, None
            if n > self.max_seqs:
                raise ValueError("q: the cache holds %d sequences" % self.max_seqs)
        else:
            n, start = self._vector(token_start, "token_start", 1), token_start.data_ptr()
        if granted is not None:
            self._expect(granted, _i32, (n,), "granted")
        if out is None:
            out = torch.empty_like(q)
        else:
            self._expect(out, self.dtype, shape, "out")
        if lse is True:
            lse = self._f32.new_empty(hq, rows)
        elif lse is not None and lse is not False:
            self._expect(lse, torch.float32, (hq, rows), "lse")
        else:
            lse = None
        a = self._attn
        with self._lock:
            a.q, a.o, a.token_start = q.data_ptr(), out.data_ptr(), start
            a.lse = None if lse is None else lse.data_ptr()
            a.granted = None if granted is None else granted.data_ptr()
            a.nseq, a.total_q, a.hq = n, rows, hq
            a.max_new, a.max_seqlen, a.softmax_scale = max_new, max_seqlen, softmax_scale
            if rows and n:
                # (held until the call is enqueued: a graph's own lives in its pool from then on)
                space = self._space(a, max_new * hq > 8 * self.hk)
                a.workspace, a.workspace_bytes, a.sync = space[2:]
            self._call("tilemix_kv4_attn")
        return out if lse is None else (out, lse)

    def _space(self, a, wide):
        """Workspace and sync words of the current stream, their addresses and size."""
        key = _stream_of(self._index), wide
        space = self._spaces.get(key)
        if space is not None and not _capturing():
            return space
        # a graph being captured gets one of its own: its replays must not share
        # one with calls outside it
        work = torch.empty(tilemix_kv4_attn_workspace_size(a), dtype=torch.uint8, device=self.device)
        sync = torch.zeros(KV4_SYNC_WORDS, dtype=_i32, device=self.device)
        space = (work, sync, work.data_ptr(), work.shape[0], sync.data_ptr())
        if not _capturing():
            self._spaces[key] = space
        return space
