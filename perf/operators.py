"""Cases of the paged 4-bit K/V cache: its page plan, append, gather and attention.

Each operator is here twice: as the library's call (``own``) and in its plain
form, elementary torch operations in 32 bits.  ``exact`` restates the results
from the definitions in 64 bits, sequence by sequence.

The cache.  A pool of ``num_pages`` pages of ``page`` tokens holds, per page,
KV head and token, a row of d 4-bit codes for K and one for V, with one scale
per ``group`` channels in the activations' type:
  k_codes, v_codes  uint8 [num_pages][hk][page][d / 2]
  k_scale, v_scale  fp16 or bf16 [num_pages][hk][page][d / group]
a = max |x| of a group, s = a / 7 rounded to the scale's type, code =
clamp(rne(x / s), -7, 7), held as code + 8; the value held is code * s.  Within
a row the 32-bit words of K (8 channels, low nibble first) and the 16-bit
halfwords of V (4 channels) are stored in a fixed order: K word w at place
(w mod 4) * (d / 32) + w / 4, V halfword h at place (h mod 8) * (d / 32) + h / 8.
Sequence s keeps its tokens in the pages block_table[s][0], [1], ...
"""
import math
import random

import torch

own = False

HEADS = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ---

def listed():
    """The 3B shape (24 query / 8 KV heads of 128), the 28/4, 4/1 and 32/8 head
    layouts and the lengths 4096, 16384 and 65536 are this repository's own
    workloads; page sizes and groups are the ones the cache is built for."""
    return [
        # a decode step of a busy server: one new token for each of 256 requests
        dict(name="plan_decode", kind="plan", nseq=256, page=16, len=4096, new=1, ragged=True, lens=1),
        # admission of 64 prompts of up to 4096 tokens beside what is running
        dict(name="plan_prompts", kind="plan", nseq=64, page=64, len=4096, new=4096, ragged=True, lens=2),
        # the rows of one decode step of eight sequences, and those sequences read back
        dict(name="append_step", kind="append", dtype="fp16", d=128, group=64, hq=24, hk=8, page=16, nseq=8,
             len=100, new=1, ragged=True, lens=3),
        # a prefilled batch (8 x 4096 tokens) written to the cache and read back
        dict(name="append_prefill", kind="append", dtype="bf16", d=128, group=32, hq=24, hk=8, page=64, nseq=8,
             len=4096, new=4096, ragged=False, lens=4),
        # one sequence handed to a path that wants 16-bit K and V
        dict(name="gather_one", kind="gather", dtype="bf16", d=64, group=32, hq=4, hk=1, page=32, nseq=1,
             len=1000, new=1, ragged=False, lens=5),
        # a ragged batch of the 28/4 layout handed over, 1024 to 16384 tokens each
        dict(name="gather_batch", kind="gather", dtype="fp16", d=128, group=128, hq=28, hk=4, page=128, nseq=12,
             len=16384, new=1, ragged=True, lens=7),
        # the smallest call: one short sequence, where latency counts
        dict(name="attend_one", kind="attend", dtype="fp16", d=128, group=32, hq=24, hk=8, page=16, nseq=1,
             len=777, new=1, ragged=False, lens=8),
        # a decode step of the 3B shape at 8 x 4096
        dict(name="attend_b8", kind="attend", dtype="fp16", d=128, group=64, hq=24, hk=8, page=64, nseq=8,
             len=4096, new=1, ragged=False, lens=9),
        # five draft tokens of each of 12 ragged sequences verified at once
        dict(name="attend_draft", kind="attend", dtype="bf16", d=128, group=32, hq=28, hk=4, page=32, nseq=12,
             len=16384, new=5, ragged=True, lens=10),
        # one long context
        dict(name="attend_long", kind="attend", dtype="bf16", d=128, group=128, hq=32, hk=8, page=128, nseq=1,
             len=65536, new=1, ragged=False, lens=11),
        # the largest: 64 ragged sequences of up to 32768 tokens
        dict(name="attend_large", kind="attend", dtype="fp16", d=128, group=32, hq=32, hk=8, page=64, nseq=64,
             len=32768, new=1, ragged=True, lens=12),
        # a whole step, as a server runs it: pages and slots for three draft tokens each, their rows
        # written, their attention, and the drafts dropped again
        dict(name="step_b16", kind="step", dtype="bf16", d=128, group=32, hq=24, hk=8, page=16, nseq=16,
             len=4096, new=3, ragged=True, lens=13),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "append", "gather", "attend", "attend", "attend", "step"])
    c = dict(kind=kind, page=rng.choice([16, 32, 64, 128, 256]), ragged=rng.random() < 0.7,
             lens=rng.randrange(1 << 20))
    if kind == "plan":
        c.update(nseq=_log(rng, 1, 1024), len=_log(rng, 1, 8192), new=_log(rng, 1, 1024))
        return c
    d = rng.choice([64, 128, 128])
    group = rng.choice([g for g in (32, 64, 128) if g <= d])
    heads = rng.choice([(24, 8), (28, 4), (32, 8), (4, 1), (8, 8), (16, 1), (6, 2)])
    c.update(dtype=rng.choice(["fp16", "bf16"]), d=d, group=group, hq=heads[0], hk=heads[1])
    if kind == "append":
        c.update(nseq=_log(rng, 1, 64), new=_log(rng, 1, 1024))
        c["len"] = c["new"] + rng.randrange(0, 512)
        return c
    new = 1 if kind == "gather" or rng.random() < 0.6 else rng.randrange(2, 17)
    top = 1 << 20  # tokens of the padded batch
    nseq = _log(rng, 1, 128)
    c.update(nseq=nseq, len=max(new, _log(rng, 1, min(65536, top // nseq))), new=new)
    return c


def _lengths(case):
    """(tokens in the cache, new tokens) of each sequence.  A ragged batch has
    lengths from a sixteenth of the longest up, and a few idle sequences."""
    rng = random.Random(case["lens"])
    n, top, new = case["nseq"], case["len"], case["new"]
    if not case["ragged"]:
        return [top] * n, [new] * n
    lens, news = [], []
    for s in range(n):
        m = rng.randint(max(1, new // 16), new) if s % 7 != 3 else 0
        if case["kind"] == "attend" and case["new"] == 1:
            m = 1
        lens.append(max(m, rng.randint(max(1, top // 16), top)))
        news.append(m)
    lens[0], news[0] = top, new
    return lens, news


def _grows(case):
    return case["kind"] in ("plan", "step")


def work(case):
    lens, news = _lengths(case)
    kind, page = case["kind"], case["page"]
    tokens, new = sum(lens), sum(news)
    if kind == "plan":
        # lengths, new lengths, offsets and grants of both calls, the slots, and each page that comes
        # and goes: its place in the stack read and written, its table entry written twice
        pages = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, news))
        return {"bytes": 2 * 4 * 5 * len(lens) + 4 * new + 16 * pages, "flops": 0}
    d, hk, hq = case["d"], case["hk"], case["hq"]
    cached = 2 * hk * (d // 2 + 2 * (d // case["group"]))  # bytes of one token's codes and scales
    plain = 2 * hk * d * 2                                 # ... of its 16-bit K and V
    if kind == "gather":
        return {"bytes": tokens * (cached + plain), "flops": 2 * tokens * hk * d}
    if kind == "append":
        return {"bytes": new * (plain + cached) + (tokens - new) * cached + tokens * plain,
                "flops": 2 * (2 * new + tokens) * hk * d}
    if kind == "step":
        lens = [a + b for a, b in zip(lens, news)]
        tokens = sum(lens)
    pairs = sum(m * a - m * (m - 1) // 2 for a, m in zip(lens, news))
    more = new * plain + new * cached if kind == "step" else 0
    live = sum(a for a, m in zip(lens, news) if m > 0)
    return {"bytes": live * cached + 2 * new * hq * d * 2 + 4 * sum(-(-a // page) for a in lens) + more,
            "flops": 4 * pairs * hq * d}


# ----------------------------------------------------------------- inputs ---

def _pack(k_codes, v_codes):
    """Offset codes (uint8 0..15, [..., d]) of K and V in the pool's order."""
    lead, d = list(k_codes.shape[:-1]), k_codes.shape[-1]
    t = d // 32
    pair = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)
    k = pair(k_codes).view(lead + [t, 4, 4]).transpose(-3, -2).reshape(lead + [d // 2])
    v = pair(v_codes).view(lead + [t, 8, 2]).transpose(-3, -2).reshape(lead + [d // 2])
    return k.contiguous(), v.contiguous()


def _quantise(x, group):
    """(offset codes uint8 [..., d], scales [..., d / group]) of x [..., d]."""
    y = x.float().unflatten(-1, (x.shape[-1] // group, group))
    s = (y.abs().amax(-1) / 7).to(x.dtype)
    q = torch.where(s.float()[..., None] > 0, y / s.float()[..., None], 0.0)
    return (q.round().clamp(-7, 7) + 8).to(torch.uint8).flatten(-2), s


def _activations(shape, gen, dtype, boost=None):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if boost is not None:
        x = x * boost
    return x.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    lens, news = _lengths(case)
    page, nseq = case["page"], case["nseq"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    grown = [a + b for a, b in zip(lens, news)] if _grows(case) else lens
    used = [-(-a // page) for a in lens]
    most = sum(-(-a // page) for a in grown)
    num_pages = most + 3
    max_pages = max(1, max(-(-a // page) for a in grown))
    order = torch.randperm(num_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((nseq, max_pages), -1, dtype=torch.int32, device="cuda")
    count = ints(used)
    start = torch.cumsum(count, 0) - count
    col = torch.arange(max_pages, device="cuda")
    inside = col[None, :] < count[:, None]
    table[inside] = order[(start[:, None] + col[None, :])[inside].long()]
    free = num_pages - sum(used)
    free_list = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    free_list[:free] = order[sum(used):]
    st = dict(case, num_pages=num_pages, max_pages=max_pages, block_table=table, free_list=free_list,
              free_count=ints([free]), seq_len=ints(lens), new_len=ints(news), drop_len=ints([-m for m in news]),
              max_tokens=sum(news), max_new=max(news), max_seqlen=max(grown))
    st["token_start"] = ints([0] + torch.tensor(news).cumsum(0).tolist())
    if case["kind"] == "plan":
        # the tables alone: the pages' contents take no part
        st.update(hk=1, d=64, group=64, dtype="fp16")
    dtype, d, hk, group = HEADS[st["dtype"]], st["d"], st["hk"], st["group"]
    pool_pages = 1 if case["kind"] == "plan" else num_pages
    codes = [torch.empty((pool_pages, hk, page, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty((pool_pages, hk, page, d // group), dtype=dtype, device="cuda") for _ in range(2)]
    # K has a few strong channels in every head, as keys have
    boost = torch.ones((hk, 1, d), device="cuda")
    boost.view(-1)[torch.randint(0, hk * d, (4 * hk,), generator=gen, device="cuda")] = 6.0
    step = max(1, (1 << 26) // (hk * page * d))
    for a in range(0, pool_pages, step):
        b = min(pool_pages, a + step)
        k, ks = _quantise(_activations((b - a, hk, page, d), gen, dtype, boost), group)
        v, vs = _quantise(_activations((b - a, hk, page, d), gen, dtype), group)
        codes[0][a:b], codes[1][a:b] = _pack(k, v)
        scales[0][a:b], scales[1][a:b] = ks, vs
    st.update(k_codes=codes[0], v_codes=codes[1], k_scale=scales[0], v_scale=scales[1])
    n = st["max_tokens"]
    if case["kind"] in ("append", "step"):
        rows = boost.view(1, hk, d)
        st["k"] = _activations((n, hk, d), gen, dtype, rows)
        st["v"] = _activations((n, hk, d), gen, dtype)
    if case["kind"] in ("attend", "step"):
        st["q"] = _activations((n, case["hq"], d), gen, dtype)
    if case["kind"] == "append":
        # the last new_len tokens of each sequence are the new ones
        s = torch.repeat_interleave(torch.arange(nseq, device="cuda"), st["new_len"].long(), output_size=n)
        pos = (st["seq_len"] - st["new_len"]).long()[s] + torch.arange(n, device="cuda") - st["token_start"].long()[s]
        st["slots"] = (table[s, pos // page] * page + (pos % page).to(torch.int32)).to(torch.int32)
    if case["kind"] in ("append", "gather"):
        st["out_start"] = (torch.cumsum(st["seq_len"], 0) - st["seq_len"]).to(torch.int32)
        st["rows"] = sum(lens)
    if own:
        import tile_routed_mixed_b200 as tm
        pool = (st["k_codes"], st["k_scale"], st["v_codes"], st["v_scale"])
        if case["kind"] == "plan":
            pool = None
        tables = (table, st["seq_len"], st["free_list"], st["free_count"])
        st["cache"] = tm.TileMixKV4Cache(num_pages, page, hk, d, nseq, max_pages, group=group, dtype=dtype,
                                         pool=pool, tables=tables)
        st["plans"] = [st["cache"].new_plan(n), st["cache"].new_plan(0)]
    return st


# ------------------------------------------------------------ plain forms ---

def _plan(st, new_len, max_tokens):
    """Pages and slots of one step.  new_len[s] tokens are added to sequence s,
    or, where it is negative, the last -new_len[s] are dropped."""
    page, nseq, max_pages = st["page"], st["nseq"], st["max_pages"]
    length, n = st["seq_len"].long(), new_len.long()
    grow, drop = n.clamp(min=0), torch.minimum((-n).clamp(min=0), length)
    end = torch.cumsum(grow, 0)
    begin = end - grow
    pages = lambda x: torch.div(x + page - 1, page, rounding_mode="floor")
    before, keep, after = pages(length), pages(length - drop), pages(length + grow)
    fits = (end <= max_tokens) & (after <= max_pages)
    need = torch.where(fits, after - before, 0)
    back = before - keep
    free = st["free_count"].long()
    have = free + back.sum()
    cum = torch.cumsum(need, 0)
    granted = (grow == 0) | (fits & ((need == 0) | (cum <= have)))
    col = torch.arange(max_pages, device=length.device)[None, :]
    # pages that come back: the k-th of them to place have - 1 - k of the stack
    leaves = (col >= keep[:, None]) & (col < before[:, None])
    k = (torch.cumsum(back, 0) - back)[:, None] + col - keep[:, None]
    stack = torch.cat([st["free_list"], st["free_list"].new_zeros(1)])
    stack.scatter_(0, torch.where(leaves, have - 1 - k, st["num_pages"]).flatten(), st["block_table"].flatten())
    st["free_list"].copy_(stack[:-1])
    # pages that go out: the k-th of them from place have - 1 - k
    comes = granted[:, None] & (col >= before[:, None]) & (col < after[:, None])
    k = (cum - need)[:, None] + col - before[:, None]
    taken = stack[torch.where(comes, have - 1 - k, st["num_pages"])]
    table = torch.where(comes, taken, torch.where(leaves, -1, st["block_table"]))
    st["block_table"].copy_(table)
    st["free_count"].copy_(have - torch.where(granted, need, 0).sum())
    st["seq_len"].copy_(length - drop + torch.where(granted, grow, 0))
    i = torch.arange(max_tokens, device=length.device)
    s = torch.searchsorted(end, i, right=True).clamp(max=nseq - 1)
    pos = length[s] + i - begin[s]
    slot = table[s, torch.div(pos, page, rounding_mode="floor").clamp(0, max_pages - 1)] * page + pos % page
    slots = torch.where((i < end[-1]) & granted[s], slot, -1).to(torch.int32)
    token_start = torch.cat([end.new_zeros(1), end]).to(torch.int32)
    return token_start, slots, granted.to(torch.int32)


def _append(st, k, v, slots):
    page = st["page"]
    kq, ks = _quantise(k, st["group"])
    vq, vs = _quantise(v, st["group"])
    kp, vp = _pack(kq, vq)
    real = (slots >= 0).nonzero().flatten()
    p, r = torch.div(slots[real], page, rounding_mode="floor").long(), (slots[real] % page).long()
    for name, x in (("k_codes", kp), ("v_codes", vp), ("k_scale", ks), ("v_scale", vs)):
        st[name][p, :, r] = x[real]


def _values(st, which, pages, dtype):
    """The values that the rows of `pages` stand for: [..., hk, page, d]."""
    d, t = st["d"], st["d"] // 32
    b = st[which + "_codes"][pages]
    lead = list(b.shape[:-1])
    b = b.view(lead + ([4, t, 4] if which == "k" else [8, t, 2])).transpose(-3, -2).reshape(lead + [d // 2])
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).to(dtype) - 8
    return (c.unflatten(-1, (d // st["group"], st["group"])) * st[which + "_scale"][pages].to(dtype)[..., None]).flatten(-2)


def _tokens(st, which):
    """[nseq][hk][max_pages * page][d] in 32 bits, page after page."""
    x = _values(st, which, st["block_table"].clamp(min=0).long(), torch.float32)
    return x.transpose(1, 2).flatten(2, 3)


def _gather(st):
    dtype, page = HEADS[st["dtype"]], st["page"]
    i = torch.arange(st["rows"], device="cuda")
    s = torch.searchsorted(torch.cumsum(st["seq_len"].long(), 0), i, right=True)
    pos = i - st["out_start"].long()[s]
    p = st["block_table"][s, torch.div(pos, page, rounding_mode="floor")].long()
    return [_rows(st, which, p, pos % page).to(dtype) for which in "kv"]


def _rows(st, which, p, r):
    """[n][hk][d] in 32 bits: row r of page p."""
    sub = dict(st)
    sub[which + "_codes"], sub[which + "_scale"] = (st[which + x][p, :, r] for x in ("_codes", "_scale"))
    return _values(sub, which, slice(None), torch.float32)


def _attend(st, token_start):
    nseq, hk, hq, d = st["nseq"], st["hk"], st["hq"], st["d"]
    q, n, mq = st["q"], st["q"].shape[0], st["max_new"]
    start = token_start.long()
    m = start[1:] - start[:-1]
    i = torch.arange(n, device="cuda")
    s = torch.searchsorted(start[1:], i, right=True)
    at = i - start[s]
    padded = torch.zeros((nseq, mq, hk, hq // hk, d), device="cuda")
    padded[s, at] = q.float().view(n, hk, hq // hk, d)
    padded = padded.permute(0, 2, 1, 3, 4).flatten(2, 3)             # [nseq, hk, mq * group, d]
    score = padded @ _tokens(st, "k").transpose(-1, -2) / math.sqrt(d)
    last = st["seq_len"].long()[:, None] - m[:, None] + torch.arange(mq, device="cuda")  # newest key each may see
    legal = torch.arange(score.shape[-1], device="cuda") <= last[..., None]
    score.unflatten(2, (mq, hq // hk)).masked_fill_(~legal[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(top).exp_()
    z = p.sum(-1, keepdim=True)
    o = (p @ _tokens(st, "v")) / z.clamp(min=1e-37)
    lse = (top + z.log()).squeeze(-1)
    o = o.unflatten(2, (mq, hq // hk)).permute(0, 2, 1, 3, 4)[s, at].reshape(n, hq, d).to(q.dtype)
    lse = lse.unflatten(2, (mq, hq // hk)).permute(0, 2, 1, 3)[s, at].reshape(n, hq)
    return o, lse.t().contiguous()


def _tables(st):
    return [st[x] for x in ("seq_len", "block_table", "free_list", "free_count")]


def run(st):
    kind = st["kind"]
    if kind == "plan":
        # tokens added, then dropped again: the tables end as they began
        if own:
            a = st["cache"].plan(st["new_len"], out=st["plans"][0])
            b = st["cache"].plan(st["drop_len"], out=st["plans"][1])
        else:
            a = _plan(st, st["new_len"], st["max_tokens"])
            b = _plan(st, st["drop_len"], 0)
        return [list(a), list(b), _tables(st)]
    if kind == "append":
        if own:
            st["cache"].append(st["k"], st["v"], st["slots"])
            return list(st["cache"].gather(st["out_start"], st["rows"]))
        _append(st, st["k"], st["v"], st["slots"])
        return _gather(st)
    if kind == "gather":
        if own:
            return list(st["cache"].gather(st["out_start"], st["rows"]))
        return _gather(st)
    if kind == "attend":
        if own:
            return list(st["cache"].attend(st["q"], st["max_seqlen"], token_start=st["token_start"],
                                           max_new=st["max_new"], lse=True))
        return list(_attend(st, st["token_start"]))
    if own:
        cache = st["cache"]
        a = cache.plan(st["new_len"], out=st["plans"][0])
        cache.append(st["k"], st["v"], a.slots)
        o, lse = cache.attend(st["q"], st["max_seqlen"], token_start=a.token_start, max_new=st["max_new"], lse=True)
        cache.plan(st["drop_len"], out=st["plans"][1])
        return [a.slots, o, lse, _tables(st)]
    token_start, slots, _ = _plan(st, st["new_len"], st["max_tokens"])
    _append(st, st["k"], st["v"], slots)
    o, lse = _attend(st, token_start)
    _plan(st, st["drop_len"], 0)
    return [slots, o, lse, _tables(st)]


# ------------------------------------------------------------------ exact ---

def _exact_row_codes(x, group):
    """Values that a row's codes stand for, in 64 bits: code * s."""
    y = x.double().unflatten(-1, (-1, group))
    s = (y.abs().amax(-1, keepdim=True) / 7).to(x.dtype).double()
    return (torch.where(s > 0, torch.round(y / s), 0.0).clamp(-7, 7) * s).flatten(-2)


def _exact_page_values(st, which, pages):
    """[tokens][hk][d] in 64 bits of one sequence's pages, nibble by nibble."""
    d, t = st["d"], st["d"] // 32
    c = torch.arange(d, device="cuda")
    if which == "k":   # channel c: nibble c % 8 of word c / 8
        w = c // 8
        byte = 4 * ((w % 4) * t + w // 4) + c % 8 // 2
    else:              # channel c: nibble c % 4 of halfword c / 4
        h = c // 4
        byte = 2 * ((h % 8) * t + h // 8) + c % 4 // 2
    b = st[which + "_codes"][pages][..., byte]                       # [pages][hk][page][d]
    code = torch.where(c % 2 == 0, b % 16, b // 16).double() - 8
    x = code * st[which + "_scale"][pages][..., c // st["group"]].double()
    return x.transpose(1, 2).flatten(0, 1)


def _exact_plan(lens, news, table, free, page, max_pages, max_tokens):
    """One plan on host lists, sequence by sequence; returns its outputs."""
    back = []
    for s, m in enumerate(news):
        if m < 0:
            keep = -(-max(0, lens[s] + m) // page)
            for j in range(keep, -(-lens[s] // page)):
                back.append(table[s][j])
                table[s][j] = -1
    stack = free[0] + back[::-1]
    start, slots, granted, need = [0], [], [], 0
    have, used = len(stack), 0
    for s, m in enumerate(news):
        g = max(0, m)
        a, b = -(-lens[s] // page), -(-(lens[s] + g) // page)
        fits = start[-1] + g <= max_tokens and b <= max_pages
        if g and fits:
            need += b - a
        ok = g == 0 or (fits and (b == a or need <= have))
        if ok:
            for j in range(a, b):
                table[s][j] = stack[have - 1 - used]
                used += 1
        for i in range(g):
            if start[-1] + i < max_tokens:
                x = lens[s] + i
                slots.append(table[s][x // page] * page + x % page if ok else -1)
        start.append(start[-1] + g)
        granted.append(int(ok))
        lens[s] = lens[s] + g * ok if m >= 0 else max(0, lens[s] + m)
    slots += [-1] * (max_tokens - len(slots))
    free[1] = have - used
    free[2] = stack + free[2][len(stack):]
    free[0] = stack[:have - used]
    return start, slots, granted


def exact(case, seed):
    st = prepare(case, seed)
    kind, page, group = case["kind"], case["page"], st["group"]
    lens, news = _lengths(case)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    tables, slots = None, None
    if _grows(case):
        table = st["block_table"].tolist()
        whole = st["free_list"].tolist()
        free = [whole[:int(st["free_count"])], 0, whole]
        cur = list(lens)
        a = _exact_plan(cur, news, table, free, page, st["max_pages"], st["max_tokens"])
        grown = ints(table)
        full = list(cur)
        b = _exact_plan(cur, [-m for m in news], table, free, page, st["max_pages"], 0)
        tables = [ints(cur), ints(table), ints(free[2]), ints([free[1]])]
        slots = ints(a[1])
        if kind == "plan":
            return [[ints(x) for x in a], [ints(x) for x in b], tables]
        st["block_table"], lens = grown, full
    dtype, n = HEADS[st["dtype"]], st["max_tokens"]
    rows = {}
    if kind in ("append", "step"):
        rows = {w: _exact_row_codes(st[w], group) for w in "kv"}
    got, first = [], 0
    for s in range(case["nseq"]):
        pages = st["block_table"][s, :-(-lens[s] // page)].long()
        kv = {}
        for w in "kv":
            kv[w] = _exact_page_values(st, w, pages)[:lens[s]]
            if rows and news[s]:
                kv[w][lens[s] - news[s]:] = rows[w][first:first + news[s]]
        if kind in ("append", "gather"):
            got.append([kv["k"], kv["v"]])
        elif news[s]:
            q = st["q"][first:first + news[s]].double()                        # [m, hq, d]
            per = case["hq"] // case["hk"]
            o = torch.empty_like(q)
            lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
            last = lens[s] - news[s] + torch.arange(news[s], device="cuda")
            dark = torch.arange(lens[s], device="cuda")[None, None, :] > last[:, None, None]
            for h in range(case["hk"]):
                sel = slice(h * per, (h + 1) * per)
                x = torch.einsum("mgd,td->mgt", q[:, sel], kv["k"][:, h]) / math.sqrt(case["d"])
                x = x.masked_fill(dark, -math.inf)
                lse[:, sel] = torch.logsumexp(x, -1)
                o[:, sel] = torch.einsum("mgt,td->mgd", torch.softmax(x, -1), kv["v"][:, h])
            got.append([o, lse])
        first += news[s]
    a, b = (torch.cat([g[i] for g in got]) for i in range(2))
    if kind in ("append", "gather"):
        return [a, b]
    out = [a, b.t().contiguous()]
    return out if kind == "attend" else [slots, out[0], out[1], tables]
