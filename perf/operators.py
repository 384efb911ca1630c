"""The operators of a decode loop over a paged 4-bit KV cache, measured at real sizes.

Between the merged QKV projection and o_proj a serving step appends the new keys and
values to the cache (`append`, with the read-back of the same rows) and attends over it
(`attend`); after the LM head a beam search picks the next tokens from the vocab shards
(`beam`) and gives every surviving beam its parent's pages (`fork`); now and then the
live pages move to the front of the pool (`compact`).

Cache of one shard and one layer: uint8 [pages, kv_heads, page_size / 16, 16 (hd + 8)].
A block of 16 tokens of one kv head holds the codes of 16 keys (hd / 2 bytes each, dim d
in the low (d even) or high half of byte d / 2), the codes of 16 values, 16 pairs (step,
base) of bfloat16 for the keys, and 16 for the values.  A row x of hd elements is held
as base = min(x), step = bf16((max(x) - min(x)) / 15) and codes
u = clamp(rint((x - base) / step), 0, 15); it stands for step u + base.
"""

import math
import random

import torch

own = False

BLOCK = 16          # tokens of a cache block


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's rows of 64 sequences, h = 8192 cut into 4 shards
        dict(name="append_decode", kind="append", t=4, kv=2, hd=128, ps=64, seqs=64, lo=1, hi=2000, rows_lo=1, rows_hi=1),
        # a prefill of 8192 tokens in four prompts
        dict(name="append_prefill", kind="append", t=8, kv=1, hd=128, ps=64, seqs=4, lo=2048, hi=4096, rows_lo=2048,
             rows_hi=2048),
        # one user's decode step: latency counts
        dict(name="attend_one", kind="attend", t=4, heads=16, kv=2, hd=128, ps=64, seqs=1, lo=4097, hi=4097, rows_lo=1,
             rows_hi=1, window=0, sinks=0),
        # a full decode batch with long contexts of all lengths
        dict(name="attend_batch", kind="attend", t=4, heads=16, kv=2, hd=128, ps=64, seqs=64, lo=4100, hi=8192, rows_lo=1,
             rows_hi=1, window=0, sinks=0),
        # long chats that keep a window and the first tokens
        dict(name="attend_window", kind="attend", t=8, heads=8, kv=1, hd=128, ps=32, seqs=32, lo=9000, hi=24001, rows_lo=1,
             rows_hi=1, window=4096, sinks=4),
        # chunked prefill: 8192 new tokens over what is cached already
        dict(name="attend_prefill", kind="attend", t=4, heads=16, kv=2, hd=128, ps=64, seqs=4, lo=2100, hi=6001,
             rows_lo=2048, rows_hi=2048, window=0, sinks=0),
        # a beam step of one short request over a small model's cache
        dict(name="fork_few", kind="fork", t=2, kv=4, hd=64, ps=16, layers=2, items=2, beams=4, prefix=100, tail=41, own_pages=8),
        # a beam step of 32 requests of 8 beams
        dict(name="fork_many", kind="fork", t=4, kv=2, hd=128, ps=64, layers=4, items=32, beams=8, prefix=1537, tail=411,
             own_pages=8),
        # defragmentation of a small pool and of a large one
        dict(name="compact_few", kind="compact", t=2, kv=4, hd=64, ps=16, layers=2, seqs=7, lo=5, hi=300, spare=2),
        dict(name="compact_many", kind="compact", t=4, kv=2, hd=128, ps=64, layers=4, seqs=96, lo=200, hi=2500, spare=2),
        # selection for one request of four beams, and for a full batch of 32 requests
        dict(name="beam_one", kind="beam", t=2, items=1, beams=4, k=4, vocab=151936, f32=False, done=0),
        dict(name="beam_batch", kind="beam", t=4, items=32, beams=8, k=8, vocab=151936, f32=True, done=1),
    ]


def _log(rng, lo, hi):
    """A whole number spread over lo..hi by its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    kind = rng.choice(["append", "attend", "attend", "attend", "fork", "compact", "beam"])
    t, kv, hd, ps = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    if kind == "append":
        rows = _log(rng, 1, 2048)
        seqs = _log(rng, 1, max(1, min(64, 4096 // rows)))
        return dict(kind=kind, t=t, kv=kv, hd=hd, ps=ps, seqs=seqs, lo=rows, hi=rows + _log(rng, 1, 2000),
                    rows_lo=max(1, rows // 3), rows_hi=rows)
    if kind == "attend":
        heads = kv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
        window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 1, 3000), rng.randint(0, 40))])
        if rng.random() < 0.6:                                           # decode, or a few rows each (speculation)
            rows = rng.choice([1, 1, 1, 2, 3, 5])
            seqs = _log(rng, 1, 128)
            hi = _log(rng, 16, min(24000, 2000000 // (seqs * t * kv)))
        else:                                                            # chunks of prompts
            rows = _log(rng, 6, 1200)
            seqs = _log(rng, 1, max(1, min(24, 3000 // rows)))
            hi = rows + _log(rng, 1, max(2, min(9000, 600000000 // (seqs * rows * t * heads))))
        return dict(kind=kind, t=t, heads=heads, kv=kv, hd=hd, ps=ps, seqs=seqs, lo=max(rows, hi // 3), hi=max(rows, hi),
                    rows_lo=max(1, rows // 2), rows_hi=rows, window=window, sinks=sinks)
    if kind == "fork":
        return dict(kind=kind, t=t, kv=kv, hd=hd, ps=ps, layers=rng.choice([1, 2, 3, 4]), items=_log(rng, 1, 24),
                    beams=rng.randint(2, 8), prefix=_log(rng, 1, 1000), tail=rng.randint(0, 300), own_pages=320 // ps + 2)
    if kind == "compact":
        return dict(kind=kind, t=t, kv=kv, hd=hd, ps=ps, layers=rng.choice([1, 2, 3]), seqs=_log(rng, 1, 64), lo=1,
                    hi=_log(rng, 2, 1500), spare=rng.randint(1, 4))
    beams = rng.randint(1, 8)
    return dict(kind=kind, t=t, items=_log(rng, 1, 30), beams=beams, k=rng.choice([beams, 2 * beams]),
                vocab=_log(rng, 40, 151936), f32=rng.random() < 0.5, done=rng.choice([0, 1]))


def _spread(i, lo, hi):
    """The i-th of a fixed sequence over lo..hi, the first one hi."""
    return hi - (i * 40503 + i * i * 977) % (hi - lo + 1)


def _lens(c):
    return [_spread(i, c["lo"], c["hi"]) for i in range(c["seqs"])]


def _rows(c):
    return [_spread(i, c["rows_lo"], c["rows_hi"]) for i in range(c["seqs"])]


def _block_bytes(c):
    return BLOCK * (c["hd"] + 8)


def _page_bytes(c):
    return c["kv"] * c["ps"] * (c["hd"] + 8)


def _seen(c):
    """(tokens that some row of each sequence sees, summed; visible (row, token) pairs, summed)."""
    w, s = c["window"], c["sinks"]
    tokens = pairs = 0
    for n, r in zip(_lens(c), _rows(c)):
        first = n - r                                                    # position of the first row
        if not w:
            tokens += n
            pairs += r * first + r * (r + 1) // 2
            continue
        tokens += n - max(0, max(0, first - w + 1) - s)
        for i in range(first, n):
            low = max(0, i - w + 1)
            pairs += i + 1 - low + min(low, s)
    return tokens, pairs


def work(c):
    kind = c["kind"]
    if kind == "append":                                                 # rows in, codes out and in, values out
        n = sum(_rows(c)) * c["t"] * c["kv"]
        return {"bytes": n * (4 * c["hd"] + 2 * (c["hd"] + 8) + 8 * c["hd"]), "flops": n * 2 * c["hd"] * 6}
    if kind == "attend":
        tokens, pairs = _seen(c)
        io = sum(_rows(c)) * c["t"] * c["heads"] * c["hd"] * 4
        return {"bytes": tokens * c["t"] * c["kv"] * (c["hd"] + 8) + io, "flops": 4 * pairs * c["t"] * c["heads"] * c["hd"]}
    if kind == "fork":
        rows = c["items"] * c["beams"]
        copies = rows - c["items"] * ((c["beams"] + 1) // 2) if (c["prefix"] + c["tail"]) % c["ps"] else 0
        cols = _fork_cols(c)
        return {"bytes": 2 * copies * _page_bytes(c) * c["t"] * c["layers"] + 8 * rows * cols, "flops": rows * cols}
    if kind == "compact":
        pages = sum(-(-n // c["ps"]) for n in _lens(c))
        moved = pages - pages // (c["spare"] + 1)                        # expected: live pages are spread evenly
        return {"bytes": 2 * moved * _page_bytes(c) * c["t"] * c["layers"] + 8 * pages, "flops": pages}
    n = c["items"] * (c["beams"] - (1 if c["done"] and c["beams"] > 1 else 0)) * c["vocab"]
    return {"bytes": n * (4 if c["f32"] else 2) + 12 * c["items"] * c["k"], "flops": 3 * n}


# ------------------------------------------------------------------ the cache, in plain torch

def _quantise(x):
    """Codes, step and base (float32 that bf16 holds) of rows x [..., hd], bf16."""
    x = x.float()
    base, top = x.amin(-1, keepdim=True) + 0.0, x.amax(-1, keepdim=True)
    step = ((top - base) * (1.0 / 15.0)).to(torch.bfloat16).float()
    u = torch.where(step > 0, torch.round((x - base) / step), torch.zeros_like(x)).clamp(0, 15)
    return u, step, base


def _codes(u):
    u = u.to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _pair(step, base):
    return torch.cat([step, base], -1).to(torch.bfloat16).contiguous().view(torch.uint8)


def _values(codes, pair):
    """float32 rows [..., hd] that codes [..., hd / 2] and pairs [..., 4] stand for."""
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    sb = pair.contiguous().view(torch.bfloat16).float()
    return u * sb[..., :1] + sb[..., 1:]


def _parts(pool, hd):
    """Views of a pool [..., 16 (hd + 8)]: key codes, value codes, key pairs, value pairs, [..., 16, bytes] each."""
    a, lead = BLOCK * hd // 2, pool.shape[:-1]
    cut = lambda lo, n: pool[..., lo:lo + BLOCK * n].unflatten(-1, (BLOCK, n))  # noqa: E731
    assert len(lead) >= 1
    return cut(0, hd // 2), cut(a, hd // 2), cut(2 * a, 4), cut(2 * a + 4 * BLOCK, 4)


def _fill(pool, c, g):
    """Random keys and values in every slot of pool [pages, kv, blocks, bytes] of one shard."""
    hd, dev = c["hd"], pool.device
    k4, v4, kp, vp = _parts(pool, hd)
    scale = 0.4 + 2.0 * torch.rand(hd, device=dev, generator=g)          # keys have loud channels
    shift = 0.7 * torch.randn(hd, device=dev, generator=g)
    step = max(1, (1 << 26) // (pool[0].numel()))
    for i in range(0, pool.shape[0], step):
        shape = (*pool[i:i + step].shape[:-1], BLOCK, hd)
        for codes, pair, key in ((k4, kp, True), (v4, vp, False)):
            x = torch.randn(shape, device=dev, generator=g)
            u, s, b = _quantise((x * scale + shift if key else x).to(torch.bfloat16))
            codes[i:i + step] = _codes(u)
            pair[i:i + step] = _pair(s, b)


def _int(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


# ------------------------------------------------------------------ inputs

def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": dict(c), "kind": c["kind"]}
    {"append": _prepare_cache, "attend": _prepare_cache, "fork": _prepare_fork, "compact": _prepare_compact,
     "beam": _prepare_beam}[c["kind"]](c, seed, s, dev, g)
    if own:                                    # the checked and marshalled call that a serving loop repeats
        s["call"] = _handle(s)
    return s


def _prepare_cache(c, seed, s, dev, g):
    lens, rows, ps, hd = _lens(c), _rows(c), c["ps"], c["hd"]
    cols = max(-(-n // ps) for n in lens) + 1
    used = [-(-n // ps) for n in lens]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).tolist()
    table, at = [], 0
    for n in used:
        table.append(order[at:at + n] + [-1] * (cols - n))
        at += n
    s["pool"] = torch.empty((c["t"], pages, c["kv"], ps // BLOCK, _block_bytes(c)), dtype=torch.uint8, device=dev)
    for r in range(c["t"]):
        _fill(s["pool"][r], c, g)
    s["pools"] = list(s["pool"].unbind())
    s["table"], s["lens"] = _int(table, dev), _int(lens, dev)
    n = sum(rows)
    s["n"], s["most"], s["long"] = n, max(rows), max(lens)
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    s["cu"] = _int(cu, dev)
    s["cu_rows"] = None if max(rows) == 1 else s["cu"]
    draw_rows = lambda heads: [torch.randn((n, heads * hd), device=dev, generator=g).to(torch.bfloat16)  # noqa: E731
                               for _ in range(c["t"])]
    if c["kind"] == "attend":
        # q is the first part of the merged QKV projection's rows
        qkv = draw_rows(c["heads"] + 2 * c["kv"])
        s["q"] = [x[:, :c["heads"] * hd] for x in qkv]
    else:
        s["k"], s["v"] = draw_rows(c["kv"]), draw_rows(c["kv"])


def _fork_cols(c):
    return -(-(c["prefix"] + c["tail"] + 1) // c["ps"]) + c["own_pages"]


def _prepare_fork(c, seed, s, dev, g):
    """Beams of an item share the prompt's full pages; each holds its own pages from there on."""
    ps, length = c["ps"], c["prefix"] + c["tail"]
    shared, held = c["prefix"] // ps, -(-length // ps)
    rows, cols = c["items"] * c["beams"], _fork_cols(c)
    pages = c["items"] * (shared + c["beams"] * (held - shared)) + rows + 5
    cpu = torch.Generator().manual_seed(int(seed))
    order = torch.randperm(pages, generator=cpu).tolist()
    table, parents, at = [], [], 0
    for i in range(c["items"]):
        front = order[at:at + shared]
        at += shared
        # half of the beams survive, the best of them in several children
        kept = torch.randperm(c["beams"], generator=cpu)[:(c["beams"] + 1) // 2].tolist()
        for b in range(c["beams"]):
            mine = order[at:at + held - shared]
            at += held - shared
            table.append(front + mine + [-1] * (cols - held))
            parents.append(i * c["beams"] + kept[b % len(kept)])
    s["pool"] = torch.randint(0, 256, (c["t"], c["layers"], pages, c["kv"], ps // BLOCK, _block_bytes(c)),
                              dtype=torch.uint8, device=dev, generator=g)
    s["pools"] = list(s["pool"].unbind())
    s["table"], s["lens"], s["parents"] = _int(table, dev), _int([length] * rows, dev), _int(parents, dev)
    s["grow"] = 1


def _prepare_compact(c, seed, s, dev, g):
    lens, ps = _lens(c), c["ps"]
    used = [-(-n // ps) for n in lens]
    pages = sum(used) * (c["spare"] + 1)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(int(seed))).tolist()
    cols, table, at = max(used) + 1, [], 0
    for n in used:
        table.append(order[at:at + n] + [-1] * (cols - n))
        at += n
    s["pool"] = torch.randint(0, 256, (c["t"], c["layers"], pages, c["kv"], ps // BLOCK, _block_bytes(c)),
                              dtype=torch.uint8, device=dev, generator=g)
    s["pools"] = list(s["pool"].unbind())
    s["table"], s["lens"] = _int(table, dev), _int(lens, dev)


def _prepare_beam(c, seed, s, dev, g):
    rows, per = c["items"] * c["beams"], -(-c["vocab"] // c["t"])
    dt = torch.float32 if c["f32"] else torch.bfloat16
    # an LM head's logits: a few loud tokens over a broad floor
    x = torch.randn((rows, c["vocab"]), device=dev, generator=g)
    x = x * 2.0 + 0.3 * x * x
    s["logits"] = [x[:, r * per:(r + 1) * per].to(dt).contiguous() for r in range(c["t"])]
    s["scores"] = -10.0 * torch.rand((c["items"], c["beams"]), device=dev, generator=g)
    s["finished"] = None
    if c["done"] and c["beams"] > 1:
        s["finished"] = torch.zeros((c["items"], c["beams"]), dtype=torch.bool, device=dev)
        s["finished"][:, 1] = True
    s["eos"], s["k"] = c["vocab"] - 1, c["k"]


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"append": _plain_append, "attend": _plain_attend, "fork": _plain_fork, "compact": _plain_compact,
            "beam": _plain_beam}[s["kind"]](s)


def _handle(s):
    """The prepared calls (each checks and marshals its arguments once) of one pass."""
    import megatron_tensor_layers_gb300 as tp
    c, kind = s["case"], s["kind"]
    if kind == "append":
        return [tp.prepare(tp.tp_kv4_append, s["k"], s["v"], s["pools"], s["table"], s["lens"], cu_rows=s["cu_rows"]),
                tp.prepare(tp.tp_kv4_load, s["pools"], s["table"], s["lens"], s["n"], cu_rows=s["cu_rows"],
                           dtype=torch.float32)]
    if kind == "attend":
        return [tp.prepare(tp.tp_kv4_attention, s["q"], s["pools"], s["table"], s["lens"], cu_rows=s["cu_rows"],
                           window=c["window"], sinks=c["sinks"])]
    if kind == "fork":
        return [tp.prepare(tp.tp_kv_fork, s["table"], s["lens"], s["parents"], s["pools"], grow=s["grow"])]
    if kind == "compact":
        return [tp.prepare(tp.tp_kv_compact, s["table"], s["lens"], s["pools"])]
    return [tp.prepare(tp.tp_beam_select, s["logits"], s["scores"], s["k"], finished=s["finished"], eos=s["eos"])]


def _run_own(s):
    call, kind = s["call"], s["kind"]
    if kind == "append":
        call[0]()
        return call[1]()
    got = call[0]()
    if kind in ("fork", "compact"):
        return {"pools": s["pools"], "tables": got}
    return got


# ------------------------------------------------------------------ plain forms

def _row_places(s):
    """Of each new row: its sequence, its number there and its position."""
    cu, lens = s["cu"].long(), s["lens"].long()
    i = torch.arange(s["n"], device=cu.device)
    seq = torch.bucketize(i, cu[1:], right=True)
    r = i - cu[seq]
    return seq, r, lens[seq] - (cu[seq + 1] - cu[seq]) + r


def _plain_append(s):
    c = s["case"]
    t, kv, hd, ps = c["t"], c["kv"], c["hd"], c["ps"]
    seq, _, pos = _row_places(s)
    page, block, slot = s["table"].long()[seq, pos // ps], pos % ps // BLOCK, pos % BLOCK
    k4, v4, kp, vp = _parts(s["pool"], hd)
    uk, sk, bk = _quantise(torch.stack(s["k"]).unflatten(-1, (kv, hd)))  # [t, n, kv, hd]
    uv, sv, bv = _quantise(torch.stack(s["v"]).unflatten(-1, (kv, hd)))
    put = lambda part, x: part.permute(1, 3, 4, 0, 2, 5).index_put_((page, block, slot), x.transpose(0, 1))  # noqa: E731
    put(k4, _codes(uk)), put(v4, _codes(uv)), put(kp, _pair(sk, bk)), put(vp, _pair(sv, bv))
    get = lambda part: part.permute(1, 3, 4, 0, 2, 5)[page, block, slot].transpose(0, 1)  # noqa: E731
    return (list(_values(get(k4), get(kp)).flatten(-2).unbind()), list(_values(get(v4), get(vp)).flatten(-2).unbind()))


def _plain_attend(s):
    c = s["case"]
    t, kv, hd, heads, ns = c["t"], c["kv"], c["hd"], c["heads"], c["seqs"]
    group, most, dev = heads // kv, s["most"], s["table"].device
    lens, cu = s["lens"].long(), s["cu"].long()
    # the sequences' keys and values [t, seqs, kv, tokens, hd]
    blocks = s["pool"][:, s["table"].long().clamp(min=0)].transpose(2, 3).flatten(3, 4)
    k4, v4, kp, vp = (x.flatten(3, 4) for x in _parts(blocks, hd))
    keys, vals = _values(k4, kp), _values(v4, vp)
    tokens = keys.shape[3]
    # the rows, padded to the longest: [t, seqs, kv, rows group, hd]
    count = cu[1:] - cu[:-1]
    r = torch.arange(most, device=dev)
    q = torch.stack(s["q"]).float()[:, (cu[:-1, None] + r).clamp(max=s["n"] - 1)]
    q = q.unflatten(-1, (kv, group, hd)).permute(0, 1, 3, 2, 4, 5).flatten(3, 4) * (1.0 / math.sqrt(hd))
    i = (lens - count)[:, None, None] + r[:, None]                       # positions of rows
    j = torch.arange(tokens, device=dev)
    see = (j <= i) & (r[:, None] < count[:, None, None])
    if c["window"]:
        see &= (j > i - c["window"]) | (j < c["sinks"])
    see = see.repeat_interleave(group, 1)[None, :, None]
    x = torch.matmul(q, keys.transpose(-1, -2)).masked_fill_(~see, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, vals) / torch.where(total > 0, total, torch.ones_like(total))
    seq, r, _ = _row_places(s)
    o = o.unflatten(3, (most, group))[:, seq, :, r]                      # [n, t, kv, group, hd]
    o = o.transpose(0, 1).flatten(2).to(torch.bfloat16)
    return list(o.unbind())


def _count(pages, entries):
    """How often each page stands among entries (negative ones do not count)."""
    entries = entries.flatten()
    return torch.zeros(pages + 1, dtype=torch.int64, device=entries.device).index_add_(
        0, torch.where(entries < 0, pages, entries), torch.ones_like(entries))[:pages]


def _plain_fork(s):
    c = s["case"]
    ps, pages = c["ps"], s["pool"].shape[2]
    table, lens, parents = s["table"].long(), s["lens"].long(), s["parents"].long()
    rows, cols = parents.shape[0], table.shape[1]
    dev = table.device
    have = lens[parents]
    new = (have + s["grow"]).clamp(0, cols * ps)
    keep = torch.minimum(have, new)
    kept, want = -(-keep // ps), -(-new // ps)
    col = torch.arange(cols, device=dev)
    out = torch.where(col < kept[:, None], table[parents], -1)
    refs = _count(pages, out)
    # a row that goes on writing inside a page needs it for itself
    writes = (keep % ps != 0) & (new > keep)
    tail = out.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0]
    place = torch.where(writes, tail, pages)
    writers = _count(pages + 1, place)
    i = torch.arange(rows, device=dev)
    first = torch.full((pages + 1,), rows, device=dev).scatter_reduce_(0, place, i, "amin")
    alone = (torch.cat([refs, refs.new_zeros(1)]) == writers)[place] & (first[place] == i)
    copies = writes & ~alone
    # free pages in ascending order, dealt out row by row: the copy first, then fresh pages
    free = refs == 0
    order = torch.argsort(~free, stable=True)
    order = torch.cat([torch.where(torch.arange(pages, device=dev) < free.sum(), order, -1), order.new_full((1,), -1)])
    need = copies.long() + want - kept
    start = need.cumsum(0) - need
    deal = lambda k: order[k.clamp(max=pages)]  # noqa: E731
    into = deal(start)
    out = torch.where(copies[:, None] & (col == kept[:, None] - 1), into[:, None], out)
    fresh = (col >= kept[:, None]) & (col < want[:, None])
    out = torch.where(fresh, deal((start + copies)[:, None] + col - kept[:, None]), out)
    move = copies & (into >= 0)
    s["pool"][:, :, into[move]] = s["pool"][:, :, tail[move]]
    refs = _count(pages, out)
    missing = ((col < want[:, None]) & (out < 0)).sum()
    info = torch.stack([(refs > 0).sum(), missing, move.sum(), torch.zeros_like(missing)])
    return {"pools": s["pools"], "tables": (out.int(), new.int(), refs.int(), info.int())}


def _plain_compact(s):
    ps, pages = s["case"]["ps"], s["pool"].shape[2]
    table, lens = s["table"].long(), s["lens"].long()
    col, page = torch.arange(table.shape[1], device=table.device), torch.arange(pages, device=table.device)
    out = torch.where(col < -(-lens[:, None] // ps), table, -1)
    refs = _count(pages, out)
    live = refs > 0
    total = live.sum()
    src, dst = page[live & (page >= total)], page[~live & (page < total)]
    dst = dst[:src.shape[0]]
    to = page.clone()
    to[src] = dst
    out = torch.where(out < 0, out, to[out.clamp(min=0)])
    s["pool"][:, :, dst] = s["pool"][:, :, src]
    refs = _count(pages, out)
    zero = torch.zeros_like(total)
    info = torch.stack([total, zero, zero + src.shape[0], zero])
    return {"pools": s["pools"], "tables": (out.int(), refs.int(), info.int())}


def _plain_beam(s):
    c, k = s["case"], s["k"]
    items, beams = c["items"], c["beams"]
    x = torch.cat(s["logits"], 1).float() + 0.0
    top = x.amax(1, keepdim=True)
    # log of the normaliser, in 64 bits: candidates of two beams can be next to each other
    norm = top[:, 0].double() + (x - top).exp_().sum(1, dtype=torch.float64).log()
    # the best k of a row by (logit, lowest token): the two as one whole number
    bits = x.view(torch.int32)
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    token = torch.arange(x.shape[1], device=x.device)
    key = torch.topk((bits << 32) | (0xFFFFFFFF - token), min(k, x.shape[1]), dim=1).values
    token = 0xFFFFFFFF - (key & 0xFFFFFFFF)
    score = (s["scores"].flatten().double() - norm)[:, None] + x.gather(1, token).double()
    if s["finished"] is not None:                                        # such a beam has one candidate: itself
        done = s["finished"].flatten()[:, None]
        first = torch.arange(token.shape[1], device=x.device) == 0
        score = torch.where(done, torch.where(first, s["scores"].flatten().double()[:, None], -math.inf), score)
        token = torch.where(done, s["eos"], token)
    row = torch.arange(items * beams, device=x.device)[:, None].expand_as(token)
    score, token, row = (v.reshape(items, -1) for v in (score, token, row))
    # ties to the lowest (beam, token): candidates stand in that order before a stable sort
    at = torch.argsort(row * c["vocab"] + token, dim=1, stable=True)
    score, token, row = (v.gather(1, at) for v in (score, token, row))
    at = torch.argsort(score, dim=1, descending=True, stable=True)[:, :k]
    score, token, row = (v.gather(1, at) for v in (score, token, row))
    none = score == -math.inf
    token, row = torch.where(none, -1, token), torch.where(none, -1, row)
    if score.shape[1] < k:
        pad = (0, k - score.shape[1])
        score = torch.nn.functional.pad(score, pad, value=-math.inf)
        token, row = (torch.nn.functional.pad(v, pad, value=-1) for v in (token, row))
    return score.float(), row.int(), token.int()


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(c, seed):
    s = prepare(c, seed)
    if c["kind"] == "append":
        return _exact_append(c, s)
    if c["kind"] == "attend":
        return _exact_attend(c, s)
    if c["kind"] == "beam":
        return _exact_beam(c, s)
    return None


def _exact_append(c, s):
    """What each row stands for: the codes from their definition (its few float32 steps), the values in 64 bits."""
    import numpy as np

    def one(x):
        x = x.float().cpu().numpy().reshape(s["n"], c["kv"], c["hd"])
        low, high = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        step = torch.from_numpy((high - low) * np.float32(1.0 / 15.0)).to(torch.bfloat16).float().numpy()
        safe = np.where(step > 0, step, np.float32(1))
        u = np.where(step > 0, np.clip(np.rint((x - low) / safe), 0, 15), 0)
        return torch.from_numpy((u.astype(np.float64) * step + low).reshape(s["n"], -1))

    return [one(x) for x in s["k"]], [one(x) for x in s["v"]]


def _exact_attend(c, s):
    kv, hd, heads, ps = c["kv"], c["hd"], c["heads"], c["ps"]
    outs = []
    for r in range(c["t"]):
        at, out = 0, []
        for i, (n, rows) in enumerate(zip(_lens(c), _rows(c))):
            pages = s["table"][i, :-(-n // ps)].long()
            rec = s["pools"][r][pages].transpose(0, 1).reshape(kv, -1, _block_bytes(c))
            half = BLOCK * hd // 2

            def side(lo, where):
                byte = rec[..., lo:lo + half].reshape(kv, -1, hd // 2)
                x = torch.empty((kv, byte.shape[1], hd), dtype=torch.float64, device=byte.device)
                x[..., 0::2], x[..., 1::2] = (byte % 16).double(), (byte // 16).double()
                sb = rec[..., where:where + 4 * BLOCK].reshape(kv, -1, 4).contiguous().view(torch.bfloat16).double()
                return (x * sb[..., 0:1] + sb[..., 1:2])[:, :n]

            keys, vals = side(0, 2 * half), side(half, 2 * half + 4 * BLOCK)
            q = s["q"][r][at:at + rows].double().reshape(rows, kv, heads // kv, hd)
            pos = torch.arange(n - rows, n, device=q.device)[:, None]
            j = torch.arange(n, device=q.device)[None]
            hidden = j > pos
            if c["window"]:
                hidden = hidden | ((j <= pos - c["window"]) & (j >= c["sinks"]))
            o = torch.empty_like(q)
            for h in range(kv):
                x = torch.einsum("rgd,jd->rgj", q[:, h], keys[h]) / math.sqrt(hd)
                x.masked_fill_(hidden[:, None], -math.inf)
                o[:, h] = torch.einsum("rgj,jd->rgd", torch.softmax(x, -1), vals[h])
            out.append(o.reshape(rows, heads * hd))
            at += rows
        outs.append(torch.cat(out))
    return outs


def _exact_beam(c, s):
    x = torch.cat([v.double() for v in s["logits"]], 1)
    logp = torch.log_softmax(x, 1).reshape(c["items"], c["beams"], c["vocab"])
    total = s["scores"].double()[..., None] + logp
    if s["finished"] is not None:
        total[s["finished"]] = -math.inf
        total[..., s["eos"]] = torch.where(s["finished"], s["scores"].double(), total[..., s["eos"]])
    got = []
    for i in range(c["items"]):
        v, at = torch.sort(total[i].flatten(), descending=True, stable=True)
        n = min(c["k"], int((v > -math.inf).sum()))
        v, at = v[:c["k"]], at[:c["k"]]
        row, token = i * c["beams"] + at // c["vocab"], at % c["vocab"]
        pad = c["k"] - n
        got.append((torch.cat([v[:n], v.new_full((pad,), -math.inf)]), torch.cat([row[:n], row.new_full((pad,), -1)]),
                    torch.cat([token[:n], token.new_full((pad,), -1)])))
    score, row, token = (torch.stack(v) for v in zip(*got))
    return score, row.int(), token.int()
