"""Decode-loop operators restated on the CPU (numpy, float64 where a value is
computed, Python integers where a page or a token is chosen), sharing no code
with the GPU path: the 4-bit cache format, attention over what it stands for,
page bookkeeping and beam selection.  The definitions are those of
include/tp.h; the few float32 steps of the format are part of it."""

from __future__ import annotations

import numpy as np

BLOCK = 16


def bf16(x: np.ndarray) -> np.ndarray:
    """float32 rounded to the nearest bfloat16 (ties to even), as float32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint32) << 16
    out = r.view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), out)


def quantise(x: np.ndarray):
    """Codes, steps and bases of rows x [..., hd] (float32 holding bf16 values)."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
        span = (hi - lo).astype(np.float32)
        good = np.isfinite(x).all(-1, keepdims=True) & np.isfinite(span)
        step = bf16(np.where(good, span, 0) * np.float32(1.0 / 15.0))
        safe = np.where(step > 0, step, np.float32(1.0))
        u = np.where(good & (step > 0), np.clip(np.rint(((x - lo).astype(np.float32) / safe)), 0, 15), 0)
    base = np.where(good, lo + np.float32(0), np.float32(np.nan))
    return u.astype(np.uint8), step, base


def values(u, step, base) -> np.ndarray:
    """float64 values that the codes stand for."""
    return u.astype(np.float64) * step.astype(np.float64) + base.astype(np.float64)


def pack_blocks(ku, ks, kb, vu, vs, vb) -> np.ndarray:
    """Blocks [..., 16 (hd + 8)] of codes [..., 16, hd] and steps, bases [..., 16, 1]."""
    def codes(u):
        return (u[..., 0::2] | (u[..., 1::2] << 4)).reshape(*u.shape[:-2], -1)

    def pairs(s, b):
        p = np.concatenate([s, b], -1).astype(np.float32)
        bits = (p.view(np.uint32) >> 16).astype(np.uint16)
        return np.ascontiguousarray(bits).view(np.uint8).reshape(*s.shape[:-2], -1)

    return np.concatenate([codes(ku), codes(vu), pairs(ks, kb), pairs(vs, vb)], -1)


def attention(q, k, v, pos, scale, window=0, sinks=0) -> np.ndarray:
    """softmax(scale q k^T) v in float64 for rows q [n, hd] at positions pos [n]
    over tokens k, v [m, hd] of one kv head; rows that see nothing give 0."""
    out = np.zeros(q.shape, dtype=np.float64)
    j = np.arange(k.shape[0])
    for i, p in enumerate(pos):
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        if not see.any():
            continue
        x = scale * (k[see] @ q[i])
        e = np.exp(x - x.max())
        out[i] = (e / e.sum()) @ v[see]
    return out


def fork(table, lens, parents, grow, page_size, pages, held=None):
    """(table, lens, refs, info, copies) of tp_kv_fork, row by row."""
    max_blocks = table.shape[1]
    held = [0] * pages if held is None else list(held)
    room = max_blocks * page_size
    rows, lens_out, bad = [], [], 0
    for i, p in enumerate(parents):
        g = grow[i] if hasattr(grow, "__len__") else grow
        if not 0 <= p < table.shape[0]:
            rows.append(dict(entries=[], keep=0, new=0))
            lens_out.append(0)
            continue
        have = min(max(int(lens[p]), 0), room)
        new = min(max(have + int(g), 0), room)
        keep = min(have, new)
        entries = [int(x) for x in table[p][:-(-keep // page_size)]]
        bad += sum(not 0 <= x < pages for x in entries)
        rows.append(dict(entries=[x if 0 <= x < pages else -1 for x in entries], keep=keep, new=new))
        lens_out.append(new)
    users = {}
    for i, r in enumerate(rows):
        for e in r["entries"]:
            users.setdefault(e, []).append(i)
    users.pop(-1, None)
    free = [p for p in range(pages) if p not in users and not held[p]]
    writes = [r["keep"] % page_size != 0 and r["new"] > r["keep"] for r in rows]
    deal, copies, missing = iter(free), [], bad
    out = [list(r["entries"]) for r in rows]
    for i, r in enumerate(rows):
        if writes[i] and r["entries"][-1] >= 0:
            page = r["entries"][-1]
            writers = [j for j in range(len(rows)) if writes[j] and rows[j]["entries"][-1] == page]
            if held[page] or len(users[page]) != len(writers) or writers[0] != i:
                to = next(deal, -1)
                out[i][-1] = to
                if to >= 0:
                    copies.append((page, to))
                else:
                    missing += 1
        for _ in range(-(-r["new"] // page_size) - len(r["entries"])):
            to = next(deal, -1)
            missing += to < 0
            out[i].append(to)
    refs = [0] * pages
    for row in out:
        for e in row:
            if e >= 0:
                refs[e] += 1
    new_table = np.array([row + [-1] * (max_blocks - len(row)) for row in out], dtype=np.int32).reshape(len(rows), max_blocks)
    used = sum(1 for p in range(pages) if refs[p] or held[p])
    return new_table, np.array(lens_out, np.int32), np.array(refs, np.int32), [used, missing, len(copies), bad], copies


def compact(table, lens, page_size, pages, held=None):
    """(table, refs, info, moves) of tp_kv_compact."""
    held = [0] * pages if held is None else list(held)
    out = np.full(table.shape, -1, dtype=np.int32)
    bad = 0
    refs = [0] * pages
    for i in range(table.shape[0]):
        n = min(max(int(lens[i]), 0), table.shape[1] * page_size)
        for c in range(-(-n // page_size)):
            p = int(table[i, c])
            if 0 <= p < pages:
                out[i, c] = p
                refs[p] += 1
            else:
                bad += 1
    used = [p for p in range(pages) if refs[p] or held[p]]
    total = len(used)
    src = [p for p in used if p >= total and not held[p]]
    holes = [p for p in range(total) if not refs[p] and not held[p]]
    moves = list(zip(src, holes))
    to = dict(moves)
    for a, b in moves:
        refs[b], refs[a] = refs[a], 0
    out = np.vectorize(lambda p: to.get(int(p), int(p)), otypes=[np.int32])(out) if out.size else out
    return out, np.array(refs, np.int32), [total, bad, len(moves), bad], moves


def beam_select(logits, scores, k, finished=None, eos=-1):
    """(scores, rows, tokens) of tp_beam_select for logits [items, beams, vocab] in float64."""
    items, beams, vocab = logits.shape
    so = np.full((items, k), -np.inf)
    ro, to = np.full((items, k), -1, np.int32), np.full((items, k), -1, np.int32)
    for i in range(items):
        cands = []
        for b in range(beams):
            s = float(scores[i, b])
            if not s > -np.inf:
                continue
            if finished is not None and finished[i, b]:
                cands.append((-s, b, eos))
                continue
            x = logits[i, b]
            with np.errstate(all="ignore"):
                top = x.max()
                lse = top + np.log(np.exp(x - top).sum())
            if not np.isfinite(lse):
                continue
            for v in np.argsort(-x, kind="stable")[:k]:
                if x[v] > -np.inf:
                    cands.append((-((s - lse) + x[v]), b, int(v)))
        for n, (s, b, v) in enumerate(sorted(cands)[:k]):
            so[i, n], ro[i, n], to[i, n] = -s, i * beams + b, v
    return so, ro, to
