"""CPU oracle of the paged cache's calls (test infrastructure only).

Plain loops over the definitions: float64 arithmetic for the numbers, Python
integers for the page tables.  Shares no code with the GPU path.

Pins (tests/test_paged_cpu.py):
  paged_prep    -- the contiguous oracle's prep (queries) and quantiser (rows)
                   on the same tokens; interleaved pairs against the half
                   layout under the permutation that maps one to the other;
                   pair norms under rotation; padding tokens.
  paged_attn    -- the contiguous oracle's attention over all cells.
  page_update   -- hand-built tables: growth, fork with a shared last page,
                   reorder, free, an exhausted pool; invariants on random ones.
  page_compact  -- a hand-built table; contents of every row kept.
"""
from __future__ import annotations

import numpy as np

NO_PAGES, BAD_ID = 4, 1


def rotate(y, pos, inv_freq, interleaved=False, mscale=1.0):
    """y [T, H, D] float64 with its first 2 len(inv_freq) dims rotated by
    pos * inv_freq."""
    n = len(inv_freq)
    out = y.copy()
    for i in range(n):
        a = np.asarray(pos, dtype=np.float64) * float(inv_freq[i])
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        out[..., p] = mscale * (y[..., p] * c - y[..., q] * s)
        out[..., q] = mscale * (y[..., q] * c + y[..., p] * s)
    return out


def norm_rotate(x, w, pos, inv_freq, interleaved=False, mscale=1.0, eps=1e-6):
    y = np.asarray(x, dtype=np.float64)
    if w is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    return rotate(y, pos, inv_freq, interleaved, mscale) if inv_freq is not None else y


def attn(q, kq, vq, ksc, vsc, page_table, seq_lens, rows=None, scale=None, gate=None):
    """q [T, H, D]; kq [pages, page, Hkv, D] ...  Returns out, lse (float64) and
    per (token, head) the sums that bound a kernel's rounding: sum w|v| / L per
    dim, sum |code| * (largest V scale) / L per dim, and the largest score
    bound scale * sum_g ksc * sum |q| (the caller multiplies by its steps)."""
    T, H, D = q.shape
    page, hkv = kq.shape[1], kq.shape[2]
    per, grp = H // hkv, D // 4
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    mag, flush, qk = np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros((T, H))
    for t in range(T):
        r = t if rows is None else int(rows[t])
        n = min(max(int(seq_lens[t]), 0), page_table.shape[1] * page) if 0 <= r < page_table.shape[0] else 0
        c = np.arange(n)
        pg = page_table[r, c // page] if n else np.zeros(0, int)
        ok = (pg >= 0) & (pg < kq.shape[0])
        pg, at = pg[ok], (c % page)[ok]
        if not len(pg):
            continue
        for h in range(H):
            k = h // per
            ks, vs = ksc[pg, at, k].astype(np.float64), vsc[pg, at, k].astype(np.float64)
            code = vq[pg, at, k].astype(np.float64)
            K = kq[pg, at, k].astype(np.float64) * np.repeat(ks, grp, -1)
            V = code * np.repeat(vs, grp, -1)
            qd = q[t, h].astype(np.float64)
            s = K @ qd * scale
            m = s.max()
            w = np.exp(s - m)
            L = w.sum()
            out[t, h] = w @ V / L
            lse[t, h] = m + np.log(L)
            mag[t, h] = w @ np.abs(V) / L
            flush[t, h] = np.abs(code).sum(0) * vs.max() / L
            qk[t, h] = abs(scale) * (ks @ np.abs(qd).reshape(4, grp).sum(-1)).max()
    if gate is not None:
        sg = 1.0 / (1.0 + np.exp(-np.asarray(gate, dtype=np.float64)))
        out, mag, flush = out * sg, mag * sg, flush * sg
    return out, lse, mag, flush, qk


def _entry(e, n_pages):
    return int(e) if 0 <= e < n_pages else -1


def page_update(page_table, seq_lens, src, n_new, n_pages, page, n_slots):
    """Returns table, lens, refs, slots, positions, copies [(src, dst, cells)], err."""
    wide = page_table.shape[1]
    rows = len(n_new)
    err = 0
    table, keep = [], []
    for r in range(rows):
        f = r if src is None else int(src[r])
        if not 0 <= f < page_table.shape[0]:
            err |= BAD_ID if f != -1 else 0
            table.append([])
            keep.append(0)
            continue
        n = int(seq_lens[f])
        if not 0 <= n <= wide * page:
            err |= BAD_ID
            n = min(max(n, 0), wide * page)
        entries = [_entry(e, n_pages) for e in page_table[f, : -(-n // page)]]
        err |= BAD_ID if -1 in entries else 0
        table.append(entries)
        keep.append(n)
    refs = [0] * n_pages
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    free = [p for p in range(n_pages) if refs[p] == 0]
    held_before = list(refs)
    slots, positions = [-1] * n_slots, [-1] * n_slots
    copies, lens = [], list(keep)
    off = asked = 0
    for r in range(rows):
        n = int(n_new[r])
        if n < 0:
            err |= BAD_ID
            n = 0
        if n == 0:
            continue
        had, want, tail = len(table[r]), -(-(keep[r] + n) // page), keep[r] % page
        copy = tail > 0 and table[r][-1] >= 0 and held_before[table[r][-1]] > 1
        need = want - had + copy
        fits = want <= wide and off + n <= n_slots
        if fits:
            asked += need
        if not fits or (need and asked > len(free)):
            err |= NO_PAGES
            off += n
            continue
        got = free[asked - need: asked]
        if copy:
            copies.append((table[r][-1], got[0], tail))
            table[r][-1] = got[0]
            got = got[1:]
        table[r] = table[r] + got
        for i in range(n):
            p = keep[r] + i
            e = table[r][p // page]
            slots[off + i] = e * page + p % page if e >= 0 else -1
            positions[off + i] = p
        lens[r] = keep[r] + n
        off += n
    refs = [0] * n_pages
    for row in table:
        for e in row:
            if e >= 0:
                refs[e] += 1
    full = np.full((rows, wide), -1, dtype=np.int32)
    for r, row in enumerate(table):
        full[r, : len(row)] = row
    i32 = lambda v: np.asarray(v, dtype=np.int32)  # noqa: E731
    return full, i32(lens), i32(refs), i32(slots), i32(positions), copies, err


def page_compact(page_table, seq_lens, n_pages, page):
    """Returns table, refs, page_map, n_live, moves [(src, dst)], err."""
    wide = page_table.shape[1]
    err = 0
    rows = []
    for r in range(page_table.shape[0]):
        n = int(seq_lens[r])
        if not 0 <= n <= wide * page:
            err |= BAD_ID
            n = min(max(n, 0), wide * page)
        entries = [_entry(e, n_pages) for e in page_table[r, : -(-n // page)]]
        err |= BAD_ID if -1 in entries else 0
        rows.append(entries)
    refs = np.zeros(n_pages, dtype=np.int32)
    for row in rows:
        for e in row:
            if e >= 0:
                refs[e] += 1
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] == 0]
    movers = [p for p in range(live, n_pages) if refs[p] > 0]
    to = {p: p for p in range(live) if refs[p] > 0}
    to.update(zip(movers, holes))
    page_map = np.array([to.get(p, -1) for p in range(n_pages)], dtype=np.int32)
    table = np.full(page_table.shape, -1, dtype=np.int32)
    new_refs = np.zeros(n_pages, dtype=np.int32)
    for r, row in enumerate(rows):
        for j, e in enumerate(row):
            table[r, j] = to[e] if e >= 0 else -1
    for p, q in to.items():
        new_refs[q] = refs[p]
    return table, new_refs, page_map, live, list(zip(movers, holes)), err
