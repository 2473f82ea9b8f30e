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
Pins (tests/test_paged_pick_cpu.py):
  page_bounds   -- hand-built pages; every key between its page's bounds, which
                   a code less or the next smaller scale would not hold.
  page_score    -- brute force over the corners of the bounds.
  page_select   -- the contiguous oracle's selection; hand-built ties and NaNs.
  sparse_cells, tree_cells, attn_cells -- paged_attn with all pages listed, with
                   a full mask, and a tree's branches as sequences of their own.
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


def _row_cells(page_table, seq_lens, rows, t, page, err):
    """Table row and length of token t as they count, and whether they were in range."""
    r = t if rows is None else int(rows[t])
    n = int(seq_lens[t])
    if not 0 <= r < page_table.shape[0]:
        return 0, 0, BAD_ID
    most = page_table.shape[1] * page
    return r, min(max(n, 0), most), err | (0 if 0 <= n <= most else BAD_ID)


def page_bounds(page_table, seq_lens, n_new, kq, ksc):
    """{page: (hi_q, lo_q, hi_sc, lo_sc)} of the written pages ([Hkv, D] and [Hkv, 4]), and err."""
    n_pages, page, hkv, d = kq.shape
    most, out, err = page_table.shape[1] * page, {}, 0
    for r in range(page_table.shape[0]):
        n = min(max(int(seq_lens[r]), 0), most)
        new = n if n_new is None else min(max(int(n_new[r]), 0), n)
        err |= BAD_ID if n != int(seq_lens[r]) or (n_new is not None and new != int(n_new[r])) else 0
        for j in range((n - new) // page, -(-n // page) if new else 0):
            p = int(page_table[r, j])
            if not 0 <= p < n_pages:
                err |= BAD_ID
                continue
            filled = min(page, n - j * page)
            sc = ksc[p, :filled].astype(np.float64)
            with np.errstate(invalid="ignore"):
                keys = (kq[p, :filled].astype(np.float64).reshape(filled, hkv, 4, d // 4) * sc[..., None])
            bad = ~np.isfinite(sc).all(0)
            keys = np.where(bad[None, ..., None], 0.0, keys)
            res = []
            for v, outwards in ((keys.max(0), np.ceil), (keys.min(0), np.floor)):
                need = np.abs(v).max(-1) / 127.0
                s16 = need.astype(np.float16)
                s16 = np.where(s16.astype(np.float64) < need, np.nextafter(s16, np.float16(np.inf)), s16).astype(np.float16)
                step = s16.astype(np.float64)[..., None]
                code = outwards(np.divide(v, step, out=np.zeros_like(v), where=step > 0)).astype(np.int8)
                res.append((code.reshape(hkv, d), np.where(bad, np.float16(np.nan), s16)))
            out[p] = (res[0][0], res[1][0], res[0][1], res[1][1])
    return out, err


def page_score(q, hi_q, lo_q, hi_sc, lo_sc, page_table, seq_lens, page, rows=None):
    """Per (token, KV head): the pages' scores, sum |terms| and sum |hi| + |lo|
    (-inf, 0, 0 of a page outside the pool); the largest sum; and err."""
    T, H, D = q.shape
    hkv, err, out = hi_q.shape[1], 0, []
    wide = lambda c, s: c.astype(np.float64) * np.repeat(s.astype(np.float64), D // 4, -1)  # noqa: E731
    hi, lo = wide(hi_q, hi_sc), wide(lo_q, lo_sc)
    for t in range(T):
        r, n, err = _row_cells(page_table, seq_lens, rows, t, page, err)
        x = q[t].astype(np.float64).reshape(hkv, -1, D)
        up, down = np.maximum(x, 0).sum(1), np.minimum(x, 0).sum(1)
        p = page_table[r, : -(-n // page)]
        ok = (p >= 0) & (p < hi_q.shape[0])
        err |= 0 if ok.all() else BAD_ID
        per = []
        for h in range(hkv):
            a, b = hi[np.where(ok, p, 0), h], lo[np.where(ok, p, 0), h]
            per.append((np.where(ok, a @ up[h] + b @ down[h], -np.inf), np.where(ok, np.abs(a) @ up[h] - np.abs(b) @ down[h], 0.0),
                        np.where(ok, (np.abs(a) + np.abs(b)).sum(-1), 0.0), max(up[h].max(), -down[h].min())))
        out.append(per)
    return out, err


def page_select(scores, seq_lens, page, budget, sink, local, width):
    """pages [T, Hkv, width], counts [T, Hkv], err."""
    T, hkv, ld = scores.shape
    pages, counts, err = np.full((T, hkv, width), -1, np.int32), np.zeros((T, hkv), np.int32), 0
    for t in range(T):
        n = -(-int(seq_lens[t]) // page)
        err |= BAD_ID if seq_lens[t] < 0 or n > ld else 0
        n = min(max(n, 0), ld)
        for h in range(hkv):
            forced = [j for j in range(n) if j < sink or j >= n - local]
            free = [j for j in range(n) if sink <= j < n - local]
            rank = lambda j: (1, 0.0, j) if np.isnan(scores[t, h, j]) else (0, -float(scores[t, h, j]), j)  # noqa: E731
            got = list(range(n)) if n <= budget else sorted(forced + sorted(free, key=rank)[: budget - len(forced)])
            pages[t, h, : len(got)] = got
            counts[t, h] = len(got)
    return pages, counts, err


def _pool_cells(page_table, r, cells, page, n_pages, err):
    out = []
    for c in cells:
        p = int(page_table[r, c // page])
        if 0 <= p < n_pages:
            out.append(p * page + c % page)
        else:
            err |= BAD_ID
    return out, err


def sparse_cells(page_table, seq_lens, pages, counts, page, n_pages, rows=None):
    """Pool cells that each (token, KV head) attends to, and err."""
    T, hkv, width = pages.shape
    out, err = [], 0
    for t in range(T):
        r, n, err = _row_cells(page_table, seq_lens, rows, t, page, err)
        per = []
        for h in range(hkv):
            k = int(counts[t, h])
            err |= 0 if 0 <= k <= width else BAD_ID
            cells = []
            for j in pages[t, h, : min(max(k, 0), width)] if n else []:
                if j < -1 or j >= page_table.shape[1]:
                    err |= BAD_ID
                elif j >= 0:
                    cells += [c for c in range(j * page, (j + 1) * page) if c < n]
            cells, err = _pool_cells(page_table, r, cells, page, n_pages, err)
            per.append(cells)
        out.append(per)
    return out, err


def tree_cells(page_table, prefix_lens, mask, hkv, page, n_pages, rows=None):
    """Pool cells that each (token, KV head) attends to, and err."""
    out, err, most = [], 0, page_table.shape[1] * page
    for t in range(len(prefix_lens)):
        r = t if rows is None else int(rows[t])
        if not 0 <= r < page_table.shape[0]:
            out.append([[]] * hkv)
            err |= BAD_ID
            continue
        n = min(max(int(prefix_lens[t]), 0), most)
        err |= 0 if n == int(prefix_lens[t]) else BAD_ID
        cells = list(range(n)) + [n + b for b in range(32 * mask.shape[1]) if int(mask[t, b // 32]) >> (b % 32) & 1]
        err |= BAD_ID if cells and cells[-1] >= most else 0
        cells, err = _pool_cells(page_table, r, [c for c in cells if c < most], page, n_pages, err)
        out.append([cells] * hkv)
    return out, err


def attn_cells(q, kq, vq, ksc, vsc, cells, scale=None, gate=None):
    """attn's numbers, of listed pool cells: cells[t][KV head]."""
    T, H, D = q.shape
    hkv = kq.shape[2]
    per = H // hkv
    scale = 1.0 / np.sqrt(D) if scale is None else scale
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    mag, flush, qk = np.zeros((T, H, D)), np.zeros((T, H, D)), np.zeros((T, H))
    flat = [x.reshape(-1, *x.shape[2:]) for x in (kq, vq, ksc, vsc)]
    for t in range(T):
        for k in range(hkv):
            at = np.asarray(cells[t][k], dtype=np.int64)
            if not len(at):
                continue
            codes, values, ks, vs = (x[at, k].astype(np.float64) for x in flat)
            heads = slice(k * per, (k + 1) * per)
            x = q[t, heads].astype(np.float64)
            keys, v = codes * np.repeat(ks, D // 4, -1), values * np.repeat(vs, D // 4, -1)
            s = x @ keys.T * scale
            m = s.max(-1, keepdims=True)
            w = np.exp(s - m)
            L = w.sum(-1, keepdims=True)
            out[t, heads], mag[t, heads] = w @ v / L, w @ np.abs(v) / L
            lse[t, heads] = (m + np.log(L))[:, 0]
            flush[t, heads] = np.abs(values).sum(0) * vs.max() / L
            qk[t, heads] = abs(scale) * (np.abs(x).reshape(per, 4, -1).sum(-1) @ ks.T).max(-1)
    if gate is not None:
        sg = 1.0 / (1.0 + np.exp(-np.asarray(gate, dtype=np.float64)))
        out, mag, flush = out * sg, mag * sg, flush * sg
    return out, lse, mag, flush, qk
