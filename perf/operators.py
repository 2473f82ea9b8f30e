"""Cases for the paged-cache operators: what a serving loop calls on them, at the sizes it calls them.

The cache is a pool of pages of int8 K/V codes with four fp16 scales per row (one per quarter of the head dim),
shared by all sequences through a page table.  Five operators work on it:

  prep     norm and rotation of the new tokens' query and key heads, and quantised K/V rows into their slots
           (with the rows read back as the values they stand for)
  gather   cached rows of listed cells as fp16, bf16 or fp32 values
  attn     attention of one new token per row over the row's whole cached length
  update   the batch's next page table: fork, reorder, free and extend, copying shared last pages before a write
  compact  live pages moved to the lowest page numbers

`own` is False for the plain form (elementary torch operations) and True for the framework's own calls.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # The next token of one conversation: what a decode step waits for first.
        {"name": "prep one token", "op": "prep", "tokens": 1, "hq": 12, "hkv": 1, "d": 128, "type": "fp16", "out": "fp16",
         "rope": 64, "layout": "half", "factor": 1.0, "norm": True, "page": 64, "pos0": 320, "skip": 0},
        # A prompt chunk of 1984 tokens at a far position, the rotation over half of the head.
        {"name": "prep prompt chunk", "op": "prep", "tokens": 1984, "hq": 12, "hkv": 1, "d": 128, "type": "bf16", "out": "fp16",
         "rope": 64, "layout": "half", "factor": 1.0, "norm": True, "page": 64, "pos0": 30000, "skip": 0},
        # Several prompts in one packed batch of wide heads, interleaved rotation stretched for long contexts,
        # and places that the batch does not use.
        {"name": "prep packed prompts", "op": "prep", "tokens": 8191, "hq": 24, "hkv": 2, "d": 256, "type": "bf16", "out": "bf16",
         "rope": 256, "layout": "interleaved", "factor": 8.0, "norm": True, "page": 32, "pos0": 100000, "skip": 17},
        # The decode window of one token, read back.
        {"name": "gather one window", "op": "gather", "cells": 321, "hkv": 1, "d": 128, "out": "fp16", "page": 64,
         "paged": True},
        # Shared prefixes of eight prompts read back for their prompt attention.
        {"name": "gather prefixes", "op": "gather", "cells": 240061, "hkv": 2, "d": 256, "out": "bf16", "page": 32,
         "paged": True},
        # The smallest decode: one conversation of 321 cells.
        {"name": "attn one row", "op": "attn", "rows": 1, "share": 1, "lo": 321, "hi": 321, "hq": 12, "hkv": 1, "d": 128,
         "type": "fp16", "page": 64, "gate": False},
        # A window of eight draft tokens of one long conversation, wide heads, gated.
        {"name": "attn draft window", "op": "attn", "rows": 8, "share": 8, "lo": 30001, "hi": 30008, "hq": 24, "hkv": 2, "d": 256,
         "type": "bf16", "page": 16, "gate": True},
        # A full decode batch, conversations of all lengths up to 32 K cells.
        {"name": "attn ragged batch", "op": "attn", "rows": 61, "share": 1, "lo": 1, "hi": 32701, "hq": 48, "hkv": 4, "d": 128,
         "type": "fp16", "page": 64, "gate": False},
        # One decode step of a batch: every row grows by one token, some into a new page.
        {"name": "update decode step", "op": "update", "rows": 64, "parents": 64, "len": 2000, "grow": 1, "layers": 4,
         "hkv": 1, "d": 128, "page": 64, "spare": 128},
        # A beam step: 256 beams take their parents' pages, and each gets its own copy of the last page.
        {"name": "update beam step", "op": "update", "rows": 256, "parents": 64, "len": 4000, "grow": 1, "layers": 16,
         "hkv": 2, "d": 128, "page": 128, "spare": 512},
        # A small pool after a few conversations ended.
        {"name": "compact small pool", "op": "compact", "rows": 9, "len": 400, "layers": 2, "hkv": 1, "d": 128, "page": 16,
         "pages": 701},
        # A large pool, half of it free, before it is cut to what is used.
        {"name": "compact large pool", "op": "compact", "rows": 120, "len": 2100, "layers": 8, "hkv": 2, "d": 128, "page": 64,
         "pages": 8000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep", "gather", "attn", "update", "compact"])
    d = rng.choice([128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op == "prep":
        hkv = rng.choice([1, 2, 4])
        per = rng.choice([1, 4, 6, 8, 12])
        tokens = _log(rng, 1, 8191 * 28 * 256 // ((per + 2) * hkv * d))
        return {"op": op, "tokens": min(tokens, 16000), "hq": per * hkv, "hkv": hkv, "d": d,
                "type": rng.choice(["fp16", "bf16", "fp32"]), "out": rng.choice(["fp16", "bf16"]),
                "rope": rng.choice([0, 32, 64, d // 2, d]), "layout": rng.choice(["half", "interleaved"]),
                "factor": rng.choice([1.0, 4.0, 8.0]), "norm": rng.choice([True, True, False]), "page": page,
                "pos0": _log(rng, 1, 200000), "skip": rng.choice([0, 7, 19])}
    if op == "gather":
        hkv = rng.choice([1, 2, 4])
        return {"op": op, "cells": _log(rng, 1, 240000 * 512 // (hkv * d)), "hkv": hkv, "d": d,
                "out": rng.choice(["fp16", "bf16"]), "page": page, "paged": rng.choice([True, False])}
    if op == "attn":
        hkv = rng.choice([1, 2, 4, 8])
        per = rng.choice([1, 2, 4, 6, 8, 12, 16])
        rows = _log(rng, 1, 200)
        most = min(32700, 61 * 16000 * 4 * 128 // (rows * hkv * d))
        hi = _log(rng, 1, max(2, most))
        return {"op": op, "rows": rows, "share": rng.choice([1, 1, 4]), "lo": rng.randint(0, hi), "hi": hi, "hq": per * hkv,
                "hkv": hkv, "d": d, "type": rng.choice(["fp16", "bf16"]), "page": page, "gate": rng.choice([False, True])}
    if op == "update":
        rows = _log(rng, 1, 200)
        return {"op": op, "rows": rows, "parents": rng.randint(1, rows), "len": _log(rng, 1, 4000), "grow": rng.choice([0, 1, 1, 7, 130]),
                "layers": rng.choice([1, 2, 4]), "hkv": rng.choice([1, 2]), "d": 128, "page": page, "spare": rng.randint(3, 600)}
    rows = _log(rng, 1, 120)
    length = _log(rng, 1, 2100)
    need = rows * (-(-length // page))
    return {"op": op, "rows": rows, "len": length, "layers": rng.choice([1, 2, 8]), "hkv": rng.choice([1, 2]), "d": 128, "page": page,
            "pages": need + rng.randint(1, max(2, min(need, 4000)))}


# ---------------------------------------------------------------- inputs

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def _spread(n, lo, hi):
    """n whole numbers over lo .. hi, mixed up, the same for every seed."""
    if n == 1:
        return np.array([hi], dtype=np.int64)
    f = (np.arange(n) * 0.6180339887498949 + 0.37) % 1.0
    v = lo + np.floor(f * (hi - lo + 1)).astype(np.int64)
    v[0], v[-1] = lo, hi
    return v


def _inv_freq(rope, factor, theta=10000.0, context=4096, fast=32.0, slow=1.0):
    """Frequencies of a rotation over `rope` dims; with factor > 1 the slow ones are stretched by it, the fast ones are
    kept, and those between (by turns over the trained context) go from one to the other."""
    i = np.arange(rope // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / max(rope, 1))
    if factor != 1.0:
        turns = context * f / (2.0 * math.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
    return f.astype(np.float32)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _pool(g, layers, pages, page, hkv, d):
    shape = (layers, pages, page, hkv)
    codes = [torch.randint(-127, 128, shape + (d,), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
    scales = [(torch.rand(shape + (4,), generator=g, device="cuda") * 0.019 + 0.001).half() for _ in range(2)]
    return {"kq": codes[0], "vq": codes[1], "ksc": scales[0], "vsc": scales[1]}


def _table(g, lens, page, pages, wide):
    """Pages for rows of these lengths, from a shuffled pool, and -1 behind them."""
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    held = -(-np.asarray(lens) // page)
    at = torch.as_tensor(np.concatenate([[0], np.cumsum(held)[:-1]]), device="cuda")
    held = torch.as_tensor(held, device="cuda")
    j = torch.arange(wide, device="cuda")
    idx = (at[:, None] + j[None]).clamp(max=pages - 1)
    return torch.where(j[None] < held[:, None], order[idx], torch.full_like(order[idx], -1)).contiguous()


def _attn_lens(c):
    """Cached cells each row attends to, and the sequence that holds them."""
    n, share = c["rows"], c["share"]
    seqs = -(-n // share)
    if share == 1:
        lens = _spread(n, c["lo"], c["hi"])
        return lens, np.arange(n), lens
    # Rows of one sequence are consecutive tokens of it: row k of `share` sees k cells more than the first.
    base = np.maximum(_spread(seqs, c["lo"], c["hi"]) - share + 1, 0)
    seq = np.arange(n) // share
    return base[seq] + np.arange(n) % share, seq, base + share - 1


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    i32 = lambda v: torch.as_tensor(np.asarray(v), device="cuda", dtype=torch.int32)  # noqa: E731
    if c["op"] == "prep":
        t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
        pages = -(-t // c["page"]) + 3
        s.update(_pool(g, 1, pages, c["page"], hkv, d))
        # One projection's output; q, k and v are views of it.
        x = torch.randn(t, hq + 2 * hkv, d, generator=g, device="cuda")
        x = x * torch.exp(torch.randn(t, hq + 2 * hkv, 1, generator=g, device="cuda"))
        x = x.to(_TYPES[c["type"]])
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        s["wq"] = torch.rand(d, generator=g, device="cuda") + 0.5 if c["norm"] else None
        s["wk"] = torch.rand(d, generator=g, device="cuda") + 0.5 if c["norm"] else None
        s["freq"] = torch.as_tensor(_inv_freq(c["rope"], c["factor"]), device="cuda") if c["rope"] else None
        s["pos"] = (c["pos0"] + torch.arange(t, device="cuda")).to(torch.int32)
        order = torch.randperm(pages, generator=g, device="cuda")
        tok = torch.arange(t, device="cuda")
        slots = order[tok // c["page"]] * c["page"] + tok % c["page"]
        if c["skip"]:
            slots = torch.where(tok % c["skip"] == c["skip"] - 1, torch.full_like(slots, -1), slots)
        s["slots"] = slots.to(torch.int32)
        s["qo"] = torch.zeros(t, hq, d, device="cuda", dtype=_TYPES[c["out"]])
        s["ko"], s["vo"] = (torch.empty(t, hkv, d, device="cuda", dtype=torch.float16) for _ in range(2))
    elif c["op"] == "gather":
        n, hkv, d = c["cells"], c["hkv"], c["d"]
        seqs = min(8, n)
        lens = np.full(seqs, n // seqs)
        lens[: n % seqs] += 1
        wide = -(-int(lens.max()) // c["page"])
        pages = int((-(-lens // c["page"])).sum()) + 5
        s.update(_pool(g, 1, pages, c["page"], hkv, d))
        s["table"] = _table(g, lens, c["page"], pages, wide)
        ids = i32(np.concatenate([np.arange(v) for v in lens]))
        rows = i32(np.repeat(np.arange(seqs), lens))
        if not c["paged"]:  # the cells' own numbers, as the update gives them
            ids = (s["table"][rows.long(), ids.long() // c["page"]] * c["page"] + ids % c["page"]).to(torch.int32)
        ids = torch.where(torch.arange(n, device="cuda") % 97 == 96, torch.full_like(ids, -1), ids)
        s["ids"], s["rows"] = ids, rows
        s["ko"], s["vo"] = (torch.empty(n, hkv, d, device="cuda", dtype=_TYPES[c["out"]]) for _ in range(2))
    elif c["op"] == "attn":
        n, hq, hkv, d = c["rows"], c["hq"], c["hkv"], c["d"]
        lens, seq, held = _attn_lens(c)
        s["most"] = max(1, int(lens.max()))
        wide = -(-max(1, int(held.max())) // c["page"])
        pages = int((-(-held // c["page"])).sum()) + 3
        s.update(_pool(g, 1, pages, c["page"], hkv, d))
        s["table"] = _table(g, held, c["page"], pages, wide)
        s["lens"] = i32(lens)
        s["rows"] = i32(seq) if c["share"] > 1 else None
        q = torch.randn(n, hq, d, generator=g, device="cuda") * (0.5 + 2.5 * torch.rand(1, hq, 1, generator=g, device="cuda"))
        s["q"] = q.to(_TYPES[c["type"]])
        s["gate"] = 2.0 * torch.randn(n, hq, d, generator=g, device="cuda") if c["gate"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(n, hq, device="cuda")
        if own:
            import sparse_selected_attention_gb300 as qsa
            s["ws"] = torch.empty(qsa.qsa_paged_attn_workspace_bytes(hq, hkv, d), dtype=torch.uint8, device="cuda")
    else:
        page, layers, hkv, d = c["page"], c["layers"], c["hkv"], c["d"]
        if c["op"] == "update":
            parents, rows = c["parents"], c["rows"]
            lens = np.maximum(_spread(parents, c["len"] // 2, c["len"]), 0)
            wide = -(-(c["len"] + c["grow"]) // page) + 1
            pages = int((-(-lens // page)).sum()) + c["spare"]
            s["src"] = i32(np.where(np.arange(rows) % 11 == 10, -1, np.arange(rows) % parents))
            s["new"] = i32(np.where(np.arange(rows) % 7 == 6, 0, c["grow"]))
            cap = max(1, int(s["new"].sum()))
            s["slots"], s["pos"] = (torch.empty(cap, device="cuda", dtype=torch.int32) for _ in range(2))
            s["lens_out"] = torch.empty(rows, device="cuda", dtype=torch.int32)
        else:
            rows, pages = c["rows"], c["pages"]
            lens = np.maximum(_spread(rows, c["len"] // 2, c["len"]), 0)
            wide = -(-c["len"] // page)
            s["map"] = torch.empty(pages, device="cuda", dtype=torch.int32)
            s["live"] = torch.empty(1, device="cuda", dtype=torch.int32)
        s.update(_pool(g, layers, pages, page, hkv, d))
        s["table"], s["lens"] = _table(g, lens, page, pages, wide), i32(lens)
        if c["op"] == "compact" and rows > 2:  # the second row is a fork of the first: it holds the same pages
            s["table"][1] = s["table"][0]
            s["lens"][1] = s["lens"][0]
        s["table_out"] = torch.empty(rows, wide, device="cuda", dtype=torch.int32)
        s["refs"] = torch.empty(pages, device="cuda", dtype=torch.int32)
        if own:
            import sparse_selected_attention_gb300 as qsa
            s["ws"] = torch.empty(qsa.qsa_pages_workspace_bytes(rows, pages), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def _rotate(y, pos, freq, layout):
    """Rotates the first 2 * len(freq) dims of y [T, H, D]; the angles in 64 bits, since far positions need them."""
    a = pos.double()[:, None] * freq.double()[None]
    cos, sin = a.cos().to(y.dtype)[:, None], a.sin().to(y.dtype)[:, None]
    n = freq.numel()
    if layout == "half":
        x0, x1 = y[..., :n], y[..., n:2 * n]
        rot = torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    else:
        x0, x1 = y[..., 0:2 * n:2], y[..., 1:2 * n:2]
        rot = torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)
    return torch.cat([rot, y[..., 2 * n:]], -1)


def _quantise(y):
    """Codes and scales of rows y [T, H, D], a scale per quarter."""
    t, h, d = y.shape
    x = y.reshape(t, h, 4, d // 4)
    sc = (x.abs().amax(-1) / 127.0).half()
    f = sc.float()[..., None]
    code = torch.where(f == 0, torch.zeros_like(x), (x / torch.where(f == 0, torch.ones_like(f), f)).round().clamp(-127, 127))
    return code.reshape(t, h, d).to(torch.int8), sc


def _values(codes, scales):
    """codes [..., D] times scales [..., 4], in fp32."""
    x = codes.float().unflatten(-1, (4, codes.shape[-1] // 4))
    return (x * scales.float()[..., None]).flatten(-2)


def _plain_prep(s):
    c = s["c"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6) * s["wq"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + 1e-6) * s["wk"]
    if c["rope"]:
        q, k = (_rotate(x, s["pos"], s["freq"], c["layout"]) for x in (q, k))
    used = s["slots"] >= 0
    at = s["slots"][used].long()
    s["qo"][used] = q[used].to(s["qo"].dtype)
    flat = {n: s[n][0].flatten(0, 1) for n in ("kq", "vq", "ksc", "vsc")}
    flat["kq"][at], flat["ksc"][at] = _quantise(k[used])
    flat["vq"][at], flat["vsc"][at] = _quantise(v[used])
    back = s["slots"].clamp(min=0).long()
    ko, vo = _values(flat["kq"][back], flat["ksc"][back]), _values(flat["vq"][back], flat["vsc"][back])
    zero = used[:, None, None]
    return s["qo"], torch.where(zero, ko, 0.0 * ko).half(), torch.where(zero, vo, 0.0 * vo).half()


def _plain_gather(s):
    c = s["c"]
    ids = s["ids"].long()
    used = (ids >= 0)[:, None, None]
    ids = ids.clamp(min=0)
    if c["paged"]:
        ids = s["table"][s["rows"].long(), ids // c["page"]].long() * c["page"] + ids % c["page"]
    flat = {n: s[n][0].flatten(0, 1) for n in ("kq", "vq", "ksc", "vsc")}
    out = []
    for codes, scales in (("kq", "ksc"), ("vq", "vsc")):
        x = _values(flat[codes][ids], flat[scales][ids])
        out.append(torch.where(used, x, torch.zeros_like(x)).to(_TYPES[c["out"]]))
    return tuple(out)


def _plain_attn(s):
    c = s["c"]
    n, hq, hkv, d = c["rows"], c["hq"], c["hkv"], c["d"]
    table = s["table"] if s["rows"] is None else s["table"][s["rows"].long()]
    page = table.clamp(min=0).long()
    most = s["most"]
    kv = []
    for codes, scales in (("kq", "ksc"), ("vq", "vsc")):
        x = s[codes][0][page].flatten(1, 2)[:, :most]
        kv.append(_values(x, s[scales][0][page].flatten(1, 2)[:, :most]).transpose(1, 2))  # [n, hkv, cells, d]
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    logits = torch.matmul(q, kv[0].transpose(-1, -2)) / math.sqrt(d)
    seen = torch.arange(most, device="cuda")[None] < s["lens"][:, None]
    logits = logits.masked_fill(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(logits - top)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, kv[1]) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (torch.log(total) + top).view(n, hq)
    o = o.reshape(n, hq, d)
    if s["gate"] is not None:
        o = o / (1.0 + torch.exp(-s["gate"]))
    return o.to(s["q"].dtype), lse


def _counts(table, pages):
    held = table.flatten()
    return torch.bincount(held[held >= 0], minlength=pages).to(torch.int32)


def _plain_update(s):
    page = s["c"]["page"]
    pages, wide, cap = s["refs"].numel(), s["table"].shape[1], s["slots"].numel()
    j = torch.arange(wide, device="cuda")[None]
    src = s["src"].long()
    keep = torch.where(src >= 0, s["lens"][src.clamp(min=0)].long(), torch.zeros_like(src))
    had = (keep + page - 1) // page
    table = torch.where(j < had[:, None], s["table"][src.clamp(min=0)].long(), torch.full_like(j, -1))
    refs = _counts(table, pages)
    new = s["new"].long()
    end = torch.cumsum(new, 0)
    tail, last = keep % page, (keep // page).clamp(max=wide - 1)
    held = table.gather(1, last[:, None])[:, 0]
    shared = (new > 0) & (tail > 0) & (refs[held.clamp(min=0)] > 1)
    want = (keep + new + page - 1) // page
    fits = (want <= wide) & (end <= cap)
    need = torch.where(fits & (new > 0), want - had + shared, torch.zeros_like(want))
    upto = torch.cumsum(need, 0)
    ok = (new > 0) & fits & ((need == 0) | (upto <= (refs == 0).sum()))
    free = torch.argsort((refs > 0).int(), stable=True)  # the free pages first, lowest first
    first = (upto - need)[:, None]
    got = first + shared[:, None] + j - had[:, None]
    out = torch.where(ok[:, None] & (j >= had[:, None]) & (j < want[:, None]), free[got.clamp(0, pages - 1)], table)
    out = torch.where((ok & shared)[:, None] & (j == last[:, None]), free[first.clamp(max=pages - 1)], out)
    s["lens_out"].copy_(keep + torch.where(ok, new, torch.zeros_like(new)))
    i = torch.arange(cap, device="cuda")
    row = torch.searchsorted(end, i, right=True).clamp(max=end.numel() - 1)
    at = keep[row] + i - (end - new)[row]
    good = ok[row] & (i < end[-1])
    cell = out[row, (at // page).clamp(0, wide - 1)] * page + at % page
    s["slots"].copy_(torch.where(good, cell, torch.full_like(cell, -1)))
    s["pos"].copy_(torch.where(good, at, torch.full_like(at, -1)))
    r = torch.nonzero(ok & shared)[:, 0]
    a, b = held[r], out[r, last[r]]
    part = (torch.arange(page, device="cuda")[None] < tail[r][:, None])[None, :, :, None, None]
    for n in ("kq", "vq", "ksc", "vsc"):
        s[n][:, b] = torch.where(part, s[n][:, a], s[n][:, b])
    s["table_out"].copy_(out)
    s["refs"].copy_(_counts(out, pages))


def _plain_compact(s):
    page, pages = s["c"]["page"], s["refs"].numel()
    had = (s["lens"].long() + page - 1) // page
    j = torch.arange(s["table"].shape[1], device="cuda")[None]
    table = torch.where(j < had[:, None], s["table"].long(), torch.full_like(j, -1))
    refs = _counts(table, pages)
    p = torch.arange(pages, device="cuda")
    live = (refs > 0).sum()
    holes, movers = p[(refs == 0) & (p < live)], p[(refs > 0) & (p >= live)]
    to = torch.where(refs > 0, p, torch.full_like(p, -1))
    to[movers] = holes
    for n in ("kq", "vq", "ksc", "vsc"):
        s[n][:, holes] = s[n][:, movers]
    out = torch.where(table >= 0, to[table.clamp(min=0)], table)
    s["table_out"].copy_(out)
    s["map"].copy_(to)
    s["live"].copy_(live[None])
    s["refs"].copy_(_counts(out, pages))


def _own(s):
    import sparse_selected_attention_gb300 as qsa
    c = s["c"]
    pool = (s["kq"], s["vq"], s["ksc"], s["vsc"])
    layer = tuple(x[0] for x in pool)
    if c["op"] == "prep":
        qsa.qsa_paged_prep(s["q"], s["k"], s["v"], s["pos"], s["slots"], *layer, s["qo"], q_norm_w=s["wq"], k_norm_w=s["wk"],
                           inv_freq=s["freq"], interleaved=c["layout"] == "interleaved")
        qsa.qsa_paged_gather(*layer, s["slots"], s["ko"], s["vo"])
        return s["qo"], s["ko"], s["vo"]
    if c["op"] == "gather":
        if c["paged"]:
            qsa.qsa_paged_gather(*layer, s["ids"], s["ko"], s["vo"], rows=s["rows"], page_table=s["table"])
        else:
            qsa.qsa_paged_gather(*layer, s["ids"], s["ko"], s["vo"])
        return s["ko"], s["vo"]
    if c["op"] == "attn":
        qsa.qsa_paged_attn(s["q"], *layer, s["table"], s["lens"], s["out"], s["ws"], rows=s["rows"], gate=s["gate"], lse=s["lse"])
        return s["out"], s["lse"]
    if c["op"] == "update":
        qsa.qsa_page_update(s["table"], s["lens"], s["src"], s["new"], *pool, s["table_out"], s["lens_out"], s["refs"], s["slots"],
                            s["pos"], s["ws"])
        return (s["table_out"], s["lens_out"], s["refs"], s["slots"], s["pos"]) + pool
    qsa.qsa_page_compact(s["table"], s["lens"], *pool, s["table_out"], s["refs"], s["map"], s["live"], s["ws"])
    return (s["table_out"], s["refs"], s["map"], s["live"]) + pool


def run(state):
    s = state
    if own:
        return _own(s)
    op = s["c"]["op"]
    if op == "prep":
        return _plain_prep(s)
    if op == "gather":
        return _plain_gather(s)
    if op == "attn":
        return _plain_attn(s)
    pool = (s["kq"], s["vq"], s["ksc"], s["vsc"])
    if op == "update":
        _plain_update(s)
        return (s["table_out"], s["lens_out"], s["refs"], s["slots"], s["pos"]) + pool
    _plain_compact(s)
    return (s["table_out"], s["refs"], s["map"], s["live"]) + pool


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    row = c["hkv"] * (2 * c["d"] + 16)  # K and V of one cell: codes and scales
    size = {"fp16": 2, "bf16": 2, "fp32": 4}
    if c["op"] == "prep":
        t = c["tokens"]
        used = t - (t // c["skip"] if c["skip"] else 0)
        a = used * (c["hq"] + 2 * c["hkv"]) * c["d"]
        return {"bytes": a * size[c["type"]] + used * (c["hq"] * c["d"] * 2 + row) + t * (2 * c["hkv"] * c["d"] * 2 + 8),
                "flops": 10 * a}
    if c["op"] == "gather":
        used = c["cells"] - c["cells"] // 97
        return {"bytes": used * row + c["cells"] * (2 * c["hkv"] * c["d"] * size[c["out"]] + 8), "flops": 2 * used * c["hkv"] * c["d"]}
    if c["op"] == "attn":
        lens, _, held = _attn_lens(c)
        read = int((held if c["share"] > 1 else lens).sum()) * row
        return {"bytes": read + c["rows"] * c["hq"] * (c["d"] * (8 if c["gate"] else 4) + 4), "flops": 4 * int(lens.sum()) * c["hq"] * c["d"]}
    page = c["page"]
    if c["op"] == "update":
        lens = _spread(c["parents"], c["len"] // 2, c["len"])
        src = np.where(np.arange(c["rows"]) % 11 == 10, -1, np.arange(c["rows"]) % c["parents"])
        new = np.where(np.arange(c["rows"]) % 7 == 6, 0, c["grow"])
        keep = np.where(src >= 0, lens[src], 0)
        holders = np.bincount(src[src >= 0], minlength=c["parents"])
        copied = np.where((new > 0) & (src >= 0) & (holders[src] > 1), keep % page, 0).sum()
        entries = -(-lens // page)
        pages = int(entries.sum()) + c["spare"]
        wide = -(-(c["len"] + c["grow"]) // page) + 1
        return {"bytes": int(entries.sum()) * 4 + c["rows"] * (wide * 4 + 16) + pages * 4 + int(new.sum()) * 8 + 2 * int(copied) * c["layers"] * row,
                "flops": 0}
    lens = _spread(c["rows"], c["len"] // 2, c["len"])
    held = -(-lens // page)
    if c["rows"] > 2:
        held[1] = 0
    live = int(held.sum())
    moved = live * (c["pages"] - live) // c["pages"]  # of a shuffled pool
    return {"bytes": c["rows"] * -(-c["len"] // page) * 8 + c["pages"] * 8 + 2 * moved * page * c["layers"] * row, "flops": 0}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_cells(s, codes, scales, cells):
    """code * scale of these cells of a pool's first layer, in 64 bits."""
    x = s[codes][0].flatten(0, 1)[cells].double()
    w = s[scales][0].flatten(0, 1)[cells].double()
    return x * w.repeat_interleave(x.shape[-1] // 4, -1)


def _exact_head(x, w, pos, freq, interleaved):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * w.double()
    if freq is not None:
        m = freq.numel()
        first = torch.arange(m, device="cuda") * (2 if interleaved else 1)
        second = first + (1 if interleaved else m)
        turn = torch.polar(torch.ones(pos.numel(), m, dtype=torch.float64, device="cuda"), torch.outer(pos.double(), freq.double()))
        z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
        x = x.clone()
        x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_kept(x):
    """What the cache holds of rows x: whole multiples of a quarter's fp16 scale."""
    parts = []
    for y in x.chunk(4, -1):
        sc = (y.abs().max(-1, keepdim=True).values / 127.0).to(torch.float16).double()
        parts.append(torch.where(sc > 0, torch.clamp(torch.round(y / sc.clamp(min=1e-30)), -127, 127) * sc, 0.0 * y))
    return torch.cat(parts, -1)


def exact(case, seed):
    c = case
    if c["op"] in ("update", "compact"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    if c["op"] == "prep":
        inter = c["layout"] == "interleaved"
        used = (s["slots"] >= 0).double()[:, None, None]
        q = _exact_head(s["q"], s["wq"], s["pos"], s["freq"], inter)
        k = _exact_head(s["k"], s["wk"], s["pos"], s["freq"], inter)
        return q * used, _exact_kept(k) * used, _exact_kept(s["v"].double()) * used
    if c["op"] == "gather":
        ids = s["ids"].long()
        at = torch.where(ids < 0, torch.zeros_like(ids), ids)
        if c["paged"]:
            at = s["table"].long()[s["rows"].long(), torch.div(at, c["page"], rounding_mode="floor")] * c["page"] + at % c["page"]
        used = (ids >= 0).double()[:, None, None]
        return _exact_cells(s, "kq", "ksc", at) * used, _exact_cells(s, "vq", "vsc", at) * used
    n, hq, hkv, d = c["rows"], c["hq"], c["hkv"], c["d"]
    lens = [int(v) for v in s["lens"].tolist()]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    for t in range(n):
        if lens[t] == 0:
            continue
        cell = torch.arange(lens[t], device="cuda")
        row = t if s["rows"] is None else t // c["share"]
        at = s["table"].long()[row, cell // c["page"]] * c["page"] + cell % c["page"]
        k, v = _exact_cells(s, "kq", "ksc", at), _exact_cells(s, "vq", "vsc", at)
        q = s["q"][t].double().view(hkv, hq // hkv, d)
        z = torch.einsum("hgd,chd->hgc", q, k) * d ** -0.5
        lse[t] = torch.logsumexp(z, -1).flatten()
        out[t] = torch.einsum("hgc,chd->hgd", torch.softmax(z, -1), v).reshape(hq, d)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].double())
    return out, lse
