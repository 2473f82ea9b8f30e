"""Cases for long conversations on the paged cache: attention over the pages that a cheap score picks, and over trees
of drafted tokens.

The cache is a pool of pages of int8 K/V codes with four fp16 scales per row (one per quarter of the head dim), shared
by all sequences through a page table.  Five operators work on it:

  bounds  each page's largest and smallest key per dim, as rows of codes and scales of their own, rounded outwards
          (with the rows read back as the values they stand for)
  score   of each page of a token's sequence, what its keys can reach at most: the products of the query heads' positive
          parts with the upper bounds and of their negative parts with the lower ones, summed over dims and a KV head's
          query heads
  select  for each token and KV head the first pages, the last ones and the best-scoring others up to a budget
  sparse  attention of each token over its listed pages
  tree    attention of drafted tokens over the whole sequence before the draft and, by a bit mask, over the drafted
          tokens that lead to them

`own` is False for the plain form (elementary torch operations) and True for the framework's own calls.
"""
import math

import numpy as np
import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # A decode step of a full batch: each row's last page has got a new key.
        {"name": "bounds decode step", "op": "bounds", "rows": 61, "lo": 1, "hi": 32701, "new": 1, "hkv": 4, "d": 128, "page": 64},
        # Eight long prompts of wide heads have just been cached: all of their pages.
        {"name": "bounds whole prompts", "op": "bounds", "rows": 8, "lo": 29000, "hi": 30008, "new": 0, "hkv": 2, "d": 256, "page": 32},
        # The next token of one long conversation.
        {"name": "score one token", "op": "score", "seqs": 1, "share": 1, "lo": 30008, "hi": 30008, "hq": 12, "hkv": 1, "d": 128,
         "type": "fp16", "page": 64},
        # A full decode batch with small pages, conversations of all lengths up to 32 K cells.
        {"name": "score batch", "op": "score", "seqs": 61, "share": 1, "lo": 1, "hi": 32701, "hq": 48, "hkv": 4, "d": 128,
         "type": "bf16", "page": 16},
        # The next token of one long conversation: 32 pages of 469.
        {"name": "select one token", "op": "select", "seqs": 1, "share": 1, "lo": 30008, "hi": 30008, "hkv": 1, "page": 64,
         "budget": 32, "sink": 1, "local": 4},
        # A prompt chunk at a far position with small pages: 128 of 1875 to 1999 for each token and KV head.
        {"name": "select prompt chunk", "op": "select", "seqs": 1, "share": 1984, "lo": 31984, "hi": 31984, "hkv": 2, "page": 16,
         "budget": 128, "sink": 4, "local": 16},
        # The next token of one long conversation over its 32 pages.
        {"name": "sparse one token", "op": "sparse", "seqs": 1, "share": 1, "lo": 30008, "hi": 30008, "hq": 12, "hkv": 1, "d": 128,
         "type": "fp16", "page": 64, "budget": 32, "gate": False},
        # A full decode batch: each KV head of each row reads pages of its own.
        {"name": "sparse batch", "op": "sparse", "seqs": 61, "share": 1, "lo": 1, "hi": 32701, "hq": 48, "hkv": 4, "d": 128,
         "type": "bf16", "page": 16, "budget": 128, "gate": False},
        # A prompt chunk at a far position: 2048 cells for each token.
        {"name": "sparse prompt chunk", "op": "sparse", "seqs": 1, "share": 1984, "lo": 31984, "hi": 31984, "hq": 12, "hkv": 1,
         "d": 128, "type": "fp16", "page": 64, "budget": 32, "gate": False},
        # A small tree after a short prompt: what a step of one young conversation waits for.
        {"name": "tree short prompt", "op": "tree", "seqs": 1, "nodes": 7, "lo": 321, "hi": 321, "hq": 12, "hkv": 1, "d": 128,
         "type": "fp16", "page": 64, "gate": False},
        # A wide tree of one long conversation, wide heads, gated.
        {"name": "tree long conversation", "op": "tree", "seqs": 1, "nodes": 63, "lo": 30001, "hi": 30001, "hq": 24, "hkv": 2, "d": 256,
         "type": "bf16", "page": 16, "gate": True},
        # A batch of conversations, each with a tree of its own.
        {"name": "tree batch", "op": "tree", "seqs": 24, "nodes": 32, "lo": 100, "hi": 8190, "hq": 32, "hkv": 8, "d": 128,
         "type": "fp16", "page": 64, "gate": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(hi, lo))))))


def draw(rng):
    op = rng.choice(["bounds", "score", "select", "sparse", "tree"])
    d = rng.choice([128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    kind = rng.choice(["fp16", "bf16"])
    if op == "bounds":
        new = rng.choice([0, 1, 1, rng.randint(2, 500)])
        rows = _log(rng, 1, 128)
        hi = _log(rng, 1, min(40000, 8 * 29500 * 512 // (rows * hkv * d)))
        return {"op": op, "rows": rows, "lo": rng.randint(0, hi), "hi": hi, "new": new, "hkv": hkv, "d": d, "page": page}
    share = rng.choice([1, 1, 1, _log(rng, 2, 2000)])
    if op == "score":
        per = rng.choice([1, 2, 4, 6, 8, 12, 16])
        seqs = _log(rng, 1, max(1, 128 // share))
        hi = _log(rng, 1, min(64 * 1024, 61 * 1000 * 4 * 128 * page // (seqs * share * hkv * d) + share))
        return {"op": op, "seqs": seqs, "share": share, "lo": rng.randint(0, hi), "hi": hi, "hq": per * hkv, "hkv": hkv, "d": d,
                "type": kind, "page": page}
    budget = rng.choice([1, 3, 8, 16, 32, 64, 100, 128])
    if op == "select":
        seqs = _log(rng, 1, max(1, 200 // share))
        hi = _log(rng, 1, min(1 << 20, 1984 * 2 * 1900 * page // (seqs * share * hkv) + share))
        sink = rng.randint(0, budget) // 2
        return {"op": op, "seqs": seqs, "share": share, "lo": rng.randint(0, hi), "hi": hi, "hkv": hkv, "page": page, "budget": budget,
                "sink": sink, "local": rng.randint(0, budget - sink)}
    per = rng.choice([1, 2, 4, 6, 8, 12, 16])
    gate = rng.choice([False, True])
    if op == "sparse":
        share = min(share, max(1, 1900 * 2048 * 128 // (hkv * budget * page * d)))
        most = 1900 * 2048 * 128 // share if share > 1 else 230_000_000 // 2
        seqs = _log(rng, 1, max(1, min(200, most // (hkv * budget * page * (d + 8)))))
        hi = _log(rng, 1, min(32701, 61 * 16000 * 512 // (seqs * hkv * d)))
        return {"op": op, "seqs": seqs, "share": share, "lo": rng.randint(0, hi), "hi": hi, "hq": per * hkv, "hkv": hkv, "d": d,
                "type": kind, "page": page, "budget": budget, "gate": gate}
    seqs, nodes = _log(rng, 1, 32), _log(rng, 1, 100)
    hi = _log(rng, 1, min(32000, 24 * 4000 * 8 * 128 // (seqs * hkv * d), 60 * 30000 * 24 * 256 // (seqs * nodes * per * hkv * d)))
    return {"op": op, "seqs": seqs, "nodes": nodes, "lo": rng.randint(0, hi), "hi": hi, "hq": per * hkv, "hkv": hkv, "d": d,
            "type": kind, "page": page, "gate": gate}


# ---------------------------------------------------------------- inputs

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _spread(n, lo, hi):
    """n whole numbers over lo .. hi, mixed up, the same for every seed."""
    if n == 1:
        return np.array([hi], dtype=np.int64)
    f = (np.arange(n) * 0.6180339887498949 + 0.37) % 1.0
    v = lo + np.floor(f * (hi - lo + 1)).astype(np.int64)
    v[0], v[-1] = lo, hi
    return v


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _pool(g, pages, page, hkv, d, names=("kq", "vq", "ksc", "vsc")):
    """One layer of a pool."""
    shape = (pages, page, hkv)
    codes = [torch.randint(-127, 128, shape + (d,), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
    scales = [(torch.rand(shape + (4,), generator=g, device="cuda") * 0.019 + 0.001).half() for _ in range(2)]
    return dict(zip(names, codes + scales))


def _table(g, lens, page, pages, wide):
    """Pages for rows of these lengths, from a shuffled pool, and -1 behind them."""
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    held = -(-np.asarray(lens) // page)
    at = torch.as_tensor(np.concatenate([[0], np.cumsum(held)[:-1]]), device="cuda")
    held = torch.as_tensor(held, device="cuda")
    j = torch.arange(wide, device="cuda")
    idx = (at[:, None] + j[None]).clamp(max=pages - 1)
    return torch.where(j[None] < held[:, None], order[idx], torch.full_like(order[idx], -1)).contiguous()


def _tokens(c):
    """Cells that each token sees, the sequence it belongs to, and the sequences' cells.  The tokens of one sequence are
    consecutive: token k of `share` sees k cells more than the first."""
    n, share = c["seqs"] * c["share"], c["share"]
    base = np.maximum(_spread(c["seqs"], c["lo"], c["hi"]) - share + 1, 0)
    seq = np.arange(n) // share
    return base[seq] + np.arange(n) % share, seq, base + share - 1


def _drafts(c):
    """Drafted tokens of each sequence, and its cells before them."""
    return _spread(c["seqs"], (c["nodes"] + 1) // 2, c["nodes"]), _spread(c["seqs"], c["lo"], c["hi"])


def _queries(g, c, n):
    q = torch.randn(n, c["hq"], c["d"], generator=g, device="cuda") * (0.5 + 2.5 * torch.rand(1, c["hq"], 1, generator=g, device="cuda"))
    return q.to(_TYPES[c["type"]])


def _scores(g, c, seq, wide):
    """Scores as the tokens of a conversation give them: pages that matter to one mostly matter to the next."""
    n = len(seq)
    base = torch.randn(c["seqs"], c["hkv"], wide, generator=g, device="cuda")
    # Every 16 tokens of a sequence have a taste of their own, and each token a little of its own too.
    block = torch.as_tensor(np.arange(n) // 16 if c["share"] > 1 else np.arange(n), device="cuda")
    near = torch.randn(int(block[-1]) + 1, c["hkv"], wide, generator=g, device="cuda")
    x = base[torch.as_tensor(seq, device="cuda")] + 0.7 * near[block]
    x += 0.3 * torch.randn(n, c["hkv"], wide, generator=g, device="cuda")
    return 40.0 + 5.0 * x


def _i32(v):
    return torch.as_tensor(np.asarray(v), device="cuda", dtype=torch.int32)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    op, page = c["op"], c["page"]
    if op == "bounds":
        hkv, d = c["hkv"], c["d"]
        lens = _spread(c["rows"], c["lo"], c["hi"])
        new = np.minimum(lens, c["new"]) if c["new"] else lens
        held = -(-lens // page)
        wide, pages = max(1, int(held.max())), int(held.sum()) + 3
        s.update(_pool(g, pages, page, hkv, d))
        s["table"], s["lens"] = _table(g, lens, page, pages, wide), _i32(lens)
        s["new"] = _i32(new) if c["new"] else None
        # The pages that the call writes, in the rows' order: what is read back.
        j = torch.arange(wide, device="cuda")[None]
        first, end = torch.as_tensor((lens - new) // page, device="cuda")[:, None], torch.as_tensor(np.where(new > 0, held, 0), device="cuda")[:, None]
        s["ids"] = s["table"][(j >= first) & (j < end)].contiguous()
        s["bq"] = [torch.zeros(pages, hkv, d, device="cuda", dtype=torch.int8) for _ in range(2)]
        s["bsc"] = [torch.zeros(pages, hkv, 4, device="cuda", dtype=torch.float16) for _ in range(2)]
        s["back"] = [torch.empty(s["ids"].numel(), hkv, d, device="cuda") for _ in range(2)]
        return s
    if op == "tree":
        nodes, prefix = _drafts(c)
        n, hq, hkv, d = int(nodes.sum()), c["hq"], c["hkv"], c["d"]
        held = prefix + nodes
        wide = -(-int(held.max()) // page)
        pages = int((-(-held // page)).sum()) + 3
        s.update(_pool(g, pages, page, hkv, d))
        s["table"] = _table(g, held, page, pages, wide)
        seq = np.repeat(np.arange(c["seqs"]), nodes)
        node = np.concatenate([np.arange(k) for k in nodes])
        words = -(-int(nodes.max()) // 32)
        # A node hangs off the prefix or one of the nodes before it, and sees itself and those that lead to it.
        rng = np.random.default_rng(int(seed))
        sees = np.zeros((n, words * 32), dtype=bool)
        for i in range(n):
            above = rng.integers(-1, node[i]) if node[i] else -1
            if above >= 0:
                sees[i] = sees[i - node[i] + above]
            sees[i, node[i]] = True
        s["mask"] = torch.as_tensor(np.packbits(sees, axis=1, bitorder="little").view(np.int32), device="cuda").contiguous()
        s["prefix"], s["rows"] = _i32(prefix[seq]), _i32(seq)
        s["node"], s["nodes"] = torch.as_tensor(node, device="cuda"), int(nodes.max())
        s["most"] = int(held.max())
    else:
        lens, seq, held = _tokens(c)
        n, hkv = len(lens), c["hkv"]
        wide = max(1, -(-int(held.max()) // page))
        s["lens"], s["most"] = _i32(lens), int(lens.max())
        if op == "select":
            s["scores"] = _scores(g, c, seq, wide)
            s["pages"] = torch.empty(n, hkv, c["budget"], device="cuda", dtype=torch.int32)
            s["counts"] = torch.empty(n, hkv, device="cuda", dtype=torch.int32)
            return s
        hq, d = c["hq"], c["d"]
        pages = int((-(-held // page)).sum()) + 3
        s["table"] = _table(g, held, page, pages, wide)
        s["rows"] = _i32(seq) if c["share"] > 1 else None
        if op == "score":
            # A page's largest keys are mostly positive, its smallest mostly negative.
            s["bq"] = [torch.randint(40, 128, (pages, hkv, d), generator=g, device="cuda", dtype=torch.int8) * v for v in (1, -1)]
            s["bsc"] = [(torch.rand(pages, hkv, 4, generator=g, device="cuda") * 0.01 + 0.01).half() for _ in range(2)]
            s["q"] = _queries(g, c, n)
            s["scores"] = torch.zeros(n, hkv, wide, device="cuda")
            return s
        s.update(_pool(g, pages, page, hkv, d))
        # Lists as select gives them, the first and the last two pages among them.
        j = torch.arange(wide, device="cuda")
        count = torch.as_tensor(-(-lens // page), device="cuda")[:, None, None]
        x = _scores(g, c, seq, wide)
        x = torch.where((j == 0) | (j >= count - 2), torch.full_like(x, 1e9), x)
        x = torch.where(j < count, x, torch.full_like(x, -1e9))
        k = min(c["budget"], wide)
        top = torch.topk(x, k, -1).indices
        top = torch.where(top < count, top, torch.full_like(top, wide)).sort(-1).values
        lists = torch.full((n, hkv, c["budget"]), -1, device="cuda", dtype=torch.int32)
        lists[..., :k] = torch.where(top < wide, top, torch.full_like(top, -1))
        s["pages"], s["counts"] = lists, (lists >= 0).sum(-1).to(torch.int32)
    s["q"] = _queries(g, c, n)
    s["gate"] = 2.0 * torch.randn(n, hq, d, generator=g, device="cuda") if c["gate"] else None
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty(n, hq, device="cuda")
    if own:
        import sparse_selected_attention_gb300 as qsa
        size = qsa.qsa_paged_sparse_attn_workspace_bytes if op == "sparse" else qsa.qsa_paged_tree_attn_workspace_bytes
        s["ws"] = torch.empty(size(hq, hkv, d), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def _values(codes, scales):
    """What codes [..., D] with scales [..., 4] stand for."""
    d = codes.shape[-1]
    return (codes.float().unflatten(-1, (4, d // 4)) * scales.float().unsqueeze(-1)).flatten(-2)


def _plain_bounds(s):
    c, page = s["c"], s["c"]["page"]
    lens = s["lens"].long()
    new = lens if s["new"] is None else s["new"].long()
    j = torch.arange(s["table"].shape[1], device="cuda")[None]
    touched = (j >= ((lens - new) // page)[:, None]) & (j < ((lens + page - 1) // page)[:, None]) & (new > 0)[:, None]
    row, at = torch.nonzero(touched, as_tuple=True)
    pages = s["table"][row, at].long()
    x = _values(s["kq"][pages], s["ksc"][pages])  # [n, page, hkv, d]
    filled = (torch.arange(page, device="cuda")[None] < (lens[row] - at * page)[:, None])[:, :, None, None]
    out = []
    for k, sign in ((0, 1.0), (1, -1.0)):  # the lower bound is the negated upper one of the negated keys
        top = torch.where(filled, sign * x, torch.full_like(x, -math.inf)).amax(1).double().unflatten(-1, (4, c["d"] // 4))
        need = top.abs().amax(-1) / 127.0
        scale = need.half()
        scale = torch.where(scale.double() < need, (scale.view(torch.int16) + 1).view(torch.float16), scale)  # the next fp16 above
        step = scale.double().unsqueeze(-1)
        code = torch.where(step > 0, torch.ceil(top / torch.where(step > 0, step, torch.ones_like(step))), torch.zeros_like(top))
        s["bq"][k][pages] = (sign * code).flatten(-2).to(torch.int8)
        s["bsc"][k][pages] = scale
        out.append(_values(s["bq"][k][pages], s["bsc"][k][pages]))
    return tuple(out)


def _plain_score(s):
    c = s["c"]
    n, hkv, d = s["q"].shape[0], c["hkv"], c["d"]
    count = (s["lens"].long() + c["page"] - 1) // c["page"]
    q = s["q"].float().view(n, hkv, -1, d)
    parts = [q.clamp(min=0).sum(2), q.clamp(max=0).sum(2)]
    share = c["share"]
    at = s["table"].clamp(min=0).long()
    total = None
    for part, codes, scales in zip(parts, s["bq"], s["bsc"]):
        bound = _values(codes[at], scales[at]).permute(0, 2, 3, 1)  # [seqs, hkv, d, pages]
        x = torch.matmul(part.view(-1, share, hkv, d).transpose(1, 2), bound)  # [seqs, hkv, share, pages]
        total = x if total is None else total + x
    total = total.transpose(1, 2).flatten(0, 1)
    seen = torch.arange(total.shape[-1], device="cuda") < count[:, None, None]
    s["scores"].copy_(torch.where(seen, total, s["scores"]))
    return s["scores"]


def _plain_select(s):
    c, x = s["c"], s["scores"]
    j = torch.arange(x.shape[-1], device="cuda")
    count = ((s["lens"].long() + c["page"] - 1) // c["page"])[:, None, None]
    x = torch.where((j < c["sink"]) | (j >= count - c["local"]), torch.full_like(x, math.inf), x)
    x = torch.where(j < count, x, torch.full_like(x, -math.inf))
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., : c["budget"]]
    k = order.shape[-1]
    take = torch.minimum(count, torch.full_like(count, c["budget"]))
    i = torch.arange(k, device="cuda")
    last = torch.full_like(order, x.shape[-1])
    chosen = torch.where(i < take, order, last).sort(-1).values
    s["pages"].fill_(-1)
    s["pages"][..., :k] = torch.where(i < take, chosen, torch.full_like(chosen, -1)).to(torch.int32)
    s["counts"].copy_(take[..., 0].expand_as(s["counts"]))
    return s["pages"], s["counts"]


def _attend(logits, seen, v, gate):
    """Outputs and log denominators of logits [..., heads, cells] over v [..., cells, d]; rows that see nothing give 0."""
    logits = logits.masked_fill(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(logits - top)
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (torch.log(total) + top)[..., 0]
    return o, lse


def _finish(s, o, lse):
    o = o.reshape(s["q"].shape)
    if s["gate"] is not None:
        o = o / (1.0 + torch.exp(-s["gate"]))
    return o.to(s["q"].dtype), lse.reshape(s["lse"].shape)


def _plain_sparse(s):
    c = s["c"]
    n, hq, hkv, d, page = s["q"].shape[0], c["hq"], c["hkv"], c["d"], c["page"]
    row = torch.arange(n, device="cuda") if s["rows"] is None else s["rows"].long()
    lists = s["pages"].long()  # [n, hkv, w]
    phys = s["table"].long()[row[:, None, None], lists.clamp(min=0)]
    i = torch.arange(page, device="cuda")
    cell = (phys.clamp(min=0)[..., None] * page + i).flatten(-2)
    at = (lists[..., None] * page + i).flatten(-2)
    used = torch.arange(lists.shape[-1], device="cuda") < s["counts"][..., None]
    seen = (at >= 0) & (at < s["lens"].long()[:, None, None]) & used.repeat_interleave(page, -1)
    head = torch.arange(hkv, device="cuda")[None, :, None]
    k, v = (_values(s[a].flatten(0, 1)[cell, head], s[b].flatten(0, 1)[cell, head]) for a, b in (("kq", "ksc"), ("vq", "vsc")))
    q = s["q"].float().view(n, hkv, hq // hkv, d)
    logits = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(d)
    return _finish(s, *_attend(logits, seen[:, :, None], v, s["gate"]))


def _plain_tree(s):
    c = s["c"]
    n, hq, hkv, d, seqs, most = s["q"].shape[0], c["hq"], c["hkv"], c["d"], c["seqs"], s["most"]
    page = s["table"].clamp(min=0).long()
    k, v = (_values(s[a][page].flatten(1, 2)[:, :most], s[b][page].flatten(1, 2)[:, :most]).transpose(1, 2)
            for a, b in (("kq", "ksc"), ("vq", "vsc")))  # [seqs, hkv, cells, d]
    seq, node = s["rows"].long(), s["node"]
    # What each drafted token sees, cell by cell.
    j = torch.arange(most, device="cuda")[None] - s["prefix"].long()[:, None]
    word = torch.gather(s["mask"].long(), 1, (j // 32).clamp(0, s["mask"].shape[1] - 1))
    seen = (j < 0) | ((j < 32 * s["mask"].shape[1]) & (((word >> (j % 32)) & 1) == 1))
    q = torch.zeros(seqs, s["nodes"], hkv, hq // hkv, d, device="cuda")
    q[seq, node] = s["q"].float().view(n, hkv, -1, d)
    sees = torch.zeros(seqs, s["nodes"], most, device="cuda", dtype=torch.bool)
    sees[seq, node] = seen
    logits = torch.matmul(q.permute(0, 2, 1, 3, 4).flatten(2, 3), k.transpose(-1, -2)) / math.sqrt(d)  # [seqs, hkv, nodes * per, cells]
    o, lse = _attend(logits, sees.repeat_interleave(hq // hkv, 1)[:, None], v, s["gate"])
    o = o.view(seqs, hkv, s["nodes"], hq // hkv, d).permute(0, 2, 1, 3, 4)[seq, node]
    lse = lse.view(seqs, hkv, s["nodes"], hq // hkv).permute(0, 2, 1, 3)[seq, node]
    return _finish(s, o, lse)


def _own(s):
    import sparse_selected_attention_gb300 as qsa
    c = s["c"]
    if c["op"] == "bounds":
        qsa.qsa_page_bounds(s["table"], s["lens"], s["kq"], s["ksc"], *s["bq"], *s["bsc"], n_new=s["new"])
        qsa.qsa_paged_gather(*s["bq"], *s["bsc"], s["ids"], *s["back"])
        return tuple(s["back"])
    if c["op"] == "score":
        qsa.qsa_page_score(s["q"], *s["bq"], *s["bsc"], s["table"], s["lens"], s["scores"], c["page"], rows=s["rows"])
        return s["scores"]
    if c["op"] == "select":
        qsa.qsa_page_select(s["scores"], s["lens"], s["pages"], s["counts"], c["page"], c["budget"], sink=c["sink"], local=c["local"])
        return s["pages"], s["counts"]
    pool = (s["kq"], s["vq"], s["ksc"], s["vsc"])
    if c["op"] == "sparse":
        qsa.qsa_paged_sparse_attn(s["q"], *pool, s["table"], s["lens"], s["pages"], s["counts"], s["out"], s["ws"], rows=s["rows"],
                                  gate=s["gate"], lse=s["lse"])
    else:
        qsa.qsa_paged_tree_attn(s["q"], *pool, s["table"], s["prefix"], s["mask"], s["out"], s["ws"], rows=s["rows"], gate=s["gate"],
                                lse=s["lse"])
    return s["out"], s["lse"]


def run(state):
    if own:
        return _own(state)
    return {"bounds": _plain_bounds, "score": _plain_score, "select": _plain_select, "sparse": _plain_sparse,
            "tree": _plain_tree}[state["c"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    page = c["page"]
    if c["op"] == "bounds":
        lens = _spread(c["rows"], c["lo"], c["hi"])
        new = np.minimum(lens, c["new"]) if c["new"] else lens
        first, end = (lens - new) // page, -(-lens // page)
        pages, cells = int(np.where(new > 0, end - first, 0).sum()), int(np.where(new > 0, lens - first * page, 0).sum())
        # Keys once, bounds out and their values read back, an entry of the table for each page.
        return {"bytes": c["hkv"] * (cells * (c["d"] + 8) + pages * (2 * (c["d"] + 8) + 8 * c["d"])) + 8 * pages + 8 * c["rows"],
                "flops": 3 * cells * c["hkv"] * c["d"]}
    if c["op"] == "tree":
        nodes, prefix = _drafts(c)
        n = int(nodes.sum())
        return {"bytes": int((prefix + nodes).sum()) * c["hkv"] * (2 * c["d"] + 16) + n * c["hq"] * (c["d"] * (8 if c["gate"] else 4) + 4),
                "flops": 4 * int((nodes * (prefix + 1)).sum()) * c["hq"] * c["d"]}
    lens, _, held = _tokens(c)
    n, count = len(lens), -(-lens // page)
    if c["op"] == "score":
        read = int((-(-held // page)).sum()) * c["hkv"] * (2 * c["d"] + 16)
        pairs = int(count.sum()) * c["hkv"]
        return {"bytes": read + 4 * pairs + n * (2 * c["hq"] * c["d"] + 4), "flops": 4 * pairs * c["d"]}
    if c["op"] == "select":
        return {"bytes": 4 * c["hkv"] * (int(count.sum()) + n * (c["budget"] + 1)) + 4 * n, "flops": 0}
    cells = np.minimum(lens, c["budget"] * page)
    rows = int(cells.sum()) if c["share"] == 1 else min(int(cells.sum()), int(held.sum()))  # tokens of one sequence read the same pages
    return {"bytes": rows * c["hkv"] * (2 * c["d"] + 16) + n * (c["hq"] * (c["d"] * (8 if c["gate"] else 4) + 4) + 4 * c["hkv"] * (c["budget"] + 1)),
            "flops": 4 * int(cells.sum()) * c["hq"] * c["d"]}


# ---------------------------------------------------------------- the definitions, in 64 bits

def _exact_rows(codes, scales):
    x = codes.double()
    return x * scales.double().repeat_interleave(x.shape[-1] // 4, -1)


def _exact_bounds(s, c):
    """Page by page: the extremes, then the least fp16 scale that 127 codes reach them with, then the nearest code outside."""
    table, lens, page = s["table"].cpu().numpy(), s["lens"].tolist(), c["page"]
    new = lens if s["new"] is None else s["new"].tolist()
    x = _exact_rows(s["kq"], s["ksc"])
    top, low = [], []
    for r, (n, m) in enumerate(zip(lens, new)):
        for j in range((n - m) // page, -(-n // page) if m else 0):
            keys = x[int(table[r, j]), : min(page, n - j * page)]
            top.append(keys.max(0).values)
            low.append(keys.min(0).values)
    out = []
    for v, outwards in ((top, np.ceil), (low, np.floor)):
        v = torch.stack(v).cpu().numpy().reshape(-1, 4, c["d"] // 4) if v else np.zeros((0, 4, c["d"] // 4))
        need = np.abs(v).max(-1, initial=0.0) / 127.0
        scale = need.astype(np.float16)
        scale = np.where(scale < need, np.nextafter(scale, np.float16(np.inf)), scale).astype(np.float64)[..., None]
        value = outwards(np.divide(v, scale, out=np.zeros_like(v), where=scale > 0)) * scale
        out.append(torch.as_tensor(value.reshape(-1, c["hkv"], c["d"])))
    return tuple(out)


def exact(case, seed):
    c = case
    if c["op"] == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    if c["op"] == "bounds":
        return _exact_bounds(s, c)
    hq, hkv, d, page, n = c["hq"], c["hkv"], c["d"], c["page"], s["q"].shape[0]
    row = list(range(n)) if s["rows"] is None else s["rows"].tolist()
    table = s["table"].long()
    if c["op"] == "score":
        out = s["scores"].double()
        for t, length in enumerate(s["lens"].tolist()):
            at = table[row[t], : -(-length // page)]
            q = s["q"][t].double().view(hkv, -1, d)
            hi, lo = (_exact_rows(b[at], w[at]) for b, w in zip(s["bq"], s["bsc"]))
            # Each query head's best product with anything between the bounds.
            best = torch.einsum("hd,phd->hp", q.clamp(min=0).sum(1), hi) + torch.einsum("hd,phd->hp", q.clamp(max=0).sum(1), lo)
            out[t, :, : at.numel()] = best
        return out
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, hq), -math.inf, dtype=torch.float64, device="cuda")
    per = hq // hkv
    for t in range(n):
        if c["op"] == "tree":
            bits = [b for w, m in enumerate(s["mask"][t].tolist()) for b in range(32 * w, 32 * w + 32) if m >> (b - 32 * w) & 1]
            cells = [torch.cat([torch.arange(int(s["prefix"][t]), device="cuda"), int(s["prefix"][t]) + torch.tensor(bits, device="cuda", dtype=torch.long)])]
            heads = [slice(None)]
        else:
            cells, heads, most = [], [[h] for h in range(hkv)], int(s["lens"][t])
            for h in range(hkv):
                at = s["pages"][t, h, : int(s["counts"][t, h])].long()
                at = (at[:, None] * page + torch.arange(page, device="cuda")).flatten()
                cells.append(at[at < most])
        for at, h in zip(cells, heads):
            if not at.numel():
                continue
            pool = table[row[t], at // page] * page + at % page
            k, v = (_exact_rows(s[a].flatten(0, 1)[pool][:, h], s[b].flatten(0, 1)[pool][:, h]) for a, b in (("kq", "ksc"), ("vq", "vsc")))
            z = torch.einsum("hgd,chd->hgc", s["q"][t].double().view(hkv, per, d)[h], k) * d ** -0.5
            lse.view(n, hkv, per)[t, h] = torch.logsumexp(z, -1)
            out.view(n, hkv, per, d)[t, h] = torch.einsum("hgc,chd->hgd", torch.softmax(z, -1), v)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].double())
    return out, lse
