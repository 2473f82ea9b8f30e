"""Picked pages and trees of drafts as a serving program uses them: the calls one
after the other, in graphs, on several streams, over pools and scores past 32-bit
offsets, with scales of all sizes, in the library's test variants, and refused.

Tolerances as tests/test_paged_pick_gpu.py, of V scales of all sizes as
tests/test_paged_vscales_gpu.py.
"""
import math

import numpy as np
import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from oracle import paged_oracle as po
from tests.test_paged_gpu import BF16, F16, F32, HALF, TINY, Serving, dev, err_word, i32, make_pool, shuffled_table
from tests.test_paged_groups_gpu import reference
from tests.test_paged_pick_gpu import alike, check_sparse, check_tree, read_together, sparse_workspace, taken_together, tree_workspace, trees
from tests.test_paged_variants_gpu import use_library, word  # noqa: F401
from tests.test_paged_vscales_gpu import scales

pytestmark = pytest.mark.gpu


def zeros(*s, t=torch.int32):
    return torch.zeros(s, dtype=t, device="cuda")


def chain(n, words=None):
    """Masks of n drafted tokens that follow one another."""
    m = np.zeros((n, (words or -(-n // 32)) * 32), bool)
    m[:, :n] = np.tril(np.ones((n, n), bool))
    return np.packbits(m, axis=1, bitorder="little").view(np.int32)


# ---------------------------------------------------------------- together

class Picking(Serving):
    """The serving loop with bounds of its pages."""

    def __init__(self, rows, **kw):
        super().__init__(rows, **kw)
        pages = self.pool[0].shape[1]
        self.bounds = [zeros(pages, self.hkv, self.d, t=torch.int8) for _ in range(2)] + [zeros(pages, self.hkv, 4, t=F16) for _ in range(2)]

    def append(self, x, new, q):
        self.update(None, i32(new))
        self.write(x, q)
        kq, _, ksc, _ = self.layer()
        qsa.qsa_page_bounds(self.table, self.lens, kq, ksc, *self.bounds, n_new=i32(new), err=self.err)

    def pick(self, q, lens, budget, rows=None, sink=1, local=2):
        n, wide = q.shape[0], self.table.shape[1]
        scores, pages, counts = zeros(n, self.hkv, wide, t=F32), zeros(n, self.hkv, budget), zeros(n, self.hkv)
        qsa.qsa_page_score(q, *self.bounds, self.table, lens, scores, self.page, rows=rows, err=self.err)
        qsa.qsa_page_select(scores, lens, pages, counts, self.page, budget, sink=sink, local=local, err=self.err)
        out = torch.empty_like(q)
        qsa.qsa_paged_sparse_attn(q, *self.layer(), self.table, lens, pages, counts, out, sparse_workspace(self.hq, self.hkv, self.d), rows=rows,
                                  err=self.err)
        return scores, pages, counts, out


def test_prompts_decode_steps_and_drafts(cuda_device):
    """Prompts in chunks, decode steps and a tree of drafts.  A budget of all pages gives what attention over
    the whole sequences gives; a small one gives the oracle's lists, and attention over them."""
    s = Picking(3, hq=12, hkv=2, page=16, pages=200, wide=64, slots=512)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda n: torch.randn(n, 16, 128, generator=gen, device="cuda").to(F16)  # noqa: E731
    for new in ([300, 0, 90], [33, 64, 200], [1, 1, 1], [1, 1, 1], [40, 1, 2], [1, 1, 1]):
        n = sum(new)
        q = zeros(n, 12, 128, t=F16)
        s.append(rand(n), new, q)
        rows = [r for r, k in enumerate(new) for _ in range(k)]
        held = s.lens.tolist()
        lens = [held[r] - k + 1 + i for r, k in enumerate(new) for i in range(k)]
        # The bounds kept up page by page are those of the whole cache.
        kq, vq, ksc, vsc = (x.cpu().numpy() for x in s.layer())
        want, werr = po.page_bounds(s.table.cpu().numpy(), held, None, kq, ksc)
        for p, parts in want.items():
            for mine, x in zip(s.bounds, parts):
                np.testing.assert_array_equal(mine[p].cpu().numpy(), x)
        _, pages, counts, out = s.pick(q, i32(lens), 64, rows=i32(rows))
        full = torch.empty_like(q)
        qsa.qsa_paged_attn(q, *s.layer(), s.table, i32(lens), full, s.aws, rows=i32(rows), err=s.err)
        torch.testing.assert_close(out.float(), full.float(), rtol=2.0 ** -9, atol=2.0 ** -10)
        scores, pages, counts, out = s.pick(q, i32(lens), 7, rows=i32(rows))
        wp, wc, werr = po.page_select(scores.cpu().numpy(), lens, 16, 7, 1, 2, 7)
        np.testing.assert_array_equal(counts.cpu().numpy(), wc)
        np.testing.assert_array_equal(pages.cpu().numpy(), wp)
        check_sparse(q, (kq, vq, ksc, vsc), s.table.cpu().numpy(), lens, wp, wc, rows=rows)
    # Drafts that follow one another are what a prompt's chunk is, and a node of a tree sees what its path is.
    new = [12, 9, 0]
    q = zeros(21, 12, 128, t=F16)
    prefix = s.lens.tolist()
    s.append(rand(21), new, q)
    rows = [0] * 12 + [1] * 9
    line, out = torch.empty_like(q), torch.empty_like(q)
    lens = [prefix[0] + i + 1 for i in range(12)] + [prefix[1] + i + 1 for i in range(9)]
    qsa.qsa_paged_attn(q, *s.layer(), s.table, i32(lens), line, s.aws, rows=i32(rows), err=s.err)
    mask = np.concatenate([chain(12), chain(9)])
    pre = [prefix[r] for r in rows]
    qsa.qsa_paged_tree_attn(q, *s.layer(), s.table, i32(pre), dev(mask), out, tree_workspace(12, 2, 128), rows=i32(rows), err=s.err)
    torch.testing.assert_close(out.float(), line.float(), rtol=2.0 ** -9, atol=2.0 ** -10)
    assert int(s.err.item()) == 0


def pick_jobs(seed=50):
    """Every new call on tensors of its own, long enough for each way of taking rows: functions of (state, stream)."""
    rng = np.random.default_rng(seed)
    pool, table, lens, rows, lists, counts = alike(rng, [160, 30], 3000, 32, 4, 128, 70, 66, seed)
    p, t, n = [dev(x) for x in pool], dev(table), len(rows)
    q = dev(rng.standard_normal((n, 16, 128)).astype(np.float16))
    tpool, ttable, prefix, mask, trows = trees(rng, [2000, 700], [63, 33], 16, 2, 256, seed)
    tp, tq = [dev(x) for x in tpool], dev(rng.standard_normal((96, 8, 256)).astype(np.float32)).to(BF16)
    args = [i32(lens), i32(rows), dev(lists), dev(counts), dev(ttable), i32(prefix), dev(mask), i32(trows), i32([3160, 3067])]

    def state():
        pages = p[0].shape[0]
        return dict(b=[zeros(pages, 4, 128, t=torch.int8) for _ in range(2)] + [zeros(pages, 4, 4, t=F16) for _ in range(2)],
                    s=zeros(n, 4, table.shape[1], t=F32), l=zeros(n, 4, 40), c=zeros(n, 4), o=[torch.zeros_like(q) for _ in range(3)],
                    to=torch.zeros_like(tq), lse=zeros(n, 16, t=F32), w=[sparse_workspace(16, 4, 128), tree_workspace(8, 2, 256)], e=err_word())

    def run(s, stream=None):
        le, ro, li, co, tt, pr, ma, tr, held = args
        kw = dict(err=s["e"], stream=stream)
        qsa.qsa_page_bounds(t, held, p[0], p[2], *s["b"], **kw)
        qsa.qsa_page_score(q, *s["b"], t, le, s["s"], 32, rows=ro, **kw)
        qsa.qsa_page_select(s["s"], le, s["l"], s["c"], 32, 40, sink=2, local=3, **kw)
        qsa.qsa_paged_sparse_attn(q, *p, t, le, s["l"], s["c"], s["o"][0], s["w"][0], rows=ro, lse=s["lse"], **kw)
        qsa.qsa_paged_sparse_attn(q, *p, t, le, li, co, s["o"][1], s["w"][0], rows=ro, **kw)
        qsa.qsa_paged_sparse_attn(q[:2], *p, t, le[::160][:2].contiguous(), li[:2], co[:2], s["o"][2][:2], s["w"][0], **kw)
        qsa.qsa_paged_tree_attn(tq, *tp, tt, pr, ma, s["to"], s["w"][1], rows=tr, **kw)

    def results(s):
        return s["b"] + [s["s"], s["l"], s["c"], *s["o"], s["to"], s["lse"], s["e"]]

    return state, run, results


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_repeats_its_bits_in_graphs_and_on_streams_at_once(cuda_device):
    state, run, results = pick_jobs()
    first = state()
    run(first)
    assert int(first["e"].item()) == 0 and all(x.any() for x in results(first)[:-1])
    again = state()
    run(again)
    torch.cuda.synchronize()
    assert same(results(first), results(again))
    # Captured, over outputs and a workspace that hold something else, replayed twice.
    s, g, side = state(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        run(s)
    for _ in range(2):
        for x in results(s)[:-1]:
            x.view(torch.uint8).fill_(7)
        g.replay()
        torch.cuda.synchronize()
        # Pages' bounds, scores and rows that no call writes keep their bytes.
        assert same([s["l"], s["c"], s["o"][0], s["o"][1], s["o"][2][:2], s["to"], s["lse"]],
                    [first["l"], first["c"], first["o"][0], first["o"][1], first["o"][2][:2], first["to"], first["lse"]])
    # Two graphs that share a workspace, one after the other, and two streams at once, each with its own.
    g2, s2 = torch.cuda.CUDAGraph(), state()
    s2["w"] = s["w"]
    torch.cuda.synchronize()
    with torch.cuda.graph(g2, stream=side):
        run(s2)
    g.replay()
    g2.replay()
    g.replay()
    torch.cuda.synchronize()
    assert same([s2["o"][0], s2["o"][1], s2["to"]], [first["o"][0], first["o"][1], first["to"]])
    streams, both = [torch.cuda.Stream() for _ in range(2)], [state() for _ in range(2)]
    for _ in range(4):
        torch.cuda.synchronize()
        for st, x in zip(streams, both):
            run(x, st)
        torch.cuda.synchronize()
        assert all(same(results(x), results(first)) for x in both)


def test_a_given_stream_is_used(cuda_device):
    """A call follows what was queued on its stream, and not on the current one."""
    state, run, results = pick_jobs(51)
    want, s, side = state(), state(), torch.cuda.Stream()
    run(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for x in results(s):
            x.zero_()
    run(s, side)
    side.synchronize()
    assert same(results(s), results(want))


def test_calls_of_no_tokens(cuda_device):
    pool = [dev(x) for x in make_pool(6, 16, 2, 128)]
    b = [zeros(6, 2, 128, t=torch.int8) for _ in range(2)] + [zeros(6, 2, 4, t=F16) for _ in range(2)]
    none, q, err = zeros(0, 2), zeros(0, 4, 128, t=F16), err_word()
    qsa.qsa_page_bounds(none, zeros(0), pool[0], pool[2], *b, err=err)
    qsa.qsa_page_bounds(none, zeros(0), pool[0], pool[2], *b, n_new=zeros(0), err=err)
    scores = zeros(0, 2, 2, t=F32)
    for rows in (None, zeros(0)):
        qsa.qsa_page_score(q, *b, none, zeros(0), scores, 16, rows=rows, err=err)
    qsa.qsa_page_select(scores, zeros(0), zeros(0, 2, 3), zeros(0, 2), 16, 3, err=err)
    for rows in (None, zeros(0)):
        qsa.qsa_paged_sparse_attn(q, *pool, none, zeros(0), zeros(0, 2, 3), zeros(0, 2), q.clone(), sparse_workspace(4, 2, 128), rows=rows, err=err)
        qsa.qsa_paged_tree_attn(q, *pool, none, zeros(0), zeros(0, 1), q.clone(), tree_workspace(4, 2, 128), rows=rows, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and not any(x.any() for x in b)


# ---------------------------------------------------------------- trees

def test_tree_one_token_each_without_rows(cuda_device):
    """The form for single tokens: a row of the table each."""
    rng = np.random.default_rng(52)
    prefix = [0, 1, 700, 3000, 15, 16, 0]
    table, pages = shuffled_table([p + 40 for p in prefix], 16, 2, rng)
    pool = make_pool(pages, 16, 2, 128, seed=52)
    mask = np.array([[1, 0], [1, 0], [-1, 3], [0, 128], [0, 0], [-2 ** 31, 0], [0, 0]], np.int32)
    check_tree(rng.standard_normal((7, 8, 128)), pool, table, prefix, mask)
    check_tree(rng.standard_normal((1, 8, 128)), pool, table[2:3], prefix[2:3], mask[2:3], rows=[0])


@pytest.mark.parametrize("d,hq,hkv,page", [(128, 8, 2, 64), (256, 16, 1, 16)])
def test_tree_padded_batch(cuda_device, d, hq, hkv, page):
    """Every tree padded to as many rows; the rows of a padding token see nothing."""
    rng = np.random.default_rng(53)
    nodes = [20, 7, 31, 1]
    pool, table, prefix, mask, rows = trees(rng, [1500, 40, 0, 2200], nodes, page, hkv, d, 53)
    at, P, M, R = 0, [], [], []
    for s, n in enumerate(nodes):
        P += prefix[at:at + n] + [0] * (32 - n)
        M += list(mask[at:at + n]) + [np.zeros_like(mask[0])] * (32 - n)
        R += [s] * 32
        at += n
    out, lse = check_tree(rng.standard_normal((128, hq, d)), pool, table, P, np.stack(M), rows=R)
    assert torch.isneginf(lse).any(1).sum() == 128 - sum(nodes)


@pytest.mark.parametrize("seqs,nodes,prefix", [(40, 37, 300), (3, 500, 600), (1300, 1, 700), (2, 1024, 20)])
def test_tree_more_tokens_than_are_looked_up_at_once(cuda_device, seqs, nodes, prefix):
    rng = np.random.default_rng(54)
    page, n = 64, seqs * nodes
    table, pages = shuffled_table([prefix + nodes] * seqs, page, 1, rng)
    pool = [dev(x) for x in make_pool(pages, page, 1, 128, seed=54)]
    rows = [s for s in range(seqs) for _ in range(nodes)]
    lens = [prefix + i + 1 for _ in range(seqs) for i in range(nodes)]
    mask = np.tile(chain(nodes), (seqs, 1))
    q = dev(rng.standard_normal((n, 4, 128)).astype(np.float16))
    out, lse, err = torch.empty_like(q), zeros(n, 4, t=F32), err_word()
    qsa.qsa_paged_tree_attn(q, *pool, dev(table), i32([prefix] * n), dev(mask), out, tree_workspace(4, 1, 128), rows=i32(rows), lse=lse, err=err)
    want, wlse = torch.empty_like(q), zeros(n, 4, t=F32)
    ws = zeros(qsa.qsa_paged_attn_workspace_bytes(4, 1, 128), t=torch.uint8)
    qsa.qsa_paged_attn(q, *pool, dev(table), i32(lens), want, ws, rows=i32(rows), lse=wlse, err=err)
    torch.testing.assert_close(out.float(), want.float(), rtol=2.0 ** -9, atol=2.0 ** -10)
    torch.testing.assert_close(lse, wlse, rtol=2.0 ** -18, atol=2.0 ** -14)
    assert int(err.item()) == 0


@pytest.mark.parametrize("hkv", [77, 160])
def test_many_kv_heads(cuda_device, hkv):
    """As many KV heads as there are places for shares, and more."""
    rng = np.random.default_rng(55)
    pool, table, prefix, mask, rows = trees(rng, [400, 333], [9, 4], 32, hkv, 128, 55)
    check_tree(rng.standard_normal((13, hkv, 128)), pool, table, prefix, mask, rows=rows)
    pool, table, lens, rows, lists, counts = alike(rng, [24], 600, 32, hkv, 128, 20, 18, 55)
    check_sparse(rng.standard_normal((24, hkv, 128)), pool, table, lens, lists, counts, rows=rows)


@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e-30, 2.0])
def test_tree_softmax_scales(cuda_device, scale):
    rng = np.random.default_rng(56)
    pool, table, prefix, mask, rows = trees(rng, [1500], [20], 32, 2, 128, 56)
    for otype in (F16, BF16):
        check_tree(rng.standard_normal((20, 16, 128)) * 0.5, pool, table, prefix, mask, rows=rows, scale=scale, otype=otype)


# ---------------------------------------------------------------- scales of all sizes

def one_sequence(form, d, seed):
    """Tokens of one sequence, all of whose pages are seen: pool, table, lengths, rows and the call."""
    rng = np.random.default_rng(seed)
    n, cells, page, hkv, hq = 72, 1700, 32, 8, 16
    table, pages = shuffled_table([cells], page, 1, rng)
    pool = [dev(x) for x in make_pool(pages, page, hkv, d, seed=seed)]
    lens, rows = [cells - n + i + 1 for i in range(n)], [0] * n

    def call(q, pool, **kw):
        out, lse, err = torch.empty_like(q), zeros(n, hq, t=F32), err_word()
        if form == "tree":
            ws = tree_workspace(hq, hkv, d)
            qsa.qsa_paged_tree_attn(q, *pool, dev(table), i32([cells - n] * n), dev(chain(n)), out, ws, rows=i32(rows), lse=lse, err=err, **kw)
            assert read_together(ws, rows, 1, table.shape[1] * page, hkv, d)
        else:
            wide = table.shape[1]
            lists = torch.arange(wide, dtype=torch.int32, device="cuda").expand(n, hkv, wide).contiguous()
            ws = sparse_workspace(hq, hkv, d)
            qsa.qsa_paged_sparse_attn(q, *pool, dev(table), i32(lens), lists, torch.full_like(lists[..., 0], wide), out, ws, rows=i32(rows), lse=lse,
                                      err=err, **kw)
            assert taken_together(ws)
        assert int(err.item()) == 0
        return out, lse

    return rng.standard_normal((n, hq, d)), pool, table, lens, rows, call


def near(otype, got, want):
    (out, lse), (ref, rlse, mag, flush, qk) = got, want
    ds = 1152 * qk * 2.0 ** -21
    tol = HALF[otype] * ref.abs() + mag * (2.0 ** -10 + 2 * torch.expm1(ds)[..., None] + 2.0 ** -16) + flush * 2.0 ** -24 + TINY[otype]
    bad = ~((out.double() - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.numel(), bad.nonzero()[:3].tolist(), out[bad][:3], ref[bad][:3], tol[bad][:3])
    assert ((lse.double() - rlse).abs() <= ds + 2.0 ** -16 + 2.0 ** -22 * rlse.abs()).all()


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("kind", ["large ones without weight", "small ones after large ones", "cell by cell", "zero ones", "largest"])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("form", ["tree", "listed"])
def test_v_scales(cuda_device, form, d, kind, otype):
    q, pool, table, lens, rows, call = one_sequence(form, d, 57)
    vs, light = scales(kind, pool[3].shape[:3], d)
    pool[3] = vs.half()
    if kind == "largest":
        pool[1] = pool[1] // (2 if otype is BF16 else 127)  # results within their type
    pool[2][:] = 2.0 ** -7
    q = dev(q) * 0.5
    q[..., 0] = 32.0  # scores 15 nats up for all cells but the light ones, 47 below those
    pool[0][..., 0] = 60 if light is None else torch.where(light[..., 0], -127, 60).to(torch.int8)
    q = q.to(otype)
    near(otype, call(q, pool, softmax_scale=1.0), reference(q, pool, table, lens, rows, 1.0))


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("kind", ["cell by cell", "small ones after large ones", "zero ones"])
@pytest.mark.parametrize("form", ["tree", "listed"])
def test_k_scales(cuda_device, form, kind, otype):
    """K scales that differ by up to 2^25 among neighbours."""
    q, pool, table, lens, rows, call = one_sequence(form, 128, 58)
    ks, _ = scales(kind, pool[2].shape[:3], 128)
    pool[2] = (ks * 2.0 ** -12).half()
    q = dev(q).to(otype)
    near(otype, call(q, pool, softmax_scale=0.3), reference(q, pool, table, lens, rows, 0.3))


# ---------------------------------------------------------------- sizes

def test_pools_and_scores_beyond_32_bit_offsets(cuda_device):
    """Pages that start past 2^32 bytes of codes, and scores past 2^31 of them, give what they give elsewhere."""
    page, d, hkv, held, n = 64, 256, 8, 30, 70
    pages = (1 << 32) // (page * hkv * d) + 16
    small = [dev(x) for x in make_pool(held, page, hkv, d, seed=59)]
    big = [torch.zeros(pages, page, hkv, x.shape[3], dtype=x.dtype, device="cuda") for x in small]
    where = [pages - 1 - 2 * i if i % 2 else i for i in range(held)]
    for t, x in zip(big, small):
        t[where] = x
    rng = np.random.default_rng(59)
    q = dev(rng.standard_normal((n, 16, d)).astype(np.float16))
    lens, rows = i32([held * page - n + 1 + i for i in range(n)]), i32([0] * n)
    lists = torch.arange(held, dtype=torch.int32, device="cuda").expand(n, hkv, held).contiguous()
    counts = torch.full((n, hkv), held, dtype=torch.int32, device="cuda")
    res = []
    for pool, tab in ((big, where), (small, list(range(held)))):
        tab, np_ = i32(tab).view(1, held), pool[0].shape[0]
        b = [zeros(np_, hkv, d, t=torch.int8) for _ in range(2)] + [zeros(np_, hkv, 4, t=F16) for _ in range(2)]
        qsa.qsa_page_bounds(tab, lens[-1:], pool[0], pool[2], *b)
        s = zeros(n, hkv, held, t=F32)
        qsa.qsa_page_score(q, *b, tab, lens, s, page, rows=rows)
        outs = [torch.empty_like(q) for _ in range(4)]
        ws = sparse_workspace(16, hkv, d)
        qsa.qsa_paged_sparse_attn(q, *pool, tab, lens, lists, counts, outs[0], ws, rows=rows)
        assert taken_together(ws)
        qsa.qsa_paged_sparse_attn(q[:1], *pool, tab, lens[:1], lists[:1], counts[:1], outs[1][:1], ws)
        qsa.qsa_paged_tree_attn(q, *pool, tab, i32([held * page - n] * n), dev(chain(n)), outs[2], tree_workspace(16, hkv, d), rows=rows)
        qsa.qsa_paged_tree_attn(q[:1], *pool, tab, lens[:1] - 1, dev(chain(1)), outs[3][:1], tree_workspace(16, hkv, d))
        res.append([s, outs[0], outs[1][:1], outs[2], outs[3][:1], *[x[tab[0].long()] for x in b]])
    assert same(*res)
    del big, res
    # Rows of scores 2^20 apart, 2^31 and more of them.
    ld, rows_n = 1 << 20, 2100
    x = torch.empty(rows_n, 1, ld, device="cuda")
    few = torch.randn(rows_n, 1, 90, device="cuda")
    x[..., :90] = few
    lens = i32([16 * 90 - i % 700 for i in range(rows_n)])
    got = []
    for sc in (x, few):
        p, c = zeros(rows_n, 1, 9), zeros(rows_n, 1)
        qsa.qsa_page_select(sc, lens, p, c, 16, 9)
        got.append((p, c))
    assert same(*got) and bool((got[0][1] == 9).all())
    b = [torch.randint(-127, 128, (90, 1, 128), dtype=torch.int8, device="cuda") for _ in range(2)] + [torch.rand(90, 1, 4, device="cuda").half() for _ in range(2)]
    q = torch.randn(rows_n, 1, 128, device="cuda").half()
    tab = torch.full((1, ld), -1, dtype=torch.int32, device="cuda")
    tab[0, :90] = torch.arange(90, device="cuda")
    for sc, tb in ((x, tab), (few, tab[:, :90].contiguous())):
        sc.zero_()
        qsa.qsa_page_score(q, *b, tb, lens, sc, 16, rows=torch.zeros_like(lens))
    assert torch.equal(x[..., :90], few) and few.any()


# ---------------------------------------------------------------- test variants of the library

def test_check_build_same_bits(cuda_device, use_library):  # noqa: F811
    state, run, results = pick_jobs(60)
    plain, checked = state(), state()
    run(plain)
    L = use_library("check")
    word(L)
    run(checked)
    torch.cuda.synchronize()
    assert word(L) == 0 and same(results(plain), results(checked))


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("form", ["tree", "listed"])
def test_time_outs(cuda_device, use_library, monkeypatch, form, d):  # noqa: F811
    """Waits that give up at once: the calls say so and leave the context usable."""
    q, pool, table, lens, rows, _ = one_sequence(form, d, 61)
    q, n = dev(q).half(), len(rows)
    out, err, ws = torch.zeros_like(q), err_word(), sparse_workspace(16, 8, d)
    wide = table.shape[1]
    lists = torch.arange(wide, dtype=torch.int32, device="cuda").expand(n, 8, wide).contiguous()

    def call():
        if form == "tree":
            qsa.qsa_paged_tree_attn(q, *pool, dev(table), i32([lens[0] - 1] * n), dev(chain(n)), out, ws, rows=i32(rows), err=err)
        else:
            qsa.qsa_paged_sparse_attn(q, *pool, dev(table), i32(lens), lists, torch.full_like(lists[..., 0], wide), out, ws, rows=i32(rows), err=err)
        torch.cuda.synchronize()
        return int(err.item())

    use_library("wait0")
    assert call() == qsa.QSA_DEVERR_TIMEOUT
    monkeypatch.undo()
    err.zero_()
    assert call() == 0
    want = torch.empty_like(q)
    qsa.qsa_paged_attn(q, *pool, dev(table), i32(lens), want, zeros(qsa.qsa_paged_attn_workspace_bytes(16, 8, d), t=torch.uint8), rows=i32(rows))
    torch.testing.assert_close(out.float(), want.float(), rtol=2.0 ** -9, atol=2.0 ** -10)


# ---------------------------------------------------------------- the binding

def test_binding_refuses(cuda_device):
    kq, ksc = zeros(4, 16, 2, 128, t=torch.int8), zeros(4, 16, 2, 4, t=F16)
    lay = (kq, kq.clone(), ksc, ksc.clone())
    b = (zeros(4, 2, 128, t=torch.int8), zeros(4, 2, 128, t=torch.int8), zeros(4, 2, 4, t=F16), zeros(4, 2, 4, t=F16))
    q, tab, lens, ws = zeros(3, 8, 128, t=F16), zeros(3, 2), zeros(3), zeros(1 << 26, t=torch.uint8)
    pages, counts, mask, scores = zeros(3, 2, 2), zeros(3, 2), zeros(3, 1), zeros(3, 2, 2, t=F32)

    def refused(match, fn, *args, **kw):
        with pytest.raises((ValueError, qsa.QSAError), match=match):
            fn(*args, **kw)

    f = qsa.qsa_page_bounds
    refused("CUDA tensor", f, tab.cpu(), lens, kq, ksc, *b)
    refused("hi_q must be", f, tab, lens, kq, ksc, b[0][:3], *b[1:])
    refused("lo_sc must be", f, tab, lens, kq, ksc, *b[:3], b[3].float())
    refused("ksc must be", f, tab, lens, kq, ksc[..., :2], *b)
    refused("n_new must be", f, tab, lens, kq, ksc, *b, n_new=zeros(2))
    refused("seq_lens must be", f, tab, lens[:2], kq, ksc, *b)
    refused("err must be", f, tab, lens, kq, ksc, *b, err=torch.zeros(1, dtype=torch.int32))
    f = qsa.qsa_page_score
    refused("float16 or bfloat16", f, q.float(), *b, tab, lens, scores, 16)
    refused("scores must be", f, q, *b, tab, lens, scores.half(), 16)
    refused("scores must be", f, q, *b, tab, lens, scores[:2], 16)
    refused("row per token", f, q, *b, tab[:2], lens, scores, 16)
    refused("rows must be", f, q, *b, tab, lens, scores, 16, rows=zeros(2))
    refused("contiguous", f, q.transpose(0, 1).contiguous().transpose(0, 1), *b, tab, lens, scores, 16)
    f = qsa.qsa_page_select
    refused("counts must be", f, scores, lens, pages, counts[:, :1], 16, 2)
    refused("pages must be", f, scores, lens, pages.long(), counts, 16, 2)
    refused("budget", f, scores, lens, pages, counts, 16, 3)
    refused("seq_lens must be", f, scores, lens.cpu(), pages, counts, 16, 2)
    f = qsa.qsa_paged_sparse_attn
    refused("pages must be", f, q, *lay, tab, lens, pages[:2], counts, q.clone(), ws)
    refused("counts must be", f, q, *lay, tab, lens, pages, counts.long(), q.clone(), ws)
    refused("out must be", f, q, *lay, tab, lens, pages, counts, q.to(BF16), ws)
    refused("workspace smaller", f, q, *lay, tab, lens, pages, counts, q.clone(), ws[:256])
    refused("gate must be", f, q, *lay, tab, lens, pages, counts, q.clone(), ws, gate=q)
    refused("lse must be", f, q, *lay, tab, lens, pages, counts, q.clone(), ws, lse=zeros(3, 7, t=F32))
    refused("row per token", f, q, *lay, tab[:2], lens, pages, counts, q.clone(), ws)
    f = qsa.qsa_paged_tree_attn
    refused("mask must be", f, q, *lay, tab, lens, mask[:2], q.clone(), ws)
    refused("mask must be", f, q, *lay, tab, lens, mask.long(), q.clone(), ws)
    refused("words", f, q, *lay, tab, lens, zeros(3, 33), q.clone(), ws)
    refused("prefix_lens must be", f, q, *lay, tab, lens[:2], mask, q.clone(), ws)
    refused("CUDA tensor", f, q, *lay, tab, lens, mask.cpu(), q.clone(), ws)
    refused("workspace", f, q, *lay, tab, lens, mask, q.clone(), ws.cpu())


def test_binding_paths_agree(cuda_device, monkeypatch):
    """A call that is as it should be goes through the compiled binding alone, and does what the checked one does."""
    from sparse_selected_attention_gb300 import paged
    state, run, results = pick_jobs(62)
    a, b = state(), state()
    with monkeypatch.context() as m:
        for n in ("bounds", "score", "select", "sparse", "tree"):
            m.setattr(paged, "_checked_" + n, None)
        run(a)

    class Never:
        def __getattr__(self, name):
            return lambda *args: -1
    with monkeypatch.context() as m:
        m.setattr(paged, "_native", Never())
        run(b)
    torch.cuda.synchronize()
    assert int(a["e"].item()) == 0 and same(results(a), results(b))
    assert math.isfinite(float(a["o"][0].float().sum()))
