"""Calls on the paged cache whose tokens are of several kinds: what each way of
taking rows reports, that rows of one kind leave others their way, and that a
call's size, order or neighbours do not change how its tokens are taken.

Tolerances as tests/test_paged_pick_gpu.py.
"""
import numpy as np
import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from oracle import paged_oracle as po
from tests.test_paged_gpu import BF16, F16, Serving, dev, i32, make_pool, shuffled_table
from tests.test_paged_pick_gpu import (alike, check_score, check_sparse, check_tree, make_bounds, sparse_workspace, tree_workspace,
                                       trees)

pytestmark = pytest.mark.gpu


def tile_parts(ws, hq, hkv, d):
    """What the groups' CTAs left to be joined, a first row (or -1) for each, by the workspace's layout."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    rows, ctas = hq // hkv, 304
    at = up(up(ctas * 16) + up(ctas * 2 * rows * 8) + ctas * 2 * rows * d * 4)
    return ws[at:at + 152 // hkv * hkv * 16].view(torch.int32)[::4]


def by_groups(ws, hq, hkv, d):
    """Whether groups went through tiles of the cache (of calls whose groups are cut over CTAs): there is a part of one."""
    return bool((tile_parts(ws, hq, hkv, d) >= 0).any())


def decided(ws, hkv):
    """What the device decided, a word for each KV head at the workspace's end: 1 by groups, 0 one by one."""
    return ws[-152 * 4:].view(torch.int32)[:hkv].tolist()


# ---------------------------------------------------------------- what trees report

@pytest.mark.parametrize("n,hq,hkv,d,otype", [(72, 16, 8, 128, F16), (64, 16, 4, 256, BF16), (3, 4, 2, 128, F16)])
def test_tree_reports_what_its_tokens_attend_to(cuda_device, n, hq, hkv, d, otype):
    """Pages that no mask reaches may be missing, whichever way rows are taken; those that one token attends to may not."""
    rng = np.random.default_rng(n)
    page, prefix, together = 16, 2000, n > 3
    table, pages = shuffled_table([prefix + 256], page, 0, rng)
    pool = make_pool(pages, page, hkv, d, seed=n)
    q = rng.standard_normal((n, hq, d))
    sees = np.zeros((n, 256), bool)
    sees[:, :16] = rng.random((n, 16)) < 0.6
    sees[:, 200:208] = rng.random((n, 8)) < 0.6
    pre, rows = [prefix - 5 * (i % 3) for i in range(n)], [0] * n

    def error(sees=sees, pre=pre, table=table, rows=rows):
        mask = np.packbits(sees, axis=1, bitorder="little").view(np.int32)
        ws = tree_workspace(hq, hkv, d)
        check_tree(q, pool, table, pre, mask, rows=rows, otype=otype, ws=ws)
        assert by_groups(ws, hq, hkv, d) == together
        return po.tree_cells(table, pre, mask, hkv, page, pages, rows)[1]

    gone = table.copy()
    gone[0, 128:136], gone[0, 130] = -1, pages  # cells 2048 .. 2175: bits 48 and more of the longest prefix, to 185 of the shortest
    assert error(table=gone) == 0
    one = sees.copy()
    one[n // 2, 70] = True
    assert error(sees=one, table=gone) == po.BAD_ID
    assert error(sees=one) == 0
    hole = table.copy()
    hole[0, 7] = -1
    assert error(table=hole) == po.BAD_ID
    # A page behind all prefixes but one, whose token's bits end before the table does.
    x, few = list(pre), sees.copy()
    x[n - 1], few[n - 1, 16:] = prefix + 70, False
    assert error(sees=few, pre=x) == 0
    assert error(sees=few, pre=x, table=gone) == po.BAD_ID
    for bad in (-4, 10 ** 9, table.shape[1] * page - 100):
        x = list(pre)
        x[1] = bad
        assert error(pre=x) == po.BAD_ID
    x = list(rows)
    x[n - 1] = 1
    assert error(rows=x) == po.BAD_ID


# ---------------------------------------------------------------- trees in any order

@pytest.mark.parametrize("d,hq,hkv,page,seqs,nodes,prefix", [(128, 32, 8, 64, 6, 16, 1500), (256, 24, 2, 16, 4, 60, 2500), (128, 100, 100, 32, 3, 40, 600),
                                                            (128, 154, 77, 128, 2, 9, 900)])
def test_tree_order_decides_how_tokens_are_taken(cuda_device, d, hq, hkv, page, seqs, nodes, prefix):
    """Neighbours of one sequence go together; given level by level, they have none and go one by one, however many there are."""
    rng = np.random.default_rng(seqs)
    pool, table, pre, mask, rows = trees(rng, [prefix + 31 * s for s in range(seqs)], [nodes] * seqs, page, hkv, d, 70)
    q = rng.standard_normal((len(rows), hq, d))
    order = np.arange(len(rows)).reshape(seqs, nodes).T.reshape(-1)
    res = []
    for o in (np.arange(len(rows)), order):
        ws = tree_workspace(hq, hkv, d)
        out, lse = check_tree(q[o], pool, table, [pre[i] for i in o], mask[o], rows=[rows[i] for i in o], ws=ws)
        res.append((out[np.argsort(o)], lse[np.argsort(o)], decided(ws, hkv)))
    assert [x[2] for x in res] == [[1] * hkv, [0] * hkv]
    torch.testing.assert_close(res[0][0].float(), res[1][0].float(), rtol=2.0 ** -8, atol=2.0 ** -9)
    torch.testing.assert_close(res[0][1], res[1][1], rtol=2.0 ** -18, atol=2.0 ** -14)


# ---------------------------------------------------------------- listed rows of several kinds

@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,page,runs,base,most,together", [
    (128, 8, 2, 64, [300] + [1] * 40, 5000, 40, 1), (128, 12, 1, 64, [1] * 17 + [500] + [1] * 8, 6000, 40, 1),
    (128, 8, 2, 64, [9] * 34, 5000, 40, 1), (256, 24, 2, 32, [1, 2, 1, 3] + [170] + [1] * 23, 4000, 60, 1), (128, 16, 1, 16, [5, 3] * 60, 4000, 99, 0),
    (128, 32, 8, 32, [1] * 70, 2000, 50, 0)])
def test_listed_rows_beside_a_chunk_leave_it_together(cuda_device, d, hq, hkv, page, runs, base, most, together, otype):
    """Rows without neighbours, in whole blocks of them, do not keep others from their groups; without others they go one by one."""
    rng = np.random.default_rng(len(runs))
    pool, table, lens, rows, lists, counts = alike(rng, runs, base, page, hkv, d, most + 2, most, 71)
    n = len(rows)
    counts[rng.integers(0, n, 4)] = 0
    lens[n // 3] = 0
    q, gate = rng.standard_normal((n, hq, d)), rng.standard_normal((n, hq, d)).astype(np.float32)

    def run(want_err, lists=lists, table=table, rows=rows):
        ws = sparse_workspace(hq, hkv, d)
        check_sparse(q, pool, table, lens, lists, counts, rows=rows, otype=otype, gate=gate, ws=ws)
        assert po.sparse_cells(table, lens, lists, counts, page, pool[0].shape[0], rows)[1] == want_err
        assert decided(ws, hkv) == [together] * hkv

    run(0)
    if n > 200 or otype is F16:
        return
    # What a row by itself reports.
    t = next(i for i in range(n - 1, -1, -1) if counts[i, 0] > 3 and lens[i])
    x = lists.copy()
    x[t, 0, 2] = table.shape[1]
    run(po.BAD_ID, lists=x)
    x = table.copy()
    x[rows[t], lists[t, 0, 1]] = -1
    run(po.BAD_ID, table=x)
    x = list(rows)
    x[t] = len(table)
    run(po.BAD_ID, rows=x)
    # A page twice in the list of a row without neighbours: it counts twice there, and says nothing about others.
    t = next((i for i in range(n) if rows.count(rows[i]) == 1 and counts[i, 0] > 3 and lens[i]), None)
    if t is not None:
        x = lists.copy()
        x[t, 0, 1] = x[t, 0, 2]
        run(0, lists=x)


@pytest.mark.parametrize("d,hq,hkv,page,runs,base,most,width,otype,last", [
    (128, 16, 8, 16, [150, 90, 60], 1800, 90, 500, F16, 1), (256, 24, 2, 32, [300], 2500, 60, 2000, BF16, 1),
    (128, 12, 1, 64, [200, 1, 1, 1, 1, 1, 60], 4000, 40, 7777, F16, 0)])
def test_listed_calls_of_more_entries_than_the_workspace_holds(cuda_device, d, hq, hkv, page, runs, base, most, width, otype, last):
    """They go in slices of tokens, each by groups where that saves enough in it (not in the last 85 rows of 80 units of a KV
    head: 10 * 85 * 80 is less than a call's cost)."""
    rng = np.random.default_rng(width)
    pool, table, lens, rows, lists, counts = alike(rng, runs, base, page, hkv, d, width, most, 72)
    n = len(rows)
    assert n * hkv * width > 1 << 20
    q, gate = rng.standard_normal((n, hq, d)), rng.standard_normal((n, hq, d)).astype(np.float32)

    def run(want_err, lists=lists, counts=counts):
        ws = sparse_workspace(hq, hkv, d)
        check_sparse(q, pool, table, lens, lists, counts, rows=rows, otype=otype, gate=gate, ws=ws)
        assert po.sparse_cells(table, lens, lists, counts, page, pool[0].shape[0], rows)[1] == want_err
        assert decided(ws, hkv) == [last] * hkv  # of the last slice

    run(0)
    x, y = lists.copy(), counts.copy()
    x[3 if d == 128 else n - 2, hkv - 1, 1] = table.shape[1]  # of the first slice, or the last one
    y[0], y[n - 1] = 0, 0
    run(po.BAD_ID, lists=x, counts=y)


@pytest.mark.parametrize("hq,hkv,width,tried", [(16, 4, 2300, False), (24, 2, 4097, False), (24, 2, 4096, True)])
def test_listed_calls_too_wide_for_groups(cuda_device, hq, hkv, width, tried):
    """Lists so wide that few rows' fill the workspace: one by one, and groups are not even looked for."""
    rng = np.random.default_rng(9)
    pool, table, lens, rows, lists, counts = alike(rng, [150], 3000, 16, hkv, 128, width, 40, 73)
    ws = sparse_workspace(hq, hkv, 128)
    check_sparse(rng.standard_normal((150, hq, 128)), pool, table, lens, lists, counts, rows=rows, ws=ws)
    assert not by_groups(ws, hq, hkv, 128) and (decided(ws, hkv) == [0] * hkv) == tried


# ---------------------------------------------------------------- scores

@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("runs,lo,hi,hkv", [
    ([1] * 300, 1, 4000, 2), ([300] + [1] * 60, 2000, 6000, 1), ([1, 2, 3, 5, 8, 13, 21, 34, 55, 89, 144], 0, 3000, 4), ([9] * 40, 1, 9000, 1),
    ([40, 1, 33, 1, 31, 32, 7] * 3, 500, 800, 8), ([1] * 2500, 1, 200, 1), ([700, 1500, 3, 60], 30, 900, 2), ([17, 260], 12, 12, 3)])
def test_score_of_many_tokens_of_all_kinds(cuda_device, d, runs, lo, hi, hkv):
    """Every page of every token once, however its tokens are shared out; the others keep what they hold."""
    rng = np.random.default_rng(len(runs))
    base = [int(v) for v in rng.integers(lo, hi + 1, len(runs))]
    lens = [b + i for b, k in zip(base, runs) for i in range(k)]
    lens[len(lens) // 2], lens[-1] = 0, 1
    rows = [s for s, k in enumerate(runs) for _ in range(k)]
    table, pages = shuffled_table([b + k for b, k in zip(base, runs)], 16, 2, rng)
    order = rng.permutation(len(runs))  # of the sequences' rows in the table
    table, rows = table[np.argsort(order)], [int(order[r]) for r in rows]
    bounds = make_bounds(pages, hkv, d, 5)
    assert check_score(rng.standard_normal((len(lens), 2 * hkv, d)), bounds, table, lens, 16, rows=rows, ld=table.shape[1] + 1) == 0
    table[rows[0], 0] = pages
    rows[7] = len(runs)
    assert check_score(rng.standard_normal((len(lens), 2 * hkv, d)), bounds, table, lens, 16, rows=rows, otype=BF16) == po.BAD_ID


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,n", [(128, 5), (256, 5), (128, 300), (256, 300)])
def test_score_of_infinite_queries(cuda_device, d, n, otype):
    """An infinite query scores what its products are: infinite by its bound's sign, NaN where that is 0, whatever its other dims hold."""
    rng = np.random.default_rng(n)
    table, pages = shuffled_table([900] * 2, 16, 0, rng)
    b = make_bounds(pages, 2, d, 79)
    b[0][::3, :, 17] = 0
    b[1][:, 0, 40] = -np.abs(b[1][:, 0, 40]) - 1
    q = (rng.standard_normal((n, 8, d)) * 300).astype(np.float32)
    q[1, 5, 17], q[2, 0, 40], q[3, 2, 9], q[3, 3, 9] = np.inf, -np.inf, np.inf, -np.inf
    q[4, 6, 17], q[4, 7, 100] = np.inf, np.nan
    rows = [i % 2 if n < 256 else int(i > n // 2) for i in range(n)]
    qd, scores = dev(q).to(otype), torch.zeros(n, 2, table.shape[1], device="cuda")
    qsa.qsa_page_score(qd, *[dev(x) for x in b], dev(table), i32([900] * n), scores, 16, rows=i32(rows))
    with np.errstate(invalid="ignore"):
        want, _ = po.page_score(qd.float().cpu().numpy(), *b, table, [900] * n, 16, rows)
    wild = 0
    for t in range(n):
        for h in range(2):
            s, a, w, m = want[t][h]
            x, fin = scores[t, h, : len(s)].cpu().numpy().astype(np.float64), np.isfinite(s)
            np.testing.assert_array_equal(x[~fin], s[~fin])
            assert (np.abs(x - s)[fin] <= (2.0 ** -19 * a + 2.0 ** -22 * m * w)[fin]).all()
            wild += int((~fin).any())
    assert wild == 4


def fastest(calls, reps=10, rounds=7):
    """The least time of each call, captured `reps` times; taken in turn."""
    graphs, best = [], [float("inf")] * len(calls)
    for f in calls:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            for _ in range(reps):
                f()
        graphs.append(g)
    for _ in range(rounds):
        for i, g in enumerate(graphs):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            g.replay()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    return best


def test_score_takes_no_longer_for_neighbours_of_other_kinds(cuda_device):
    """Rows of one token each, with and without a table row each said, and beside a prompt's chunk: in the time that they take
    by themselves, a few times over at most (eight and seven times, where tokens were shared out by their number alone)."""
    rng = np.random.default_rng(77)
    page, hkv, hq, d = 16, 2, 12, 128
    lens = [int(v) for v in rng.integers(1, 30000, 256)]
    table, pages = shuffled_table([31984] + lens, page, 0, rng)
    bounds = [dev(x) for x in make_bounds(pages, hkv, d, 78)]
    n = 1024
    q, t = torch.randn(n + 256, hq, d, device="cuda").half(), dev(table)
    held = i32([31984 - n + 1 + i for i in range(n)] + lens)
    rows = i32([0] * n + list(range(1, 257)))
    scores = torch.zeros(n + 256, hkv, table.shape[1], device="cuda")

    def call(a, b, rows, table=t):
        return lambda: qsa.qsa_page_score(q[a:b], *bounds, table, held[a:b], scores[a:b], page, rows=rows)

    own = t[1:].contiguous()
    chunk, single, given, both = fastest([call(0, n, rows[:n]), call(n, n + 256, None, own), call(n, n + 256, rows[n:]), call(0, n + 256, rows)])
    assert given < 4 * single and both < 2 * (chunk + given), (chunk, single, given, both)


# ---------------------------------------------------------------- which kernels ran

@pytest.mark.parametrize("form,otype", [("tree", F16), ("listed", BF16)])
@pytest.mark.parametrize("d,hq,hkv,page,n,cells,together", [
    (128, 16, 8, 32, 72, 1700, 1), (256, 16, 8, 32, 72, 1700, 1), (128, 12, 1, 64, 340, 2600, 1), (256, 24, 2, 16, 130, 1800, 1), (128, 32, 8, 32, 90, 1600, 1),
    (128, 8, 1, 128, 200, 500, 0), (128, 12, 1, 64, 190, 190, 0), (128, 12, 1, 64, 40, 2000, 0), (256, 8, 8, 64, 3, 900, 0)])
def test_groups_are_taken_where_they_save_time(cuda_device, form, d, hq, hkv, page, n, cells, together, otype):
    """Tokens of one sequence, all of whose pages they see: by the partials that each kind leaves and by what the device wrote down."""
    rng = np.random.default_rng(n)
    table, pages = shuffled_table([cells], page, 1, rng)
    pool = make_pool(pages, page, hkv, d, seed=80)
    lens, rows, wide = [cells - n + i + 1 for i in range(n)], [0] * n, table.shape[1]
    q = rng.standard_normal((n, hq, d))
    if form == "tree":
        ws = tree_workspace(hq, hkv, d)
        mask = np.packbits(np.tril(np.ones((n, -(-n // 32) * 32), bool)), axis=1, bitorder="little").view(np.int32)
        check_tree(q, pool, table, [cells - n] * n, mask, rows=rows, otype=otype, ws=ws)
    else:
        ws = sparse_workspace(hq, hkv, d)
        lists = np.broadcast_to(np.arange(wide, dtype=np.int32), (n, hkv, wide)).copy()
        check_sparse(q, pool, table, lens, lists, np.full((n, hkv), wide, np.int32), rows=rows, otype=otype, ws=ws)
    assert by_groups(ws, hq, hkv, d) == bool(together)
    if together:  # then the kernel of rows one by one has none
        assert decided(ws, hkv) == [1] * hkv and bool((ws[: 304 // hkv * hkv * 16].view(torch.int32)[::4] == -1).all())
    else:
        assert 1 not in decided(ws, hkv)


# ---------------------------------------------------------------- digits

@pytest.mark.parametrize("form", ["listed", "tree"])
@pytest.mark.parametrize("d,hq,hkv,n", [(128, 12, 2, 5), (256, 6, 2, 5), (128, 16, 1, 200), (256, 6, 2, 90)])
def test_short_rows_have_exact_scores_behind_wide_lists_and_long_rows(cuda_device, form, d, hq, hkv, n):
    """As tests/test_paged_accuracy_gpu.py derives for short tables: whole-number scores have no rounding but the scale's.
    A row of one cell has them whatever its list's width, its table's and its neighbours' lengths are."""
    rng = np.random.default_rng(81)
    long = 1200
    table, pages = shuffled_table([long] + [1] * (n - 1), 16, 1, rng)
    pool = make_pool(pages, 16, hkv, d, seed=82)
    pool[2][:] = 2.0 ** -7
    q = rng.integers(0, 2048, (n, hq, d)).astype(np.float64)
    scale, per = 2.0 ** -12, hq // hkv
    prod = q * np.repeat(pool[0][table[:, 0], 0].astype(np.float64), per, 1)
    assert np.abs(prod.reshape(n, hq, 4, -1)).sum(-1).max() < 2 ** 24 and np.abs(np.cumsum(prod, -1)).max() < 2 ** 24
    s = torch.from_numpy(prod.sum(-1) * 2.0 ** -19).cuda()[1:]
    qd = dev(q.astype(np.float16))
    out, lse = torch.empty_like(qd), torch.empty(n, hq, device="cuda")
    args = [qd, *[dev(x) for x in pool], dev(table)]
    if form == "listed":
        lists = np.full((n, hkv, table.shape[1]), -1, np.int32)
        lists[:, :, 0], lists[0] = 0, np.arange(table.shape[1])
        counts = np.ones((n, hkv), np.int32)
        counts[0] = -(-long // 16)
        qsa.qsa_paged_sparse_attn(*args, i32([long] + [1] * (n - 1)), dev(lists), dev(counts), out, sparse_workspace(hq, hkv, d), lse=lse,
                                  softmax_scale=scale)
    else:
        qsa.qsa_paged_tree_attn(*args, i32([long - 1] + [0] * (n - 1)), dev(np.ones((n, 1), np.int32)), out, tree_workspace(hq, hkv, d), lse=lse,
                                softmax_scale=scale)
    assert ((lse[1:].double() - s).abs() <= 2.0 ** -21 * s.abs() + 2.0 ** -21).all(), ((lse[1:].double() - s).abs() / s.abs()).max()


# ---------------------------------------------------------------- after a tree

def test_an_accepted_path_is_moved_behind_its_prefix(cuda_device):
    """A tree's cells lie as its nodes were numbered.  Copied one after the other behind the prefix, the accepted ones are
    what the same tokens make when they are appended, and the sequence goes on from there."""
    make = lambda: Serving(2, hq=12, hkv=2, page=16, pages=40, wide=16)  # noqa: E731
    a, b = make(), make()
    gen = torch.Generator(device="cuda").manual_seed(4)
    rand = lambda n: torch.randn(n, 16, 128, generator=gen, device="cuda").half()  # noqa: E731
    empty = lambda n: torch.empty(n, 12, 128, dtype=F16, device="cuda")  # noqa: E731
    prompts = rand(37 + 46)
    for s in (a, b):
        s.update(None, i32(37, 46))
        s.write(prompts, empty(len(prompts)))
    parent, path = [-1, 0, 0, 1, 2, 2, 5, -1, 7, 6], [0, 2, 5, 6, 9]
    depth, sees = [], np.zeros((len(parent), 32), bool)
    for i, p in enumerate(parent):
        depth.append(depth[p] + 1 if p >= 0 else 0)
        sees[i] = sees[p] if p >= 0 else False
        sees[i, i] = True
    x, n = rand(len(parent)), len(parent)
    a.update(None, i32(0, n))
    q, out, err = empty(n), empty(n), a.err
    qsa.qsa_paged_prep(x[:, :12], x[:, 12:14], x[:, 14:], i32([46 + k for k in depth]), a.slots[:n], *a.layer(), q, q_norm_w=a.w, k_norm_w=a.w,
                       inv_freq=a.freq, err=err)
    mask = dev(np.packbits(sees, axis=1, bitorder="little").view(np.int32))
    qsa.qsa_paged_tree_attn(q, *a.layer(), a.table, i32([46] * n), mask, out, tree_workspace(12, 2, 128), rows=i32([1] * n), err=err)

    def cells(c):
        c = torch.as_tensor(c, device="cuda")
        return a.table[1].long()[c // 16] * 16 + c % 16

    src, dst = cells([46 + i for i in path]), cells([46 + k for k in range(len(path))])
    for t in a.pool:
        rows = t.flatten(1, 2)
        rows[:, dst] = rows[:, src]
    a.lens[1] = 46 + len(path)
    # The same tokens appended, each attending to what is before it.
    b.update(None, i32(0, len(path)))
    qb, ob = empty(len(path)), empty(len(path))
    b.write(x[path], qb)
    qsa.qsa_paged_attn(qb, *b.layer(), b.table, i32([47 + k for k in range(len(path))]), ob, b.aws, rows=i32([1] * len(path)), err=b.err)
    assert torch.equal(q[path], qb)
    torch.testing.assert_close(out[path].float(), ob.float(), rtol=2.0 ** -9, atol=2.0 ** -10)
    for _ in range(3):
        for r in range(2):
            assert all(torch.equal(y, z) for y, z in zip(a.kv(r), b.kv(r)))
        y = rand(2)
        for s in (a, b):
            s.update(None, i32(1, 1))
            s.q, s.o = empty(2), empty(2)
            s.write(y, s.q)
            s.attend(s.q, s.o)
        assert torch.equal(a.o, b.o) and a.lens.tolist() == b.lens.tolist()
    assert int(a.err.item()) == 0 and int(b.err.item()) == 0
