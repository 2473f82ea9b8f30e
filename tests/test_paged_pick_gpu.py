"""Picked pages and trees of drafts on the GPU against their float64 oracle.

Tolerances:
  bounds, lists, counts   exact, bit for bit;
  scores   a term is q sum * bound.  The sums of up to 16 heads are added in fp32
           (15 * 2^-24 of the terms), go as two fp16 parts under a power of two
           (each off by up to 2^-22 of the token's largest sum `m`), and their
           products are added in up to 4 + 2 + 8 steps of a quarter's k-steps, the
           parts and the quarters (tensor cores truncate: 2^-23 of the terms each):
           2^-19 sum |terms| + 2^-22 m sum (|hi| + |lo|);
  attention  as tests/test_paged_gpu.py derives for rows one by one; rows taken
           together are off by less (tests/test_paged_groups_gpu.py).
"""
import numpy as np
import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from oracle import paged_oracle as po
from tests.test_paged_gpu import BF16, F16, HALF, TINY, dev, err_word, host, i32, make_pool, shuffled_table
from tests.test_paged_pick_cpu import random_tree

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- bounds

def run_bounds(table, lens, new, pool, sentinel=77):
    pages, _, hkv, d = pool[0].shape
    q = [torch.full((pages, hkv, d), sentinel, dtype=torch.int8, device="cuda") for _ in range(2)]
    sc = [torch.full((pages, hkv, 4), 9.0, dtype=F16, device="cuda") for _ in range(2)]
    err = err_word()
    qsa.qsa_page_bounds(dev(table), i32(lens), dev(pool[0]), dev(pool[2]), *q, *sc, n_new=None if new is None else i32(new), err=err)
    return q + sc, int(err.item())


def check_bounds(table, lens, new, pool):
    got, err = run_bounds(table, lens, new, pool)
    want, werr = po.page_bounds(table, lens, new, pool[0], pool[2])
    assert err == werr
    full = [np.full(x.shape, 77 if i < 2 else 9.0, np.int8 if i < 2 else np.float16) for i, x in enumerate(got)]
    for p, parts in want.items():
        for f, x in zip(full, parts):
            f[p] = x
    for f, x in zip(full, got):
        np.testing.assert_array_equal(x.cpu().numpy(), f)
    return want, err


@pytest.mark.parametrize("d,hkv,page", [(128, 1, 64), (256, 2, 16), (128, 4, 16), (256, 1, 32), (128, 3, 128), (256, 5, 256), (128, 8, 256)])
@pytest.mark.parametrize("fresh", [None, 1, 5, 300])
def test_bounds(cuda_device, d, hkv, page, fresh):
    rng = np.random.default_rng(page)
    lens = [0, 1, 7, 15, 16, 17, 63, 64, 65, 129, 255, 256, 257, 600]
    table, pages = shuffled_table(lens, page, 4, rng)
    pool = make_pool(pages, page, hkv, d, seed=page)
    new = None if fresh is None else [min(n, fresh) if i % 5 else 0 for i, n in enumerate(lens)]
    want, err = check_bounds(table, lens, new, pool)
    assert err == 0 and want


@pytest.mark.parametrize("rows,hi,page", [(1, 30008, 64), (300, 200, 16), (1100, 40, 32), (40, 3000, 256)])
def test_bounds_many_rows(cuda_device, rows, hi, page):
    rng = np.random.default_rng(rows)
    lens = [int(v) for v in rng.integers(0, hi + 1, rows)]
    lens[-1] = hi
    table, pages = shuffled_table(lens, page, 2, rng)
    pool = make_pool(pages, page, 2, 128, seed=rows)
    check_bounds(table, lens, None, pool)
    check_bounds(table, lens, [min(n, int(v)) for n, v in zip(lens, rng.integers(0, 90, rows))], pool)


def test_bounds_extreme_scales(cuda_device):
    """Zero, subnormal, largest, negative, infinite and NaN scales."""
    pool = make_pool(12, 16, 2, 128, seed=1)
    ksc = pool[2]
    ksc[0] = 0
    ksc[1] = np.float16(6e-8)
    ksc[2] = np.float16(65504)
    ksc[3] *= np.float16(-1)
    ksc[4, 3, 1, 2] = np.float16(np.inf)
    ksc[5, 0, 0, 0], ksc[5, 1, 1, 3] = np.float16(np.nan), np.float16(-np.inf)
    ksc[6, 9:] = np.float16(np.nan)  # behind the last cell of its row
    pool[0][7] = -128
    pool[0][8], pool[0][9] = 127, -127
    ksc[10, ::2], ksc[10, 1::2] = np.float16(1e-7), np.float16(2e4)
    table = np.arange(12, dtype=np.int32).reshape(12, 1)
    lens = [16] * 12
    lens[6] = 9
    got, err = run_bounds(table, lens, None, pool)
    pool[0][7] = -127  # a code of -128 is no code of this cache: not compared
    want, _ = po.page_bounds(table, lens, None, pool[0], pool[2])
    assert err == 0
    for p in set(want) - {7}:
        for g, w in zip(got, want[p]):
            np.testing.assert_array_equal(g[p].cpu().numpy(), w)
    assert torch.isnan(got[2][4, 1, 2]) and not torch.isnan(got[2][4, 1, :2]).any() and not torch.isnan(got[2][6]).any()


def test_bounds_bad_inputs(cuda_device):
    rng = np.random.default_rng(3)
    lens = [40, 33, 20, 48, 10]
    table, pages = shuffled_table(lens, 16, 3, rng)
    pool = make_pool(pages, 16, 1, 128, seed=2)
    table[0, 1] = pages + 5
    table[1, 2] = -3
    assert check_bounds(table, lens, None, pool)[1] == po.BAD_ID
    assert check_bounds(table, lens, [1] * 5, pool)[1] == po.BAD_ID
    table, _ = shuffled_table(lens, 16, 3, rng)
    assert check_bounds(table, lens, [0, 40, 3, -4, 2], pool)[1] == po.BAD_ID
    assert check_bounds(table, [40, -7, 20, 9, 10], None, pool)[1] == po.BAD_ID
    lens[3] = 49
    assert check_bounds(table, lens, [1] * 5, pool)[1] == po.BAD_ID
    assert not check_bounds(table, [0] * 5, None, pool)[0]


def test_bounds_of_forked_rows_and_read_back(cuda_device):
    """Rows that hold the same pages; qsa_paged_gather reads the bounds as a cache."""
    rng = np.random.default_rng(5)
    table, pages = shuffled_table([100, 100, 100], 32, 1, rng)
    table[1], table[2, :3] = table[0], table[0, :3]
    pool = make_pool(pages, 32, 2, 256, seed=7)
    want, err = check_bounds(table, [100, 100, 97], None, [pool[0], pool[1], pool[2], pool[3]])
    (hi, lo, hs, ls), _ = run_bounds(table, [100, 100, 97], None, pool)
    ids = i32(table[0])
    a, b = (torch.empty(4, 2, 256, device="cuda") for _ in range(2))
    qsa.qsa_paged_gather(hi, lo, hs, ls, ids, a, b)
    for out, q, sc in ((a, hi, hs), (b, lo, ls)):
        assert torch.equal(out, q[ids.long()].float() * sc[ids.long()].float().repeat_interleave(64, -1))
    assert err == 0 and (a >= b).all()


# ---------------------------------------------------------------- score

def make_bounds(pages, hkv, d, seed, lo=0.01, hi=0.02):
    rng = np.random.default_rng(seed)
    hq, lq = rng.integers(-30, 128, (pages, hkv, d)).astype(np.int8), rng.integers(-127, 31, (pages, hkv, d)).astype(np.int8)
    sc = [rng.uniform(lo, hi, (pages, hkv, 4)).astype(np.float16) for _ in range(2)]
    return [hq, lq, *sc]


def check_score(q, bounds, table, lens, page, rows=None, ld=None, otype=F16):
    T, H, D = q.shape
    hkv = bounds[0].shape[1]
    qd = dev(q.astype(np.float32)).to(otype)
    scores = torch.full((T, hkv, ld or table.shape[1]), 12345.0, device="cuda")
    err = err_word()
    qsa.qsa_page_score(qd, *[dev(x) for x in bounds], dev(table), i32(lens), scores, page, rows=None if rows is None else i32(rows), err=err)
    want, werr = po.page_score(host(qd), *bounds, table, lens, page, rows)
    got = scores.cpu().numpy().astype(np.float64)
    for t in range(T):
        for h in range(hkv):
            s, a, b, m = want[t][h]
            tol = 2.0 ** -19 * a + 2.0 ** -22 * m * b
            x = got[t, h, : len(s)]
            ok = (np.abs(x - s) <= tol) | (x == s)
            assert ok.all(), (t, h, np.argwhere(~ok)[:5].tolist(), x[~ok][:5], s[~ok][:5], tol[~ok][:5])
            assert (got[t, h, len(s):] == 12345.0).all()
    assert int(err.item()) == werr
    return werr


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,page", [(128, 12, 1, 64), (256, 24, 2, 16), (128, 32, 8, 32), (128, 16, 1, 256), (128, 2, 2, 128),
                                           (256, 1, 1, 256), (256, 9, 3, 32)])
def test_score_shapes(cuda_device, d, hq, hkv, page, otype):
    rng = np.random.default_rng(1)
    lens = [0, 1, page, page + 1, 15 * page, 16 * page, 16 * page + 1, 33 * page - 1, 700]
    table, pages = shuffled_table(lens, page, 3, rng)
    q = rng.standard_normal((len(lens), hq, d)) * 2
    assert check_score(q, make_bounds(pages, hkv, d, 2), table, lens, page, otype=otype, ld=table.shape[1] + 3) == 0


@pytest.mark.parametrize("n,lo,hi,hkv", [(1, 30008, 30008, 1), (61, 1, 9000, 4), (700, 1, 300, 2), (3, 1, 60000, 1)])
def test_score_ragged(cuda_device, n, lo, hi, hkv):
    rng = np.random.default_rng(n)
    lens = [int(v) for v in rng.integers(lo, hi + 1, n)]
    table, pages = shuffled_table(lens, 16, 3, rng)
    q = rng.standard_normal((n, 4 * hkv, 128))
    assert check_score(q, make_bounds(pages, hkv, 128, 3), table, lens, 16) == 0


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("runs,base", [([1, 2, 3, 4, 5, 9], 500), ([300], 2500), ([31, 33, 64, 1, 200, 7], 900), ([0, 257], 0)])
def test_score_tokens_of_one_sequence(cuda_device, d, runs, base):
    """Draft windows, chunks, and both ways that tokens are taken together."""
    rng = np.random.default_rng(len(runs))
    held = [base + k for k in runs]
    table, pages = shuffled_table(held, 16, 1, rng)
    rows = [s for s, k in enumerate(runs) for _ in range(k)]
    lens = [base + i for k in runs for i in range(k)]
    q = rng.standard_normal((len(rows), 6, d)) * 1.5
    assert check_score(q, make_bounds(pages, 2, d, 4), table, lens, 16, rows=rows) == 0


@pytest.mark.parametrize("size", [1e-6, 1e-3, 300.0, 60000.0])
def test_score_query_magnitudes(cuda_device, size):
    rng = np.random.default_rng(6)
    lens = [300, 900, 40, 77]
    table, pages = shuffled_table(lens, 32, 1, rng)
    q = rng.uniform(-1, 1, (4, 16, 128)) * size
    q[1, :, 64:] = 0
    q[2] = 0
    q[3, :, ::2] *= 1e-4
    check_score(q, make_bounds(pages, 1, 128, 5, 1e-3, 30.0), table, lens, 32, otype=F16 if size > 1 else BF16)
    check_score(q, make_bounds(pages, 1, 128, 5, 1e-3, 30.0), table, lens, 32, otype=BF16)


def test_score_bad_inputs(cuda_device):
    rng = np.random.default_rng(7)
    lens = [500, 80, 333]
    table, pages = shuffled_table(lens, 16, 1, rng)
    b, q = make_bounds(pages, 2, 128, 6), rng.standard_normal((3, 8, 128))
    table[0, 3], table[0, 20] = pages, -1
    assert check_score(q, b, table, lens, 16) == po.BAD_ID
    assert check_score(q, b, table, [10, -1, 10 ** 6], 16) == po.BAD_ID
    assert check_score(q, b, table, lens, 16, rows=[1, 3, -1]) == po.BAD_ID
    assert check_score(q, b, table, [0, 0, 0], 16) == 0


def test_score_nan_pages_and_queries(cuda_device):
    """A NaN scale makes its page's score NaN, a NaN or infinite query its token's, and no other."""
    rng = np.random.default_rng(8)
    table, pages = shuffled_table([400] * 3, 16, 0, rng)
    b, q = make_bounds(pages, 2, 128, 9), rng.standard_normal((3, 8, 128))
    b[2][table[1, 4], 1, 2] = np.nan
    q[2, 5, 17] = np.nan
    q[0, 1, 100] = np.inf
    scores = torch.zeros(3, 2, 25, device="cuda")
    qsa.qsa_page_score(dev(q.astype(np.float16)), *[dev(x) for x in b], dev(table), i32([400] * 3), scores, 16)
    bad = ~torch.isfinite(scores)
    want = torch.zeros_like(bad)
    want[1, 1, 4] = True
    want[2, 1] = True
    want[0, 0] = True
    assert torch.equal(bad, want)


# ---------------------------------------------------------------- select

def check_select(scores, lens, page, budget, sink, local, width=None):
    T, hkv, _ = scores.shape
    width = width or budget
    pages = torch.full((T, hkv, width), 99, dtype=torch.int32, device="cuda")
    counts = torch.full((T, hkv), 99, dtype=torch.int32, device="cuda")
    err = err_word()
    qsa.qsa_page_select(dev(scores), i32(lens), pages, counts, page, budget, sink=sink, local=local, err=err)
    want, wcount, werr = po.page_select(scores, lens, page, budget, sink, local, width)
    np.testing.assert_array_equal(pages.cpu().numpy(), want)
    np.testing.assert_array_equal(counts.cpu().numpy(), wcount)
    assert int(err.item()) == werr
    return werr


@pytest.mark.parametrize("ld", [5, 32, 33, 500, 512, 513, 2000, 2048, 2049, 9001, 16384, 16385, 40000])
@pytest.mark.parametrize("budget,sink,local", [(1, 0, 0), (4, 1, 2), (32, 1, 4), (128, 0, 16), (1000, 500, 500)])
def test_select(cuda_device, ld, budget, sink, local):
    rng = np.random.default_rng(ld)
    n = [0, 1, budget - 1, budget, budget + 1, ld // 2, ld - 1, ld]
    lens = [max(0, min(v, ld)) * 16 - (7 if 0 < v else 0) for v in n]
    lens = [max(v, 0) for v in lens]
    scores = rng.standard_normal((len(lens), 2, ld)).astype(np.float32)
    scores[:, 1] = rng.integers(0, 40, scores[:, 1].shape)  # many ties
    assert check_select(scores, lens, 16, budget, sink, local, width=budget + 3) == 0


@pytest.mark.parametrize("ld", [70, 700, 7000, 20000])
def test_select_special_values(cuda_device, ld):
    rng = np.random.default_rng(ld)
    pick = np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-40, -1e-40, 3.4e38, -3.4e38, 1.0], np.float32)
    scores = pick[rng.integers(0, len(pick), (6, 3, ld))]
    scores[1] = np.nan
    scores[2] = -np.inf
    scores[3, 0] = 7.0
    scores[3, 1, : ld // 2] = np.nan
    scores[4] = np.where(rng.random((3, ld)) < 0.9, np.nan, scores[4])
    for budget, sink, local in ((2, 0, 1), (40, 3, 5), (ld - 2, 1, 1), (33, 0, 0)):
        assert check_select(scores, [ld * 64] * 6, 64, budget, sink, local) == 0


def test_select_skewed_scores(cuda_device):
    """Scores over all exponents, and a few that lie far above the rest."""
    rng = np.random.default_rng(11)
    scores = (rng.choice([-1.0, 1.0], (5, 2, 1500)) * 2.0 ** rng.uniform(-140, 127, (5, 2, 1500))).astype(np.float32)
    scores[3] = 40 + 1e-5 * rng.standard_normal((2, 1500))
    scores[4, :, :20] = 1e30
    for budget in (1, 7, 20, 21, 64, 1400):
        assert check_select(scores, [1500 * 16 - 3 * i for i in range(5)], 16, budget, 0, 0) == 0


def test_select_bad_lengths_and_neighbours(cuda_device):
    rng = np.random.default_rng(12)
    scores = rng.standard_normal((4, 3, 21)).astype(np.float32)
    assert check_select(scores, [-5, 400, 16 * 21, 2 ** 31 - 1], 16, 9, 1, 1, width=20) == po.BAD_ID


# ---------------------------------------------------------------- attention

def check_cells(fn, q, pool, args, cells, werr, scale=None, gate=None, otype=F16, rows=None, ws=None):
    """Compares a call with the oracle's attention over `cells`."""
    T, H, D = q.shape
    hkv = pool[0].shape[2]
    qd = q if isinstance(q, torch.Tensor) else dev(q.astype(np.float32)).to(otype)
    out, lse, err = torch.full_like(qd, 9.0), torch.full((T, H), 9.0, device="cuda"), err_word()
    if ws is None:
        ws = torch.full((getattr(qsa, fn + "_workspace_bytes")(H, hkv, D),), 0xA5, dtype=torch.uint8, device="cuda")
    getattr(qsa, fn)(qd, *[dev(x) for x in pool], *args, out, ws, rows=None if rows is None else i32(rows), softmax_scale=scale,
                     gate=None if gate is None else dev(gate), lse=lse, err=err)
    ref, rlse, mag, flush, qk = po.attn_cells(host(qd), *pool, cells, scale, gate)
    ds = 1152 * qk * 2.0 ** -21
    tol = HALF[qd.dtype] * np.abs(ref) + mag * (2.0 ** -10 + 2 * np.expm1(ds)[..., None] + 2.0 ** -16) + flush * 2.0 ** -24 + TINY[qd.dtype]
    got, g = host(out), lse.cpu().numpy().astype(np.float64)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), got[bad][:5], ref[bad][:5], tol[bad][:5])
    assert np.array_equal(np.isneginf(g), np.isneginf(rlse)) and not got[np.isneginf(rlse)].any()
    fin = np.isfinite(rlse)
    assert np.all(np.abs(g[fin] - rlse[fin]) <= ds[fin] + 2.0 ** -16 + 2.0 ** -22 * np.abs(rlse[fin]))
    assert int(err.item()) == werr
    return out, lse


def random_lists(rng, lens, hkv, page, width, most):
    """Lists of up to `most` of each row's pages, ascending, -1 padded, with their counts."""
    pages, counts = np.full((len(lens), hkv, width), -1, np.int32), np.zeros((len(lens), hkv), np.int32)
    for t, n in enumerate(lens):
        have = -(-n // page)
        for h in range(hkv):
            k = min(have, most)
            got = np.sort(rng.permutation(have)[:k])
            if k and rng.random() < 0.7:
                got[-1] = have - 1
            pages[t, h, :k], counts[t, h] = got, k
    return pages, counts


def check_sparse(q, pool, table, lens, pages, counts, **kw):
    cells, werr = po.sparse_cells(table, lens, pages, counts, pool[0].shape[1], pool[0].shape[0], kw.get("rows"))
    return check_cells("qsa_paged_sparse_attn", q, pool, (dev(table), i32(lens), dev(pages), dev(counts)), cells, werr, **kw)


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,page,width", [(128, 12, 1, 64, 6), (256, 24, 2, 16, 5), (128, 32, 8, 32, 12), (128, 16, 1, 16, 40),
                                                 (128, 2, 2, 128, 9), (256, 1, 1, 256, 3), (256, 9, 3, 32, 33), (128, 8, 4, 16, 1)])
def test_sparse_shapes(cuda_device, d, hq, hkv, page, width, otype):
    rng = np.random.default_rng(width)
    lens = [0, 1, 15, 16, 17, 33, 64, 65, 129, 257, 700, 1500, 2222]
    table, pages = shuffled_table(lens, page, 3, rng)
    pool = make_pool(pages, page, hkv, d, seed=12)
    lists, counts = random_lists(rng, lens, hkv, page, width, width)
    q = rng.standard_normal((len(lens), hq, d)) * 2
    check_sparse(q, pool, table, lens, lists, counts, otype=otype)


@pytest.mark.parametrize("n,hkv,hi,page,width", [(1, 1, 30008, 64, 32), (3, 2, 9000, 16, 100), (50, 4, 3000, 16, 64), (400, 1, 900, 64, 4),
                                                 (330, 2, 400, 16, 2), (170, 2, 5000, 16, 4), (130, 1, 4000, 32, 30)])
def test_sparse_shared_out(cuda_device, n, hkv, hi, page, width):
    """Rows whose heads have lists of other lengths, over all ways that work is shared out."""
    rng = np.random.default_rng(n)
    lens = [int(v) for v in rng.integers(0, hi + 1, n)]
    lens[0] = hi
    table, pages = shuffled_table(lens, page, 3, rng)
    pool = make_pool(pages, page, hkv, 128, seed=n)
    lists, counts = random_lists(rng, lens, hkv, page, width, width)
    for t in range(n):
        for h in range(hkv):
            if rng.random() < 0.4:
                k = int(rng.integers(0, counts[t, h] + 1))
                lists[t, h, k:], counts[t, h] = -1, k
    gate = rng.standard_normal((n, 4 * hkv, 128)).astype(np.float32) * 2
    q = rng.standard_normal((n, 4 * hkv, 128)) * 2
    check_sparse(q, pool, table, lens, lists, counts, gate=gate)
    check_sparse(q, pool, table, lens, lists, counts, otype=BF16, scale=0.2)


def test_sparse_chunk_with_rows(cuda_device):
    """Tokens of two sequences, each token with pages of its own."""
    rng = np.random.default_rng(21)
    held = [1500, 700]
    table, pages = shuffled_table(held, 16, 3, rng)
    rows = [0] * 90 + [1] * 60
    lens = [1500 - 89 + i for i in range(90)] + [700 - 59 + i for i in range(60)]
    pool = make_pool(pages, 16, 2, 128, seed=21)
    lists, counts = random_lists(rng, lens, 2, 16, 40, 37)
    check_sparse(rng.standard_normal((150, 24, 128)), pool, table, lens, lists, counts, rows=rows)


@pytest.mark.parametrize("page", [16, 64])
def test_sparse_any_order_twice_and_gaps(cuda_device, page):
    rng = np.random.default_rng(22)
    lens = [10 * page - 5, 6 * page, 4 * page - 1, 40, page]
    table, pages = shuffled_table(lens, page, 3, rng, wide=12)
    pool = make_pool(pages, page, 2, 128, seed=22)
    lists = np.array([[9, 0, -1, 3, 3, 9, -1, 2], [-1, -1, 5, 1, -1, 0, 0, 0], [3, -1, 3, 2, 1, 0, 3, 3], [0, 1, 2, -1, -1, -1, -1, 3],
                      [-1] * 8], np.int32)
    lists = np.stack([lists, lists[:, ::-1]], 1).copy()
    lists[4, 1, 2] = 0
    counts = np.array([[8, 6], [8, 3], [7, 8], [8, 8], [8, 8]], np.int32)
    check_sparse(rng.standard_normal((5, 8, 128)), pool, table, lens, lists, counts)


def test_sparse_bad_inputs(cuda_device):
    rng = np.random.default_rng(23)
    lens = [300, 500, 100, 250]
    table, pages = shuffled_table(lens, 32, 3, rng)
    pool = make_pool(pages, 32, 1, 128, seed=23)
    q = rng.standard_normal((4, 12, 128))
    lists, counts = random_lists(rng, lens, 1, 32, 6, 4)

    def both(lists=lists, counts=counts, table=table, lens=lens, rows=None):
        cells, err = po.sparse_cells(table, lens, lists, counts, 32, pages, rows)
        check_sparse(q, pool, table, lens, lists, counts, rows=rows)
        return err

    assert both() == 0
    for at, v in (((0, 0, 1), table.shape[1]), ((1, 0, 0), -2), ((2, 0, 2), 2 ** 31 - 1), ((3, 0, 3), -2 ** 31)):
        x = lists.copy()
        x[at] = v
        assert both(lists=x) == po.BAD_ID
    x = counts.copy()
    x[0], x[1] = 7, -1
    assert both(counts=x) == po.BAD_ID
    x = table.copy()
    x[1, lists[1, 0, 0]] = pages
    assert both(table=x) == po.BAD_ID
    assert both(lens=[300, -1, 10 ** 7, 250]) == po.BAD_ID
    assert both(rows=[0, 4, -1, 3]) == po.BAD_ID


def alike_lists(rng, lens, rows, hkv, page, width, most, spread=0.3):
    """Lists of up to `most` pages by scores that the tokens of a sequence mostly share, the first and the last page among them."""
    have = -(-max(lens) // page)
    base = rng.standard_normal((max(rows) + 1, hkv, have))
    pages, counts = np.full((len(lens), hkv, width), -1, np.int32), np.zeros((len(lens), hkv), np.int32)
    for t, (n, r) in enumerate(zip(lens, rows)):
        own = -(-n // page)
        for h in range(hkv):
            x = (base[r, h] + spread * rng.standard_normal(have))[:own]
            if own:
                x[[0, -1]] = 99.0
            k = min(own, most)
            pages[t, h, :k], counts[t, h] = np.sort(np.argsort(-x)[:k]), k
    return pages, counts


def alike(rng, runs, base, page, hkv, d, width, most, seed, spread=0.3):
    """Pool, table, lengths, rows and lists: runs[s] tokens of sequence s, of base cells and on."""
    rows = [s for s, n in enumerate(runs) for _ in range(n)]
    lens = [base + 37 * s + i for s, n in enumerate(runs) for i in range(n)]
    table, pages = shuffled_table([base + 37 * s + n for s, n in enumerate(runs)], page, 3, rng)
    lists, counts = alike_lists(rng, lens, rows, hkv, page, width, most, spread)
    return make_pool(pages, page, hkv, d, seed=seed), table, lens, rows, lists, counts


def sparse_workspace(hq, hkv, d):
    return torch.full((qsa.qsa_paged_sparse_attn_workspace_bytes(hq, hkv, d),), 0xA5, dtype=torch.uint8, device="cuda")


def taken_together(ws):
    """Whether a call on long rows took them by groups: then no row is shared out one by one."""
    return not bool((ws[: 304 * 16].view(torch.int32)[::4] >= 0).any())


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,page,runs,base,most", [
    (128, 12, 1, 64, [340], 9000, 40), (128, 12, 1, 64, [177, 140, 1, 9, 60], 5000, 40), (128, 32, 8, 32, [90], 2500, 50),
    (128, 16, 2, 16, [180, 175], 4000, 100), (128, 2, 2, 256, [71], 9000, 30), (256, 24, 2, 16, [130], 4000, 110),
    (256, 16, 1, 128, [190, 63], 9000, 30), (256, 5, 5, 64, [75], 3000, 40), (128, 8, 1, 128, [200], 300, 3), (128, 12, 1, 64, [190], 3, 99)])
def test_sparse_alike_lists_taken_together(cuda_device, d, hq, hkv, page, runs, base, most, otype):
    rng = np.random.default_rng(most)
    pool, table, lens, rows, lists, counts = alike(rng, runs, base, page, hkv, d, most + 4, most, 37)
    ws = sparse_workspace(hq, hkv, d)
    gate = rng.standard_normal((len(rows), hq, d)).astype(np.float32) if otype == F16 else None
    check_sparse(rng.standard_normal((len(rows), hq, d)), pool, table, lens, lists, counts, rows=rows, otype=otype, gate=gate, ws=ws)
    assert taken_together(ws)  # or rows so short that none is shared out


@pytest.mark.parametrize("d,hq,hkv,page", [(128, 12, 1, 64), (256, 24, 2, 16)])
def test_sparse_groups_with_gaps_ends_and_bad_inputs(cuda_device, d, hq, hkv, page):
    """Rows that see nothing, lists in any order with gaps, counts of junk, tables and rows out of range, in groups."""
    rng = np.random.default_rng(38)
    n, most = 190 if hkv == 2 else 420, 2048 // page
    pool, table, lens, rows, lists, counts = alike(rng, [n], 4000, page, hkv, d, most + 3, most, 38)
    lists[:, :, most:] = 10 ** 6  # past the counts
    for t in range(n):
        if t % 3 == 0:
            lists[t, :, :most] = lists[t, :, rng.permutation(most)].T
        if t % 4 == 1:
            lists[t, :, rng.integers(0, most, 5)] = -1
    lens[3], lens[20], lens[21], lens[40], lens[41] = 0, 1, page, 17, 1000
    counts[5], counts[6], counts[7, 0] = 0, 1, 3
    q = rng.standard_normal((n, hq, d))

    def run(want_err, lists=lists, counts=counts, table=table, lens=lens, rows=rows, together=True, **kw):
        ws = sparse_workspace(hq, hkv, d)
        check_sparse(q, pool, table, lens, lists, counts, rows=rows, ws=ws, **kw)
        assert po.sparse_cells(table, lens, lists, counts, page, pool[0].shape[0], rows)[1] == want_err
        assert taken_together(ws) == together

    run(0)
    run(0, scale=-0.15)
    run(0, scale=0.0, otype=BF16)
    x = lists.copy()
    x[9, 0, 2], x[10, hkv - 1, 0], x[11, 0, 1], x[12, 0, 4] = table.shape[1], -2, 2 ** 31 - 1, -2 ** 31
    run(po.BAD_ID, lists=x)
    x = counts.copy()
    x[30], x[31] = -1, 0
    run(po.BAD_ID, counts=x)
    x = table.copy()
    x[0, lists[50, 0, 3]], x[0, 0] = pool[0].shape[0], -1
    run(po.BAD_ID, table=x)
    x = list(lens)
    x[60] = -5
    run(po.BAD_ID, lens=x)
    x = list(rows)
    x[70], x[80] = 1, -1
    run(po.BAD_ID, rows=x)
    # A page that a list holds twice counts twice: then rows go one by one, all of that KV head's.
    x = lists.copy()
    x[2, :, 1] = x[2, :, 0]
    run(0, lists=x, together=False)


def test_sparse_groups_are_left_where_they_save_nothing(cuda_device):
    rng = np.random.default_rng(39)
    pool, table, lens, rows, lists, counts = alike(rng, [100], 30000, 64, 1, 128, 32, 32, 39, spread=50.0)
    ws = sparse_workspace(12, 1, 128)
    check_sparse(rng.standard_normal((100, 12, 128)), pool, table, lens, lists, counts, rows=rows, ws=ws)
    assert not taken_together(ws)
    rows = [i % 10 for i in range(100)]
    table = np.repeat(table, 10, 0)
    ws = sparse_workspace(12, 1, 128)
    check_sparse(rng.standard_normal((100, 12, 128)), pool, table, lens, lists, counts, rows=rows, ws=ws)
    assert not taken_together(ws)


def test_sparse_junk_past_the_counts(cuda_device):
    rng = np.random.default_rng(40)
    lens = [3000, 20, 700]
    table, pages = shuffled_table(lens, 16, 3, rng)
    pool = make_pool(pages, 16, 1, 128, seed=40)
    lists, counts = random_lists(rng, lens, 1, 16, 80, 71)
    for t in range(3):
        lists[t, 0, counts[t, 0]:] = 10 ** 6 if t else -9
    check_sparse(rng.standard_normal((3, 12, 128)), pool, table, lens, lists, counts)


@pytest.mark.parametrize("d,page,otype", [(128, 64, F16), (128, 16, BF16), (256, 32, F16)])
def test_sparse_groups_nan_scales_and_queries_reach_only_rows_that_see_them(cuda_device, d, page, otype):
    rng = np.random.default_rng(41)
    n, hq, hkv, most = 200, 24, 2, 2560 // page
    pool, table, lens, rows, lists, counts = alike(rng, [n], 6000, page, hkv, d, most, most, 41)
    counts[17] = 0
    q = rng.standard_normal((n, hq, d)).astype(np.float32)

    def run(p, q=q):
        ws = sparse_workspace(hq, hkv, d)
        qd = dev(q).to(otype)
        out, lse, err = torch.empty_like(qd), torch.empty(n, hq, device="cuda"), err_word()
        qsa.qsa_paged_sparse_attn(qd, *[dev(x) for x in p], dev(table), i32(lens), dev(lists), dev(counts), out, ws, rows=i32(rows), lse=lse,
                                  err=err)
        assert taken_together(ws) and not int(err.item())
        return out, lse

    want = run(pool)
    lists_some = [j for j in range(lens[0] // page) if 3 < sum(j in lists[t, 1, :counts[t, 1]] for t in range(n)) < n - 10]
    heads = torch.arange(hq, device="cuda") // (hq // hkv) == 1
    for j, part, value in ((lists_some[0], 2, np.inf), (lists_some[1], 3, np.nan), (lists_some[-1], 3, np.inf), (lists_some[-2], 2, np.nan)):
        p = [x.copy() for x in pool]
        p[part][table[0, j], 5, 1, 1] = value
        out, lse = run(p)
        hit = torch.tensor([j in lists[t, 1, :counts[t, 1]] for t in range(n)], device="cuda")
        assert hit.any() and not hit.all()
        assert torch.equal(out[:, ~heads], want[0][:, ~heads])
        # Their tile's powers of two may be others without that scale.
        torch.testing.assert_close(out[~hit].float(), want[0][~hit].float(), rtol=2.0 ** -7, atol=2.0 ** -9)
        torch.testing.assert_close(lse[~hit], want[1][~hit], rtol=2.0 ** -18, atol=2.0 ** -16)
        got = out[hit][:, heads]
        assert not torch.isfinite(got if part == 2 else got[..., d // 4:d // 2]).any()
    x = q.copy()
    x[17], x[40, 3] = np.nan, np.inf
    out, lse = run(pool, x)
    assert not out[17].any() and torch.isneginf(lse[17]).all() and not torch.isfinite(out[40, 3]).any()
    rest = torch.ones(n, hq, dtype=torch.bool, device="cuda")
    rest[17], rest[40, 3] = False, False
    assert torch.equal(out[rest], want[0][rest]) and torch.equal(lse[rest], want[1][rest])


def check_tree(q, pool, table, prefix, mask, **kw):
    cells, werr = po.tree_cells(table, prefix, mask, pool[0].shape[2], pool[0].shape[1], pool[0].shape[0], kw.get("rows"))
    return check_cells("qsa_paged_tree_attn", q, pool, (dev(table), i32(prefix), dev(mask)), cells, werr, **kw)


def trees(rng, prefix, nodes, page, hkv, d, seed, extra=2):
    """Pool, table, prefix lengths, masks and rows of drafted trees after prefixes."""
    table, pages = shuffled_table([p + n for p, n in zip(prefix, nodes)], page, extra, rng)
    pool = make_pool(pages, page, hkv, d, seed=seed)
    words = -(-max(nodes) // 32)
    mask = np.zeros((sum(nodes), words), np.int32)
    at = 0
    for n in nodes:
        m = random_tree(rng, n)[1]
        mask[at:at + n, : m.shape[1]] = m
        at += n
    rows = [s for s, n in enumerate(nodes) for _ in range(n)]
    return pool, table, [prefix[s] for s in rows], mask, rows


def tree_workspace(hq, hkv, d):
    return torch.full((qsa.qsa_paged_tree_attn_workspace_bytes(hq, hkv, d),), 0xA5, dtype=torch.uint8, device="cuda")


def read_together(ws, rows, n_rows, cells, hkv, d):
    """Whether a call on rows of a table of n_rows by `cells` took the tokens of one sequence together: where
    there are eight and more for each row of the table, unasked; else the call leaves a word for each KV head."""
    most = len(rows) * hkv * (cells // (32 if d == 128 else 16)) * 10
    if cells <= 512 or most <= 130000:
        return False
    return len(rows) >= 8 * n_rows and most > 260000 or bool((ws[-608:].view(torch.int32)[:hkv] == 1).all())


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,page", [(128, 12, 1, 64), (256, 24, 2, 16), (128, 32, 8, 32), (128, 16, 1, 16), (128, 2, 2, 128),
                                           (256, 1, 1, 256), (256, 9, 3, 32)])
def test_tree_shapes(cuda_device, d, hq, hkv, page, otype):
    rng = np.random.default_rng(d + hq)
    prefix, nodes = [0, 1, 15, 16, 31, 40, 63, 64, 127, 300, 1000], [1, 2, 7, 33, 5, 40, 1, 9, 20, 70, 12]
    pool, table, pre, mask, rows = trees(rng, prefix, nodes, page, hkv, d, 31)
    check_tree(rng.standard_normal((len(rows), hq, d)) * 2, pool, table, pre, mask, rows=rows, otype=otype)


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,page,prefix,nodes", [
    (128, 12, 1, 64, [17001], [70]), (256, 24, 2, 16, [3001, 2500], [63, 30]), (128, 32, 8, 64, [900, 1630, 1400], [32, 17, 60]),
    (128, 16, 8, 128, [577], [130]), (256, 8, 4, 32, [1000, 515, 2000], [31, 33, 90]), (128, 8, 8, 16, [560], [256]),
    (128, 16, 8, 32, [6000, 5000, 4000, 900], [7, 7, 7, 2]), (256, 24, 2, 64, [12000, 9000, 100], [9, 7, 1]), (128, 12, 4, 64, [30000], [7])])
def test_trees_taken_together(cuda_device, d, hq, hkv, page, prefix, nodes, otype):
    rng = np.random.default_rng(hq)
    pool, table, pre, mask, rows = trees(rng, prefix, nodes, page, hkv, d, 32)
    gate = rng.standard_normal((len(rows), hq, d)).astype(np.float32) * 2
    q = rng.standard_normal((len(rows), hq, d)) * 2
    ws = tree_workspace(hq, hkv, d)
    check_tree(q, pool, table, pre, mask, rows=rows, otype=otype, gate=gate, ws=ws)
    assert read_together(ws, rows, len(prefix), table.shape[1] * page, hkv, d)


@pytest.mark.parametrize("d,hq,hkv,page,prefix,nodes", [(128, 12, 2, 64, [3000] * 40, [1] * 40), (256, 24, 2, 16, [2500, 3000] * 6, [2, 1] * 6),
                                                        (128, 32, 8, 32, [900] * 30, [1, 2, 3] * 10)])
def test_trees_of_few_tokens_go_one_by_one(cuda_device, d, hq, hkv, page, prefix, nodes):
    rng = np.random.default_rng(hq)
    pool, table, pre, mask, rows = trees(rng, prefix, nodes, page, hkv, d, 43)
    ws = tree_workspace(hq, hkv, d)
    check_tree(rng.standard_normal((len(rows), hq, d)), pool, table, pre, mask, rows=rows, ws=ws)
    assert not read_together(ws, rows, len(prefix), table.shape[1] * page, hkv, d)


@pytest.mark.parametrize("together", [False, True])
def test_tree_any_masks(cuda_device, together):
    """Bits at random, none, all; rows that see nothing; prefixes of their own."""
    rng = np.random.default_rng(33)
    n, hkv = (130, 8) if together else (20, 2)
    table, pages = shuffled_table([1100, 200] if together else [500, 200], 32, 3, rng)
    pool = make_pool(pages, 32, hkv, 128, seed=33)
    rows = [0] * (n - 4) + [1] * 4
    prefix = [int(v) for v in rng.integers(*((600, 900) if together else (0, 300)), n - 4)] + [0, 0, 100, 7]
    mask = rng.integers(-2 ** 31, 2 ** 31, (n, 6), dtype=np.int64).astype(np.int32)
    mask[3], mask[4], mask[5, 1:], mask[6, :5] = 0, -1, 0, 0
    mask[n - 4:] = 0
    mask[n - 3, 3] = 1 << 5
    mask[n - 2, 0] = -2 ** 31
    prefix[7], mask[7] = 0, 0
    prefix[8], mask[8] = 0, 0
    mask[8, 0] = 1
    ws = tree_workspace(16 if together else 4, hkv, 128)
    out, lse = check_tree(rng.standard_normal((n, (16 if together else 4), 128)), pool, table, prefix, mask, rows=rows, ws=ws)
    assert read_together(ws, rows, 2, table.shape[1] * 32, hkv, 128) == together
    assert not out[7].any() and torch.isneginf(lse[7]).all() and not out[n - 4].any()


def test_tree_bad_inputs(cuda_device):
    rng = np.random.default_rng(34)
    table, pages = shuffled_table([100, 60], 16, 3, rng)
    pool = make_pool(pages, 16, 1, 128, seed=34)
    q = rng.standard_normal((3, 12, 128))
    full = np.array([[3, 0], [1, 0], [0xFF, 0]], np.int32)

    def error(prefix, mask=full, table=table, rows=(0, 1, 0)):
        check_tree(q, pool, table, prefix, mask, rows=list(rows))
        return po.tree_cells(table, prefix, mask, 1, 16, pages, list(rows))[1]

    assert error([90, 50, 0]) == 0
    assert error([111, 50, 3]) == po.BAD_ID          # a bit at the table's end
    assert error([90, -1, 3]) == po.BAD_ID
    assert error([90, 10 ** 9, 2 ** 31 - 1]) == po.BAD_ID
    assert error([90, 50, 3], rows=(0, 2, -1)) == po.BAD_ID
    high = full.copy()
    high[2] = [0, -2 ** 31]
    assert error([90, 50, 60], mask=high) == po.BAD_ID
    bad = table.copy()
    bad[0, 2] = pages
    assert error([90, 50, 3], table=bad) == po.BAD_ID


@pytest.mark.parametrize("together", [False, True])
def test_nan_and_inf_scales_reach_only_rows_that_see_them(cuda_device, together):
    rng = np.random.default_rng(35)
    hkv, d, hq = (8, 128, 16) if together else (2, 128, 8)
    nodes, pre = (130, 900) if together else (9, 300)
    pool, table, prefix, mask, rows = trees(rng, [pre], [nodes], 32, hkv, d, 35)
    sees = np.array([[int(m[b // 32]) >> (b % 32) & 1 for b in range(nodes)] for m in mask], bool)
    q = dev(rng.standard_normal((nodes, hq, d)).astype(np.float16))
    ws = torch.empty(qsa.qsa_paged_tree_attn_workspace_bytes(hq, hkv, d), dtype=torch.uint8, device="cuda")

    def run(p):
        out, lse = torch.empty_like(q), torch.empty(nodes, hq, device="cuda")
        qsa.qsa_paged_tree_attn(q, *[dev(x) for x in p], dev(table), i32(prefix), dev(mask), out, ws, rows=i32(rows), lse=lse)
        return out, lse

    want = run(pool)
    assert read_together(ws, rows, 1, table.shape[1] * 32, hkv, d) == together
    for node, part, value in ((2, 2, np.inf), (5, 3, np.nan), (nodes - 1, 3, np.inf), (3, 2, np.nan)):
        p = [x.copy() for x in pool]
        c = pre + node
        p[part][table[0, c // 32], c % 32, 1, 1] = value
        out, lse = run(p)
        hit = torch.from_numpy(sees[:, node]).cuda()
        heads = torch.arange(hq, device="cuda") // (hq // hkv) == 1
        assert torch.equal(out[:, ~heads], want[0][:, ~heads]) and torch.equal(out[~hit], want[0][~hit])
        assert torch.equal(lse[~hit], want[1][~hit])
        got = out[hit][:, heads]
        assert not torch.isfinite(got if part == 2 else got[..., d // 4:d // 2]).any()
        if part == 3:
            rest = torch.ones(d, dtype=torch.bool, device="cuda")
            rest[d // 4:d // 2] = False
            assert torch.isfinite(got[..., rest]).all()


@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 4), (256, 16, 2)])
def test_tree_of_many_infinite_and_nan_v_scales(cuda_device, d, hq, hkv):
    """One half of a tile's cells is then slower than the other, over many tiles in a row."""
    rng = np.random.default_rng(42)
    pool, table, prefix, mask, rows = trees(rng, [9000], [24], 64, hkv, d, 42)
    q = dev(rng.standard_normal((24, hq, d)).astype(np.float16))

    def run(p):
        ws = torch.empty(qsa.qsa_paged_tree_attn_workspace_bytes(hq, hkv, d), dtype=torch.uint8, device="cuda")
        out, lse, err = torch.empty_like(q), torch.empty(24, hq, device="cuda"), err_word()
        qsa.qsa_paged_tree_attn(q, *[dev(x) for x in p], dev(table), i32(prefix), dev(mask), out, ws, rows=i32(rows), lse=lse, err=err)
        assert int(err.item()) == 0
        return out, lse

    want, wlse = run(pool)
    for offset in (0, 40, 64, 100):
        p = [x.copy() for x in pool]
        for c in range(offset, 9000, 128):
            p[3][table[0, c // 64], c % 64, :, 2] = (np.nan, np.inf, -np.inf)[c // 128 % 3]
        out, lse = run(p)
        quarter = slice(d // 2, 3 * d // 4)
        assert torch.isnan(out[..., quarter]).all()
        out[..., quarter] = want[..., quarter]
        torch.testing.assert_close(out.float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -9)
        torch.testing.assert_close(lse, wlse, rtol=2.0 ** -18, atol=2.0 ** -16)


def test_sparse_nan_scales_reach_only_their_lists(cuda_device):
    rng = np.random.default_rng(36)
    lens = [900, 640, 33]
    table, pages = shuffled_table(lens, 32, 3, rng)
    pool = make_pool(pages, 32, 2, 128, seed=36)
    lists, counts = random_lists(rng, lens, 2, 32, 40, 12)
    q = dev(rng.standard_normal((3, 8, 128)).astype(np.float16))
    ws = torch.empty(qsa.qsa_paged_sparse_attn_workspace_bytes(8, 2, 128), dtype=torch.uint8, device="cuda")

    def run(p):
        out = torch.empty_like(q)
        qsa.qsa_paged_sparse_attn(q, *[dev(x) for x in p], dev(table), i32(lens), dev(lists), dev(counts), out, ws)
        return out

    want = run(pool)
    unlisted = next(j for j in range(28) if j not in lists[0, 0])
    for j, reached in ((unlisted, False), (int(lists[0, 0, 3]), True)):
        p = [x.copy() for x in pool]
        p[2][table[0, j], 5, 0, 3] = np.nan
        p[3][table[0, j], 6, 0, 3] = np.inf
        out = run(p)
        assert torch.equal(out[1:], want[1:]) and torch.equal(out[0, 4:], want[0, 4:])
        assert torch.isnan(out[0, :4]).all() if reached else torch.equal(out[0], want[0])
    # Behind the row's last cell, in a listed page.
    p = [x.copy() for x in pool]
    last = table[2, 1]
    lists[2], counts[2] = -1, 2
    lists[2, :, :2] = [0, 1]
    want = run(pool)
    for x in p[2:]:
        x[last, 1:] = np.nan
    assert torch.equal(run(p), want)
