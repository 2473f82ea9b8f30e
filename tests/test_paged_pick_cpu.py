"""Picked pages and trees of drafts without a GPU: pins of their oracle, and the
refusals of their calls, which make no CUDA call."""
import ctypes
import itertools

import numpy as np
import pytest

from oracle import paged_oracle as po
from oracle import select_ids
from sparse_selected_attention_gb300 import _abi
from sparse_selected_attention_gb300 import workloads as wl
from tests.test_paged_cpu import FAKE, INV, L, UNS, _make, _status  # noqa: F401


def pool(pages, page, hkv, d, seed=3):
    c = wl.make_cache(pages * page * hkv, seed=seed, head_dim=d, group=d // 4)
    return [x.reshape(pages, page, hkv, -1) for x in (c.kq, c.vq, c.ksc, c.vsc)]


# ---------------------------------------------------------------- oracle pins

def test_bounds_by_hand():
    kq, _, ksc, _ = pool(3, 16, 1, 128)
    kq[:], ksc[:] = 0, 0
    ksc[1, :, 0, 0] = np.float16([0.5, 0.25, 1.0] + [2.0] * 13)
    kq[1, :, 0, 0] = [-100, 127, -3] + [99] * 13   # the cells behind the third are not filled
    kq[1, :, 0, 1] = [-1, -1, -1] + [0] * 13
    got, err = po.page_bounds(np.array([[1, 2]], np.int32), [3], None, kq, ksc)
    assert err == 0 and list(got) == [1]
    hi_q, lo_q, hi_sc, lo_sc = got[1]
    # Dim 0: -50, 31.75, -3.  31.75 / 127 = 0.25; 50 / 127 rounded up to fp16's 2^-12 there.
    assert hi_sc[0].tolist() == [0.25, 0, 0, 0] and hi_q[0, 0] == 127
    assert lo_sc[0, 0] == np.ceil(50 / 127 * 4096) / 4096 and lo_q[0, 0] == -127
    # Dim 1: -0.5, -0.25, -1: the upper one is exact, the lower a code or less below.
    assert hi_q[0, 1] == -1 and lo_q[0, 1] == np.floor(-1 / float(lo_sc[0, 0])) == -3
    assert not hi_q[0, 2:].any() and not lo_q[0, 2:].any()


@pytest.mark.parametrize("d,page", [(128, 16), (256, 32)])
def test_bounds_hold_every_key_and_no_less_would(d, page):
    kq, _, ksc, _ = pool(9, page, 2, d, seed=4)
    ksc[::2] *= np.float16(1e-4)  # subnormal scales among them
    table = np.array([[3, 1, 0], [8, 5, -1]], np.int32)
    lens = [2 * page + 5, page + 1]
    got, err = po.page_bounds(table, lens, None, kq, ksc)
    assert err == 0 and sorted(got) == [0, 1, 3, 5, 8]
    for r, j in itertools.product(range(2), range(3)):
        filled = min(page, lens[r] - j * page)
        if filled <= 0:
            continue
        hi_q, lo_q, hi_sc, lo_sc = got[int(table[r, j])]
        k = kq[table[r, j], :filled].astype(np.float64) * np.repeat(ksc[table[r, j], :filled].astype(np.float64), d // 4, -1)
        for code, sc, ext in ((hi_q, hi_sc, k.max(0)), (-lo_q.astype(int), lo_sc, -k.min(0))):
            s = np.repeat(sc.astype(np.float64), d // 4, -1)
            assert (code * s >= ext).all() and ((code - 1) * s < ext).all()
            need = np.abs(ext).reshape(2, 4, -1).max(-1)
            less = np.nextafter(sc, np.float16(0)).astype(np.float64)
            assert (127 * sc.astype(np.float64) >= need).all() and (127 * less < need).all()


def test_score_is_the_best_corner():
    rng = np.random.default_rng(0)
    d, q = 128, np.zeros((1, 3, 128))
    q[0, :, :5] = rng.standard_normal((3, 5))
    hi_q = rng.integers(-20, 128, (4, 1, d)).astype(np.int8)
    lo_q = np.minimum(hi_q, rng.integers(-127, 40, (4, 1, d))).astype(np.int8)
    sc = np.full((4, 1, 4), 0.25, np.float16)
    got, _ = po.page_score(q, hi_q, lo_q, sc, sc, np.array([[2, 0]], np.int32), [20], 16)
    for j, p in enumerate((2, 0)):
        best = sum(max(sum(q[0, h, i] * 0.25 * (hi_q, lo_q)[c[i]][p, 0, i] for i in range(5)) for c in itertools.product((0, 1), repeat=5))
                   for h in range(3))
        assert abs(got[0][0][0][j] - best) < 1e-9


def test_score_bounds_the_products():
    kq, _, ksc, _ = pool(6, 16, 2, 128, seed=6)
    table, lens = np.array([[4, 2, 5]], np.int32), [43]
    b, _ = po.page_bounds(table, lens, None, kq, ksc)
    arr = [np.stack([b[p][i] if p in b else np.zeros_like(b[4][i]) for p in range(6)]) for i in range(4)]
    q = wl.queries_f16(1, seed=6)[:, :12]
    got, _ = po.page_score(q, *arr, table, lens, 16)
    for h, j in itertools.product(range(2), range(3)):
        filled = min(16, 43 - 16 * j)
        k = kq[table[0, j], :filled, h] * np.repeat(ksc[table[0, j], :filled, h].astype(np.float64), 32, -1)
        assert got[0][h][0][j] >= (k @ q[0, 6 * h:6 * h + 6].astype(np.float64).T).sum(-1).max()


def test_select_is_the_cells_selection():
    rng = np.random.default_rng(2)
    scores = rng.integers(0, 30, (7, 1, 40)).astype(np.float32)
    for t, n in enumerate([1, 5, 12, 13, 39, 40, 26]):
        ids, _, _ = po.page_select(scores[t:t + 1], [n * 16], 16, 12, 3, 4, 16)
        # One token at position n - 1 that sees n cells: 3 first, the 3 before it and itself.
        want = select_ids(np.concatenate([np.zeros((1, 0), np.float32), scores[t]], -1), n - 1, 64, budget=12, sink=3, local=3)
        assert ids[0, 0, :12].tolist() == want[0, :12].tolist()


def test_select_by_hand():
    nan, inf = np.nan, np.inf
    s = np.array([[[5, 1, nan, -inf, 1, 0.0, -0.0, 9, nan, 2]]], np.float32)
    take = lambda b, sink, local: po.page_select(s, [159], 16, b, sink, local, b)[0][0, 0].tolist()  # noqa: E731
    assert take(3, 0, 0) == [0, 7, 9] and take(4, 0, 0) == [0, 1, 7, 9] and take(6, 0, 0) == [0, 1, 4, 5, 7, 9]
    assert take(8, 0, 0) == [0, 1, 3, 4, 5, 6, 7, 9] and take(9, 0, 0) == [0, 1, 2, 3, 4, 5, 6, 7, 9]
    assert take(2, 2, 0) == [0, 1] and take(3, 0, 3) == [7, 8, 9] and take(3, 1, 1) == [0, 7, 9]
    got = po.page_select(s, [33], 16, 4, 1, 1, 5)
    assert got[0][0, 0].tolist() == [0, 1, 2, -1, -1] and got[1].tolist() == [[3]] and got[2] == 0
    got = po.page_select(s, [-1], 16, 4, 1, 1, 5)
    assert got[1].tolist() == [[0]] and got[2] == po.BAD_ID
    assert po.page_select(s, [161], 16, 4, 1, 1, 5)[2] == po.BAD_ID


def random_tree(rng, n):
    """Parents (-1: the prefix) and the mask rows of n nodes."""
    parents = [int(rng.integers(-1, i)) if i else -1 for i in range(n)]
    sees = np.zeros((n, -(-n // 32) * 32), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            sees[i] = sees[p]
        sees[i, i] = True
    return parents, np.packbits(sees, axis=1, bitorder="little").view(np.int32)


def test_all_pages_and_full_masks_are_the_whole_attention():
    p = pool(8, 16, 2, 128, seed=8)
    table, lens = np.array([[5, 0, 3], [1, 2, 4]], np.int32), [37, 48]
    q = wl.queries_f16(2, seed=8)
    want = po.attn(q, *p, table, lens)
    pages = np.tile(np.array([2, -1, 0, 1], np.int32), (2, 2, 1))
    cells, err = po.sparse_cells(table, lens, pages, np.full((2, 2), 4), 16, 8)
    assert err == 0
    for a, b in zip(want, po.attn_cells(q, *p, cells)):
        np.testing.assert_allclose(a, b, rtol=1e-9, atol=1e-12)
    cells, err = po.tree_cells(table, [30, 48], np.array([[0x7F], [0]], np.int32), 2, 16, 8)
    assert err == 0
    for a, b in zip(want, po.attn_cells(q, *p, cells)):
        np.testing.assert_allclose(a, b, rtol=1e-9, atol=1e-12)


def test_a_trees_branch_is_a_sequence_of_its_own():
    rng = np.random.default_rng(9)
    p = pool(6, 16, 1, 128, seed=9)
    table, n = np.array([[4, 1, 3, 0]], np.int32), 20
    parents, mask = random_tree(rng, n)
    q = wl.queries_f16(n, seed=9)
    cells, err = po.tree_cells(table, [27] * n, mask, 1, 16, 6, rows=[0] * n)
    got = po.attn_cells(q, *p, cells)[0]
    flat = [x.reshape(96, 1, -1) for x in p]
    for i in range(n):
        path = [i]
        while parents[path[-1]] >= 0:
            path.append(parents[path[-1]])
        at = [int(table[0, c // 16]) * 16 + c % 16 for c in list(range(27)) + [27 + v for v in reversed(path)]]
        own = [np.zeros((4, 16, 1, x.shape[-1]), x.dtype) for x in flat]
        for o, x in zip(own, flat):
            o.reshape(64, 1, -1)[: len(at)] = x[at]
        want = po.attn(q[i:i + 1], *own, np.array([[0, 1, 2, 3]], np.int32), [len(at)])[0]
        np.testing.assert_allclose(got[i:i + 1], want, rtol=1e-9, atol=1e-12)
    assert err == 0 and po.tree_cells(table, [60], np.array([[0x1F]], np.int32), 1, 16, 6)[1] == po.BAD_ID


# ---------------------------------------------------------------- refusals

BOUNDS = dict(n_rows=2, max_pages=4, n_pages=8, page_size=16, n_kv_heads=1, head_dim=128, group=32)
SCORE = dict(n_tokens=3, n_q_heads=12, n_kv_heads=1, head_dim=128, group=32, page_size=16, n_pages=8, n_rows=3, max_pages=2, dtype=1, ld=2)
SELECT = dict(n_tokens=3, n_kv_heads=2, page_size=16, width=8, budget=6, sink=1, local=2, ld=50)
SPARSE = dict(n_tokens=3, n_q_heads=12, n_kv_heads=1, head_dim=128, group=32, page_size=16, n_pages=8, n_rows=3, max_pages=2, width=2,
              dtype=1, softmax_scale=0.1, workspace_bytes=1 << 30)
TREE = {**{k: v for k, v in SPARSE.items() if k != "width"}, "words": 1}
TOKENS = [(dict(head_dim=192, group=48), UNS), (dict(n_q_heads=17), UNS), (dict(n_kv_heads=5), UNS), (dict(n_kv_heads=0), UNS),
          (dict(page_size=8), UNS), (dict(page_size=100), UNS), (dict(dtype=0), INV), (dict(n_tokens=-2), INV), (dict(n_pages=0), INV),
          (dict(max_pages=0), INV), (dict(rows=None, n_rows=2), INV), (dict(n_pages=1 << 28), INV), (dict(max_pages=1 << 28), INV),
          (dict(max_pages=(1 << 26) + 1, page_size=16, ld=1 << 30), UNS), (dict(n_tokens=1 << 30, n_rows=1 << 30, n_q_heads=4, n_kv_heads=4), UNS),
          (dict(page_table=None), INV), (dict(q=None), INV), (dict(q=FAKE + 4), INV), (dict(rows=FAKE + 2), INV), (dict(err=FAKE + 1), INV)]
ATTN = [(dict(softmax_scale=float("inf")), INV), (dict(softmax_scale=float("nan")), INV), (dict(workspace_bytes=16), INV),
        (dict(workspace=FAKE + 16), INV), (dict(workspace=None), INV), (dict(out=None), INV), (dict(out=FAKE + 8), INV),
        (dict(lse=FAKE + 2), INV), (dict(gate=FAKE + 4), INV), (dict(ksc=FAKE + 4), INV), (dict(vq=FAKE + 8), INV), (dict(vsc=None), INV)]


def _without(case, cls):
    kw, want = case
    names = {n for n, _ in cls._fields_}
    return {k: v for k, v in kw.items() if k in names}, want


@pytest.mark.parametrize("fn,cls,base,kw,want", [
    ("qsa_page_bounds", _abi.PageBoundsArgs, BOUNDS, kw, want) for kw, want in [
        (dict(page_size=24), UNS), (dict(head_dim=128, group=64), UNS), (dict(n_kv_heads=0), UNS), (dict(n_kv_heads=1 << 16), UNS),
        (dict(n_rows=-1), INV), (dict(max_pages=0), INV), (dict(n_pages=0), INV), (dict(n_pages=1 << 28), INV), (dict(max_pages=1 << 28), INV),
        (dict(page_table=None), INV), (dict(kq=None), INV), (dict(lo_sc=None), INV), (dict(kq=FAKE + 8), INV), (dict(ksc=FAKE + 4), INV),
        (dict(hi_q=FAKE + 8), INV), (dict(hi_sc=FAKE + 2), INV), (dict(n_new=FAKE + 2), INV), (dict(err=FAKE + 1), INV)]
] + [
    ("qsa_page_score", _abi.PageScoreArgs, SCORE, *_without(c, _abi.PageScoreArgs)) for c in TOKENS + [
        (dict(ld=1), INV), (dict(hi_q=FAKE + 8), INV), (dict(lo_sc=FAKE + 4), INV), (dict(scores=FAKE + 2), INV), (dict(scores=None), INV),
        (dict(seq_lens=None), INV), (dict(lo_q=None), INV)]
] + [
    ("qsa_page_select", _abi.PageSelectArgs, SELECT, kw, want) for kw, want in [
        (dict(page_size=48), UNS), (dict(n_tokens=-1), INV), (dict(n_kv_heads=0), INV), (dict(ld=0), INV), (dict(budget=0), INV),
        (dict(budget=9), INV), (dict(sink=-1), INV), (dict(local=-1), INV), (dict(sink=4, local=3), INV),
        (dict(sink=2 ** 31 - 1, local=2 ** 31 - 1), INV), (dict(n_tokens=1 << 30, n_kv_heads=4), UNS), (dict(scores=None), INV),
        (dict(counts=None), INV), (dict(pages=FAKE + 2), INV), (dict(seq_lens=FAKE + 2), INV)]
] + [
    ("qsa_paged_sparse_attn", _abi.PagedSparseAttnArgs, SPARSE, *_without(c, _abi.PagedSparseAttnArgs)) for c in TOKENS + ATTN + [
        (dict(width=0), INV), (dict(width=(1 << 26) + 1), UNS), (dict(pages=None), INV), (dict(counts=FAKE + 2), INV), (dict(seq_lens=None), INV)]
] + [
    ("qsa_paged_tree_attn", _abi.PagedTreeAttnArgs, TREE, *_without(c, _abi.PagedTreeAttnArgs)) for c in TOKENS + ATTN + [
        (dict(words=0), UNS), (dict(words=33), UNS), (dict(mask=None), INV), (dict(mask=FAKE + 2), INV), (dict(prefix_lens=None), INV)]
])
def test_refusals(L, fn, cls, base, kw, want):  # noqa: F811
    s, msg = _status(L, fn, _make(cls, base, kw))
    assert s == want and msg.startswith(fn + ":"), (s, msg)


@pytest.mark.parametrize("fn,cls,base,kw", [
    ("qsa_page_bounds", _abi.PageBoundsArgs, BOUNDS, dict(n_rows=0, page_table=None, seq_lens=None)),
    ("qsa_page_score", _abi.PageScoreArgs, SCORE, dict(n_tokens=0, n_rows=0, q=None, scores=None)),
    ("qsa_page_select", _abi.PageSelectArgs, SELECT, dict(n_tokens=0, scores=None, pages=None)),
    ("qsa_paged_sparse_attn", _abi.PagedSparseAttnArgs, SPARSE, dict(n_tokens=0, n_rows=0, q=None, out=None, pages=None)),
    ("qsa_paged_tree_attn", _abi.PagedTreeAttnArgs, TREE, dict(n_tokens=0, n_rows=0, q=None, out=None, mask=None))])
def test_nothing_to_do_is_a_no_op(L, fn, cls, base, kw):  # noqa: F811
    assert _status(L, fn, _make(cls, base, kw))[0] == _abi.QSA_OK


def test_null_args_and_workspace_sizes(L):  # noqa: F811
    for fn in ("qsa_page_bounds", "qsa_page_score", "qsa_page_select", "qsa_paged_sparse_attn", "qsa_paged_tree_attn"):
        assert getattr(L, fn)(None, None) == INV
    for fn in (L.qsa_paged_sparse_attn_workspace_bytes, L.qsa_paged_tree_attn_workspace_bytes):
        assert fn(12, 1, 128) > 0 and fn(24, 2, 256) > 0
        for bad in ((12, 1, 64), (17, 1, 128), (12, 5, 128), (0, 1, 128), (12, 0, 256)):
            assert fn(*bad) == 0


def test_structs_are_the_headers():
    """Field by field as include/qsa.h lists them."""
    import re
    text = open(_abi.HEADER).read()
    for cls, name in ((_abi.PageBoundsArgs, "qsa_page_bounds_args"), (_abi.PageScoreArgs, "qsa_page_score_args"),
                      (_abi.PageSelectArgs, "qsa_page_select_args"), (_abi.PagedSparseAttnArgs, "qsa_paged_sparse_attn_args"),
                      (_abi.PagedTreeAttnArgs, "qsa_paged_tree_attn_args")):
        end = text.index("} " + name + ";")
        body = text[text.rindex("typedef struct {", 0, end) + len("typedef struct {"):end]
        names, kinds = [], []
        for line in body.split(";"):
            m = re.match(r"\s*((?:const\s+)?\w+(?:\s+int)?)\s+(.*)", line.strip(), re.S)
            if not m:
                continue
            for part in m.group(2).split(","):
                part = part.strip()
                names.append(part.lstrip("*"))
                kinds.append(ctypes.c_void_p if part.startswith("*") or m.group(1).endswith("*") else
                             {"int": ctypes.c_int, "float": ctypes.c_float, "int64_t": ctypes.c_int64, "size_t": ctypes.c_size_t}[m.group(1)])
        assert [(n, k) for n, k in cls._fields_] == list(zip(names, kinds))


def test_binding_refuses_cpu_tensors():
    import torch

    import sparse_selected_attention_gb300 as qsa
    z = lambda *v, t=torch.int32: torch.zeros(v, dtype=t)  # noqa: E731
    kq, ksc, hi, hs = z(4, 16, 1, 128, t=torch.int8), z(4, 16, 1, 4, t=torch.float16), z(4, 1, 128, t=torch.int8), z(4, 1, 4, t=torch.float16)
    q, tab, lens, ws = z(2, 12, 128, t=torch.float16), z(2, 2), z(2), z(1 << 20, t=torch.uint8)
    for call in (lambda: qsa.qsa_page_bounds(tab, lens, kq, ksc, hi, hi, hs, hs),
                 lambda: qsa.qsa_page_score(q, hi, hi, hs, hs, tab, lens, z(2, 1, 2, t=torch.float32), 16),
                 lambda: qsa.qsa_page_select(z(2, 1, 2, t=torch.float32), lens, z(2, 1, 2), z(2, 1), 16, 2),
                 lambda: qsa.qsa_paged_sparse_attn(q, kq, kq, ksc, ksc, tab, lens, z(2, 1, 2), z(2, 1), q.clone(), ws),
                 lambda: qsa.qsa_paged_tree_attn(q, kq, kq, ksc, ksc, tab, lens, z(2, 1), q.clone(), ws)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
