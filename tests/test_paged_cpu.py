"""The paged cache without a GPU: pins of its oracle, and the refusals of its
calls, which make no CUDA call."""
import ctypes

import numpy as np
import pytest

from oracle import attention, prep_queries, rope_inv_freq
from oracle import paged_oracle as po
from sparse_selected_attention_gb300 import _abi, build
from sparse_selected_attention_gb300 import workloads as wl


# ---------------------------------------------------------------- oracle pins

def test_prep_is_the_contiguous_preps_for_one_sequence():
    inp = wl.prep_inputs(5, seed=3)
    f = rope_inv_freq(64, 10000.0)
    want = prep_queries(inp.q_in, inp.norm_w, 700, rope_dims=64)[0]
    got = po.norm_rotate(inp.q_in, inp.norm_w, np.arange(700, 705), np.asarray(f, dtype=np.float32))
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("n", [4, 64])
def test_interleaved_is_the_half_layout_permuted(n):
    y = wl.normal(4, 1, (3, 2, 128))
    f = (10000.0 ** (-np.arange(n) / n)).astype(np.float32)
    order = np.r_[np.ravel(np.column_stack([np.arange(n), np.arange(n) + n])), np.arange(2 * n, 128)]
    half = po.rotate(y, [5, 9, 100000], f)
    inter = po.rotate(y[..., order], [5, 9, 100000], f, interleaved=True)
    np.testing.assert_allclose(inter, half[..., order], rtol=0, atol=0)
    np.testing.assert_allclose(half[..., :n] ** 2 + half[..., n:2 * n] ** 2, y[..., :n] ** 2 + y[..., n:2 * n] ** 2, rtol=1e-9)


def test_attn_is_the_contiguous_attention_over_all_cells():
    c = wl.make_cache(96, seed=6)
    q = wl.queries_f16(2, seed=6)
    table = np.array([[5, 0, 3], [1, 2, 4]], dtype=np.int32)
    shape = lambda x: x.reshape(6, 16, 1, -1)  # noqa: E731
    out, lse, _, _, _ = po.attn(q, shape(c.kq), shape(c.vq), shape(c.ksc), shape(c.vsc), table, [37, 48])
    ids = np.full((2, 64), -1, dtype=np.int32)
    for t, n in enumerate([37, 48]):
        ids[t, :n] = table[t, np.arange(n) // 16] * 16 + np.arange(n) % 16
    want, _, m, l = attention(q, c.kq, c.vq, c.ksc, c.vsc, ids, 1 / np.sqrt(128))
    np.testing.assert_allclose(out, want, rtol=1e-10, atol=1e-12)


def test_update_by_hand():
    # Pages of 16: row 0 has 20 cells in pages 2, 5; row 1 has 32 in 0, 1.
    table = np.array([[2, 5, -1], [0, 1, 9]], dtype=np.int32)
    # Two beams from row 0, one empty new row of 17 tokens; row 1 is freed.
    got = po.page_update(table, [20, 32], [0, 0, -1], [1, 0, 17], 8, 16, 18)
    assert got[0].tolist() == [[2, 0, -1], [2, 5, -1], [1, 3, -1]]
    assert got[1].tolist() == [21, 20, 17]
    assert got[2].tolist() == [1, 1, 2, 1, 0, 1, 0, 0]
    assert got[3].tolist() == [4] + [16 + i for i in range(16)] + [48]
    assert got[4].tolist() == [20] + list(range(17))
    assert got[5] == [(5, 0, 4)] and got[6] == 0
    # Not enough pages: the second row stays, the third needs none and grows.
    got = po.page_update(np.array([[0], [-1], [1]], dtype=np.int32), [16, 0, 3], None, [0, 1, 1], 2, 16, 2)
    assert got[1].tolist() == [16, 0, 4] and got[3].tolist() == [-1, 19] and got[6] == po.NO_PAGES


def test_compact_by_hand():
    table = np.array([[6, 1, -1], [6, 4, 7]], dtype=np.int32)
    got = po.page_compact(table, [17, 48], 8, 16)
    assert got[3] == 4 and got[4] == [(4, 0), (6, 2), (7, 3)]
    assert got[0].tolist() == [[2, 1, -1], [2, 0, 3]]
    assert got[1].tolist() == [1, 1, 2, 1, 0, 0, 0, 0]
    assert got[2].tolist() == [-1, 1, -1, -1, 0, -1, 2, 3]


@pytest.mark.parametrize("seed", range(6))
def test_update_invariants(seed):
    rng = np.random.default_rng(seed)
    page, n_pages, wide = 16, 40, 6
    table, lens = np.zeros((0, wide), dtype=np.int32), np.zeros(0, dtype=np.int32)
    for _ in range(12):
        rows = int(rng.integers(1, 7))
        src = rng.integers(-1, len(lens), rows)
        new = rng.integers(0, 40, rows)
        t, ln, refs, slots, pos, copies, err = po.page_update(table, lens, src, new, n_pages, page, int(new.sum()))
        used = slots[slots >= 0]
        assert len(set(used.tolist())) == len(used)
        # A page that is written is held once.
        assert all(refs[s // page] == 1 for s in used)
        assert np.bincount(t[t >= 0], minlength=n_pages).tolist() == refs.tolist()
        assert all((t[r] >= 0).sum() == -(-int(ln[r]) // page) for r in range(rows))
        table, lens = t, ln


# ---------------------------------------------------------------- refusals

@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


FAKE = 1 << 20  # an aligned non-null address; never dereferenced (validation fails first)


def _status(L, fn, args):
    import torch
    if torch.cuda.is_available():
        pytest.skip("argument-rejection checks use fake device addresses: run them on a machine without a GPU")
    s = getattr(L, fn)(ctypes.byref(args), None)
    return s, L.qsa_last_error().decode()


def _make(cls, base, kw):
    a = cls()
    for n, t in cls._fields_:
        setattr(a, n, FAKE if t is ctypes.c_void_p else 0)
    for k, v in {**base, **kw}.items():
        setattr(a, k, v)
    return a


INV, UNS = _abi.QSA_ERR_INVALID_ARG, _abi.QSA_ERR_UNSUPPORTED
PREP = dict(ntok=4, n_q_heads=12, n_kv_heads=1, head_dim=128, group=32, rope_dims=64, cache_cells=64, in_dtype=1,
            q_out_dtype=1, eps=1e-6, rope_mscale=1.0, q_stride=1792, k_stride=1792, v_stride=1792)
GATHER = dict(n_ids=5, n_kv_heads=1, head_dim=128, group=32, cache_cells=64, page_size=16, n_rows=2, max_pages=2,
              out_dtype=1)
ATTN = dict(n_tokens=3, n_q_heads=12, n_kv_heads=1, head_dim=128, group=32, page_size=16, n_pages=8, n_rows=3,
            max_pages=2, dtype=1, softmax_scale=0.1, workspace_bytes=1 << 30)
UPDATE = dict(n_rows_in=2, n_rows=2, max_pages=4, n_layers=1, n_pages=8, page_size=16, n_kv_heads=1, head_dim=128,
              group=32, n_slots=4, workspace_bytes=1 << 20, page_table_out=FAKE + 4096, seq_lens_out=FAKE + 8192)
COMPACT = dict(n_rows=2, max_pages=4, n_layers=1, n_pages=8, page_size=16, n_kv_heads=1, head_dim=128, group=32,
               workspace_bytes=1 << 20)


@pytest.mark.parametrize("fn,cls,base,kw,want", [
    ("qsa_paged_prep", _abi.PagedPrepArgs, PREP, kw, want) for kw, want in [
        (dict(head_dim=64, group=16), UNS), (dict(group=64), UNS), (dict(n_q_heads=0), UNS), (dict(n_kv_heads=40000), UNS),
        (dict(rope_dims=60), UNS), (dict(rope_dims=136), UNS), (dict(head_dim=256, group=64, rope_dims=24), UNS),
        (dict(in_dtype=3), INV), (dict(q_out_dtype=0), INV), (dict(interleaved=2), INV), (dict(ntok=-1), INV),
        (dict(cache_cells=0), INV), (dict(eps=-1.0), INV), (dict(rope_mscale=float("nan")), INV),
        (dict(q_stride=1535), INV), (dict(q_stride=1540), INV), (dict(k_stride=0), INV), (dict(v_stride=100), INV),
        (dict(inv_freq=None), INV), (dict(slots=None), INV), (dict(q_in=FAKE + 8), INV), (dict(k_norm_w=FAKE + 4), INV),
        (dict(ksc=FAKE + 4), INV), (dict(q_out=FAKE + 2), INV), (dict(err=FAKE + 1), INV)]
] + [
    ("qsa_paged_gather", _abi.PagedGatherArgs, GATHER, kw, want) for kw, want in [
        (dict(head_dim=96, group=24), UNS), (dict(n_kv_heads=0), UNS), (dict(out_dtype=5), INV), (dict(n_ids=-1), INV),
        (dict(cache_cells=0), INV), (dict(page_size=48), UNS), (dict(page_size=512), UNS), (dict(rows=None), INV),
        (dict(n_rows=0), INV), (dict(max_pages=0), INV), (dict(ids=None), INV), (dict(k_out=FAKE + 8), INV),
        (dict(vsc=FAKE + 2), INV), (dict(n_ids=2 ** 31 - 1, n_kv_heads=60000), UNS)]
] + [
    ("qsa_paged_attn", _abi.PagedAttnArgs, ATTN, kw, want) for kw, want in [
        (dict(head_dim=192, group=48), UNS), (dict(n_q_heads=17), UNS), (dict(n_kv_heads=5), UNS), (dict(n_kv_heads=0), UNS),
        (dict(page_size=8), UNS), (dict(page_size=100), UNS), (dict(dtype=0), INV), (dict(n_tokens=-2), INV),
        (dict(n_pages=0), INV), (dict(max_pages=0), INV), (dict(rows=None, n_rows=2), INV),
        (dict(n_pages=1 << 28), INV), (dict(max_pages=1 << 28), INV), (dict(max_pages=(1 << 26) + 1, page_size=16), UNS),
        (dict(softmax_scale=float("inf")), INV),
        (dict(workspace_bytes=16), INV), (dict(workspace=FAKE + 16), INV), (dict(workspace=None), INV),
        (dict(seq_lens=None), INV), (dict(q=FAKE + 4), INV), (dict(lse=FAKE + 2), INV), (dict(gate=FAKE + 4), INV), (dict(ksc=FAKE + 4), INV)]
] + [
    ("qsa_page_update", _abi.PageUpdateArgs, UPDATE, kw, want) for kw, want in [
        (dict(page_size=24), UNS), (dict(head_dim=128, group=64), UNS), (dict(n_kv_heads=0), UNS), (dict(n_rows=-1), INV),
        (dict(n_layers=0), INV), (dict(n_pages=1 << 28), INV), (dict(workspace_bytes=64), INV), (dict(refs=None), INV),
        (dict(src=None, n_rows_in=1), INV), (dict(n_slots=-1), INV), (dict(slots=None), INV), (dict(ksc=FAKE + 8), INV),
        (dict(page_table_out=FAKE), INV), (dict(seq_lens_out=FAKE + 4), INV),
        (dict(src=None, page_table_out=FAKE + 16), INV), (dict(workspace=FAKE + 128), INV), (dict(n_new=None), INV)]
] + [
    ("qsa_page_compact", _abi.PageCompactArgs, COMPACT, kw, want) for kw, want in [
        (dict(page_size=0), UNS), (dict(n_pages=0), INV), (dict(page_map=None), INV), (dict(n_live=None), INV),
        (dict(page_table_out=FAKE + 16), INV), (dict(kq=FAKE + 8), INV), (dict(workspace_bytes=0), INV)]
])
def test_refusals(L, fn, cls, base, kw, want):
    s, msg = _status(L, fn, _make(cls, base, kw))
    assert s == want and msg.startswith(fn + ":"), (s, msg)


@pytest.mark.parametrize("fn,cls,base,kw", [
    ("qsa_paged_prep", _abi.PagedPrepArgs, PREP, dict(ntok=0, q_in=None, slots=None)),
    ("qsa_paged_gather", _abi.PagedGatherArgs, GATHER, dict(n_ids=0, ids=None, k_out=None)),
    ("qsa_paged_attn", _abi.PagedAttnArgs, ATTN, dict(n_tokens=0, q=None, out=None))])
def test_nothing_to_do_is_a_no_op(L, fn, cls, base, kw):
    assert _status(L, fn, _make(cls, base, kw))[0] == _abi.QSA_OK


def test_null_args_and_workspace_sizes(L):
    for fn in ("qsa_paged_prep", "qsa_paged_gather", "qsa_paged_attn", "qsa_page_update", "qsa_page_compact"):
        assert getattr(L, fn)(None, None) == INV
    assert L.qsa_pages_workspace_bytes(-1, 5) == 0 and L.qsa_pages_workspace_bytes(3, 0) == 0
    assert L.qsa_pages_workspace_bytes(10, 1000) > L.qsa_pages_workspace_bytes(10, 100) > 0
    assert L.qsa_paged_attn_workspace_bytes(12, 1, 128) > 0
    for bad in ((12, 1, 64), (17, 1, 128), (12, 5, 128), (0, 1, 128), (12, 0, 256)):
        assert L.qsa_paged_attn_workspace_bytes(*bad) == 0


def test_binding_refuses_cpu_tensors():
    import torch

    import sparse_selected_attention_gb300 as qsa
    kq = torch.zeros(4, 16, 1, 128, dtype=torch.int8)
    ksc = torch.zeros(4, 16, 1, 4, dtype=torch.float16)
    q = torch.zeros(2, 12, 128, dtype=torch.float16)
    tab, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    for call in (lambda: qsa.qsa_paged_attn(q, kq, kq, ksc, ksc, tab, lens, q.clone(), ws),
                 lambda: qsa.qsa_paged_prep(q, q[:, :1], q[:, :1], lens, lens, kq, kq, ksc, ksc, q.clone()),
                 lambda: qsa.qsa_paged_gather(kq, kq, ksc, ksc, lens, q[:, :1], q[:, :1]),
                 lambda: qsa.qsa_page_update(tab, lens, None, lens, kq, kq, ksc, ksc, tab, lens, lens, lens, lens, ws),
                 lambda: qsa.qsa_page_compact(tab, lens, kq, kq, ksc, ksc, tab, lens, lens, lens[:1], ws)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(AttributeError):
        qsa.no_such_call


def test_packed_arguments_are_the_structs():
    """The bytes that the binding packs are the ctypes mirrors' bytes."""
    from sparse_selected_attention_gb300 import paged
    for cls, fmt in paged._FORMAT.items():
        assert fmt.size == ctypes.sizeof(cls)
        vals = [float(i) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
        assert bytes(cls(*vals)) == fmt.pack(*vals)
