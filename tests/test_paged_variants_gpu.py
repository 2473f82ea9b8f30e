"""The paged calls in the library's test variants: the device bounds-check build
(the same bits, a clear check word) and the build whose bounded waits give up
at once (the attention reports it and leaves the context usable)."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from sparse_selected_attention_gb300 import _abi
from tests.test_paged_gpu import BF16, F16, check_attn, dev, i32, make_pool, shuffled_table

pytestmark = pytest.mark.gpu


@pytest.fixture
def use_library(monkeypatch):
    """Routes the binding's calls to a variant of the library."""
    def use(name):
        L = _abi.variant(name)
        monkeypatch.setattr(_abi, "lib", lambda: L)
        monkeypatch.setattr(_abi, "_packed", {})
        monkeypatch.setattr(_abi, "_entries", {})
        return L
    yield use


def word(L):
    out = ctypes.c_uint(7)
    assert L.qsa_check_word(ctypes.byref(out)) == _abi.QSA_OK
    return out.value


def every_call(d, hkv, per, page):
    rng = np.random.default_rng(3)
    lens = [700, 0, 33, 1, 2 * page, 2 * page + 1]
    table, pages = shuffled_table(lens, page, 9, rng, wide=-(-760 // page))
    pool = [dev(x) for x in make_pool(pages, page, hkv, d, seed=40, layers=2)]
    layer = [x[1] for x in pool]
    rows, hq = len(lens), hkv * per
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    err = z(1)
    src, new = i32(0, 0, 2, -1, 4, 5, 1), i32(1, 1, 40, 17, 0, 3, 2)
    tout, lout, refs, slots, pos = z(7, table.shape[1]), z(7), z(pages), z(70), z(70)
    ws = z(qsa.qsa_pages_workspace_bytes(7, pages), t=torch.uint8)
    qsa.qsa_page_update(dev(table), i32(lens), src, new, *pool, tout, lout, refs, slots, pos, ws, err=err)
    x = torch.from_numpy(rng.standard_normal((70, hq + 2 * hkv, d))).cuda().to(BF16)
    q = z(70, hq, d, t=BF16)
    w = torch.ones(d, device="cuda")
    qsa.qsa_paged_prep(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, *layer, q, q_norm_w=w, k_norm_w=w,
                       inv_freq=torch.ones(d // 4, device="cuda"), err=err)
    out, lse = z(7, hq, d, t=BF16), z(7, hq, t=torch.float32)
    qsa.qsa_paged_attn(q[:7], *layer, tout, lout, out, z(qsa.qsa_paged_attn_workspace_bytes(hq, hkv, d), t=torch.uint8), lse=lse,
                       gate=torch.ones(7, hq, d, device="cuda"), err=err)
    grp = z(7, hq, d, t=BF16)
    qsa.qsa_paged_attn(q[:7], *layer, tout, i32(900, 701, 702, 703, 20, 0, 35), grp, z(qsa.qsa_paged_attn_workspace_bytes(hq, hkv, d), t=torch.uint8),
                       rows=i32(0, 0, 0, 0, 2, 2, 2), err=z(1))
    ko, vo = z(70, hkv, d, t=F16), z(70, hkv, d, t=F16)
    qsa.qsa_paged_gather(*layer, slots, ko, vo, err=err)
    pmap, live, t2, r2 = z(pages), z(1), z(7, table.shape[1]), z(pages)
    qsa.qsa_page_compact(tout, lout, *pool, t2, r2, pmap, live, ws, err=err)
    torch.cuda.synchronize()
    return [tout, lout, refs, slots, pos, q, out, lse, grp, ko, vo, t2, r2, pmap, live, err] + pool


@pytest.mark.parametrize("d,hkv,per,page", [(128, 1, 12, 16), (128, 3, 5, 64), (256, 2, 12, 32)])
def test_check_build_same_bits(cuda_device, use_library, d, hkv, per, page):
    plain = every_call(d, hkv, per, page)
    L = use_library("check")
    word(L)
    checked = every_call(d, hkv, per, page)
    assert word(L) == 0
    for i, (a, b) in enumerate(zip(plain, checked)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


@pytest.mark.parametrize("d,page,rows", [(128, 64, None), (128, 16, None), (256, 32, None), (128, 64, [0, 0, 0]), (256, 16, [0, 0, 0])])
def test_attn_time_out(cuda_device, use_library, monkeypatch, d, page, rows):
    rng = np.random.default_rng(5)
    lens = [3000, 5, 400]
    table, pages = shuffled_table(lens, page, 1, rng)
    pool = make_pool(pages, page, 1, d, seed=41)
    q = rng.standard_normal((3, 6, d))
    use_library("wait0")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(3, 6, d, dtype=F16, device="cuda")
    ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(6, 1, d), dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_attn(dev(q.astype(np.float16)), *[dev(x) for x in pool], dev(table), i32(lens), out, ws, err=err,
                       rows=None if rows is None else i32(rows))
    torch.cuda.synchronize()
    assert int(err.item()) == qsa.QSA_DEVERR_TIMEOUT
    monkeypatch.undo()
    check_attn(q, pool, table, lens, rows=rows)


def together(d):
    """Rows of one sequence that are taken by groups, few cells for many heads."""
    rng = np.random.default_rng(6)
    lens = [560 + i for i in range(64)]
    table, pages = shuffled_table(lens[-1:], 32, 1, rng)
    return rng.standard_normal((64, 16, d)), make_pool(pages, 32, 8, d, seed=42), table, lens, [0] * 64


@pytest.mark.parametrize("d", [128, 256])
def test_check_build_rows_taken_together(cuda_device, use_library, d):
    q, pool, table, lens, rows = together(d)
    plain, _ = check_attn(q, pool, table, lens, rows=rows)
    L = use_library("check")
    word(L)
    checked, _ = check_attn(q, pool, table, lens, rows=rows)
    assert word(L) == 0 and torch.equal(plain, checked)


@pytest.mark.parametrize("d", [128, 256])
def test_time_out_of_rows_taken_together(cuda_device, use_library, monkeypatch, d):
    q, pool, table, lens, rows = together(d)
    use_library("wait0")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(64, 16, d, dtype=F16, device="cuda")
    ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(16, 8, d), dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_attn(dev(q.astype(np.float16)), *[dev(x) for x in pool], dev(table), i32(lens), out, ws, err=err, rows=i32(rows))
    torch.cuda.synchronize()
    assert int(err.item()) == qsa.QSA_DEVERR_TIMEOUT
    monkeypatch.undo()
    check_attn(q, pool, table, lens, rows=rows)
