"""Scores that are no numbers, in every form that qsa_paged_attn takes rows in:
a warp each, whole, shared out over the chip, and together (in one CTA, and
joined).  The result of a NaN score is NaN, in `out` and in `lse`; -inf in
`lse` is the mark of a row without cells."""
import numpy as np
import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from tests.test_paged_gpu import BF16, F16, dev, i32, make_pool, shuffled_table, taken_together

pytestmark = pytest.mark.gpu

FORMS = ["a warp each", "whole", "shared out", "together", "together, many"]


def batch(form, d, hkv=4, per=4):
    """q, pool, table, lens and rows of one form; some row is empty."""
    rng = np.random.default_rng(50)
    page, rows = 16, None
    if form == "a warp each":  # more rows and heads than CTAs, two units at most
        lens = [int(n) for n in rng.integers(1, 33, 90)]
        lens[1] = 0
    elif form == "whole":
        lens = [200, 0, 33, 256]
    elif form == "shared out":
        lens = [2900, 0, 40, 700]
    elif form == "together":  # one sequence's, over the chip
        rows, lens = [0] * 32 + [1, 2], [2900 + i for i in range(32)] + [0, 5]
    else:  # more groups than CTAs
        rows = [s for s in range(60) for _ in range(16)] + [60]
        lens = [640 + (7 * s) % 90 + i for s in range(60) for i in range(16)] + [0]
    if rows is None:
        table, pages = shuffled_table(lens, page, 1, rng)
    else:
        held = [max(n for n, r in zip(lens, rows) if r == s) for s in range(max(rows) + 1)]
        table, pages = shuffled_table(held, page, 1, rng)
        assert taken_together(rows, lens, hkv * per, hkv, d)
    q = rng.standard_normal((len(lens), hkv * per, d)).astype(np.float32)
    return q, make_pool(pages, page, hkv, d, seed=51), table, lens, rows


def attend(q, pool, table, lens, rows, otype):
    T, H, D = q.shape
    out, lse = torch.full((T, H, D), 9.0, dtype=otype, device="cuda"), torch.full((T, H), 9.0, device="cuda")
    ws = torch.full((qsa.qsa_paged_attn_workspace_bytes(H, pool[0].shape[2], D),), 0xA5, dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    qsa.qsa_paged_attn(dev(q).to(otype), *[dev(x) for x in pool], dev(table), i32(lens), out, ws,
                       rows=None if rows is None else i32(rows), lse=lse, err=err)
    assert int(err.item()) == 0
    return out, lse


def row_cells(table, lens, rows, t):
    r = t if rows is None else rows[t]
    c = np.arange(lens[t])
    return table[r, c // 16], c % 16


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("form", FORMS)
def test_all_scores_nan(cuda_device, form, d, otype):
    """A NaN query: its head's scores are all NaN, so out and lse are; the other
    heads and rows keep their bits, and an empty row is 0 and -inf whatever its
    query holds."""
    q, pool, table, lens, rows = batch(form, d)
    want, wlse = attend(q, pool, table, lens, rows, otype)
    q = q.copy()
    hit = [0, 3, len(lens) - 1] + [lens.index(0)]
    q[hit, 5] = np.nan
    q[2, 9, 17] = np.nan
    out, lse = attend(q, pool, table, lens, rows, otype)
    nan = torch.zeros_like(lse, dtype=torch.bool)
    nan[hit, 5], nan[2, 9] = True, True
    nan[[t for t, n in enumerate(lens) if n == 0]] = False
    assert torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()
    assert torch.equal(out[~nan], want[~nan]) and torch.equal(lse[~nan], wlse[~nan])
    empty = lens.index(0)
    assert not out[empty].any() and torch.isneginf(lse[empty]).all()


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("codes", ["zero", "against", "along"])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("form", FORMS)
def test_k_scale_not_finite(cuda_device, form, d, codes, value):
    """A K scale that is infinite or NaN (as a quantised row with an infinite or
    NaN value has it, its codes 0) makes its cell's scores NaN whatever their
    sign would be: out and lse of its KV head are NaN in the rows that attend
    to the cell, and nothing else changes."""
    q, pool, table, lens, rows = batch(form, d)
    otype, per, head = F16, 4, 2
    t = 3 if form != "whole" else 0
    page, at = (x[lens[t] - 1] for x in row_cells(table, lens, rows, t))
    # Every row attends with one sign of q in the scale's dims, so that a score
    # with this scale outside of the sum would be infinite of the other or the same sign.
    q[..., d // 4:d // 2] = np.abs(q[..., d // 4:d // 2])
    pool = [x.copy() for x in pool]
    pool[0][page, at, head, d // 4:d // 2] = {"zero": 0, "against": -3, "along": 3}[codes]
    want, wlse = attend(q, pool, table, lens, rows, otype)
    pool[2][page, at, head, 1] = value
    out, lse = attend(q, pool, table, lens, rows, otype)
    nan = torch.zeros_like(lse, dtype=torch.bool)
    for u, n in enumerate(lens):
        p, a = row_cells(table, lens, rows, u)
        if ((p == page) & (a == at)).any():
            nan[u, head * per:(head + 1) * per] = True
    assert nan.any() and torch.isnan(out[nan]).all() and torch.isnan(lse[nan]).all()
    assert torch.equal(out[~nan], want[~nan]) and torch.equal(lse[~nan], wlse[~nan])


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("form", FORMS)
def test_every_k_scale_nan(cuda_device, form, d):
    """All cells of the pool: every row with cells is NaN, an empty one is not."""
    q, pool, table, lens, rows = batch(form, d)
    pool[2][:] = np.nan
    out, lse = attend(q, pool, table, lens, rows, F16)
    some = torch.tensor([n > 0 for n in lens], device="cuda")
    assert torch.isnan(out[some]).all() and torch.isnan(lse[some]).all()
    assert not out[~some].any() and torch.isneginf(lse[~some]).all()
