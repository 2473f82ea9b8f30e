"""Rows of qsa_paged_attn that are taken together (paged_group.cu): each case
says so (taken_together), and covers a path of the kernel: groups that lie
whole in a CTA's share, several to a share, with many tiles each, gated and
not; groups shared out; rows that name no table row; queries of any size.

The reference is the definition in 64 bits, a matrix product per row.  The
tolerance counts the roundings, relative to the sum of weight * |value| of a
dim (`mag`): V's code * scale to fp16 2^-11; a weight in two parts 2^-22 (fp16
results), in one 2^-11 (bf16 results); what underflows, half of fp16's least
step of a weight in units of the largest weight * V scale, 2^-24 of that *
|code| (`flush`; a cell's largest scale is in [1, 2) of its exponent's); the scores' error ds once for the numerator and once for the
denominator; the result's own half step.  ds: K's products are exact in their
two parts, so D/8 steps of sixteen products are summed, each off by at most
2^-23 (tensor cores truncate) of 128 sum_g ksc sum|q| (`qk`), and the scale,
the exponent and the subtraction by 2^-24 of the same or of lse: D/8 * 2^-23 +
2^-21 times 128 qk.
"""
import math

import numpy as np
import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from tests.test_paged_gpu import BF16, F16, HALF, TINY, dev, i32, make_pool, shuffled_table, taken_together

pytestmark = pytest.mark.gpu


def reference(q, pool, table, lens, rows, scale=None, gate=None):
    """out, lse, mag, flush (T, H, D; lse T, H) and qk (T, H) in 64 bits, where q is."""
    (T, H, D), on = q.shape, q.device
    page, hkv = pool[0].shape[1:3]
    per, scale = H // hkv, D ** -0.5 if scale is None else scale
    kq, vq, ksc, vsc = (x.flatten(0, 1) for x in pool)
    out, mag, flush = (torch.zeros(T, H, D, dtype=torch.float64, device=on) for _ in range(3))
    lse, qk = torch.full((T, H), -math.inf, dtype=torch.float64, device=on), torch.zeros(T, H, dtype=torch.float64, device=on)
    wide = lambda s: s.double().repeat_interleave(D // 4, -1)  # noqa: E731
    c = np.arange(table.shape[1] * page)
    t0 = 0
    while t0 < T:  # a run of rows of one sequence at a time
        r, t1 = rows[t0], t0 + 1
        while t1 < T and rows[t1] == r and t1 - t0 < 64:
            t1 += 1
        run, t0 = slice(t0, t1), t1
        n = torch.tensor([min(max(v, 0), len(c)) if 0 <= r < table.shape[0] else 0 for v in lens[run]], device=on)
        most = int(n.max())
        if most == 0:
            continue
        e = table[r, c[:most] // page].astype(np.int64)
        there = (e >= 0) & (e < pool[0].shape[0])
        at = torch.from_numpy(np.where(there, e, 0) * page + c[:most] % page).to(on)
        ok = (torch.arange(most, device=on) < n[:, None]) & torch.from_numpy(there).to(on)  # [t, c]
        k, code, vs, ks = kq[at].double() * wide(ksc[at]), vq[at].double(), wide(vsc[at]), ksc[at].double()
        top, v = vsc[at].double().amax(-1), code * vs
        x = q[run].double().view(-1, hkv, per, D)
        s = (torch.einsum("thpd,chd->thpc", x, k) * scale).masked_fill(~ok[:, None, None], -math.inf)
        some = ok.any(-1)[:, None, None, None]
        w = torch.where(some, torch.softmax(s, -1), 0.0)
        shape = (-1, H, D)
        out[run] = torch.einsum("thpc,chd->thpd", w, v).reshape(shape)
        lse[run] = torch.logsumexp(s, -1).flatten(1)
        mag[run] = torch.einsum("thpc,chd->thpd", w, v.abs()).reshape(shape)
        flush[run] = ((w * top.T[None, :, None]).amax(-1)[..., None] * torch.einsum("tc,chd->thd", ok.double(), code.abs())[:, :, None]).reshape(shape)
        each = torch.einsum("chg,thpg->tchp", ks, x.abs().unflatten(-1, (4, D // 4)).sum(-1))
        qk[run] = ((each * ok[..., None, None]).amax(1) * abs(scale)).flatten(1)
    if gate is not None:
        sg = torch.sigmoid(gate.double())
        out, mag, flush = out * sg, mag * sg, flush * sg
    return out, lse, mag, flush, qk


def run(q, pool, table, lens, rows, scale=None, gate=None):
    T, H, D = q.shape
    out, lse = torch.full_like(q, 9.0), torch.full((T, H), 9.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.full((qsa.qsa_paged_attn_workspace_bytes(H, pool[0].shape[2], D),), 0xA5, dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_attn(q, *pool, dev(table), i32(lens), out, ws, rows=i32(rows), softmax_scale=scale, gate=gate, lse=lse, err=err)
    return out, lse, int(err.item())


def bounds(ref, lse, mag, flush, qk, otype, d, v_exact=False):
    ds = 128 * qk * (d / 8 * 2.0 ** -23 + 2.0 ** -21)
    w = 2.0 ** -21 if otype is F16 else 2.0 ** -11
    v = 0.0 if v_exact else 2.0 ** -11
    tol = HALF[otype] * ref.abs() + mag * (w + v + 2 * torch.expm1(ds)[..., None] + 2.0 ** -20) + flush * 2.0 ** -24 + TINY[otype]
    return tol, ds + 2.0 ** -20 + 2.0 ** -21 * lse.abs()


def check(q, pool, table, lens, rows, scale=None, gate=None, error=0, valid=None, v_exact=False):
    """Compares a call with the reference; rows: as given, valid: as they count."""
    T, H, D = q.shape
    hkv = pool[0].shape[2]
    use = lens if valid is None else [n if v else 0 for n, v in zip(lens, valid)]
    assert taken_together(rows, use, H, hkv, D)
    out, lse, err = run(q, pool, table, lens, rows, scale, gate)
    assert err == error
    ref = reference(q, pool, table, lens, rows, scale, gate)
    tol, ltol = bounds(*ref, q.dtype, D, v_exact)
    bad = ~((out.double() - ref[0]).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), out[bad][:5], ref[0][bad][:5], tol[bad][:5])
    empty = torch.isneginf(ref[1])
    assert torch.equal(torch.isneginf(lse), empty) and not out[empty].any()
    bad = ~((lse.double() - ref[1]).abs() <= ltol) & ~empty
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist(), lse[bad][:5], ref[1][bad][:5], ltol[bad][:5])
    return out, lse


def windows(held, window, page, hkv, d, seed, extra=2):
    """Each sequence's last `window` tokens, one after the other."""
    rng = np.random.default_rng(seed)
    table, pages = shuffled_table(held, page, extra, rng)
    pool = [dev(x) for x in make_pool(pages, page, hkv, d, seed=seed)]
    rows = [s for s in range(len(held)) for _ in range(window)]
    lens = [n - window + 1 + i for n in held for i in range(window)]
    return pool, table, lens, rows


def queries(T, H, D, otype, seed, size=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, H, D, generator=g, device="cuda") * size).to(otype)


def gates(T, H, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 2.0 * torch.randn(T, H, D, generator=g, device="cuda")


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("d,hq,hkv,page,seqs,window,lo,hi", [
    (128, 8, 1, 64, 220, 16, 560, 640),     # groups of ten tiles, fifteen to a share: whole ones and shared ones
    (256, 4, 1, 32, 200, 16, 500, 610), (128, 24, 2, 16, 160, 8, 1000, 1100), (256, 16, 4, 16, 70, 16, 300, 900),
    (128, 16, 8, 128, 300, 32, 40, 700),    # short and long windows mixed
    (128, 16, 1, 256, 900, 8, 1, 1500)])
def test_many_groups_whole_in_a_share(cuda_device, d, hq, hkv, page, seqs, window, lo, hi, gated, otype):
    rng = np.random.default_rng(seqs)
    held = [max(int(n), window) for n in rng.integers(lo, hi + 1, seqs)]
    pool, table, lens, rows = windows(held, window, page, hkv, d, seqs)
    tiles = sum(-(-n // 64) for n in held)
    share = -(-tiles // (152 // hkv))
    assert share >= max(-(-n // 64) for n in held) + 2 or hkv > 2  # a CTA ends one group and has another whole
    T = len(rows)
    check(queries(T, hq, d, otype, 1), pool, table, lens, rows, gate=gates(T, hq, d, 2) if gated else None)


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,window,cells", [(128, 4, 1, 16, 20000), (256, 12, 2, 8, 9000), (128, 64, 4, 8, 9001), (256, 32, 8, 31, 1100)])
def test_one_group_over_the_chip(cuda_device, d, hq, hkv, window, cells, otype):
    pool, table, lens, rows = windows([cells], window, 64, hkv, d, window)
    check(queries(window, hq, d, otype, 3), pool, table, lens, rows, gate=gates(window, hq, d, 4) if hkv == 2 else None)


@pytest.mark.parametrize("d,n", [(128, 8), (128, 40), (256, 8)])
def test_rows_that_name_no_table_row(cuda_device, d, n):
    """Windows of rows outside the table (empty, and reported) beside long valid
    ones; up to 32 rows of q, and more."""
    pool, table, lens, _ = windows([2600, 2300], n, 32, 8, d, 60)
    rows = [0] * n + [7] * n + [-3] * n + [1] * n
    lens = lens[:n] + [1500 + i for i in range(n)] + [9] * n + lens[n:]
    valid = [0 <= r < 2 for r in rows]
    for otype in (F16, BF16):
        out, lse = check(queries(4 * n, 16, d, otype, 5), pool, table, lens, rows, error=qsa.QSA_DEVERR_BAD_ID, valid=valid)
        assert not out[n:3 * n].any() and torch.isneginf(lse[n:3 * n]).all()


def test_lengths_out_of_range_and_missing_pages(cuda_device):
    pool, table, lens, rows = windows([2600, 2600], 16, 32, 8, 128, 61)
    table = table.copy()
    table[0, 5], table[1, 0], table[1, 81] = -2, pool[0].shape[0], 1 << 30
    lens[3], lens[7], lens[20] = -5, 1 << 20, 0
    use = [min(max(n, 0), 2624) for n in lens]
    assert taken_together(rows, use, 16, 8, 128)
    q = queries(32, 16, 128, BF16, 6)
    out, lse, err = run(q, pool, table, lens, rows)
    assert err == qsa.QSA_DEVERR_BAD_ID and not out[3].any() and not out[20].any()
    ref = reference(q, pool, table, use, rows)
    tol, _ = bounds(*ref, BF16, 128)
    assert ((out.double() - ref[0]).abs() <= tol).all() and torch.isneginf(lse[[3, 20]]).all()


@pytest.mark.parametrize("otype,size,scale", [(BF16, 1e8, 1e-9), (BF16, 1e30, 1e-31), (BF16, 1e-20, 1e19), (BF16, 1e-38, 1e37), (F16, 8000.0, 1e-5),
                                              (F16, 1e-4, 900.0), (F16, 1.0, -0.05), (BF16, 1.0, 0.0)])
@pytest.mark.parametrize("d", [128, 256])
def test_query_sizes(cuda_device, d, otype, size, scale):
    """Queries far outside fp16's range and at both ends of it, with the scale
    that undoes it; one head of zeros."""
    pool, table, lens, rows = windows([1300, 900], 32, 32, 8, d, 62)
    g = torch.Generator(device="cuda").manual_seed(7)
    q = (torch.randn(64, 16, d, generator=g, device="cuda", dtype=torch.float64) * size).to(otype)
    q[:, 3] = 0
    check(q, pool, table, lens, rows, scale=scale)


def test_v_scales_of_all_sizes(cuda_device):
    """V scales from fp16's least to 100, cell by cell and zero ones among them:
    the sum has an exponent per cell, so a cell's size does not cost another's
    digits where it has the weight."""
    pool, table, lens, rows = windows([900], 100, 32, 8, 128, 63)
    g = torch.Generator(device="cuda").manual_seed(8)
    size = torch.exp(torch.rand(*pool[3].shape[:3], 1, generator=g, device="cuda") * (math.log(100.0) - math.log(1e-6)) + math.log(1e-6))
    pool[3] = (size * (1 + torch.rand(pool[3].shape, generator=g, device="cuda"))).half()
    pool[3][::5] = 0
    check(queries(100, 16, 128, F16, 9), pool, table, lens, rows)
