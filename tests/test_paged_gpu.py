"""The paged cache's calls on the GPU against their float64 oracle.

Tolerances, derived from the number formats (a rounding is off by at most half
a step, relative 2^-11 in fp16 and 2^-8 in bf16):
  query rows   half a step of the output, plus 2^-19 of the row's entries that
               meet in it: at most 20 fp32 roundings (sum of squares, root,
               products, rotation) and angles to 2^-22 rad;
  cached rows  |code * s - y| <= s (1/2 + 2^-10): half a code, and the fp32
               error of y (2^-19 of at most 128 codes = 2^-12) with the largest
               code's own excess, where s = fp16(max/127) is rounded down by up
               to 2^-11 (127 * 2^-11 = 2^-4 of a code, for the codes at +-127
               only, below the half);
               rows that are stored as given are exact, bit for bit;
  attention    half a step of the output, plus per cell weight * |v| * 2^-10
               (weight to fp16, weight * scale to fp16: two half steps) or,
               where that underflows, |code| * 2^-24 of the largest V scale,
               plus the scores' error twice (numerator and denominator): fp32
               sums of 32 products of q with codes shifted by 1152, each step
               off by at most 2^-21 of 1152 * sum|q| (tensor cores truncate),
               plus 2^-16 for exponentials and sums;
  everything else (tables, slots, counts, copies, gathered values) is exact.
"""
import math

import numpy as np
import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from oracle import paged_oracle as po
from oracle import quantize_rows
from sparse_selected_attention_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
HALF = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
TINY = {F16: 2.0 ** -25, BF16: 0.0}


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def i32(*v):
    return dev(np.asarray(v, dtype=np.int32).reshape(-1))


def make_pool(pages, page, hkv, d, seed=5, layers=None, scale_lo=1e-3, scale_hi=2e-2):
    c = wl.make_cache((layers or 1) * pages * page * hkv, seed=seed, head_dim=d, group=d // 4, scale_lo=scale_lo, scale_hi=scale_hi)
    lead = (pages, page, hkv) if layers is None else (layers, pages, page, hkv)
    return [x.reshape(*lead, -1) for x in (c.kq, c.vq, c.ksc, c.vsc)]


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- prep

def run_prep(T, hq, hkv, d, itype, otype, rope, inter, norm, pos, slots, page=32, mscale=1.0, strided=True, seed=7):
    cells = max(64, -(-(max(slots) + 1) // page) * page)
    x = wl.normal(seed, 1, (T, hq + 2 * hkv, d)) * np.exp(wl.normal(seed, 2, (T, hq + 2 * hkv, 1)))
    xd = dev(x.astype(np.float32)).to(itype)
    q, k, v = xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:]
    if not strided:
        q, k, v = (z.contiguous() for z in (q, k, v))
    wq = wl.uniform(seed, 3, (d,), 0.5, 1.5).astype(np.float32) if norm else None
    wk = wl.uniform(seed, 4, (d,), 0.5, 1.5).astype(np.float32) if norm else None
    freq = (10000.0 ** (-2.0 * np.arange(rope // 2) / rope)).astype(np.float32) if rope else None
    pool = [torch.full(s, 77, dtype=t, device="cuda") for s, t in
            (((cells, hkv, d), torch.int8), ((cells, hkv, d), torch.int8), ((cells, hkv, 4), F16), ((cells, hkv, 4), F16))]
    qo = torch.full((T, hq, d), 55.0, dtype=otype, device="cuda")
    err = err_word()
    qsa.qsa_paged_prep(q, k, v, i32(pos), i32(slots), *pool, qo, q_norm_w=None if wq is None else dev(wq),
                       k_norm_w=None if wk is None else dev(wk), inv_freq=None if freq is None else dev(freq),
                       interleaved=inter, rope_mscale=mscale, err=err)
    torch.cuda.synchronize()
    x64 = host(xd)
    used = [t for t in range(T) if 0 <= slots[t] < cells]
    qr = po.norm_rotate(x64[:, :hq], wq, pos, freq, inter, mscale)
    kr = po.norm_rotate(x64[:, hq:hq + hkv], wk, pos, freq, inter, mscale)
    # Entries that meet in one rotated value: bounded by the pair's magnitude.
    mag = lambda w, z: np.sqrt(2.0) * np.abs(po.norm_rotate(z, w, pos, None)).max(-1, keepdims=True) * abs(mscale) + np.abs(z * 0)  # noqa: E731
    got = host(qo)
    tol = HALF[otype] * np.abs(qr) + 2.0 ** -19 * mag(wq, x64[:, :hq]) + TINY[otype]
    assert np.all(np.abs(got - qr)[used] <= tol[used])
    unused = [t for t in range(T) if t not in used]
    assert np.all(got[unused] == 55.0)
    kq, vq, ksc, vsc = (z.cpu().numpy() for z in pool)
    at = np.array([slots[t] for t in used], dtype=int)
    if used:
        vcode, vscale = quantize_rows(x64[used, hq + hkv:].astype(np.float32), d // 4)
        assert np.array_equal(vq[at], vcode.reshape(vq[at].shape))
        assert np.array_equal(vsc[at].view(np.int16), np.asarray(vscale, dtype=np.float16).reshape(vsc[at].shape).view(np.int16))
        if not rope and not norm:
            kcode, kscale = quantize_rows(x64[used, hq:hq + hkv].astype(np.float32), d // 4)
            assert np.array_equal(kq[at], kcode.reshape(kq[at].shape))
        y = kr[used].reshape(len(used), hkv, 4, d // 4)
        s = ksc[at].astype(np.float64)
        top = np.abs(y).max(-1) / 127
        assert np.all(np.abs(s - top) <= 2.0 ** -11 * top + 2.0 ** -18 * top + 2.0 ** -25)
        back = kq[at].reshape(y.shape).astype(np.float64) * s[..., None]
        assert np.all(np.abs(back - y) <= s[..., None] * (0.5 + 2.0 ** -10) + 2.0 ** -25 * 127 * (s[..., None] < 2.0 ** -14))
    left = np.setdiff1d(np.arange(cells), at)
    assert np.all(kq[left] == 77) and np.all(vq[left] == 77) and np.all(ksc[left] == 77) and np.all(vsc[left] == 77)
    return int(err.item()), qo, pool


@pytest.mark.parametrize("d,hq,hkv", [(128, 12, 1), (256, 24, 2), (128, 1, 1), (128, 8, 8), (256, 5, 5), (128, 33, 3)])
@pytest.mark.parametrize("itype,otype", [(F32, F16), (F16, F16), (BF16, BF16)])
@pytest.mark.parametrize("inter", [False, True])
def test_prep_shapes_and_types(cuda_device, d, hq, hkv, itype, otype, inter):
    T = 9
    slots = [(5 * t + 3) % 64 for t in range(T)]
    err, _, _ = run_prep(T, hq, hkv, d, itype, otype, 64, inter, True, list(range(30000, 30000 + T)), slots)
    assert err == 0


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("rope", [0, "least", "full"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("inter", [False, True])
def test_prep_rotated_part(cuda_device, d, rope, norm, inter):
    n = {0: 0, "least": d // 16, "full": d}[rope]
    run_prep(4, 3, 2, d, BF16, F16, n, inter, norm, [0, 1, 131071, 1 << 24], [7, 0, 63, 20], mscale=1.25)


def test_prep_far_positions(cuda_device):
    """Angles of the first frequency (1 rad per position) up to 2^31 - 1."""
    pos = [0, 1, 2 ** 20 + 1, 2 ** 29 - 3, 2 ** 31 - 1]
    run_prep(5, 2, 1, 128, F32, F16, 128, False, True, pos, [4, 3, 2, 1, 0])


def test_prep_one_token_and_strides(cuda_device):
    run_prep(1, 12, 1, 128, F16, F16, 64, False, True, [320], [63], strided=False)
    run_prep(1, 12, 1, 128, F16, F16, 64, False, True, [320], [63])
    run_prep(70, 4, 2, 128, F32, BF16, 32, True, True, list(range(70)), list(range(70)), page=16, strided=False)


def test_prep_padding_and_bad_slots(cuda_device):
    """-1 is padding; other slots outside are padding that is reported."""
    err, _, _ = run_prep(5, 2, 1, 128, BF16, F16, 64, False, True, [1, 2, 3, 4, 5], [3, -1, 9, -1, 0])
    assert err == 0
    x = torch.ones(2, 4, 128, dtype=F16, device="cuda")
    pool = [torch.zeros(s, dtype=t, device="cuda") for s, t in (((32, 1, 128), torch.int8),) * 2 + (((32, 1, 4), F16),) * 2]
    qo, err = torch.full((2, 2, 128), 3.0, dtype=F16, device="cuda"), err_word()
    qsa.qsa_paged_prep(x[:, :2], x[:, 2:3], x[:, 3:], i32(0, 1), i32(32, -7), *pool, qo, err=err)
    assert int(err.item()) == qsa.QSA_DEVERR_BAD_ID
    assert (qo == 3.0).all() and not any(p.any() for p in pool)


def test_prep_extreme_rows(cuda_device):
    """Zero groups, groups that hold an infinity or a NaN (poisoned, the others
    untouched), values at the fp16 scale's limits."""
    x = np.zeros((4, 3, 128), dtype=np.float32)
    x[0, 2, 0:32] = np.linspace(-3, 3, 32)
    x[1, 2, 5], x[1, 2, 40] = np.inf, 2.0
    x[2, 2, 100], x[2, 2, 1] = np.nan, -1.0
    x[3, 2, 64], x[3, 2, 96] = 127 * 65504.0, 3e-6
    x[:, 1] = x[:, 2]
    xd = dev(x)
    pool = [torch.zeros(s, dtype=t, device="cuda") for s, t in (((16, 1, 128), torch.int8),) * 2 + (((16, 1, 4), F16),) * 2]
    qo = torch.zeros(4, 1, 128, dtype=F16, device="cuda")
    qsa.qsa_paged_prep(xd[:, :1], xd[:, 1:2], xd[:, 2:], i32(0, 1, 2, 3), i32(0, 1, 2, 3), *pool, qo)
    back = [torch.empty(4, 1, 128, device="cuda") for _ in range(2)]
    qsa.qsa_paged_gather(*pool, i32(0, 1, 2, 3), *back)
    for b in back:
        b = b.cpu().numpy()[:, 0].reshape(4, 4, 32)
        assert np.all(np.abs(b[0, 0] - x[0, 2, :32]) <= 3.0 / 127 * 0.501 + 1e-6) and not b[0, 1:].any()
        assert np.isnan(b[1, 0]).any() and not np.isfinite(b[1, 0]).any() and b[1, 1, 8] == pytest.approx(2.0, rel=2 ** -10)
        assert np.isnan(b[2, 3]).all() and b[2, 0, 1] == pytest.approx(-1.0, rel=2 ** -10)
        assert b[3, 2, 0] == 127 * 65504.0 and b[3, 3, 0] <= 4e-6


# ---------------------------------------------------------------- gather

@pytest.mark.parametrize("d,hkv,page", [(128, 1, 64), (256, 2, 16), (128, 3, 256)])
@pytest.mark.parametrize("otype", [F32, F16, BF16])
def test_gather(cuda_device, d, hkv, page, otype):
    pages = 6
    pool = make_pool(pages, page, hkv, d, seed=11)
    n = 157
    cells = np.arange(n) * 37 % (pages * page)
    cells[5], cells[9] = -1, pages * page - 1
    ko, vo = (torch.full((n, hkv, d), 9.0, dtype=otype, device="cuda") for _ in range(2))
    err = err_word()
    pd = [dev(x) for x in pool]
    qsa.qsa_paged_gather(*pd, i32(cells), ko, vo, err=err)
    assert int(err.item()) == 0
    for codes, scales, got in ((pool[0], pool[2], ko), (pool[1], pool[3], vo)):
        v = codes.reshape(-1, hkv, d).astype(np.float32) * np.repeat(scales.reshape(-1, hkv, 4).astype(np.float32), d // 4, -1)
        v = v[np.maximum(cells, 0)] * (cells >= 0)[:, None, None]
        assert torch.equal(got, dev(v).to(otype) + 0.0)
    # The same cells through a table, rows given out of order.
    table = np.array([[4, 1], [0, 5], [2, 3]], dtype=np.int32)
    rows = np.arange(n) % 3
    ids = np.arange(n) * 29 % (2 * page)
    flat = table[rows, ids // page] * page + ids % page
    a, b = [torch.empty_like(ko) for _ in range(2)], [torch.empty_like(ko) for _ in range(2)]
    qsa.qsa_paged_gather(*pd, i32(ids), *a, rows=i32(rows), page_table=dev(table), err=err)
    qsa.qsa_paged_gather(*pd, i32(flat), *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and int(err.item()) == 0


def test_gather_bad_ids(cuda_device):
    pd = [dev(x) for x in make_pool(2, 16, 1, 128)]
    table = i32(0, 5, 1, -1).view(2, 2)
    for ids, rows in (((-2, 3), None), ((32, 3), None), ((16, 3), (0, 0)), ((16, 3), (1, 0)), ((32, 3), (0, 0)),
                      ((0, 3), (2, 0)), ((0, 3), (-1, 0))):
        ko, vo = (torch.full((2, 1, 128), 9.0, device="cuda") for _ in range(2))
        err = err_word()
        kw = {} if rows is None else dict(rows=i32(*rows), page_table=table)
        qsa.qsa_paged_gather(*pd, i32(*ids), ko, vo, err=err, **kw)
        assert int(err.item()) == qsa.QSA_DEVERR_BAD_ID, (ids, rows)
        assert not ko[0].any() and not vo[0].any() and ko[1].any()
    qsa.qsa_paged_gather(*pd, i32()[:0], ko[:0], vo[:0])


# ---------------------------------------------------------------- attention

def shuffled_table(lens, page, extra, rng, wide=None):
    held = [-(-max(n, 0) // page) for n in lens]
    pages = sum(held) + extra
    order = rng.permutation(pages)
    table = np.full((len(lens), wide or max(held + [1])), -1, dtype=np.int32)
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = order[at:at + h]
        at += h
    return table, max(pages, 1)


def check_attn(q, pool, table, lens, rows=None, scale=None, gate=None, otype=F16, lse=True, ws=None, what=""):
    """q float64 [T, H, D]; returns the output tensor and the error word."""
    T, H, D = q.shape
    hkv = pool[0].shape[2]
    qd = dev(q.astype(np.float32)).to(otype)
    out = torch.full((T, H, D), 9.0, dtype=otype, device="cuda")
    ls = torch.full((T, H), 9.0, device="cuda") if lse else None
    err = err_word()
    if ws is None:
        ws = torch.full((qsa.qsa_paged_attn_workspace_bytes(H, hkv, D),), 0xA5, dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_attn(qd, *[dev(x) for x in pool], dev(table), i32(lens), out, ws, rows=None if rows is None else i32(rows),
                       softmax_scale=scale, gate=None if gate is None else dev(gate), lse=ls, err=err)
    torch.cuda.synchronize()
    ref, rlse, mag, flush, qk = po.attn(host(qd), *pool, table, lens, rows, scale, gate)
    ds = 1152 * qk * 2.0 ** -21
    tol = HALF[otype] * np.abs(ref) + mag * (2.0 ** -10 + 2 * np.expm1(ds)[..., None] + 2.0 ** -16) + flush * 2.0 ** -24 + TINY[otype]
    got = host(out)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5].tolist(), got[bad][:5], ref[bad][:5], tol[bad][:5])
    if lse:
        g = ls.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isneginf(g), np.isneginf(rlse))
        fin = np.isfinite(rlse)
        assert np.all(np.abs(g[fin] - rlse[fin]) <= ds[fin] + 2.0 ** -16 + 2.0 ** -22 * np.abs(rlse[fin]))
    return out, int(err.item())


LENS = [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 321, 1000]


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,page", [(128, 12, 1, 64), (256, 24, 2, 16), (128, 32, 8, 32), (128, 16, 1, 16), (128, 2, 2, 128),
                                           (256, 1, 1, 256), (256, 9, 3, 32)])
def test_attn_shapes(cuda_device, d, hq, hkv, page, otype):
    rng = np.random.default_rng(1)
    lens = LENS + [0, 700]
    table, pages = shuffled_table(lens, page, 3, rng)
    pool = make_pool(pages, page, hkv, d, seed=12)
    q = rng.standard_normal((len(lens), hq, d)) * 2
    out, err = check_attn(q, pool, table, lens, otype=otype)
    assert err == 0 and not out[lens.index(0)].any()


@pytest.mark.parametrize("rows_n,lo,hi", [(1, 30008, 30008), (3, 5000, 20000), (40, 1, 2500), (700, 1, 90), (1, 1, 1), (1, 700, 700)])
@pytest.mark.parametrize("page", [16, 64])
def test_attn_split_lengths(cuda_device, rows_n, lo, hi, page):
    """Few long rows (their cells shared out over the chip and joined), many
    short ones (several to a block), and both kinds of boundary between."""
    rng = np.random.default_rng(rows_n)
    lens = [int(v) for v in rng.integers(lo, hi + 1, rows_n)]
    lens[-1] = hi
    table, pages = shuffled_table(lens, page, 1, rng)
    pool = make_pool(pages, page, 1, 128, seed=13)
    q = rng.standard_normal((rows_n, 4, 128)) * 3
    _, err = check_attn(q, pool, table, lens)
    assert err == 0


@pytest.mark.parametrize("d,hq,hkv,page,n,most", [
    (128, 8, 8, 16, 40, 16), (128, 16, 1, 64, 320, 64), (128, 24, 4, 128, 160, 128), (256, 12, 4, 16, 90, 16), (256, 16, 2, 32, 170, 32),
    (256, 10, 10, 64, 70, 64), (128, 320, 160, 16, 3, 16)])
def test_attn_many_short_rows(cuda_device, d, hq, hkv, page, n, most):
    """More short rows than blocks: a warp each, several rows to a warp, with
    empty rows, bad pages and all head counts; gated and with lse."""
    rng = np.random.default_rng(n)
    lens = [int(v) for v in rng.integers(0, most + 1, n)]
    lens[:3] = [most, 0, 1]
    table, pages = shuffled_table(lens, page, 1, rng, wide=most // page)
    pool = make_pool(pages, page, hkv, d, seed=40)
    q = rng.standard_normal((n, hq, d)) * 2
    gate = wl.gates_f32(n, seed=6, heads=hq, head_dim=d)
    for otype in (F16, BF16):
        _, err = check_attn(q, pool, table, lens, gate=gate, otype=otype)
        assert err == 0
    table[0, 0] = -7
    out, err = check_attn(q, pool, table, lens, rows=list(range(n)))
    assert err == qsa.QSA_DEVERR_BAD_ID and not out[1].any()


def test_attn_draft_window_shares_a_sequence(cuda_device):
    """Eight rows of one sequence, each a cell longer, and the order of rows
    and columns unlike the table's; gated, wide heads."""
    rng = np.random.default_rng(4)
    base = 2990
    table, pages = shuffled_table([100, base + 8, 50], 64, 2, rng)
    pool = make_pool(pages, 64, 2, 256, seed=14)
    rows = [1] * 8 + [2, 0, 0]
    lens = [base + 1 + i for i in range(8)] + [50, 99, 0]
    q = rng.standard_normal((11, 24, 256))
    gate = wl.gates_f32(11, seed=3, heads=24, head_dim=256)
    _, err = check_attn(q, pool, table, lens, rows=rows, gate=gate, otype=BF16)
    assert err == 0


@pytest.mark.parametrize("d,hq,hkv,page,window,base", [
    (128, 12, 1, 64, 8, 700), (256, 24, 2, 16, 8, 1300), (128, 32, 8, 32, 4, 500), (128, 4, 4, 16, 130, 63), (256, 16, 1, 256, 5, 1),
    (128, 8, 1, 128, 16, 9000), (256, 6, 3, 64, 3, 64)])
def test_attn_groups(cuda_device, d, hq, hkv, page, window, base):
    """Windows of consecutive tokens of several sequences, which are taken
    together: sizes below and past a group's, alone and beside single rows."""
    rng = np.random.default_rng(window)
    held = [base + window, 40, base // 2 + 3, 2 * base + window]
    table, pages = shuffled_table(held, page, 2, rng)
    pool = make_pool(pages, page, hkv, d, seed=22)
    rows, lens = [], []
    for s in (0, 1, 3, 2, 0):
        n = window if s != 1 else 1
        rows += [s] * n
        lens += [max(held[s] - n + 1 + i, 0) for i in range(n)]
    q = rng.standard_normal((len(rows), hq, d)) * 1.5
    otype = F16 if hkv % 2 else BF16
    gate = wl.gates_f32(len(rows), seed=4, heads=hq, head_dim=d) if hkv == 2 else None
    _, err = check_attn(q, pool, table, lens, rows=rows, gate=gate, otype=otype)
    assert err == 0


def test_attn_group_lengths_and_scales(cuda_device):
    """Rows of a group in any order of lengths, empty ones among them; wide K
    and V scales, zero ones, a negative softmax scale; missing pages."""
    rng = np.random.default_rng(23)
    table, pages = shuffled_table([1000, 64], 32, 2, rng)
    pool = make_pool(pages, 32, 2, 128, seed=23)
    for i in (2, 3):
        pool[i] = np.exp(wl.uniform(24 + i, 1, pool[i].shape, math.log(1e-5), math.log(0.5 if i == 2 else 100.0))).astype(np.float16)
        pool[i][::3, ::2] = 0
    rows = [0] * 7 + [1] * 5
    lens = [1000, 0, 3, 129, 64, 999, 65, 0, 64, 1, 63, 33]
    q = rng.standard_normal((12, 24, 128))
    for scale in (None, -0.03, 0.0):
        out, err = check_attn(q, pool, table, lens, rows=rows, scale=scale, otype=BF16)
        assert err == 0 and not out[1].any() and not out[7].any()
    check_attn(q * 1e8, pool, table, lens, rows=rows, scale=1e-10, otype=BF16)
    table[0, 3], table[1, 1] = -4, pages
    _, err = check_attn(q, pool, table, lens, rows=rows)
    assert err == qsa.QSA_DEVERR_BAD_ID
    out, err = check_attn(q, pool, table, lens, rows=[9] * 12)
    assert err == qsa.QSA_DEVERR_BAD_ID and not out.any()


def test_attn_many_groups(cuda_device):
    """More groups than CTAs, and one group over the whole chip."""
    rng = np.random.default_rng(25)
    for seqs, window, lo, hi in ((90, 4, 1, 300), (1, 8, 20000, 20000), (5, 3, 2000, 4000)):
        held = [int(v) + window for v in rng.integers(lo, hi + 1, seqs)]
        table, pages = shuffled_table(held, 64, 1, rng)
        pool = make_pool(pages, 64, 1, 128, seed=26)
        rows = [s for s in range(seqs) for _ in range(window)]
        lens = [held[s] - window + 1 + i for s in range(seqs) for i in range(window)]
        q = rng.standard_normal((len(rows), 4, 128)) * 2
        _, err = check_attn(q, pool, table, lens, rows=rows)
        assert err == 0


def taken_together(rows, lens, hq, hkv, d):
    """Whether the call's rows are taken by groups: the units of 32 (of 256
    dims 16) cells that rows alone and the longest of each group have."""
    unit, block = 32 if d == 128 else 16, 1
    while 2 * block * (hq // hkv) <= 128:
        block *= 2
    units = [max(-(-n // unit), 1) for n in lens]
    together, start = 0, 0
    for t in range(len(rows)):
        if t % max(block, 64) == 0 or rows[t] != rows[t - 1]:
            start = t
        if (t - start) % block == 0:
            end = t
            while end < len(rows) and end - t < block and rows[end] == rows[t] and (end == t or end % max(block, 64)):
                end += 1
            together += max(units[t:end])
    return max(units) > 16 and (2 * sum(units) - (8 if d == 128 else 7) * together) * hkv > 8192


@pytest.mark.parametrize("d,hq,hkv,page,windows,cells", [
    (128, 8, 8, 64, [128], 600), (128, 12, 1, 64, [8], 33001), (256, 24, 2, 16, [8, 8, 1], 7900), (256, 16, 1, 256, [40], 2950),
    (128, 32, 8, 32, [4, 5, 7, 1, 8, 2, 6, 9, 5, 4, 3, 6], 2000), (256, 6, 3, 64, [67], 700), (128, 15, 3, 128, [90, 1, 30], 1300),
    (256, 8, 8, 32, [300, 210], 290), (128, 2, 2, 16, [512, 188], 1030)])
def test_attn_rows_taken_together(cuda_device, d, hq, hkv, page, windows, cells):
    """Windows of consecutive tokens of sequences, long enough to be taken by
    groups: groups cut by a block, by a span and by the rows' end, heads that do
    not fill a tile, shares that end inside a group; empty outputs' neighbours."""
    rng = np.random.default_rng(len(windows) + d)
    held = [cells - 3 * i for i in range(len(windows))]
    table, pages = shuffled_table(held, page, 2, rng)
    pool = make_pool(pages, page, hkv, d, seed=27)
    rows = [s for s, n in enumerate(windows) for _ in range(n)]
    lens = [max(held[s] - n + 1 + i, 0) for s, n in enumerate(windows) for i in range(n)]
    assert taken_together(rows, lens, hq, hkv, d)
    q = rng.standard_normal((len(rows), hq, d)) * 1.5
    gate = wl.gates_f32(len(rows), seed=5, heads=hq, head_dim=d) if hkv == 2 else None
    for otype in (F16, BF16):
        _, err = check_attn(q, pool, table, lens, rows=rows, gate=gate, otype=otype)
        assert err == 0


def test_attn_together_lengths_and_scales(cuda_device):
    """Rows taken together with any order of lengths, empty ones among them;
    wide K and V scales, zero ones, a negative softmax scale; missing pages."""
    rng = np.random.default_rng(28)
    table, pages = shuffled_table([700, 64], 32, 2, rng)
    pool = make_pool(pages, 32, 8, 128, seed=29)
    for i in (2, 3):
        pool[i] = np.exp(wl.uniform(30 + i, 1, pool[i].shape, math.log(1e-5), math.log(0.5 if i == 2 else 100.0))).astype(np.float16)
        pool[i][::3, ::2] = 0
    rows = [0] * 128 + [1] * 5
    lens = [int(n) for n in rng.integers(0, 701, 128)] + [64, 1, 63, 33, 0]
    lens[:9] = [700, 0, 3, 129, 64, 699, 65, 0, 1]
    assert taken_together(rows, lens, 8, 8, 128)
    q = rng.standard_normal((133, 8, 128))
    for otype in (F16, BF16):
        for scale in (None, -0.03, 0.0):
            out, err = check_attn(q, pool, table, lens, rows=rows, scale=scale, otype=otype)
            assert err == 0 and not out[1].any() and not out[7].any() and not out[132].any()
    check_attn(q * 1e8, pool, table, lens, rows=rows, scale=1e-10, otype=BF16)
    table[0, 3], table[1, 1] = -4, pages
    _, err = check_attn(q, pool, table, lens, rows=rows)
    assert err == qsa.QSA_DEVERR_BAD_ID


def test_attn_together_repeats_its_bits(cuda_device):
    """The same call twice, and captured and replayed, gives the same bits."""
    rng = np.random.default_rng(31)
    table, pages = shuffled_table([900], 64, 1, rng)
    pd = [dev(x) for x in make_pool(pages, 64, 8, 128, seed=32)]
    q = dev(rng.standard_normal((100, 8, 128)).astype(np.float16))
    lens, rows = i32(list(range(801, 901))), i32([0] * 100)
    ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(8, 8, 128), dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(q) for _ in range(3)]
    for o in out[:2]:
        qsa.qsa_paged_attn(q, *pd, dev(table), lens, o, ws, rows=rows)
    td, g, s = dev(table), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        qsa.qsa_paged_attn(q, *pd, td, lens, out[2], ws, rows=rows)
    for _ in range(2):
        out[2].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("d,hq,hkv,n,base", [(128, 8, 8, 128, 600), (256, 16, 8, 64, 560), (128, 12, 1, 8, 700)])
def test_attn_nan_and_inf_reach_only_their_rows(cuda_device, d, hq, hkv, n, base):
    """A NaN or infinite scale of a window's later token: rows that end before
    its cell are as without it, to the last bit where the division of work is
    the same; a V scale makes its own dims of the others NaN or infinite, a K
    scale a whole head of them."""
    rng = np.random.default_rng(33)
    table, pages = shuffled_table([base + n], 32, 1, rng)
    pool = make_pool(pages, 32, hkv, d, seed=34)
    rows, lens = [0] * n, [base + 1 + i for i in range(n)]
    q = rng.standard_normal((n, hq, d))
    per, cut = hq // hkv, n // 2
    cell = base + cut  # of row cut's own token
    page, at = table[0, cell // 32], cell % 32
    # Two runs, each off by two roundings of at most 2^-11 of each term.
    most = 2 * 2.0 ** -10 * float(np.abs(pool[1].astype(np.float64) * np.repeat(pool[3].astype(np.float64), d // 4, -1)).max())
    for otype in (F16, BF16):
        plain, _ = check_attn(q, pool, table, lens, rows=rows, otype=otype)
        for value in (np.nan, np.inf, -np.inf):
            bad = [x.copy() for x in pool]
            bad[3][page, at, hkv - 1, 2] = value
            bad[1][page, at, hkv - 1] = 3
            out = torch.empty_like(plain)
            ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(hq, hkv, d), dtype=torch.uint8, device="cuda")
            args = (dev(table), i32(lens), out, ws)
            qd = dev(q.astype(np.float32)).to(otype)
            good = [x.copy() for x in bad]
            good[3][page, at, hkv - 1, 2] = 0.01
            qsa.qsa_paged_attn(qd, *[dev(x) for x in good], *args, rows=i32(rows))
            want = out.clone()
            qsa.qsa_paged_attn(qd, *[dev(x) for x in bad], *args, rows=i32(rows))
            head, dims = slice((hkv - 1) * per, hq), slice(d // 2, 3 * d // 4)
            assert not torch.isfinite(out[cut:, head, dims]).any()
            assert torch.equal(out[:cut], want[:cut]) and torch.equal(out[:, :hq - per], want[:, :hq - per])
            for part in (slice(0, d // 2), slice(3 * d // 4, d)):
                assert torch.isfinite(out[cut:, head, part]).all()
                assert torch.allclose(out[cut:, head, part].float(), want[cut:, head, part].float(), rtol=2.0 ** -7, atol=most)
        bad = [x.copy() for x in pool]
        bad[2][page, at, 0, 1] = np.nan
        out = torch.empty_like(plain)
        qsa.qsa_paged_attn(qd, *[dev(x) for x in bad], dev(table), i32(lens), out, ws, rows=i32(rows))
        assert torch.equal(out[:cut], plain[:cut]) and torch.equal(out[:, per:], plain[:, per:])
        assert torch.isnan(out[cut:, :per]).all()


def test_attn_together_beyond_32_bit_offsets(cuda_device):
    """Rows taken together whose pages start past 2^32 bytes of codes."""
    page, d, hkv, n, held = 64, 256, 8, 64, 9
    pages = (1 << 32) // (page * hkv * d) + 16
    small = make_pool(held, page, hkv, d, seed=35)
    big = [torch.zeros(pages, page, hkv, x.shape[3], dtype=dev(x).dtype, device="cuda") for x in small]
    where = [pages - 1 - 2 * i if i % 2 else i for i in range(held)]
    for t, x in zip(big, small):
        t[where] = dev(x)
    q = dev(np.random.default_rng(12).standard_normal((n, hkv * 2, d)).astype(np.float16))
    lens = [held * page - n + 1 + i for i in range(n)]
    assert taken_together([0] * n, lens, hkv * 2, hkv, d)
    ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(hkv * 2, hkv, d), dtype=torch.uint8, device="cuda")
    outs = []
    for pool, tab in ((big, where), ([dev(x) for x in small], list(range(held)))):
        out = torch.empty_like(q)
        qsa.qsa_paged_attn(q, *pool, i32(tab).view(1, held), i32(lens), out, ws, rows=i32([0] * n))
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("scale", [0.0, -0.05, 1.0, 1e-30])
def test_attn_scales_and_peaks(cuda_device, scale):
    """Uniform weights, reversed ones, and ones so peaked that nearly every
    weight underflows."""
    rng = np.random.default_rng(5)
    table, pages = shuffled_table([800, 5], 32, 1, rng)
    pool = make_pool(pages, 32, 1, 128, seed=15)
    check_attn(rng.standard_normal((2, 12, 128)), pool, table, [800, 5], scale=scale, otype=F16)


@pytest.mark.parametrize("lo,hi", [(1e-6, 2e-6), (1e-5, 1e-2), (1.0, 30.0), (1e-4, 100.0)])
def test_attn_v_scales(cuda_device, lo, hi):
    """V scales from the smallest to large ones, mixed in one row."""
    rng = np.random.default_rng(6)
    table, pages = shuffled_table([1500], 64, 1, rng)
    pool = make_pool(pages, 64, 1, 128, seed=16)
    sc = np.exp(wl.uniform(9, 1, pool[3].shape, math.log(lo), math.log(hi)))
    pool[3] = sc.astype(np.float16)
    check_attn(rng.standard_normal((1, 12, 128)), pool, table, [1500], what=(lo, hi))


def test_attn_query_magnitudes(cuda_device):
    """bf16 queries beyond the fp16 range in both directions, and zeros."""
    rng = np.random.default_rng(7)
    table, pages = shuffled_table([300] * 5, 64, 1, rng)
    pool = make_pool(pages, 64, 1, 128, seed=17)
    q = rng.standard_normal((5, 12, 128)) * np.array([1e-30, 1e6, 1e-8, 0.0, 1.0])[:, None, None]
    check_attn(q, pool, table, [300] * 5, otype=BF16, scale=1e-6)


def test_attn_zero_scales(cuda_device):
    """Cells whose scales are 0 score 0 and add nothing to the values."""
    rng = np.random.default_rng(8)
    table, pages = shuffled_table([200, 64], 16, 1, rng)
    pool = make_pool(pages, 16, 1, 128, seed=18)
    pool[2][::2] = 0
    pool[3][table[1, :4]] = 0
    out, _ = check_attn(rng.standard_normal((2, 12, 128)), pool, table, [200, 64])
    assert not out[1].any()


def test_attn_bad_tables_and_lengths(cuda_device):
    """Entries outside the pool leave their cells out, lengths are cut, rows
    outside the table are empty; all of it is reported."""
    rng = np.random.default_rng(9)
    table, pages = shuffled_table([320] * 3, 32, 1, rng)
    pool = make_pool(pages, 32, 1, 128, seed=19)
    q = rng.standard_normal((3, 12, 128))
    table[0, 3], table[1, 0], table[1, 9] = -1, pages, 1 << 30
    _, err = check_attn(q, pool, table, [320, 320, 320])
    assert err == qsa.QSA_DEVERR_BAD_ID
    table[2, :] = -5
    out, err = check_attn(q, pool, table, [31, 5000, 100])
    assert err == qsa.QSA_DEVERR_BAD_ID and not out[2].any()
    out, err = check_attn(q, pool, table, [31, -1, 64], rows=[0, 1, 3])
    assert err == qsa.QSA_DEVERR_BAD_ID and not out[1:].any()
    # An entry past a row's length is not looked at.
    table[0, 1:] = 1 << 30
    _, err = check_attn(q[:1], pool, table, [32], rows=[0])
    assert err == 0


def test_attn_pool_beyond_32_bit_offsets(cuda_device):
    """Pages whose rows start past 2^32 bytes of codes."""
    page, d, hkv = 64, 256, 8
    pages = (1 << 32) // (page * hkv * d) + 8
    kq = torch.zeros(pages, page, hkv, d, dtype=torch.int8, device="cuda")
    vq = torch.zeros_like(kq)
    ksc = torch.zeros(pages, page, hkv, 4, dtype=F16, device="cuda")
    vsc = torch.zeros_like(ksc)
    small = make_pool(3, page, hkv, d, seed=20)
    where = [pages - 1, 2, pages - 5]
    for t, x in zip((kq, vq, ksc, vsc), small):
        t[where] = dev(x)
    rng = np.random.default_rng(10)
    q = rng.standard_normal((2, hkv * 2, d))
    ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(hkv * 2, hkv, d), dtype=torch.uint8, device="cuda")
    outs = []
    for pool, tab in (((kq, vq, ksc, vsc), [where, where[::-1]]), ([dev(x) for x in small], [[0, 1, 2], [2, 1, 0]])):
        out = torch.empty(2, hkv * 2, d, dtype=F16, device="cuda")
        qsa.qsa_paged_attn(dev(q.astype(np.float16)), *pool, i32(tab).view(2, 3), i32(150, 192), out, ws)
        outs.append(out)
    assert torch.equal(*outs)
    ko, vo = (torch.empty(4, hkv, d, device="cuda") for _ in range(2))
    ko2, vo2 = torch.empty_like(ko), torch.empty_like(vo)
    qsa.qsa_paged_gather(kq, vq, ksc, vsc, i32([(pages - 1) * page + i for i in range(4)]), ko, vo)
    qsa.qsa_paged_gather(*[dev(x) for x in small], i32(0, 1, 2, 3), ko2, vo2)
    assert torch.equal(ko, ko2) and torch.equal(vo, vo2)


def test_attn_repeats_bit_for_bit(cuda_device):
    rng = np.random.default_rng(11)
    lens = [9000, 17, 2500, 1]
    table, pages = shuffled_table(lens, 64, 1, rng)
    pool = [dev(x) for x in make_pool(pages, 64, 2, 128, seed=21)]
    q = dev(rng.standard_normal((4, 8, 128)).astype(np.float16))
    ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(8, 2, 128), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(5):
        out = torch.empty_like(q)
        ws.random_()
        qsa.qsa_paged_attn(q, *pool, dev(table), i32(lens), out, ws)
        outs.append(out)
    assert all(torch.equal(outs[0], o) for o in outs)


# ---------------------------------------------------------------- page update

def run_update(table, lens, src, new, pages, page, n_slots, layers=1, hkv=1, d=128, in_place=False, seed=30):
    pool = make_pool(pages, page, hkv, d, seed=seed, layers=layers)
    pd = [dev(x) for x in pool]
    rows, wide = len(new), table.shape[1]
    td, ld = dev(table), i32(lens)
    tout, lout = (td, ld) if in_place else (torch.full((rows, wide), 99, dtype=torch.int32, device="cuda"),
                                            torch.full((rows,), 99, dtype=torch.int32, device="cuda"))
    refs = torch.full((pages,), 99, dtype=torch.int32, device="cuda")
    slots, pos = (torch.full((n_slots,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.full((qsa.qsa_pages_workspace_bytes(rows, pages),), 0x5A, dtype=torch.uint8, device="cuda")
    err = err_word()
    qsa.qsa_page_update(td, ld, None if src is None else i32(src), i32(new), *pd, tout, lout, refs, slots, pos, ws, err=err)
    torch.cuda.synchronize()
    want = po.page_update(np.asarray(table), lens, src, new, pages, page, n_slots)
    for name, g, w in zip(("table", "lens", "refs", "slots", "positions"), (tout, lout, refs, slots, pos), want):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert int(err.item()) == want[6]
    for x, g in zip(pool, pd):
        for a, b, cells in want[5]:
            x[:, b, :cells] = x[:, a, :cells]
        assert np.array_equal(x.view(np.int8), g.cpu().numpy().view(np.int8))
    return want


@pytest.mark.parametrize("layers,hkv,page", [(1, 1, 16), (3, 2, 64), (2, 1, 256)])
def test_update_decode_step(cuda_device, layers, hkv, page):
    """Every row grows by one: in its page, into a new page, from nothing."""
    rng = np.random.default_rng(12)
    lens = [0, 1, page - 1, page, page + 1, 2 * page, 5 * page - 1]
    table, pages = shuffled_table(lens, page, 5, rng, wide=7)
    for in_place in (False, True):
        w = run_update(table, lens, None, [1] * len(lens), pages, page, len(lens), layers, hkv, in_place=in_place)
        assert w[6] == 0 and not w[5]


def test_update_forks_copy_shared_last_pages(cuda_device):
    rng = np.random.default_rng(13)
    page = 32
    lens = [70, 64, 5]
    table, pages = shuffled_table(lens, page, 12, rng, wide=5)
    # Forks of a partly filled and of a full last page, one that does not grow, a freed row, a new prompt.
    w = run_update(table, lens, [0, 0, 1, 1, 0, -1, 0], [1, 3, 1, 0, 0, 50, 40], pages, page, 200, layers=2, hkv=3)
    assert len(w[5]) == 3 and w[6] == 0


@pytest.mark.parametrize("hkv,cells", [(1, 1), (1, 15), (3, 7)])
def test_update_odd_tails(cuda_device, hkv, cells):
    """A copied part whose scales end in half a 16-byte word."""
    rng = np.random.default_rng(14)
    table, pages = shuffled_table([cells], 16, 4, rng, wide=2)
    w = run_update(table, [cells], [0, 0], [1, 1], pages, 16, 2, layers=2, hkv=hkv)
    assert len(w[5]) == 2


def test_update_runs_out(cuda_device):
    """Pages, table columns and slots run out: a row grows whole or not at all."""
    rng = np.random.default_rng(15)
    table, pages = shuffled_table([16, 16, 10, 16], 16, 2, rng, wide=3)
    lens = [16, 16, 10, 16]
    assert run_update(table, lens, None, [1, 40, 1, 1], pages, 16, 43)[6] == po.NO_PAGES      # row 1 too wide
    assert run_update(table, lens, None, [1, 17, 1, 1], pages, 16, 20)[6] == po.NO_PAGES      # row 1 finds one page
    assert run_update(table, lens, None, [1, 1, 2, 0], pages, 16, 3)[6] == po.NO_PAGES        # slots end inside row 2
    assert run_update(table, lens, [0, 1, 2, 2, 2], [16, 16, 0, 1, 1], pages, 16, 99)[6] == po.NO_PAGES  # no page to copy to
    assert run_update(table, lens, None, [0, 0, 0, 0], pages, 16, 0)[6] == 0


def test_update_bad_inputs(cuda_device):
    rng = np.random.default_rng(16)
    table, pages = shuffled_table([40, 40, 40], 16, 6, rng, wide=4)
    table[0, 1], table[1, 2] = 1 << 20, -3
    for lens, src, new in (([40, 20, 40], [0, 2], [1, 1]), ([40, 40, 40], [1, 2], [5, 1]), ([-4, 900, 40], [0, 1, 2], [1, 1, 1]),
                           ([16, 16, 40], [7, -2, 2], [1, 1, 1]), ([16, 16, 40], [0, 1, 2], [-1, 1, -9])):
        w = run_update(table, lens, src, new, pages, 16, 8)
        assert w[6] & po.BAD_ID


def test_update_large(cuda_device):
    """More columns than a warp takes at once, more pages and rows than one
    round of the cluster, a prompt of thousands of tokens."""
    rng = np.random.default_rng(17)
    page = 16
    lens = [int(v) for v in rng.integers(0, 40, 1500)] + [16 * 700 + 3, 16 * 520]
    table, pages = shuffled_table(lens, page, 9000, rng, wide=1100)
    src = list(rng.integers(-1, len(lens), 2100)) + [1500, 1500, 1501]
    new = list(rng.integers(0, 20, 2100)) + [4000, 1, 0]
    run_update(table, lens, src, new, pages, page, int(sum(new)) + 5)


@pytest.mark.parametrize("seed", range(8))
def test_update_random(cuda_device, seed):
    rng = np.random.default_rng(100 + seed)
    page = int(rng.choice([16, 32, 64]))
    n = int(rng.integers(1, 30))
    lens = [int(v) for v in rng.integers(0, 5 * page, n)]
    table, pages = shuffled_table(lens, page, int(rng.integers(0, 25)), rng, wide=6)
    rows = int(rng.integers(1, 50))
    new = [int(v) for v in rng.integers(0, 2 * page, rows)] if seed % 2 else [1] * rows
    src = [int(v) for v in rng.integers(-1, n, rows)]
    run_update(table, lens, src, new, pages, page, max(0, sum(new) - (seed == 3)), layers=2, hkv=2)


# ---------------------------------------------------------------- compaction

def run_compact(table, lens, pages, page, layers=1, hkv=1, d=128, in_place=False):
    pool = make_pool(pages, page, hkv, d, seed=31, layers=layers)
    pd = [dev(x) for x in pool]
    td = dev(table)
    tout = td if in_place else torch.full_like(td, 99)
    refs, pmap = (torch.full((pages,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    live, err = torch.full((1,), 99, dtype=torch.int32, device="cuda"), err_word()
    ws = torch.full((qsa.qsa_pages_workspace_bytes(len(lens), pages),), 0x5A, dtype=torch.uint8, device="cuda")
    qsa.qsa_page_compact(td, i32(lens), *pd, tout, refs, pmap, live, ws, err=err)
    torch.cuda.synchronize()
    wt, wr, wm, wl_, moves, werr = po.page_compact(np.asarray(table), lens, pages, page)
    assert np.array_equal(tout.cpu().numpy(), wt) and np.array_equal(refs.cpu().numpy(), wr)
    assert np.array_equal(pmap.cpu().numpy(), wm) and int(live.item()) == wl_ and int(err.item()) == werr
    for x, g in zip(pool, pd):
        for a, b in moves:
            x[:, b] = x[:, a]
        assert np.array_equal(x.view(np.int8), g.cpu().numpy().view(np.int8))
    return moves


@pytest.mark.parametrize("pages_extra,rows", [(0, 5), (1, 1), (40, 7), (9000, 300)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(cuda_device, pages_extra, rows, in_place):
    rng = np.random.default_rng(pages_extra + rows)
    lens = [int(v) for v in rng.integers(0, 200, rows)]
    lens[0] = 16
    table, pages = shuffled_table(lens, 16, pages_extra, rng)
    if rows > 4:  # a fork, and a row that holds only the first half of its pages
        table[1], lens[1] = table[0], lens[0]
        lens[2] //= 2
    run_compact(table, lens, pages, 16, layers=1 if pages > 5000 else 3, hkv=1 if pages > 5000 else 2, in_place=in_place)


def test_compact_edges(cuda_device):
    t = lambda *v: np.array(v, dtype=np.int32)  # noqa: E731
    assert run_compact(t([-1, -1]), [0], 5, 16) == []                    # nothing is held
    assert run_compact(t([0, 1, 2]), [48], 3, 16) == []                  # everything is
    assert run_compact(t([4, 2, 1]), [96], 5, 32, layers=2) == [(4, 0)]  # two of three stay
    assert run_compact(t([4, -1]), [10], 5, 64) == [(4, 0)]
    run_compact(t([9, 3, -7], [1, 900, 0]), [48, 40], 5, 16)             # entries outside the pool
    run_compact(t([3, 4], [1, 2]), [-3, 500], 5, 16)                     # lengths outside


# ---------------------------------------------------------------- together

class Serving:
    """A small decode loop over the paged calls and the selected attention."""

    def __init__(self, rows, hq=12, hkv=1, d=128, page=16, pages=64, wide=24, slots=256):
        z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
        self.page, self.hq, self.hkv, self.d = page, hq, hkv, d
        self.pool = [z(1, pages, page, hkv, d, t=torch.int8) for _ in range(2)] + [z(1, pages, page, hkv, 4, t=F16) for _ in range(2)]
        self.table, self.lens = torch.full((rows, wide), -1, dtype=torch.int32, device="cuda"), z(rows)
        self.refs, self.slots, self.pos = z(pages), z(slots), z(slots)
        self.ws = z(qsa.qsa_pages_workspace_bytes(rows, pages), t=torch.uint8)
        self.aws = z(qsa.qsa_paged_attn_workspace_bytes(hq, hkv, d), t=torch.uint8)
        self.err = err_word()
        self.freq = dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
        self.w = dev(wl.uniform(2, 1, (d,), 0.5, 1.5).astype(np.float32))

    def layer(self):
        return [x[0] for x in self.pool]

    def update(self, src, new):
        t, n = (torch.empty_like(self.table), torch.empty_like(self.lens)) if src is not None else (self.table, self.lens)
        qsa.qsa_page_update(self.table, self.lens, src, new, *self.pool, t, n, self.refs, self.slots, self.pos, self.ws, err=self.err)
        self.table, self.lens = t, n

    def write(self, x, q_out):
        q, k, v = x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]
        n = x.shape[0]
        qsa.qsa_paged_prep(q, k, v, self.pos[:n], self.slots[:n], *self.layer(), q_out, q_norm_w=self.w, k_norm_w=self.w,
                           inv_freq=self.freq, err=self.err)

    def attend(self, q, out):
        qsa.qsa_paged_attn(q, *self.layer(), self.table, self.lens, out, self.aws, err=self.err)

    def kv(self, r):
        n = int(self.lens[r])
        ko, vo = (torch.empty(n, self.hkv, self.d, device="cuda") for _ in range(2))
        ids = torch.arange(n, dtype=torch.int32, device="cuda")
        qsa.qsa_paged_gather(*self.layer(), ids, ko, vo, rows=torch.full_like(ids, r), page_table=self.table)
        return ko, vo


def dense(q, ko, vo):
    """Attention of q [H, D] over one sequence's values, in 64 bits."""
    q, k, v = host(q), host(ko), host(vo)
    per = q.shape[0] // k.shape[1]
    out = np.zeros_like(q)
    for h in range(q.shape[0]):
        s = k[:, h // per] @ q[h] / math.sqrt(q.shape[1])
        w = np.exp(s - s.max())
        out[h] = w @ v[:, h // per] / w.sum()
    return out


def test_serving_loop(cuda_device):
    """Prompts, decode steps, a fork, a reorder, a free and a compaction; each
    row's cache read back and its attention must be what the tokens it was
    given make, and the selected attention over all its cells agrees."""
    s = Serving(4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda n: torch.randn(n, 14, 128, generator=gen, device="cuda", dtype=F32).to(F16)  # noqa: E731
    history = [[], [], [], []]

    def step(src, new):
        nonlocal history
        history = [list(history[f]) if f >= 0 else [] for f in (src or range(4))]
        x = rand(sum(new))
        s.update(None if src is None else i32(src), i32(new))
        q = torch.zeros(len(x), 12, 128, dtype=F16, device="cuda")
        s.write(x, q)
        at = 0
        for r, n in enumerate(new):
            history[r] += [x[at + i] for i in range(n)]
            at += n
        assert [int(v) for v in s.lens] == [len(h) for h in history]
        return q

    step(None, [20, 1, 33, 16])
    for src, new in ((None, [1, 1, 1, 1]), ([0, 0, 2, 0], [1, 1, 1, 1]), ([3, 2, -1, 1], [1, 2, 5, 0]), ([0, 1, 2, 2], [1, 1, 1, 1]),
                     (None, [1, 1, 1, 1])):
        step(src, new)
    q = step(None, [1, 1, 1, 1])
    for compacted in (False, True):
        if compacted:
            pmap, live, t = torch.empty_like(s.refs), err_word(), torch.empty_like(s.table)
            qsa.qsa_page_compact(s.table, s.lens, *s.pool, t, s.refs, pmap, live, s.ws, err=s.err)
            s.table = t
            assert int(t.max()) < int(live) == int((s.refs > 0).sum())
        out = torch.empty_like(q)
        s.attend(q, out)
        for r, h in enumerate(history):
            x = host(torch.stack(h))
            w = s.w.cpu().numpy()
            k64 = po.norm_rotate(x[:, 12:13], w, np.arange(len(h)), s.freq.cpu().numpy())
            ko, vo = s.kv(r)
            step_k = np.repeat(np.abs(k64).reshape(len(h), 1, 4, 32).max(-1) / 127, 32, -1)
            step_v = np.repeat(np.abs(x[:, 13:]).reshape(len(h), 1, 4, 32).max(-1) / 127, 32, -1)
            assert np.all(np.abs(host(ko) - k64) <= step_k * 0.51) and np.all(np.abs(host(vo) - x[:, 13:]) <= step_v * 0.51)
            ref = dense(q[r], ko, vo)
            assert np.all(np.abs(host(out[r]) - ref) <= 2e-3 + 1e-2 * np.abs(ref))
            # qsa_attn over the same cells, by their pool numbers.
            n, wide = len(h), -(-len(h) // 64) * 64
            c = torch.arange(n, device="cuda")
            ids = torch.full((1, wide), -1, dtype=torch.int32, device="cuda")
            ids[0, :n] = s.table[r, c // s.page] * s.page + (c % s.page).int()
            kq, vq, ksc, vsc = (z.flatten(0, 2) for z in s.layer())
            o2 = torch.empty(1, 12, 128, dtype=F16, device="cuda")
            qsa.qsa_attn(q[r:r + 1].contiguous(), kq, vq, ksc, vsc, ids, o2)
            assert np.all(np.abs(host(o2[0]) - ref) <= 2e-3 + 1e-2 * np.abs(ref))
    assert int(s.err.item()) == 0


def test_decode_step_in_a_graph(cuda_device):
    """Update in place, prep and attention captured once and replayed: the same
    tables and outputs as the calls made one by one on another stream."""
    x = torch.randn(40, 3, 14, 128, device="cuda").to(BF16)
    runs = []
    for graphed in (False, True):
        s = Serving(3)
        new, xin = i32(1, 1, 1), torch.zeros(3, 14, 128, dtype=BF16, device="cuda")
        q, out = (torch.zeros(3, 12, 128, dtype=BF16, device="cuda") for _ in range(2))

        def one():
            s.update(None, new)
            s.write(xin, q)
            s.attend(q, out)

        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        outs = []
        with torch.cuda.stream(stream):
            if graphed:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=stream):
                    one()
            for i in range(40):
                xin.copy_(x[i])
                g.replay() if graphed else one()
                outs.append(out.clone())
        torch.cuda.synchronize()
        assert int(s.err.item()) == 0 and s.lens.tolist() == [40, 40, 40]
        runs.append((s.table, torch.stack(outs), s.pool))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    assert all(torch.equal(a, b) for a, b in zip(runs[0][2], runs[1][2]))


def test_binding_streams(cuda_device):
    """A given stream is used; a call on it follows what was queued there."""
    pd = [dev(x) for x in make_pool(2, 16, 1, 128)]
    side = torch.cuda.Stream()
    ids = i32(3, 4)
    a, b = (torch.zeros(2, 1, 128, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        ids.fill_(7)
    qsa.qsa_paged_gather(*pd, ids, a, b, stream=side)
    side.synchronize()
    assert torch.equal(a[0], a[1]) and a.any()


def test_binding_refuses(cuda_device):
    """What only the binding can see: devices, dtypes, shapes, contiguity."""
    z = lambda *v, t=torch.int32: torch.zeros(v, dtype=t, device="cuda")  # noqa: E731
    kq, ksc = z(2, 4, 16, 1, 128, t=torch.int8), z(2, 4, 16, 1, 4, t=F16)
    lay = (kq[0], kq[1], ksc[0], ksc[1])
    q, tab, lens, ws = z(2, 12, 128, t=F16), z(2, 2), z(2), z(1 << 24, t=torch.uint8)

    def refused(match, fn, *args, **kw):
        with pytest.raises((ValueError, qsa.QSAError), match=match):
            fn(*args, **kw)

    attn = qsa.qsa_paged_attn
    refused("CUDA tensor", attn, q, *lay, tab, lens, q.cpu(), ws)
    refused("CUDA tensor", attn, q, *lay, tab, lens.cpu(), q, ws)
    refused("vq must be", attn, q, lay[0], lay[1][:2], *lay[2:], tab, lens, q, ws)
    refused("ksc must be", attn, q, *lay[:2], lay[2][..., :2], lay[3], tab, lens, q, ws)
    refused("kq must be", attn, q, *[x.flatten(0, 1) for x in lay], tab, lens, q, ws)
    refused("seq_lens must be", attn, q, *lay, tab, lens[:1], q, ws)
    refused("seq_lens must be", attn, q, *lay, tab, lens.long(), q, ws)
    refused("rows must be", attn, q, *lay, tab, lens, q, ws, rows=z(3))
    refused("float16 or bfloat16", attn, q.float(), *lay, tab, lens, q.float(), ws)
    refused("out must be", attn, q, *lay, tab, lens, q.to(BF16), ws)
    refused("contiguous", attn, q.transpose(0, 1).contiguous().transpose(0, 1), *lay, tab, lens, q, ws)
    refused("gate must be", attn, q, *lay, tab, lens, q, ws, gate=q)
    refused("page_table must be", attn, q, *lay, tab[0], lens, q, ws)
    refused("workspace", attn, q, *lay, tab, lens, q, ws.cpu())
    refused("workspace smaller", attn, q, *lay, tab, lens, q, ws[:256])
    refused("row per token", attn, q, *lay, tab[:1], lens, q, ws)
    refused("err must be", attn, q, *lay, tab, lens, q, ws, err=torch.zeros(1, dtype=torch.int32))
    prep = qsa.qsa_paged_prep
    x = z(2, 14, 128, t=F16)
    a = (x[:, :12], x[:, 12:13], x[:, 13:])
    refused("k_in must be", prep, a[0], a[1].float(), a[2], lens, lens, *lay, q)
    refused("k_in must be", prep, a[0], x[:, 11:13], a[2], lens, lens, *lay, q)
    refused("contiguous", prep, x[:, ::2][:, :6], a[1], a[2], lens, lens, *lay, q[:, :6].contiguous())
    refused("slots must be", prep, *a, lens, lens[:1], *lay, q)
    refused("q_norm_w must be", prep, *a, lens, lens, *lay, q, q_norm_w=z(64, t=F32))
    refused("inv_freq", prep, *a, lens, lens, *lay, q, inv_freq=z(2, 2, t=F32))
    refused("rope_dims", prep, *a, lens, lens, *lay, q, inv_freq=z(3, t=F32))
    refused("q_out", prep, *a, lens, lens, *lay, q.float())
    refused("strides", prep, x[:1, :12].expand(2, 12, 128), a[1], a[2], lens, lens, *lay, q)
    out = z(2, 1, 128, t=F32)
    refused("go together", qsa.qsa_paged_gather, *lay, lens, out, out, rows=lens)
    refused("v_out must be", qsa.qsa_paged_gather, *lay, lens, out, out.half())
    refused("k_out must be", qsa.qsa_paged_gather, *lay, lens, z(2, 2, 128, t=F32), out)
    pool = (kq, kq.clone(), ksc, ksc.clone())
    upd = lambda **kw: {**dict(page_table=tab, seq_lens=lens, src=None, n_new=lens, page_table_out=z(2, 2), seq_lens_out=z(2),  # noqa: E731
                               refs=z(4), slots=lens, positions=z(2), workspace=ws), **kw}
    call = lambda kq=None, **kw: qsa.qsa_page_update(kq=pool[0], vq=pool[1], ksc=pool[2], vsc=pool[3], **upd(**kw))  # noqa: E731
    refused("page_table_out must be", call, page_table_out=z(2, 3))
    refused("refs must be", call, refs=z(5))
    refused("positions must be", call, positions=z(3))
    refused("src must be", call, src=z(3))
    refused("may be the old ones only without src", call, src=lens, page_table_out=tab)
    refused("may be the old ones only without src", call, src=lens, seq_lens_out=lens)
    refused("page_map must be", qsa.qsa_page_compact, tab, lens, *pool, z(2, 2), z(4), z(3), z(1), ws)
    refused("n_live must be", qsa.qsa_page_compact, tab, lens, *pool, z(2, 2), z(4), z(4), z(2), ws)


def test_binding_paths_agree(cuda_device, monkeypatch):
    """A call that is as it should be goes through the compiled binding alone,
    and does what the checked one does, to the bit."""
    from sparse_selected_attention_gb300 import paged
    rng = np.random.default_rng(36)
    T, hq, hkv, d, page, pages = 5, 6, 2, 128, 16, 12
    z = lambda *v, t=torch.int32: torch.zeros(v, dtype=t, device="cuda")  # noqa: E731
    q, k, v = (dev(rng.standard_normal((T, h, d)).astype(np.float16)) for h in (hq, hkv, hkv))
    w, freq = dev(rng.random(d).astype(np.float32)), dev(rng.random(d // 4).astype(np.float32))
    gate = dev(rng.standard_normal((T, hq, d)).astype(np.float32))
    first = [dev(x) for x in make_pool(pages, page, hkv, d, seed=37)]
    table, lens = i32(3, 5, -1, 7, 1, 2).view(2, 3), i32(20, 40)
    side = torch.cuda.Stream()

    def everything(stream):
        lay = [x.clone() for x in first]
        qo, ko, vo, out, lse = torch.empty_like(q), *(torch.empty(T, hkv, d, device="cuda") for _ in range(2)), torch.empty_like(q), z(T, hq, t=F32)
        to, lo, refs, sl, po_, tc, mp, nl, err = z(2, 3), z(2), z(pages), z(T), z(T), z(2, 3), z(pages), z(1), z(1)
        wa, wp = (z(n, t=torch.uint8) for n in (qsa.qsa_paged_attn_workspace_bytes(hq, hkv, d), qsa.qsa_pages_workspace_bytes(2, pages)))
        torch.cuda.synchronize()
        kw = dict(err=err, stream=stream)
        qsa.qsa_page_update(table, lens, i32(0, 1), i32(3, 2), *lay, to, lo, refs, sl, po_, wp, **kw)
        qsa.qsa_paged_prep(q, k, v, po_, sl, *lay, qo, q_norm_w=w, k_norm_w=w, inv_freq=freq, interleaved=True, eps=1e-5, rope_mscale=0.5, **kw)
        qsa.qsa_paged_gather(*lay, i32(0, 19, 39, -1, 2), ko, vo, rows=i32(0, 0, 1, 1, 1), page_table=to, **kw)
        qsa.qsa_paged_attn(qo, *lay, to, i32(21, 22, 23, 41, 42), out, wa, rows=i32(0, 0, 0, 1, 1), softmax_scale=0.1, gate=gate, lse=lse, **kw)
        qsa.qsa_page_compact(to, lo, *lay, tc, refs, mp, nl, wp, **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return lay + [qo, ko, vo, out, lse, to, lo, refs, sl, po_, tc, mp, nl]

    checked = {n: getattr(paged, "_checked_" + n) for n in ("prep", "gather", "attn", "update", "compact")}
    with monkeypatch.context() as m:
        for n in checked:
            m.setattr(paged, "_checked_" + n, None)
        a = [everything(s) for s in (None, side)]

    class Never:
        def __getattr__(self, name):
            return lambda *args: -1
    with monkeypatch.context() as m:
        m.setattr(paged, "_native", Never())
        a += [everything(s) for s in (None, side)]
    for other in a[1:]:
        for i, (x, y) in enumerate(zip(a[0], other)):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), i


def test_binding_says_what_the_library_says(cuda_device):
    """A refusal by the library, through the compiled binding."""
    pd = [dev(x) for x in make_pool(2, 16, 1, 128)]
    ko, vo = (torch.empty(1, 1, 128, device="cuda") for _ in range(2))
    shifted = torch.empty(129, device="cuda")[1:].view(1, 1, 128)
    with pytest.raises(qsa.QSAError, match="qsa_paged_gather: misaligned"):
        qsa.qsa_paged_gather(*pd, i32(0), shifted, vo)
    with pytest.raises((ValueError, TypeError, AttributeError)):
        qsa.qsa_paged_gather(*pd, [0], ko, vo)
    with pytest.raises((ValueError, TypeError)):
        qsa.qsa_paged_gather(*pd, i32(0).expand(2)[:1].to_sparse(), ko, vo)


def test_two_calls_at_once(cuda_device):
    """Calls on two streams, each with its own workspace and outputs, beside
    one another: rows taken together, rows one by one, and a page table's
    update, give the bits that they give alone."""
    rng = np.random.default_rng(38)
    jobs = []
    for d, n, held in ((256, 64, 900), (128, 100, 900), (128, 0, 5000)):
        table, pages = shuffled_table([held] * (1 if n else 6), 32, 4, rng)
        pool = [dev(x) for x in make_pool(pages, 32, 8, d, seed=39)]
        rows = [0] * n if n else list(range(6))
        lens = [held - n + 1 + i for i in range(n)] if n else [held - 700 * i for i in range(6)]
        assert taken_together(rows, lens, 16, 8, d) == bool(n)
        q = dev(rng.standard_normal((len(rows), 16, d)).astype(np.float16))
        jobs.append((q, pool, dev(table), i32(lens), i32(rows), d))

    def state():
        out = []
        for q, pool, table, lens, rows, d in jobs:
            ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(16, 8, d), dtype=torch.uint8, device="cuda")
            r = table.shape[0]
            up = [torch.zeros_like(table), i32([0] * r), torch.zeros(pool[0].shape[0], dtype=torch.int32, device="cuda"), i32([0] * r), i32([0] * r),
                  torch.empty(qsa.qsa_pages_workspace_bytes(r, pool[0].shape[0]), dtype=torch.uint8, device="cuda")]
            out.append((torch.empty_like(q), ws, up))
        return out

    def run(state, stream):
        for (q, pool, table, lens, rows, d), (out, ws, up) in zip(jobs, state):
            r = table.shape[0]
            qsa.qsa_paged_attn(q, *pool, table, lens, out, ws, rows=rows, stream=stream)
            qsa.qsa_page_update(table, i32([table.shape[1] * 32 - 32] * r), None, i32([1] * r), *pool, *up, stream=stream)

    alone = state()
    torch.cuda.synchronize()
    run(alone, None)
    torch.cuda.synchronize()
    streams, both = [torch.cuda.Stream() for _ in range(2)], [state() for _ in range(2)]
    for _ in range(5):
        torch.cuda.synchronize()
        for s, st in zip(streams, both):
            with torch.cuda.stream(s):
                run(st, s)
        torch.cuda.synchronize()
        for st in both:
            for (out, _, up), (want, _, wup) in zip(st, alone):
                assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(up[:5], wup[:5]))
