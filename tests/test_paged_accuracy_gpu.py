"""What qsa_paged_attn keeps of its numbers, form by form, on inputs made so
that the roundings that a form does without would show.

  exact codes   (tables of up to 16 units, a unit being 32 cells of 128 dims or
                16 of 256) scores of whole-number queries whose sums stay below
                2^24 under K scales of a power of two have no rounding but the
                scale's: lse of one cell is off by at most 8 * 2^-24 of itself
                (scale, its product with log2 e, the score's with both, the
                subtraction, the logarithm's sum, the product with ln 2) and
                by 2^-21 (the exponential's 2^-22 of the weight, wherever the
                reference maximum lies, and the logarithm's 2^-24 of up to 1);
  two parts     (the same tables) weight * V scale keeps 22 bits: `out` is off
                by its own half step and 2^-20 of the sum of weight * |value|
                (2^-22 for the parts, 2^-22 each for exponential, division and
                what the sums of 8 K dims truncate), and what underflows;
  two parts     (rows taken together) K's code * scale is exact, so that a score
                of one product is exact; and of fp16 results the weights keep
                22 bits: with V scales of a power of two `out` is off as above.

tests/test_paged_bounds_cpu.py plants the roundings in the definition.
"""
import numpy as np
import pytest
import torch

from tests.test_paged_gpu import BF16, F16, HALF, TINY, dev, i32, make_pool, shuffled_table, taken_together
from tests.test_paged_groups_gpu import check, reference, run

pytestmark = pytest.mark.gpu


def short_rows(d, hkv, n, seed, most=None):
    """Rows that go whole, a warp or a block each by their number."""
    unit = 4096 // d
    rng = np.random.default_rng(seed)
    most = most or (2 if n * hkv > 304 else 16) * unit
    lens = [int(v) for v in rng.integers(1, most + 1, n)]
    lens[0], lens[-1] = most, 2
    table, pages = shuffled_table(lens, 16, 1, rng, wide=most // 16)
    return table, pages, lens


@pytest.mark.parametrize("n", [5, 200])
@pytest.mark.parametrize("d,hq,hkv", [(128, 12, 2), (256, 6, 2), (128, 16, 1)])
def test_short_tables_have_exact_scores(cuda_device, d, hq, hkv, n):
    table, pages, _ = short_rows(d, hkv, n, 70)
    lens = [1] * n
    pool = make_pool(pages, 16, hkv, d, seed=70)
    pool[2][:] = 2.0 ** -7
    rng = np.random.default_rng(71)
    q = rng.integers(0, 2048, (n, hq, d)).astype(np.float64)
    scale = 2.0 ** -12
    per, code = hq // hkv, pool[0][table[:, 0], 0].astype(np.float64)  # [n, hkv, d]
    prod = q * np.repeat(code, per, 1)
    assert np.abs(prod.reshape(n, hq, 4, -1)).sum(-1).max() < 2 ** 24 and np.abs(np.cumsum(prod, -1)).max() < 2 ** 24
    s = torch.from_numpy(prod.sum(-1) * 2.0 ** -19).cuda()
    out, lse, err = run(dev(q.astype(np.float16)), [dev(x) for x in pool], table, lens, list(range(n)), scale)
    assert err == 0
    assert ((lse.double() - s).abs() <= 2.0 ** -21 * s.abs() + 2.0 ** -21).all(), ((lse.double() - s).abs() / s.abs()).max()


def short_case(d, hq, hkv, n, device):
    table, pages, lens = short_rows(d, hkv, n, 72)
    pool = [torch.from_numpy(x).to(device) for x in make_pool(pages, 16, hkv, d, seed=73)]
    q = torch.from_numpy(np.random.default_rng(74).standard_normal((n, hq, d)) * 0.02).to(device).half()
    return q, pool, table, lens


def short_bound(ref, lse, mag, flush, qk, vtop):
    """Codes of at most 128 in place of 1152 + code: 2^-20 and 2^-22 of 128 qk
    for the sums and the scale; flush by the row's largest V scale."""
    ds = 128 * qk * 2.0 ** -19
    return HALF[F16] * ref.abs() + mag * (2.0 ** -20 + 2 * torch.expm1(ds)[..., None]) + vtop * flush * 2.0 ** -24 + TINY[F16]


def vtop_of(pool):
    """How far a row's largest V scale can be above the one with the largest weight."""
    return float(pool[3].max() / pool[3].min())


@pytest.mark.parametrize("n", [6, 200])
@pytest.mark.parametrize("d,hq,hkv", [(128, 12, 2), (256, 6, 2)])
def test_short_tables_have_weights_in_two_parts(cuda_device, d, hq, hkv, n):
    q, pool, table, lens = short_case(d, hq, hkv, n, "cuda")
    rows = list(range(n))
    out, lse, err = run(q, pool, table, lens, rows)
    ref = reference(q, pool, table, lens, rows)
    bad = ~((out.double() - ref[0]).abs() <= short_bound(*ref, vtop_of(pool)))
    assert err == 0 and not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist())


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("d,hq,hkv,n,cells", [(128, 16, 8, 64, 700), (256, 8, 4, 32, 1500)])
def test_rows_taken_together_have_exact_scores(cuda_device, d, hq, hkv, n, cells, otype):
    """Queries of one dim each; a cell of the largest code there carries all of
    the weight, so lse is its score."""
    rng = np.random.default_rng(75)
    table, pages = shuffled_table([cells], 32, 1, rng)
    pool = make_pool(pages, 32, hkv, d, seed=76)
    pool[2] = (2.0 ** -7 * (1 + rng.integers(0, 1024, pool[2].shape) / 1024)).astype(np.float16)
    pool[0] = (pool[0] // 8).astype(np.int8)
    rows, lens = [0] * n, [cells - n + 1 + i for i in range(n)]
    assert taken_together(rows, lens, hq, hkv, d)
    per = hq // hkv
    dims = rng.permutation(d)[:hq]
    where = rng.integers(0, cells - n, hq)
    q, s = np.zeros((n, hq, d)), np.zeros(hq)
    for h in range(hq):
        page, at, x = table[0, where[h] // 32], where[h] % 32, dims[h]
        pool[0][page, at, h // per, x] = 127 if h % 2 else -125
        q[:, h, x] = 64.0 if h % 2 else -64.0
        s[h] = (127 if h % 2 else 125) * float(pool[2][page, at, h // per, x // (d // 4)]) * 64.0
    qd = dev(q.astype(np.float32)).to(otype)
    out, lse, err = run(qd, [dev(x) for x in pool], table, lens, rows, 1.0)
    want = torch.from_numpy(s).cuda().expand(n, hq)
    ref = reference(qd, [dev(x) for x in pool], table, lens, rows, 1.0)[1]
    assert err == 0 and (ref - want).abs().max() < 1e-8  # the rest of the cells add nothing
    assert ((lse.double() - want).abs() <= 2.0 ** -21 * want).all(), ((lse.double() - want).abs() / want).max()


def group_case(d, hq, hkv, n, cells, device):
    rng = np.random.default_rng(77)
    table, pages = shuffled_table([cells], 32, 1, rng)
    pool = make_pool(pages, 32, hkv, d, seed=78)
    pool[3][:] = 2.0 ** rng.integers(-9, -6, (*pool[3].shape[:3], 1))
    q = torch.from_numpy(rng.standard_normal((n, hq, d)) * 0.005).to(device).half()
    rows, lens = [0] * n, [cells - n + 1 + i for i in range(n)]
    assert taken_together(rows, lens, hq, hkv, d)
    return q, [torch.from_numpy(x).to(device) for x in pool], table, lens, rows


@pytest.mark.parametrize("d,hq,hkv,n,cells", [(128, 16, 8, 64, 700), (256, 8, 4, 32, 1500)])
def test_rows_taken_together_have_weights_in_two_parts(cuda_device, d, hq, hkv, n, cells):
    check(*group_case(d, hq, hkv, n, cells, "cuda"), v_exact=True)
