"""The bounds of tests/test_paged_accuracy_gpu.py against the roundings that
they are there to notice, planted in the definition, on the CPU."""
import numpy as np
import pytest
import torch

from tests import test_paged_accuracy_gpu as acc
from tests import test_paged_groups_gpu as groups


def weights(q, pool, table, lens, t, h):
    """Weights (largest 1), codes and V scales of one head of row t of table row t or 0."""
    page, hkv, d = pool[0].shape[1], pool[0].shape[2], q.shape[2]
    c = np.arange(lens[t])
    at = torch.from_numpy(table[min(t, len(table) - 1), c // page].astype(np.int64) * page + c % page)
    k = h // (q.shape[1] // hkv)
    kq, vq, ksc, vsc = (x.flatten(0, 1)[at, k].double() for x in pool)
    s = (kq * ksc.repeat_interleave(d // 4, -1)) @ q[t, h].double() / d ** 0.5
    return torch.exp(s - s.max()), vq, vsc.repeat_interleave(d // 4, -1)


def half(x):
    return x.half().double()


def two(x):
    return half(x) + half(x - half(x))


@pytest.mark.parametrize("d,hq,hkv", [(128, 12, 2), (256, 6, 2)])
def test_one_part_of_a_weight_times_scale_is_noticed(d, hq, hkv):
    q, pool, table, lens = acc.short_case(d, hq, hkv, 6, "cpu")
    ref = groups.reference(q, pool, table, lens, list(range(6)))
    tol = acc.short_bound(*ref, acc.vtop_of(pool))
    seen = 0
    for t in range(6):
        for h in range(hq):
            w, code, vs = weights(q, pool, table, lens, t, h)
            unit = 2.0 ** torch.floor(torch.log2(vs.max()))
            for part, notice in ((two, False), (half, True)):
                out = (part(w[:, None] * vs / unit) * unit * code).sum(0) / w.sum()
                over = ((half(out) - ref[0][t, h]).abs() > tol[t, h]).any()
                seen += bool(over) and notice
                assert notice or not over
    assert seen > 3 * hq  # of the six rows' heads


@pytest.mark.parametrize("d,hq,hkv,n,cells", [(128, 16, 8, 64, 700), (256, 8, 4, 32, 1500)])
def test_one_part_of_a_weight_is_noticed(d, hq, hkv, n, cells):
    q, pool, table, lens, rows = acc.group_case(d, hq, hkv, n, cells, "cpu")
    few = [0, n // 2, n - 1]
    q, lens, rows = q[few], [lens[t] for t in few], [0] * 3
    ref = groups.reference(q, pool, table, lens, rows)
    tol, _ = groups.bounds(*ref, torch.float16, d, v_exact=True)
    seen = 0
    for t in range(3):
        for h in range(hq):
            w, code, vs = weights(q, pool, table, lens, t, h)
            # In units of a power of two near the largest weight * V scale, as the running maximum is.
            p = w[:, None] * vs / (w[:, None] * vs).max() * 1.37
            for part, notice in ((two, False), (half, True)):
                out = (part(p) * code).sum(0) * (w[:, None] * vs).max() / 1.37 / w.sum()
                over = ((half(out) - ref[0][t, h]).abs() > tol[t, h]).any()
                seen += bool(over) and notice
                assert notice or not over
    assert seen > 2 * hq


@pytest.mark.parametrize("d", [128, 256])
def test_a_sum_over_shifted_codes_is_noticed(d):
    """fp32 sums of q (1152 + code) from -1152 sum q, truncated at each step."""
    rng = np.random.default_rng(79)
    n, off = 500, 0
    for _ in range(n):
        q, code = rng.integers(0, 2048, d), rng.integers(-127, 128, d)
        s = 0.0
        for g in range(4):
            x, c = (v[g * d // 4:(g + 1) * d // 4].astype(np.float64) for v in (q, code))
            a = np.float32(-1152 * x.sum())
            for k in range(0, d // 4, 16):
                y = float(a) + (x[k:k + 16] * (1152 + c[k:k + 16])).sum()
                a = np.float32(y)
                if abs(float(a)) > abs(y):
                    a = np.nextafter(a, np.float32(0))
            s += float(a)
        want = float((q * code).sum())
        off += abs(s - want) > 2.0 ** -21 * abs(want) + 2.0 ** -21 * 2.0 ** 19
    assert off > n // 10
