"""V scales of all sizes in one row of qsa_paged_attn, in every form that it
takes rows in: what a cell adds is kept to the digits of the largest weight *
V scale, however large a scale is that has no weight, and however many cells
have a scale of 0.

Tolerance: that of tests/test_paged_groups_gpu.py, for the form with the
coarsest steps: scores over codes shifted by 1152, each off by 2^-21 of
1152 qk; a weight and its product with a scale off by 2^-11 each; 2^-24 of
|code| * the largest weight * scale for what underflows.
"""
import math

import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from tests.test_paged_gpu import BF16, F16, HALF, TINY, dev, i32
from tests.test_paged_groups_gpu import reference
from tests.test_paged_nan_gpu import FORMS, batch

pytestmark = pytest.mark.gpu


def scales(kind, shape, d):
    g = torch.Generator(device="cuda").manual_seed(80)
    u = torch.rand(*shape, 1, generator=g, device="cuda")
    within = 1 + torch.rand(*shape, 4, generator=g, device="cuda")  # a cell's four, within a factor of two
    between = lambda lo, hi: torch.exp(u * math.log(hi / lo)) * lo  # noqa: E731
    rare = torch.rand(*shape, 1, generator=g, device="cuda") < 0.03
    if kind == "large ones without weight":
        return torch.where(rare, 100 * within, between(1e-5, 2e-5) * within), rare
    if kind == "small ones after large ones":
        # The pages' order in a row is mixed, so these meet in both orders.
        return torch.where(torch.rand(shape[0], 1, 1, 1, generator=g, device="cuda") < 0.5, between(20, 50), between(1e-5, 2e-5)) * within, None
    if kind == "cell by cell":
        return between(1e-6, 100) * within, None
    if kind == "zero ones":
        return torch.where(torch.rand(*shape, 1, generator=g, device="cuda") < 0.3, 0.0, between(1e-6, 1e-5)) * within, None
    assert kind == "largest"
    return between(2e4, 3.2e4) * within.clamp(max=2.0), None


@pytest.mark.parametrize("otype", [F16, BF16])
@pytest.mark.parametrize("kind", ["large ones without weight", "small ones after large ones", "cell by cell", "zero ones", "largest"])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("form", FORMS)
def test_v_scales(cuda_device, form, d, kind, otype):
    q, pool, table, lens, rows = batch(form, d)
    pool = [dev(x) for x in pool]
    vs, light = scales(kind, pool[3].shape[:3], d)
    pool[3] = vs.half()
    if kind == "largest":
        pool[1] = pool[1] // (2 if otype is BF16 else 127)  # results within their type
    pool[2][:] = 2.0 ** -7
    q = dev(q) * 0.5
    q[..., 0] = 32.0  # scores 15 nats up for all cells but the light ones, 47 below those
    pool[0][..., 0] = 60 if light is None else torch.where(light[..., 0], -127, 60).to(torch.int8)
    q = q.to(otype)
    T, H, D = q.shape
    out, lse = torch.empty_like(q), torch.empty(T, H, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(qsa.qsa_paged_attn_workspace_bytes(H, pool[0].shape[2], D), dtype=torch.uint8, device="cuda")
    qsa.qsa_paged_attn(q, *pool, dev(table), i32(lens), out, ws, rows=None if rows is None else i32(rows), softmax_scale=1.0, lse=lse, err=err)
    ref, rlse, mag, flush, qk = reference(q, pool, table, lens, rows or list(range(T)), 1.0)
    ds = 1152 * qk * 2.0 ** -21
    tol = HALF[otype] * ref.abs() + mag * (2.0 ** -10 + 2 * torch.expm1(ds)[..., None] + 2.0 ** -16) + flush * 2.0 ** -24 + TINY[otype]
    bad = ~((out.double() - ref).abs() <= tol)
    assert int(err.item()) == 0
    assert not bad.any(), (int(bad.sum()), bad.numel(), bad.nonzero()[:3].tolist(), out[bad][:3], ref[bad][:3], tol[bad][:3])
    some = torch.isfinite(rlse)
    assert torch.equal(torch.isneginf(lse), ~some)
    assert ((lse.double() - rlse).abs() <= ds + 2.0 ** -16 + 2.0 ** -22 * rlse.abs())[some].all()
