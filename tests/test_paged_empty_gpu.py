"""A serving step of a batch that has become empty, and of one that begins."""
import pytest
import torch

import sparse_selected_attention_gb300 as qsa
from tests.test_paged_gpu import F16, dev, i32, make_pool

pytestmark = pytest.mark.gpu


def test_a_batch_without_rows(cuda_device):
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    pool = [dev(x) for x in make_pool(6, 16, 2, 128)]
    before = [x.clone() for x in pool]
    table, lens, none = i32(3, 1, 0, -1).view(2, 2), i32(20, 9), z(0, 2)
    refs, slots, pos, err = z(6) + 9, z(3) + 9, z(3) + 9, z(1)
    ws = z(qsa.qsa_pages_workspace_bytes(0, 6), t=torch.uint8)
    qsa.qsa_page_update(table, lens, z(0), z(0), *pool, none, z(0), refs, slots, pos, ws, err=err)
    assert not refs.any() and (slots == -1).all() and (pos == -1).all()
    q = z(0, 4, 128, t=F16)
    qsa.qsa_paged_prep(q, z(0, 2, 128, t=F16), z(0, 2, 128, t=F16), z(0), z(0), *pool, q, err=err)
    aws = z(qsa.qsa_paged_attn_workspace_bytes(4, 2, 128), t=torch.uint8)
    qsa.qsa_paged_attn(q, *pool, none, z(0), q.clone(), aws, err=err)
    qsa.qsa_paged_attn(q, *pool, none, z(0), q.clone(), aws, rows=z(0), lse=z(0, 4, t=torch.float32), err=err)
    out = z(0, 2, 128, t=F16)
    qsa.qsa_paged_gather(*pool, z(0), out, out.clone(), rows=z(0), page_table=none, err=err)
    pmap, live, refs = z(6) + 9, z(1) + 9, z(6) + 9
    qsa.qsa_page_compact(none, z(0), *pool, none.clone(), refs, pmap, live, ws, err=err)
    assert not refs.any() and (pmap == -1).all() and int(live) == 0 and int(err) == 0
    # From nothing: a first row of 20 tokens.
    t, n = z(1, 2), z(1)
    slots, pos = z(20), z(20)
    ws = z(qsa.qsa_pages_workspace_bytes(1, 6), t=torch.uint8)
    qsa.qsa_page_update(none, z(0), i32(-1), i32(20), *pool, t, n, refs, slots, pos, ws, err=err)
    assert t.tolist() == [[0, 1]] and n.tolist() == [20] and slots.tolist() == list(range(20)) and int(err) == 0
    assert all(torch.equal(a, b) for a, b in zip(pool, before))
