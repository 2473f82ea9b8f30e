"""A batch without rows: its table has no rows, and calls that have nothing to
do say so before they look at it."""
import ctypes

import pytest

from sparse_selected_attention_gb300 import _abi, build
from tests.test_paged_cpu import ATTN, GATHER, INV, _make, _status


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


@pytest.mark.parametrize("kw", [dict(n_rows=0, page_table=None), dict(n_rows=0, rows=None, seq_lens=None, q=None, out=None)])
def test_attn_of_no_tokens(L, kw):
    assert _status(L, "qsa_paged_attn", _make(_abi.PagedAttnArgs, ATTN, dict(n_tokens=0, **kw))) == (_abi.QSA_OK, "")


def test_gather_of_no_cells(L):
    kw = dict(n_ids=0, n_rows=0, rows=None, ids=None, k_out=None, v_out=None)
    assert _status(L, "qsa_paged_gather", _make(_abi.PagedGatherArgs, GATHER, kw)) == (_abi.QSA_OK, "")


@pytest.mark.parametrize("n,rows", [(3, 0), (0, -1), (3, -1)])
def test_rows_below_what_is_read(L, n, rows):
    for fn, cls, base, kw in (("qsa_paged_attn", _abi.PagedAttnArgs, ATTN, dict(n_tokens=n)),
                              ("qsa_paged_gather", _abi.PagedGatherArgs, GATHER, dict(n_ids=n))):
        s, msg = _status(L, fn, _make(cls, base, dict(n_rows=rows, **kw)))
        assert s == INV and "n_rows" in msg, (fn, s, msg)
