"""The largest sizes that the paged calls take, and what their Python side
refuses; nothing here touches a device."""
import ctypes as C

import pytest
import torch

import lightning_indexer_top_index_b200 as L
from test_paged_host import _attn, _pages, lib  # noqa: F401


def _status(lib, args):
    n = C.c_size_t(0)
    return lib.lidx_workspace_size(L.OP_PAGED_ATTN, C.byref(args), C.byref(n))


def _table_of(pages):
    return _pages(page_rows=16, n_pages=1 << 20, ld_table=pages, max_pages=pages)


@pytest.mark.parametrize("pages,status", [((1 << 27) - 4, L.OK), ((1 << 27) - 3, L.ERR_UNSUPPORTED),
                                          ((1 << 27) - 1, L.ERR_UNSUPPORTED)])
def test_rows_of_a_query(lib, pages, status):  # noqa: F811
    """The end of a job's last chunk of 64 entries stays below 2^31."""
    assert ((pages * 16 + 63) // 64 * 64 < 2 ** 31) == (status == L.OK)
    assert _status(lib, _attn(B=1, cache=_table_of(pages))) == status
    listed = _attn(B=1, cache=_table_of(10), blocks=0x9000, n_blocks=pages, ld_blocks=pages)
    assert _status(lib, listed) == status
    assert lib.lidx_paged_attn(C.byref(_attn(B=1, cache=_table_of(pages))), C.c_void_p(0x100000), 0, None) == (
        L.ERR_WORKSPACE if status == L.OK else status)
