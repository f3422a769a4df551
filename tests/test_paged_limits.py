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


@pytest.mark.parametrize("scale,status", [(1e38, L.OK), (-1e38, L.OK), (0.0, L.OK), (2e38, L.ERR_INVALID_ARG),
                                          (-3e38, L.ERR_INVALID_ARG)])
def test_attention_scale(lib, scale, status):  # noqa: F811
    """log2(e) times the scale stays finite."""
    assert _status(lib, _attn(scale=scale)) == status


def _cache(dim, table):
    return L.PagedKV(L.DeviceKV(L.BF16, dim, torch.zeros(64, dim, dtype=torch.bfloat16)), table, 16)


def test_layer_wants_one_table():
    """Views that begin at the same entry but are laid out otherwise are not the same table."""
    whole = torch.zeros(2, 8, dtype=torch.int32)
    for other in (whole[:, :4], whole.t().reshape(8, 2)[:2], whole[:1], whole.as_strided((2, 8), (4, 1))):
        with pytest.raises(ValueError, match="share pages and table"):
            L.PagedLayer(_cache(512, whole), _cache(128, other), 64, 4)


def test_layer_refuses_inputs_of_other_shapes():
    """A step's data for one sequence, or one token, is not spread over the batch."""
    B, T, H = 3, 2, 8
    layer = L.PagedLayer.__new__(L.PagedLayer)
    layer.B, layer.T = B, T
    shapes = dict(x_rows=(B * T, 512), x_keys=(B * T, 128), q_idx=(B, T, H, 128), w=(B, T, H), q_attn=(B, T, H, 512),
                  length=(B,), pos=(B * T,))
    ints = ("length", "pos")
    for name, shape in shapes.items():
        setattr(layer, {"length": "first"}.get(name, name), torch.zeros(shape, dtype=torch.int32 if name in ints else torch.float32))
    layer.length, layer.row = torch.zeros(B, dtype=torch.int32), torch.zeros(B * T, dtype=torch.int32)
    good = {n: torch.full(s, 5, dtype=torch.int32) if n in ints else torch.ones(s) for n, s in shapes.items()}
    layer.set_inputs(**good)
    assert layer.length.tolist() == [7] * B and layer.row.tolist() == [5, 6] * B and layer.pos.tolist() == [5] * (B * T)
    for name, t in good.items():
        for bad in (t[:1], t[0], torch.cat([t, t])):
            with pytest.raises(ValueError, match=name):
                layer.set_inputs(**{**good, name: bad})
    layer.set_inputs(**{n: t for n, t in good.items() if n != "pos"})
    assert layer.pos.tolist() == [5, 6] * B
