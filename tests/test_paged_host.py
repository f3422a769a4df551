"""The paged-cache calls' refusals (before anything touches a device) and the
plain forms the GPU tests use, on hand values."""
import ctypes as C

import numpy as np
import pytest
import torch

import _paged_ref as ref
import lightning_indexer_top_index_b200 as L

WS = C.c_void_p(0x100000)


@pytest.fixture(scope="module")
def lib():
    from lightning_indexer_top_index_b200 import build
    build.build()
    return L.lib()


def _rows(dtype=L.E2M1, dim=512, **kw):
    q = dim - 64
    ld = {L.E2M1: q // 2, L.E4M3: q}.get(dtype, dim)
    a = dict(dtype=dtype, dim=dim, data=0x1000, scale=0x2000, rope=0x3000, ld=ld, ld_scale=16, ld_rope=64, batch_rows=0)
    a.update(kw)
    return L.KVArgs(*[a[n] for n, _ in L.KVArgs._fields_])


def _pages(rows=None, page_rows=64, n_pages=100, table=0x4000, ld_table=50, max_pages=50):
    return L.PagesArgs(rows if rows is not None else _rows(), page_rows, n_pages, table, ld_table, max_pages)


def _make(cls, base, **kw):
    a = dict(base)
    a.update(kw)
    return cls(*[a[n] for n, _ in cls._fields_])


def _append(**kw):
    return _make(L.PagedAppendArgs, dict(n=5, B=2, x_dtype=L.F32, x=0x10000, ld_x=512, cache=_pages(), seq=0x5000,
                                         row=0x6000, pos=0x7000, inv_freq=0x8000, rope_pairs=0, flags=0), **kw)


def _read(**kw):
    return _make(L.PagedReadArgs, dict(n=5, B=2, cache=_pages(), seq=0x5000, row=0x6000, out_dtype=L.F32, out=0x10000,
                                       ld_out=512, flags=0), **kw)


def _pool(**kw):
    return _make(L.BlockPoolArgs, dict(B=2, keys=_pages(_rows(L.E4M3, 128)), len=0x5000, first=None, codes=0x10000,
                                       scale=0x20000, flags=0), **kw)


def _select(**kw):
    return _make(L.BlockSelectArgs, dict(B=2, T=1, H=64, k=16, n_first=1, n_last=2, q=0x10000, w=0x20000, codes=0x30000,
                                         scale=0x40000, page_rows=64, n_pages=100, table=0x4000, ld_table=50,
                                         max_pages=50, len=0x5000, ids=0x50000, n_sel=None, flags=0), **kw)


def _attn(**kw):
    return _make(L.PagedAttnArgs, dict(B=2, T=1, H=64, q=0x10000, cache=_pages(), len=0x5000, blocks=None, n_blocks=0,
                                       ld_blocks=0, n_sel=None, scale=0.04, out=0x20000, lse=None, flags=0), **kw)


CALLS = [("lidx_paged_append", L.OP_PAGED_APPEND, _append), ("lidx_paged_read", L.OP_PAGED_READ, _read),
         ("lidx_block_pool", L.OP_BLOCK_POOL, _pool), ("lidx_block_select", L.OP_BLOCK_SELECT, _select),
         ("lidx_paged_attn", L.OP_PAGED_ATTN, _attn)]

BAD_PAGES = [dict(page_rows=0), dict(page_rows=8), dict(page_rows=48), dict(page_rows=512), dict(n_pages=0),
             dict(max_pages=0), dict(table=None), dict(table=0x4002), dict(ld_table=49), dict(n_pages=1 << 26),
             dict(max_pages=1 << 26, ld_table=1 << 26)]
BAD_ROWS = [dict(data=None), dict(data=0x1008), dict(scale=None), dict(rope=None), dict(rope=0x3004), dict(ld=208),
            dict(ld=232), dict(ld_scale=13), dict(ld_rope=56), dict(ld_rope=68)]

INVALID = ([("lidx_paged_append", _append(cache=_pages(**kw))) for kw in BAD_PAGES] +
           [("lidx_paged_attn", _attn(cache=_pages(**kw))) for kw in BAD_PAGES] +
           [("lidx_paged_attn", _attn(cache=_pages(_rows(**kw)))) for kw in BAD_ROWS] +
           [("lidx_paged_read", _read(cache=_pages(_rows(**kw)))) for kw in BAD_ROWS] +
           [("lidx_block_select", _select(**kw)) for kw in BAD_PAGES] +
           [("lidx_paged_append", _append(**kw)) for kw in (
               dict(n=0), dict(n=-1), dict(B=0), dict(x=None), dict(x=0x10004), dict(ld_x=511), dict(ld_x=514),
               dict(x_dtype=L.BF16, ld_x=516), dict(seq=None), dict(row=None), dict(row=0x6001), dict(pos=0x7001),
               dict(inv_freq=0x8002), dict(rope_pairs=2))] +
           [("lidx_paged_read", _read(**kw)) for kw in (dict(n=0), dict(out=None), dict(out=0x10004), dict(ld_out=508),
                                                        dict(seq=None), dict(row=None))] +
           [("lidx_block_pool", _pool(**kw)) for kw in (dict(B=0), dict(len=None), dict(codes=None), dict(codes=0x10008),
                                                        dict(scale=None), dict(first=0x5001))] +
           [("lidx_block_select", _select(**kw)) for kw in (
               dict(B=0), dict(T=0), dict(H=0), dict(k=0), dict(n_first=-1), dict(n_first=9, n_last=8), dict(q=None),
               dict(q=0x10008), dict(w=None), dict(codes=None), dict(scale=None), dict(len=None), dict(ids=None),
               dict(n_sel=0x5002))] +
           [("lidx_paged_attn", _attn(**kw)) for kw in (
               dict(B=0), dict(T=0), dict(H=0), dict(q=None), dict(q=0x10008), dict(out=None), dict(out=0x20008),
               dict(len=None), dict(lse=0x3), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(blocks=0x9000, n_blocks=0), dict(blocks=0x9000, n_blocks=4, ld_blocks=3), dict(blocks=0x9002, n_blocks=4,
                                                                                                  ld_blocks=4))])
UNSUPPORTED = ([("lidx_paged_append", _append(cache=_pages(_rows(dim=256)))), ("lidx_paged_append", _append(x_dtype=L.F16)),
                ("lidx_paged_append", _append(cache=_pages(_rows(L.F16)))), ("lidx_paged_read", _read(out_dtype=L.E4M3)),
                ("lidx_block_pool", _pool(keys=_pages())), ("lidx_block_select", _select(H=65)),
                ("lidx_block_select", _select(k=257)),
                ("lidx_block_select", _select(max_pages=131073, ld_table=131073, page_rows=16)),
                ("lidx_paged_attn", _attn(H=129)), ("lidx_paged_attn", _attn(cache=_pages(_rows(L.F32)))),
                ("lidx_paged_attn", _attn(cache=_pages(_rows(dim=128))))])


@pytest.mark.parametrize("status,name,args", [(L.ERR_INVALID_ARG, *x) for x in INVALID] +
                         [(L.ERR_UNSUPPORTED, *x) for x in UNSUPPORTED])
def test_refusals(lib, status, name, args):
    assert getattr(lib, name)(C.byref(args), WS, 1 << 40, None) == status


@pytest.mark.parametrize("name,op,make", CALLS)
def test_workspace_and_launches(lib, name, op, make):
    n, c = C.c_size_t(0), C.c_int(0)
    assert lib.lidx_workspace_size(op, C.byref(make()), C.byref(n)) == L.OK and n.value >= 256
    assert lib.lidx_launch_count(op, C.byref(make()), C.byref(c)) == L.OK and c.value >= 1
    f = getattr(lib, name)
    assert f(C.byref(make()), None, 0, None) == L.ERR_WORKSPACE
    assert f(C.byref(make()), WS, n.value - 1, None) == L.ERR_WORKSPACE
    assert f(C.byref(make()), C.c_void_p(0x100010), 1 << 40, None) == L.ERR_WORKSPACE
    assert f(None, WS, 1 << 40, None) == L.ERR_INVALID_ARG
    assert lib.lidx_workspace_size(op, None, C.byref(n)) == L.ERR_INVALID_ARG


def test_other_calls_refuse_four_bits(lib):
    """E2M1 rows belong to paged caches."""
    kv = _rows(L.E2M1, 512)
    a = L.AttnArgs(1, 64, L.BF16, 0x1000, kv, 1000, 0x2000, 512, 512, None, kv, 0, 0.04, 0x3000, None)
    assert lib.lidx_sparse_attn_decode(C.byref(a), WS, 1 << 40, None) == L.ERR_UNSUPPORTED
    s = L.ScoreArgs(1, 1, 64, 100, L.BF16, 0x1000, 0x2000, _rows(L.E2M1, 128), 0x3000, 100)
    assert lib.lidx_index_score(C.byref(s), None) == L.ERR_UNSUPPORTED
    p = L.AppendArgs(1, 1, 0x1000, kv, 10, 0x2000, 0, 0)
    assert lib.lidx_cache_append(C.byref(p), WS, 1 << 40, None) == L.ERR_UNSUPPORTED


def test_host_tensors_are_refused():
    c = L.PagedKV(L.DeviceKV(L.BF16, 512, torch.zeros(64, 512, dtype=torch.bfloat16)), torch.zeros(1, 1, dtype=torch.int32), 64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        L.paged_append_call(torch.zeros(1, 512), c, i, i)
    with pytest.raises(ValueError, match="CUDA"):
        L.paged_attn_call(torch.zeros(1, 1, 64, 512, dtype=torch.bfloat16), c, i)
    with pytest.raises(ValueError):
        L.block_select_call(torch.zeros(1, 1, 64, 64), None, None, None, None, 64, i, 4)
    with pytest.raises(ValueError):
        L.paged_append_call(torch.zeros(3, 100), c, i, i)


# ------------------------------------------------- the plain forms, by hand
def test_ref_e2m1():
    x = np.zeros((1, 64))
    x[0, :12] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.0, 0.26, np.nan]
    x[0, 32] = 13.0  # 6 * 2^1 < 13 <= 6 * 2^2
    x[0, 33] = np.inf
    codes, scale = ref.encode_e2m1(x)
    n = [int(codes[0, i // 2] >> (4 * (i % 2))) & 15 for i in range(64)]
    assert n[:12] == [7, 15, 0, 2, 2, 4, 4, 6, 6, 8, 1, 7]
    assert list(scale[0]) == [127, 129] and n[32] == 5 and n[33] == 7  # 13 / 4 = 3.25 -> 3
    v = ref.decode(np.concatenate([codes, codes[:, :0]], 1), scale, np.zeros((1, 64), np.uint16), "e2m1", 128)
    assert v[0, 1] == -6 and v[0, 32] == 12 and v[0, 33] == 24


def test_ref_rotation():
    x = np.zeros((1, 128))
    x[0, 64], x[0, 65], x[0, 96] = 1.0, 2.0, 3.0
    f = np.zeros(32)
    f[0] = np.pi / 2
    out, _ = ref.rotate(x, [1], f, 0)
    assert np.allclose(out[0, :2], [-2, 1]) and out[0, 32] == 3
    out, _ = ref.rotate(x, [1], f, 1)
    assert np.allclose([out[0, 0], out[0, 32]], [-3, 1]) and out[0, 1] == 2


def test_ref_select_and_attend():
    q = np.ones((1, 1, 1, 128), np.float32)
    codes = np.zeros((5, 128), np.int8)
    codes[:, 0] = [10, 50, 20, 50, 1]
    table = np.arange(5, dtype=np.int32).reshape(1, 5)
    one = np.ones(5, np.float32)
    ids, n = ref.select(q, np.ones((1, 1, 1), np.float32), codes, one, table, 16, 5, [80], 3, 1, 0)
    assert list(ids[0, 0]) == [0, 1, 3] and n[0, 0] == 3
    ids, n = ref.select(q, np.ones((1, 1, 1), np.float32), codes, one, table, 16, 5, [33], 4, 1, 1)
    assert list(ids[0, 0]) == [0, 1, 2, -1]
    vals = np.zeros((32, 512))
    vals[1] = 1.0
    out, lse, _, _ = ref.attend(np.zeros((1, 1, 1, 512)), vals, np.array([[0, 1]], np.int32), 16, 2, [2], 1.0)
    assert np.allclose(out, 0.5) and np.allclose(lse, np.log(2))
