"""The paged-cache calls against plain 64-bit forms: append with rotation and
read back, block summaries, block selection, attention over pages, and a
decode step of all of them.

Tolerances.  Codes, scales, summaries and selections are whole numbers and
equal.  A rotated value is off by the angle's and the sine's rounding (below
2^-25 turns and 2^-22) and three fp32 roundings, together below 2^-20 (|u| +
|v|), before it is rounded to its format (half a step: 2^-8 of the value in
bf16).  Attention: the logits are fp32 sums of 512 products (error d <= 512 *
2^-24 * scale * sum |q x|), which moves each probability by a factor within
exp(+-2d); a probability may be rounded to bf16 (2^-8 of itself) and the
output is (2^-8 of itself)."""
import numpy as np
import pytest
import torch

import _paged_ref as ref
import lightning_indexer_top_index_b200 as L
import oracle

pytestmark = pytest.mark.gpu

FMT = {"f32": L.F32, "bf16": L.BF16, "e4m3": L.E4M3, "e2m1": L.E2M1}
DEV = "cuda"


def _np(t):
    if t.dtype == torch.bfloat16:
        return t.cpu().view(torch.int16).numpy().view(np.uint16).copy()
    return t.cpu().numpy().copy()


def _table(g, lens, page_rows, spare=3, width=None):
    need = [-(-n // page_rows) for n in lens]
    pages = g.permutation(sum(need) + spare)
    width = max(max(need), 1) if width is None else width
    t = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, m in enumerate(need):
        t[b, :m] = pages[at:at + m]
        at += m
    return t, sum(need) + spare


def _cache(g, fmt, dim, n_pages, page_rows, table, pad=0):
    """A pool of random bytes (finite values), its planes `pad` columns wider than a row."""
    rows = n_pages * page_rows
    q = dim - 64
    if fmt == "f32":
        kv = L.DeviceKV(L.F32, dim, torch.from_numpy(g.standard_normal((rows, dim + 4 * pad)).astype(np.float32)).to(DEV))
    elif fmt == "bf16":
        kv = L.DeviceKV(L.BF16, dim, torch.from_numpy(g.standard_normal((rows, dim + 8 * pad)).astype(np.float32)).to(DEV).bfloat16())
    else:
        width = q if fmt == "e4m3" else q // 2
        n_scale = q // 64 if fmt == "e4m3" else q // 32
        data = g.integers(0, 256, (rows, width + 16 * pad), dtype=np.uint8)
        if fmt == "e4m3":
            data[(data & 0x7F) >= 0x50] &= 0xBF  # no NaN codes, magnitudes of a few
        scale = g.integers(124, 129, (rows, n_scale + pad), dtype=np.uint8)
        rope = torch.from_numpy(g.standard_normal((rows, 64 + 8 * pad)).astype(np.float32)).to(DEV).bfloat16()
        kv = L.DeviceKV(FMT[fmt], dim, torch.from_numpy(data).to(DEV), torch.from_numpy(scale).to(DEV), rope)
    return L.PagedKV(kv, torch.from_numpy(table).to(DEV), page_rows)


def _planes(c):
    r = c.rows
    return [_np(t) for t in (r.data, r.scale, r.rope) if t is not None]


def _values(c, fmt):
    p = _planes(c)
    dim = c.rows.dim
    if fmt in ("f32", "bf16"):
        return ref.decode(p[0][:, :dim], None, None, fmt, dim)
    return ref.decode(p[0], p[1], p[2], fmt, dim)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


# ------------------------------------------------------------------ append
def _hard_rows(g, n, dim):
    x = g.standard_normal((n, dim)) * np.exp2(g.integers(-30, 30, (n, dim // 32))).repeat(32, axis=1)
    x[:, -64:] = g.standard_normal((n, 64)) * 3
    x = x.astype(np.float32)
    if n >= 6:
        x[0, :32] = 0.0
        x[1, :8] = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]) * 2.0 ** 4  # every midpoint, and the top
        x[1, 8:32] = -x[1, 31:7:-1] * 0
        x[2, :32] = np.float32(2.0 ** -140)
        x[3, 0] = np.float32(-0.0)
        x[4] = -x[4]
        x[5, 32:64] = np.float32(6.0000005) * 2.0 ** 3  # just above 6 * 2^3: the next scale
    return x


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3", "bf16", "f32"])
@pytest.mark.parametrize("dim", [512, 128])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("pairs", [None, L.ROPE_ADJACENT, L.ROPE_HALVES])
def test_append(cuda_device, fmt, dim, xt, pairs):
    g = np.random.default_rng(dim + 7 * len(fmt) + (pairs or 0))
    P = 16
    lens = [40, 1, 33]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, fmt, dim, n_pages, P, table, pad=1)
    todo = [(b, r) for b, n in enumerate(lens) for r in range(n) if g.random() < 0.7]
    todo.insert(3, (-1, 5))  # padding
    n = len(todo)
    seq, row = np.array(todo, np.int32).T.copy()
    pos = g.integers(0, 1 << 20, n).astype(np.int32)
    pos[0], pos[1] = 2 ** 31 - 1, 0
    x = torch.from_numpy(_hard_rows(g, n, dim))
    x = x.bfloat16() if xt == "bf16" else x
    wide = torch.zeros(n, dim + 8, dtype=x.dtype, device=DEV)  # rows further apart than they are wide
    wide[:, :dim] = x.to(DEV)
    xv = x.double().numpy()
    freq = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    before = _planes(c)
    call = L.paged_append_call(wide[:, :dim], c, _i32(seq), _i32(row), _i32(pos), None if pairs is None else
                               torch.from_numpy(freq).to(DEV), pairs or 0)
    call()
    assert call.status() == 0
    after = _planes(c)
    rows = np.array([table[b, r // P] * P + r % P for b, r in todo if b >= 0])
    at = np.array([i for i, (b, _) in enumerate(todo) if b >= 0])
    rot, mag = (xv[:, -64:], np.zeros((n, 64))) if pairs is None else ref.rotate(xv, pos, freq, pairs)
    rot, mag, body = rot[at], mag[at], xv[at][:, :-64]
    q = dim - 64
    untouched = np.setdiff1d(np.arange(n_pages * P), rows)
    for was, now in zip(before, after):
        assert np.array_equal(was[untouched], now[untouched])
    if fmt in ("f32", "bf16"):
        assert np.array_equal(before[0][:, dim:], after[0][:, dim:])
        got = ref.decode(after[0][rows][:, :dim], None, None, fmt, dim)
        want = body.astype(np.float32)
        if fmt == "bf16":
            want = torch.from_numpy(want).bfloat16().double().numpy()
        assert np.array_equal(got[:, :q], want.astype(np.float64))
        got_rot, step = got[:, q:], 2.0 ** -8 if fmt == "bf16" else 2.0 ** -24
    else:
        if fmt == "e2m1":
            codes, scale = ref.encode_e2m1(body)
        else:
            enc = oracle.encode_rows(np.concatenate([body, np.zeros((len(rows), 64))], 1).astype(np.float32), "e4m3")
            codes, scale = enc["data"].view(np.uint8).reshape(len(rows), -1), enc["scale"].reshape(len(rows), -1)
        assert np.array_equal(after[0][rows][:, : codes.shape[1]], codes)
        assert np.array_equal(after[1][rows][:, : scale.shape[1]], scale)
        for k, w in ((0, codes.shape[1]), (1, scale.shape[1]), (2, 64)):
            assert np.array_equal(before[k][:, w:], after[k][:, w:])
        got_rot, step = ref.bf16_value(after[2][rows][:, :64]), 2.0 ** -8
    assert (np.abs(got_rot - rot) <= step * np.abs(rot) + 2.0 ** -20 * mag + 1e-38).all()
    # and read back: the values that the planes stand for
    out = L.paged_read(c, _i32(seq), _i32(row))
    vals = _values(c, fmt)[rows]
    assert np.array_equal(out.cpu().double().numpy()[at], vals)
    assert torch.equal(out.cpu()[3], torch.zeros(dim))  # padding: left as it was
    if fmt != "f32":
        assert np.array_equal(L.paged_read(c, _i32(seq), _i32(row), dtype=torch.bfloat16).cpu().double().numpy()[at], vals)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_append_skips_what_does_not_exist(cuda_device, fmt):
    """Rows beyond the table, negative rows, sequences beyond the batch and
    missing pages are skipped and reported; nothing else changes."""
    g = np.random.default_rng(5)
    P = 16
    table = np.array([[1, 99, -1], [0, 2, 3]], np.int32)
    c = _cache(g, fmt, 512, 4, P, table)
    bad = [(0, 16), (0, 47), (0, 48), (0, -1), (2, 0), (2 ** 31 - 1, 0), (0, 2 ** 31 - 1), (-5, 0), (0, 32)]
    good = [(0, 3), (1, 47)]
    seq, row = np.array(bad + good, np.int32).T.copy()
    x = g.standard_normal((len(seq), 512)).astype(np.float32)
    before = _planes(c)
    call = L.paged_append_call(torch.from_numpy(x).to(DEV), c, _i32(seq), _i32(row))
    call()
    assert call.status() == L.DEV_BOUNDS
    rows = np.array([1 * P + 3, 3 * P + 15])
    after = _planes(c)
    keep = np.setdiff1d(np.arange(4 * P), rows)
    for was, now in zip(before, after):
        assert np.array_equal(was[keep], now[keep])
        assert not np.array_equal(was[rows], now[rows])
    read = L.paged_read_call(c, _i32(seq), _i32(row))
    out = read().cpu().numpy()
    assert read.status() == L.DEV_BOUNDS
    assert (out[: len(bad)] == 0).all()
    assert np.array_equal(out[len(bad):].astype(np.float64), _values(c, fmt)[rows])


def test_append_nonfinite(cuda_device):
    g = np.random.default_rng(6)
    c = _cache(g, "e2m1", 512, 1, 16, np.zeros((1, 1), np.int32))
    x = g.standard_normal((4, 512)).astype(np.float32)
    x[1, 3], x[1, 5], x[2, 40], x[3, 500] = np.nan, np.inf, -np.inf, np.inf
    call = L.paged_append_call(torch.from_numpy(x).to(DEV), c, _i32([0] * 4), _i32(range(4)))
    call()
    assert call.status() == L.DEV_NAN
    codes, scale = ref.encode_e2m1(x[:, :448].astype(np.float64))
    p = _planes(c)
    assert np.array_equal(p[0][:4], codes) and np.array_equal(p[1][:4], scale)
    assert ref.bf16_value(p[2][3])[52] == np.inf


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("dim", [512, 128])
@pytest.mark.parametrize("n", [7, 9000])
def test_read_bf16_every_scale(cuda_device, fmt, dim, n):
    """Rows read as bf16 under every scale byte: the exact products, rounded once; few rows and many, some of
    them padding or not there."""
    g = np.random.default_rng(dim + n)
    P = 16
    table = g.permutation(40).astype(np.int32).reshape(2, 20)
    table[1, 19] = -1
    c = _cache(g, fmt, dim, 40, P, table, pad=1)
    if fmt != "bf16":
        c.rows.scale.copy_(torch.from_numpy(g.permutation(c.rows.scale.numel()).astype(np.uint8).reshape(c.rows.scale.shape)))
    seq, row = g.integers(0, 2, n).astype(np.int32), g.integers(0, 20 * P, n).astype(np.int32)
    seq[3] = -1
    seq[5], row[5] = 1, 19 * P + 2
    out = torch.full((n, dim + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    call = L.paged_read_call(c, _i32(seq), _i32(row), out=out[:, :dim])
    call()
    assert call.status() == L.DEV_BOUNDS
    page = table[np.maximum(seq, 0), row // P]
    with np.errstate(all="ignore"):
        want = torch.from_numpy(_values(c, fmt)[np.maximum(page, 0) * P + row % P].astype(np.float64)).to(torch.bfloat16).float().numpy()
    want[(page < 0) & (seq >= 0)] = 0.0
    want[seq < 0] = 7.0
    got = out.float().cpu().numpy()
    assert np.array_equal(got[:, :dim], want, equal_nan=True)
    assert (got[:, dim:] == 7.0).all()


# -------------------------------------------------------------------- pool
@pytest.mark.parametrize("fmt", ["e4m3", "e2m1", "bf16", "f32"])
@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("tail", [False, True])
def test_pool(cuda_device, fmt, P, tail):
    g = np.random.default_rng(10 + P)
    lens = [3 * P + 1, 0, 1, P, 2 * P - 1]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, fmt, 128, n_pages, P, table, pad=1)
    first = np.array([2 * P, 0, 0, P - 1, -4], np.int32) if tail else None
    codes = torch.full((n_pages, 128), 55, dtype=torch.int8, device=DEV)
    scale = torch.full((n_pages,), 7.0, device=DEV)
    call = L.block_pool_call(c, _i32(lens), codes, scale, None if first is None else _i32(first))
    call()
    assert call.status() == 0
    want = ref.pool(_values(c, fmt), table, P, n_pages, lens, first)
    assert len(want) > 3
    for p in range(n_pages):
        wc, ws = want.get(p, (np.full(128, 55, np.int8), np.float32(7.0)))
        assert np.array_equal(codes[p].cpu().numpy(), wc), p
        assert scale[p].item() == ws, p


def test_pool_hard_values(cuda_device):
    """Subnormals, a block of zeros, sums that cancel, non-finite rows, lens
    beyond the table and missing pages."""
    g = np.random.default_rng(11)
    P = 16
    table = np.array([[0, 1, 2, 3], [4, 5, -1, 77]], np.int32)
    c = _cache(g, "f32", 128, 7, P, table)
    d = c.rows.data
    d[0:P] = 0.0
    d[P:2 * P] = torch.from_numpy((g.standard_normal((P, 128)) * 1e-41).astype(np.float32)).to(DEV)
    d[2 * P:3 * P] = 3e38
    d[2 * P + 1:3 * P:2] = -3e38
    d[2 * P, 5] = 1.0
    d[3 * P + 15, 100] = float("inf")
    d[4 * P + 3, 0] = float("nan")
    codes = torch.full((7, 128), 55, dtype=torch.int8, device=DEV)
    scale = torch.full((7,), 7.0, device=DEV)
    lens = [10 ** 6, 64]
    call = L.block_pool_call(c, _i32(lens), codes, scale)
    call()
    assert call.status() == L.DEV_BOUNDS | L.DEV_NAN
    want = ref.pool(_values(c, "f32"), table, P, 7, lens)
    for p in range(7):
        wc, ws = want.get(p, (np.full(128, 55, np.int8), np.float32(7.0)))
        assert np.array_equal(codes[p].cpu().numpy(), wc), p
        assert scale[p].item() == ws or (np.isnan(ws) and np.isnan(scale[p].item())), p


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1", "bf16", "f32"])
@pytest.mark.parametrize("P", [16, 64, 256])
def test_pool_long_tables(cuda_device, fmt, P):
    """Tables with room for many blocks (a warp sums one by itself), most of them not there yet."""
    g = np.random.default_rng(40 + P)
    lens = [5 * P + 1, 0, 1, P, 2 * P - 1, 37 * P - 3]
    table, n_pages = _table(g, lens, P)
    wide = np.full((len(lens), 500), -1, np.int32)
    wide[:, :table.shape[1]] = table
    c = _cache(g, fmt, 128, n_pages, P, wide, pad=1)
    codes = torch.full((n_pages, 128), 55, dtype=torch.int8, device=DEV)
    scale = torch.full((n_pages,), 7.0, device=DEV)
    if fmt != "f32":  # a block of zeros
        for plane in (t for t in (c.rows.data, c.rows.scale, c.rows.rope) if t is not None):
            plane.view(n_pages, P, -1)[int(table[5, 3])] = 0
    else:  # ... and sums that cancel, subnormals, a NaN
        d = c.rows.data.view(n_pages, P, -1)
        d[int(table[5, 3])] = 0.0
        d[int(table[5, 4])] = torch.from_numpy((g.standard_normal((P, d.shape[2])) * 1e-41).astype(np.float32)).to(DEV)
        d[int(table[5, 5]), 0::2] = 3e38
        d[int(table[5, 5]), 1::2] = -3e38
        d[int(table[5, 5]), 0, 5] = 1.0
        d[int(table[5, 6]), P - 1, 100] = float("nan")
    call = L.block_pool_call(c, _i32(lens), codes, scale)
    call()
    assert call.status() == (L.DEV_NAN if fmt == "f32" else 0)
    want = ref.pool(_values(c, fmt), wide, P, n_pages, lens)
    for p in range(n_pages):
        wc, ws = want.get(p, (np.full(128, 55, np.int8), np.float32(7.0)))
        assert np.array_equal(codes[p].cpu().numpy(), wc), p
        assert scale[p].item() == ws or (np.isnan(ws) and np.isnan(scale[p].item())), p


def test_pool_borders(cuda_device):
    """Means on and next to the middle between two codes, and quotients next to a border of fp32."""
    g = np.random.default_rng(47)
    P, n_pages = 16, 2400
    table = np.arange(n_pages, dtype=np.int32)[None]
    c = _cache(g, "f32", 128, n_pages, P, table)
    x = np.rint(g.uniform(-127, 127, (n_pages, 128)) * 2) / 2  # whole and half codes of a largest mean of 127
    x[:, 7] = 127.0
    x = x.astype(np.float32)
    half = n_pages // 2
    x[half:] = np.nextafter(x[half:], (np.where(g.random((n_pages - half, 128)) < 0.5, -1e9, 1e9)).astype(np.float32))
    x *= (2.0 ** g.integers(-140, 100, (n_pages, 1))).astype(np.float32)
    c.rows.data[:, :128] = torch.from_numpy(np.repeat(x, P, axis=0)).to(DEV)
    codes = torch.zeros((n_pages, 128), dtype=torch.int8, device=DEV)
    scale = torch.zeros(n_pages, device=DEV)
    call = L.block_pool_call(c, _i32([n_pages * P]), codes, scale)
    call()
    assert call.status() == 0
    want = ref.pool(_values(c, "f32"), table, P, n_pages, [n_pages * P])
    assert np.array_equal(codes.cpu().numpy(), np.stack([want[p][0] for p in range(n_pages)]))
    assert np.array_equal(scale.cpu().numpy(), np.array([want[p][1] for p in range(n_pages)], np.float32))


# ------------------------------------------------------------------ select
def _summaries(g, n_pages):
    codes = np.clip(np.rint(g.standard_normal((n_pages, 128)) * 40), -127, 127).astype(np.int8)
    return codes, (g.random(n_pages) * 0.02 + 0.01).astype(np.float32)


def _select(q, w, codes, scale, table, P, lens, k, **kw):
    qt = torch.from_numpy(q).to(DEV).bfloat16()
    call = L.block_select_call(qt, torch.from_numpy(w).to(DEV), torch.from_numpy(codes).to(DEV),
                               torch.from_numpy(scale).to(DEV), _i32(table), P, _i32(lens), k, **kw)
    ids, n_sel = call()
    return ids.cpu().numpy(), n_sel.cpu().numpy(), call.status(), qt.float().cpu().numpy()


@pytest.mark.parametrize("H,T,B,P,rows,k", [
    (64, 1, 1, 64, 64 * 300 + 5, 16), (1, 1, 3, 16, 200, 4), (17, 3, 2, 32, 1000, 8), (64, 5, 2, 128, 128 * 9, 5),
    (8, 1, 1, 16, 16 * 3000, 48), (64, 2, 1, 16, 16 * 20011, 200), (40, 1, 2, 64, 64 * 256, 256), (33, 1, 4, 256, 1, 3)])
def test_select(cuda_device, H, T, B, P, rows, k):
    g = np.random.default_rng(H * 1000 + rows)
    lens = [rows] + [int(rows * g.random()) for _ in range(B - 1)]
    if B > 2:
        lens[1] = 0
    table, n_pages = _table(g, lens, P)
    codes, scale = _summaries(g, n_pages)
    q = g.standard_normal((B, T, H, 128)).astype(np.float32)
    w = (g.random((B, T, H)) - 0.3).astype(np.float32)
    ids, n_sel, status, qb = _select(q, w, codes, scale, table, P, lens, k)
    assert status == 0
    want, wn = ref.select(qb, w, codes, scale, table, P, n_pages, lens, k, 1, 2)
    assert np.array_equal(n_sel, wn)
    assert np.array_equal(ids, want)


@pytest.mark.parametrize("B,n_blocks,k", [(1, 1025, 16), (4, 1100, 100), (7, 8300, 30), (10, 8300, 30), (2, 131072, 256),
                                          (40, 16390, 5)])
def test_select_long_rows(cuda_device, B, n_blocks, k):
    """Rows that clusters of every size share, up to the longest; pages shared by the sequences."""
    g = np.random.default_rng(B + n_blocks)
    P = 16
    n_pages = 5000
    table = g.integers(0, n_pages, (B, n_blocks)).astype(np.int32)
    codes, scale = _summaries(g, n_pages)
    q = g.standard_normal((B, 1, 3, 128)).astype(np.float32)
    w = (g.random((B, 1, 3)) - 0.3).astype(np.float32)
    lens = [n_blocks * P] + [int(n_blocks * P * g.random()) for _ in range(B - 1)]
    ids, n_sel, status, qb = _select(q, w, codes, scale, table, P, lens, k)
    assert status == 0
    want, wn = ref.select(qb, w, codes, scale, table, P, n_pages, lens, k, 1, 2)
    assert np.array_equal(n_sel, wn)
    assert np.array_equal(ids, want)


@pytest.mark.parametrize("n_blocks", [700, 5000])
@pytest.mark.parametrize("n_first,n_last,k", [(0, 0, 7), (1, 2, 3), (0, 9, 20), (4, 0, 256)])
def test_select_ties(cuda_device, n_blocks, n_first, n_last, k):
    """Equal scores go to the lower index, also across the CTAs of a row: all
    blocks alike, a few distinct values, and zero weights."""
    g = np.random.default_rng(n_blocks + k)
    P = 16
    table = g.permutation(n_blocks).astype(np.int32).reshape(1, -1).repeat(3, 0)
    codes = np.full((n_blocks, 128), 3, np.int8)
    scale = g.choice(np.array([0.5, 1.0, 2.0], np.float32), n_blocks)
    q = g.standard_normal((3, 1, 4, 128)).astype(np.float32)
    q[0] = 1.0
    w = np.ones((3, 1, 4), np.float32)
    w[1] = 0.0
    w[2] = -1.0
    lens = [n_blocks * P] * 3
    ids, n_sel, status, qb = _select(q, w, codes, scale, table, P, lens, k, n_first=n_first, n_last=n_last)
    want, wn = ref.select(qb, w, codes, scale, table, P, n_blocks, lens, k, n_first, n_last)
    assert np.array_equal(ids, want) and np.array_equal(n_sel, wn) and status == 0


def test_select_nan_and_missing_pages(cuda_device):
    """Blocks without a page or with a NaN score are taken only where they
    must be; lens beyond the table are cut; all is reported."""
    g = np.random.default_rng(3)
    P, nb = 32, 40
    table = g.permutation(nb).astype(np.int32).reshape(1, -1)
    codes, scale = _summaries(g, nb)
    scale[table[0, 3]] = np.nan
    scale[table[0, 39]] = np.nan  # the last block: always taken
    table[0, 7], table[0, 8] = -1, nb
    q = g.standard_normal((1, 1, 64, 128)).astype(np.float32)
    w = g.random((1, 1, 64)).astype(np.float32)
    ids, n_sel, status, qb = _select(q, w, codes, scale, table, P, [nb * P + 1], 38, n_first=1, n_last=1)
    assert status == L.DEV_NAN | L.DEV_BOUNDS
    want, wn = ref.select(qb, w, codes, scale, table, P, nb, [nb * P + 1], 38, 1, 1)
    assert np.array_equal(ids, want) and np.array_equal(n_sel, wn)
    assert n_sel[0, 0] == 37 and 3 not in ids and 7 not in ids and 39 in ids
    q[0, 0, 5, 7] = np.nan  # a query that is not a number scores nothing
    ids, n_sel, status, _ = _select(q, w, codes, scale, table, P, [nb * P], 10, n_first=1, n_last=1)
    assert status & L.DEV_NAN and n_sel[0, 0] == 2 and list(ids[0, 0, :3]) == [0, 39, -1]


# ------------------------------------------------------------------ attend
def _check_attn(out, lse, want):
    wo, wl, mag, big = want
    d = 512 * 2.0 ** -24 * big[..., None]
    o, l = out.cpu().double().numpy(), lse.cpu().double().numpy()
    assert np.isfinite(o).all()
    tol = 2.0 ** -8 * np.abs(wo) + (2.0 ** -8 + np.expm1(2 * d)) * 1.02 * mag + 1e-30
    worst = (np.abs(o - wo) / tol).max()
    assert worst <= 1.0, f"out off by {worst:.2f} of its bound"
    empty = np.isneginf(wl)
    assert np.array_equal(np.isneginf(l), empty)
    assert (o[empty] == 0).all()
    # the sum of exponentials: fp32 terms and sums (2^-20 of it), and the logits' own error
    lt = d[..., 0] + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, wl)))
    assert (np.abs(l - wl)[~empty] <= lt[~empty]).all()


def _q(g, B, T, H, mul=2.0):
    q = torch.from_numpy((mul * g.standard_normal((B, T, H, 512))).astype(np.float32)).to(DEV).bfloat16()
    return q, q.float().cpu().numpy()


def _poison(c, fmt, table, P, lens):
    """Rows that no query sees hold NaN (or the largest bytes)."""
    used = np.zeros(c.rows.data.shape[0], bool)
    for b, n in enumerate(lens):
        for r in range(min(n, table.shape[1] * P)):
            p = table[b, r // P]
            if 0 <= p < c.n_pages:
                used[p * P + r % P] = True
    idle = torch.from_numpy(~used).to(DEV)
    if fmt == "bf16":
        c.rows.data[idle] = float("nan")
    else:
        c.rows.data[idle] = 0xFF
        c.rows.scale[idle] = 0xFF
        c.rows.rope[idle] = float("nan")


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("H", [64, 1, 40, 65, 128])
@pytest.mark.parametrize("P,lens,T", [(64, [700, 1, 0, 64, 65], 1), (16, [333, 63], 3), (256, [1000], 2), (32, [5], 5)])
def test_attn_dense(cuda_device, fmt, H, P, lens, T):
    g = np.random.default_rng(100 + H + P)
    table, n_pages = _table(g, lens, P)
    c = _cache(g, fmt, 512, n_pages, P, table, pad=1)
    _poison(c, fmt, table, P, lens)
    B = len(lens)
    q, qn = _q(g, B, T, H)
    call = L.paged_attn_call(q, c, _i32(lens))
    out, lse = call()
    assert call.status() == 0
    vals = np.nan_to_num(_values(c, fmt))
    _check_attn(out, lse, ref.attend(qn, vals, table, P, n_pages, lens, 512 ** -0.5))
    again, _ = call()  # a second call on the same workspace
    assert torch.equal(out, again)


@pytest.mark.parametrize("fmt", ["e2m1", "bf16"])
@pytest.mark.parametrize("P,T,k,use_n", [(64, 1, 16, False), (16, 3, 9, True), (128, 2, 2, False), (32, 1, 1, True)])
def test_attn_blocks(cuda_device, fmt, P, T, k, use_n):
    g = np.random.default_rng(200 + P)
    lens = [20 * P + 7, 3 * P, P // 2, 0]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, fmt, 512, n_pages, P, table)
    B = len(lens)
    q, qn = _q(g, B, T, 64)
    blocks = np.full((B, T, k), -1, np.int32)
    n_sel = np.zeros((B, T), np.int32)
    for b, n in enumerate(lens):
        nb = -(-n // P)
        for t in range(T):
            m = min(k, nb)
            blocks[b, t, :m] = np.sort(g.permutation(nb)[:m])
            n_sel[b, t] = g.integers(0, m + 1)
    if k > 2:
        blocks[0, 0, 1] = blocks[0, 0, 0]  # twice: counts twice
    call = L.paged_attn_call(q, c, _i32(lens), _i32(blocks), _i32(n_sel) if use_n else None)
    out, lse = call()
    assert call.status() == 0
    _check_attn(out, lse, ref.attend(qn, _values(c, fmt), table, P, n_pages, lens, 512 ** -0.5, blocks,
                                     n_sel if use_n else None))


def test_attn_bad_blocks_and_pages(cuda_device):
    g = np.random.default_rng(7)
    P = 32
    lens = [10 * P - 3, 6 * P, 999 * P]
    table, n_pages = _table(g, [10 * P, 10 * P, 10 * P], P)
    table[0, 4], table[1, 0], table[1, 5] = n_pages, -1, 2 ** 31 - 1
    c = _cache(g, "e2m1", 512, n_pages, P, table)
    q, qn = _q(g, 3, 1, 64)
    call = L.paged_attn_call(q, c, _i32(lens))
    out, lse = call()
    assert call.status() == L.DEV_BOUNDS
    _check_attn(out, lse, ref.attend(qn, _values(c, "e2m1"), table, P, n_pages, lens, 512 ** -0.5))
    blocks = np.array([[[0, 10, -2, 4, 9]], [[-1, -1, -1, -1, -1]], [[9, 9, 2 ** 31 - 1, 1 << 27, 0]]], np.int32)
    call = L.paged_attn_call(q, c, _i32([10 * P - 3, 6 * P, 10 * P]), _i32(blocks))
    out, lse = call()
    assert call.status() == L.DEV_BOUNDS
    _check_attn(out, lse, ref.attend(qn, _values(c, "e2m1"), table, P, n_pages, [10 * P - 3, 6 * P, 10 * P], 512 ** -0.5,
                                     blocks))
    # a bad -1 alone is no error
    call = L.paged_attn_call(q, c, _i32(lens[:2] + [5]), _i32(np.full((3, 1, 4), -1)))
    out, lse = call()
    assert call.status() == 0 and (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("scale,mul", [(-0.05, 2.0), (0.5, 8.0), (0.0, 1.0)])
def test_attn_far_apart_logits(cuda_device, scale, mul):
    """Logits hundreds apart (the running maximum moves again and again), a
    negative scale, and a zero one."""
    g = np.random.default_rng(9)
    P = 64
    lens = [1500, 640]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, "e2m1", 512, n_pages, P, table)
    ramp = torch.from_numpy(np.linspace(0.05, 1.5, n_pages * P).astype(np.float32)).to(DEV)
    order = torch.from_numpy(np.concatenate([table[b, : -(-n // P)] for b, n in enumerate(lens)])).to(DEV).long()
    rows = (order.unsqueeze(1) * P + torch.arange(P, device=DEV)).reshape(-1)
    c.rows.rope[rows] = (c.rows.rope[rows].float() * ramp[: rows.numel()].unsqueeze(1) * 2).bfloat16()
    q, qn = _q(g, 2, 1, 64, mul)
    call = L.paged_attn_call(q, c, _i32(lens), scale=scale)
    out, lse = call()
    _check_attn(out, lse, ref.attend(qn, _values(c, "e2m1"), table, P, n_pages, lens, scale))


def test_attn_scale_extremes(cuda_device):
    """Block scales from 2^-127 up to 2^10, as the format allows them."""
    g = np.random.default_rng(12)
    P = 16
    table = np.arange(4, dtype=np.int32).reshape(1, 4)
    c = _cache(g, "e2m1", 512, 4, P, table)
    c.rows.scale[:] = torch.from_numpy(g.choice(np.array([0, 1, 100, 120, 127, 130, 137], np.uint8),
                                                tuple(c.rows.scale.shape))).to(DEV)
    q, qn = _q(g, 1, 1, 64, 0.01)
    out, lse = L.paged_attn(q, c, _i32([64]))
    _check_attn(out, lse, ref.attend(qn, _values(c, "e2m1"), table, P, 4, [64], 512 ** -0.5))
    vals = L.paged_read(c, _i32([0] * 64), _i32(range(64))).cpu().double().numpy()
    assert np.array_equal(vals, _values(c, "e2m1"))


def test_attn_nan_stays_with_its_head(cuda_device):
    """A NaN in one query head leaves the other heads alone; a NaN in a row
    that is attended to reaches all of them."""
    g = np.random.default_rng(13)
    P, lens = 64, [200]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, "bf16", 512, n_pages, P, table)
    q, qn = _q(g, 1, 1, 64)
    clean, _ = L.paged_attn(q, c, _i32(lens))
    q[0, 0, 7, 100] = float("nan")
    out, lse = L.paged_attn(q, c, _i32(lens))
    assert torch.isnan(out[0, 0, 7]).all() and torch.isnan(lse[0, 0, 7])
    others = [h for h in range(64) if h != 7]
    assert torch.equal(out[0, 0, others], clean[0, 0, others])


@pytest.mark.parametrize("B,T,rows,k", [(1, 1, 16384, 0), (32, 1, 1000, 0), (2, 130, 2000, 4), (150, 2, 64, 0)])
def test_attn_many_chunks(cuda_device, B, T, rows, k):
    """Sizes at which a sequence is split over many CTAs, a CTA serves many
    sequences, and partial results are joined."""
    g = np.random.default_rng(B + rows)
    P = 64
    lens = [rows] + [int(g.integers(0, rows + 1)) for _ in range(B - 1)]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, "e2m1", 512, n_pages, P, table)
    H = 16
    q, qn = _q(g, B, T, H)
    blocks = None
    if k:
        blocks = np.full((B, T, k), -1, np.int32)
        for b, n in enumerate(lens):
            for t in range(T):
                nb = -(-max(0, n - T + 1 + t) // P)
                m = min(k, nb)
                blocks[b, t, :m] = np.sort(g.permutation(nb)[:m])
    call = L.paged_attn_call(q, c, _i32(lens), None if blocks is None else _i32(blocks))
    out, lse = call()
    assert call.status() == 0
    _check_attn(out, lse, ref.attend(qn, _values(c, "e2m1"), table, P, n_pages, lens, 512 ** -0.5, blocks))


# -------------------------------------------------------- the calls together
def _layer(g, B, P, width, H, k, T=1, pdl=True):
    n_pages = B * width + 2
    table = torch.from_numpy(g.permutation(n_pages)[: B * width].astype(np.int32).reshape(B, width)).to(DEV)
    rows = L.PagedKV.empty(L.E2M1, 512, n_pages, P, table)
    keys = L.PagedKV.empty(L.E4M3, 128, n_pages, P, table)
    freq = torch.from_numpy((10000.0 ** (-np.arange(32) / 32)).astype(np.float32)).to(DEV)
    return L.PagedLayer(rows, keys, H, k, T, inv_freq=freq, pdl=pdl), freq


def _step_inputs(g, B, T, H):
    f = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32))  # noqa: E731
    return (f(B * T, 512).bfloat16(), f(B * T, 128).bfloat16(), f(B, T, H, 128).bfloat16(),
            torch.rand(B, T, H), f(B, T, H, 512).bfloat16())


def _check_layer(layer, lens):
    """The layer's outputs from its caches as they are now."""
    keys, rows = layer.keys, layer.rows
    table, P = keys.table.cpu().numpy(), keys.page_rows
    want = ref.pool(_values(keys, "e4m3"), table, P, keys.n_pages, lens)
    codes, scale = layer.codes.cpu().numpy(), layer.scale.cpu().numpy()
    for p, (wc, ws) in want.items():
        assert np.array_equal(codes[p], wc) and scale[p] == ws
    ids, n_sel = ref.select(layer.q_idx.float().cpu().numpy(), layer.w.cpu().numpy(), codes, scale, table, P,
                            keys.n_pages, lens, layer.ids.shape[2], 1, 2)
    assert np.array_equal(layer.ids.cpu().numpy(), ids) and np.array_equal(layer.n_sel.cpu().numpy(), n_sel)
    _check_attn(layer.out, layer.lse, ref.attend(layer.q_attn.float().cpu().numpy(), _values(rows, "e2m1"), table, P,
                                                 rows.n_pages, lens, 512 ** -0.5, ids, n_sel))


@pytest.mark.parametrize("T,pdl", [(1, True), (3, True), (1, False)])
def test_layer_steps(cuda_device, T, pdl):
    """A prefill by paged_append, then decode steps through the prepared calls
    and through the captured graph."""
    g = np.random.default_rng(21)
    B, P, width, H, k = 3, 16, 40, 64, 6
    layer, freq = _layer(g, B, P, width, H, k, T, pdl)
    lens = np.array([300, 17, 0], np.int32)
    seq = np.repeat(np.arange(B), lens).astype(np.int32)
    row = np.concatenate([np.arange(n) for n in lens]).astype(np.int32)
    for cache, dim in ((layer.rows, 512), (layer.keys, 128)):
        x = torch.from_numpy(g.standard_normal((len(seq), dim)).astype(np.float32)).to(DEV)
        L.paged_append(x, cache, _i32(seq), _i32(row), inv_freq=freq)
    layer.summarise(_i32(lens))
    assert layer.kernel_launches() == sum(c.launches for c in layer._calls)
    for step in range(4):
        layer.set_inputs(*_step_inputs(g, B, T, H), torch.from_numpy(lens))
        if step < 2:
            layer.enqueue()
        else:
            layer.replay()
        lens = lens + T
        torch.cuda.synchronize()
        _check_layer(layer, lens)
    assert layer.status() == 0


def test_two_graphs_and_streams(cuda_device):
    """Two layers' graphs replayed at the same time on two streams give what
    each gives alone."""
    g = np.random.default_rng(22)
    layers = [_layer(g, 2, 32, 12, 64, 5)[0] for _ in range(2)]
    lens = torch.tensor([200, 77], dtype=torch.int32)
    alone = []
    for layer in layers:
        for cache in (layer.rows, layer.keys):
            cache.rows.data.copy_(torch.from_numpy(g.integers(0, 120, tuple(cache.rows.data.shape), dtype=np.uint8)))
            cache.rows.scale.fill_(126)
        layer.summarise((lens + 1).to(DEV))
        layer.set_inputs(*_step_inputs(g, 2, 1, 64), lens)
        layer.capture()
        layer.replay()
        torch.cuda.synchronize()
        alone.append((layer.out.clone(), layer.ids.clone()))
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(20):
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):
                layer.replay()
    torch.cuda.synchronize()
    for layer, (out, ids) in zip(layers, alone):
        assert torch.equal(layer.out, out) and torch.equal(layer.ids, ids)


def test_one_shot_on_another_stream(cuda_device):
    """stream= (an object or a raw handle) allocates, runs and returns on that stream."""
    g = np.random.default_rng(23)
    P, lens = 64, [500]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, "e2m1", 512, n_pages, P, table)
    q, _ = _q(g, 1, 1, 64)
    n = _i32(lens)
    want = L.paged_attn(q, c, n)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        out, lse = L.paged_attn(q, c, n, stream=stream)
        s.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("call", ["append", "read", "pool", "select", "attn"])
def test_launch_count_matches_graph(cuda_device, call):
    from _helpers import graph_kernel_count
    g = np.random.default_rng(24)
    layer, freq = _layer(g, 2, 16, 8, 16, 4)
    calls = dict(append=layer._calls[0], pool=layer._calls[2], select=layer._calls[3], attn=layer._calls[4],
                 read=L.paged_read_call(layer.rows, _i32([0, 1]), _i32([0, 3])))
    assert graph_kernel_count(lambda s: calls[call](s)) == calls[call].launches


def test_workspace_too_small(cuda_device):
    g = np.random.default_rng(25)
    layer, _ = _layer(g, 2, 16, 8, 16, 4)
    with pytest.raises(L.LidxError) as e:
        L.paged_attn(layer.q_attn, layer.rows, layer.length, ws=torch.zeros(16, dtype=torch.uint8, device=DEV))
    assert e.value.status == L.ERR_WORKSPACE
