"""Paged-cache calls where they can go wrong beside the ordinary cases: what
the attention's probabilities keep, calls from several host threads and
streams, selections among many near scores, values that are not numbers.

Tolerances as derived in test_gpu_paged.py, but for the probabilities: they
enter the second product as a bf16 value and the bf16 value of what its
rounding left, together within 2^-16 of each."""
import gc
import threading
import weakref

import numpy as np
import pytest
import torch

import _paged_ref as ref
import lightning_indexer_top_index_b200 as L
from test_gpu_paged import DEV, FMT, _cache, _i32, _select, _summaries, _table, _values

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attend
def cancelling_case(g, rows, heads):
    """Rows in pairs (x, -x) in all but the first 16 dims, which alone meet the
    queries: outputs nearly cancel, so that an error of a probability shows
    beside the output's own rounding.  Values are exact in every format."""
    x = g.choice(np.array([1.0, 2.0, 3.0, 4.0, 6.0]), (rows, 512)) * g.choice(np.array([-1.0, 1.0]), (rows, 512))
    x[1::2, 16:] = -x[: rows - rows % 2: 2, 16:]
    q = np.zeros((heads, 512))
    q[:, :16] = g.standard_normal((heads, 16)) * 2.0 ** -8
    return x, torch.from_numpy(q).bfloat16()


def attn_bound(want, rows):
    """Largest errors of out: its rounding, 2^-16 of each probability, what the
    logits' error does to them, and two fp32 sums over the rows."""
    wo, _, mag, big = want
    d = 512 * 2.0 ** -24 * big[..., None]
    return 2.0 ** -8 * np.abs(wo) + (2.0 ** -16 + np.expm1(2 * d) + 2 * rows * 2.0 ** -24) * 1.02 * mag + 1e-30


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("rows,heads", [(6, 64), (64, 70), (300, 16), (3000, 5)])
def test_attn_probabilities_keep_16_bits(cuda_device, fmt, rows, heads):
    g = np.random.default_rng(rows + heads)
    P = 64
    table, n_pages = _table(g, [rows], P)
    c = L.PagedKV.empty(FMT[fmt], 512, n_pages, P, torch.from_numpy(table).to(DEV))
    x, q = cancelling_case(g, rows, heads)
    L.paged_append(torch.from_numpy(x.astype(np.float32)).to(DEV), c, _i32([0] * rows), _i32(range(rows)))
    vals = _values(c, fmt)
    assert np.array_equal(vals[[table[0, r // P] * P + r % P for r in range(rows)]], x)
    want = ref.attend(q.double().numpy()[None, None], vals, table, P, n_pages, [rows], 1.0)
    out, _ = L.paged_attn(q.to(DEV)[None, None], c, _i32([rows]), scale=1.0)
    worst = (np.abs(out.cpu().double().numpy() - want[0]) / attn_bound(want, rows)).max()
    assert worst <= 1.0, f"out off by {worst:.2f} of its bound"


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3", "bf16"])
@pytest.mark.parametrize("rows,bad", [(50, [3]), (50, range(50)), (700, [0]), (700, [650]), (700, range(64))])
def test_attn_nan_in_an_attended_row(cuda_device, fmt, rows, bad):
    """A NaN in a row that is attended to reaches all heads and dims, whether the job
    is one chunk or split over CTAs, also where a chunk holds nothing else; the
    batch's other sequence stays as it was."""
    g = np.random.default_rng(60 + rows)
    P, lens, H = 64, [rows, 130], 70
    table, n_pages = _table(g, lens, P)
    c = _cache(g, fmt, 512, n_pages, P, table)
    q = torch.from_numpy(g.standard_normal((2, 1, H, 512)).astype(np.float32)).to(DEV).bfloat16()
    clean, clean_lse = L.paged_attn(q, c, _i32(lens))
    at = [int(table[0, r // P]) * P + r % P for r in bad]
    if fmt == "bf16":
        c.rows.data[at, 100] = float("nan")
    else:
        c.rows.scale[at, 2] = 0xFF
    out, lse = L.paged_attn(q, c, _i32(lens))
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.equal(out[1], clean[1]) and torch.equal(lse[1], clean_lse[1])


@pytest.mark.parametrize("rows", [40, 700])
def test_attn_infinite_value(cuda_device, rows):
    """A row with an infinite value: heads whose score of it is -inf lose that dim
    only (0 * inf), the others are NaN, as the formula has it."""
    g = np.random.default_rng(61)
    P, lens = 64, [rows]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, "bf16", 512, n_pages, P, table)
    c.rows.data[int(table[0, 0]) * P + 7, 33] = float("inf")
    q = torch.from_numpy(g.standard_normal((1, 1, 64, 512)).astype(np.float32)).to(DEV).bfloat16()
    out, lse = L.paged_attn(q, c, _i32(lens))
    vals, qn = _values(c, "bf16"), q.double().cpu().numpy()
    with np.errstate(all="ignore"):
        want, want_lse, _, _ = ref.attend(qn, vals, table, P, n_pages, lens, 512 ** -0.5)
    assert np.array_equal(torch.isnan(out).cpu().numpy(), np.isnan(want))
    assert np.array_equal(torch.isnan(lse).cpu().numpy(), np.isnan(want_lse))
    assert 0 < np.isnan(want_lse).sum() < 64
    # where its probability is 0, the values are those of the other rows
    others = np.zeros((n_pages * P, 512))
    others[: rows - 1] = vals[[int(table[0, r // P]) * P + r % P for r in range(rows) if r != 7]]
    without = ref.attend(qn, others, np.arange(n_pages, dtype=np.int32)[None], P, n_pages, [rows - 1], 512 ** -0.5)
    off = np.abs(out.double().cpu().numpy() - without[0]) / attn_bound(without, rows)
    assert off[~np.isnan(want)].max() <= 1.0


@pytest.mark.parametrize("scale", [0.0, -0.0, 2.0 ** -130, -2.0 ** -140])
def test_attn_scale_of_nothing(cuda_device, scale):
    """A zero scale makes every logit zero however large the products are, and a tiny one keeps its share."""
    g = np.random.default_rng(62)
    P, lens = 64, [300]
    table, n_pages = _table(g, lens, P)
    c = _cache(g, "bf16", 512, n_pages, P, table)
    c.rows.data.mul_(2.0 ** 59)
    q = torch.from_numpy((g.standard_normal((1, 1, 64, 512)) * 2.0 ** 60).astype(np.float32)).to(DEV).bfloat16()
    out, lse = L.paged_attn(q, c, _i32(lens), scale=scale)
    want = ref.attend(q.double().cpu().numpy(), _values(c, "bf16"), table, P, n_pages, lens, float(np.float32(scale)))
    assert (np.abs(out.double().cpu().numpy() - want[0]) <= attn_bound(want, lens[0])).all()
    d = 512 * 2.0 ** -24 * want[3]
    assert (np.abs(lse.double().cpu().numpy() - want[1]) <= d + 2.0 ** -20 * (1 + np.abs(want[1]))).all()


# ------------------------------------------------- several threads and streams
def _many_threads(calls, times):
    """Every call `times` times, each from a thread and on a stream of its own; the errors."""
    errors, start = [], threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        start.wait()
        for _ in range(times):
            try:
                call(stream)
            except Exception as e:
                errors.append(str(e))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


def test_select_from_several_threads(cuda_device):
    """Calls whose shared memory differs, from several host threads at once."""
    g = np.random.default_rng(50)
    P, n_pages = 16, 300
    codes = torch.from_numpy(g.integers(-127, 128, (n_pages, 128), dtype=np.int8)).to(DEV)
    scale = torch.rand(n_pages, device=DEV) + 0.5
    calls, want = [], []
    for width, k in ((131072, 256), (40, 4), (16000, 200), (300, 16)):
        lens = _i32([min(width, 500) * P])
        table = _i32(g.integers(0, n_pages, (1, width)))
        q = torch.from_numpy(g.standard_normal((1, 1, 8, 128)).astype(np.float32)).to(DEV).bfloat16()
        w = torch.rand(1, 1, 8, device=DEV)
        call = L.block_select_call(q, w, codes, scale, table, P, lens, k)
        want.append(call()[0].clone())
        calls.append(call)
    torch.cuda.synchronize()
    errors = _many_threads(calls, 4000)
    assert not errors, f"{len(errors)} calls failed: {errors[0]}"
    for call, ids in zip(calls, want):
        assert torch.equal(call.out[0], ids)


def _small(g, rows=500, heads=64):
    """A cache, a query and lens of one sequence."""
    P = 64
    table, n_pages = _table(g, [rows], P)
    c = _cache(g, "e2m1", 512, n_pages, P, table)
    q = torch.from_numpy(g.standard_normal((1, 1, heads, 512)).astype(np.float32)).to(DEV).bfloat16()
    return c, q, _i32([rows])


def test_prepared_on_a_busy_stream(cuda_device):
    """A call prepared on a stream with work before it, then called on another:
    what preparing does to its memory does not come after the call."""
    c, q, n = _small(np.random.default_rng(51))
    seq, row = _i32([0] * 400), _i32(range(400))
    want_rows, (want, want_lse) = L.paged_read(c, seq, row), L.paged_attn(q, c, n)
    busy, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(busy):
        torch.cuda._sleep(200_000_000)
        read, attn = L.paged_read_call(c, seq, row), L.paged_attn_call(q, c, n)
    got = read(stream=other)
    out, lse = attn(stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got, want_rows)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert read.status() == 0 and attn.status() == 0


def test_prepared_call_dropped_while_another_stream_runs_it(cuda_device):
    """The workspace is not given away before the work on another stream that uses it is done."""
    c, q, n = _small(np.random.default_rng(52))
    want, _ = L.paged_attn(q, c, n)
    call = L.paged_attn_call(q, c, n)
    size, other = call.ws.numel(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(200_000_000)
        out, _ = call()
    del call
    mine = torch.full((size,), 0x5A, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    assert (mine == 0x5A).all()
    assert torch.equal(out, want)


@pytest.mark.parametrize("fmt", ["e2m1", "bf16"])
def test_prepared_call_keeps_a_replaced_cache(cuda_device, fmt):
    """A cache object may be given a longer table or a larger pool: a call that was
    prepared before keeps the tensors that its pointers name."""
    g = np.random.default_rng(53)
    P, n = 64, _i32([100])
    table, n_pages = _table(g, [100], P)
    c, k = _cache(g, fmt, 512, n_pages, P, table), _cache(g, fmt, 128, n_pages, P, table)
    q = torch.zeros(1, 1, 64, 512, dtype=torch.bfloat16, device=DEV)
    codes, scale = torch.zeros(n_pages, 128, dtype=torch.int8, device=DEV), torch.zeros(n_pages, device=DEV)
    seq = _i32([0])
    calls = [L.paged_attn_call(q, c, n), L.paged_read_call(c, seq, seq), L.block_pool_call(k, n, codes, scale),
             L.paged_append_call(torch.zeros(1, 512, device=DEV), c, seq, seq)]
    held = [weakref.ref(t) for x in (c, k) for t in x.tensors()]
    for x in (c, k):
        x.table = x.table.clone()
        for plane in ("data", "scale", "rope"):
            if getattr(x.rows, plane) is not None:
                setattr(x.rows, plane, getattr(x.rows, plane).clone())
    gc.collect()
    assert all(r() is not None for r in held)
    del calls
    gc.collect()
    assert all(r() is None for r in held)


# ------------------------------------------------------------------ select
def near_scores(g, kind, n):
    """Block scales, to which the scores are in proportion: a few far ones
    stretch the range, so that most of the others share a bin of it."""
    near = {"near": lambda: 1.0 + g.random(n) * 2.0 ** -7, "infinite": lambda: g.random(n),
            "signs": lambda: (g.random(n) - 0.5) * 2.0 ** -5,
            "low bits": lambda: 1.0 + g.integers(0, 4 * n, n) * 2.0 ** -23,
            "duplicates": lambda: np.where(g.random(n) < 0.4, 1.0 + 2.0 ** -9, 1.0 + g.random(n) * 1.01 * 2.0 ** -9)}[kind]()
    far = g.permutation(n)[:4]
    near[far] = [1000.0, -1000.0, 999.0, 998.5] if kind != "infinite" else [np.inf, -np.inf, np.inf, 5.0]
    return near.astype(np.float32)


NEAR = [(kind, *size) for kind in ("near", "signs", "low bits", "duplicates", "infinite")
        for size in ((1, 20000, 16), (2, 20000, 256), (80, 3001, 40), (10, 40000, 250))]


def near_case(kind, B, n_blocks, k):
    g = np.random.default_rng(n_blocks + k + len(kind))
    scale = near_scores(g, kind, n_blocks)
    codes = np.full((n_blocks, 128), 3, np.int8)
    table = np.stack([g.permutation(n_blocks) for _ in range(B)]).astype(np.int32)
    q, w = np.ones((B, 1, 1, 128), np.float32), g.random((B, 1, 1)).astype(np.float32) + 0.1
    return q, w, codes, scale, table


@pytest.mark.parametrize("kind,B,n_blocks,k", NEAR)
def test_select_near_scores(cuda_device, kind, B, n_blocks, k):
    """More than 256 scores in the bin of the k-th: the digits of the scores decide, down to the last
    where many are equal, in a CTA's slice of a row and among the lists of a cluster."""
    q, w, codes, scale, table = near_case(kind, B, n_blocks, k)
    lens = [16 * n_blocks] * B
    ids, n_sel, status, qb = _select(q, w, codes, scale, table, 16, lens, k)
    want, wn = ref.select(qb, w, codes, scale, table, 16, n_blocks, lens, k, 1, 2)
    assert status == 0 and np.array_equal(n_sel, wn)
    assert np.array_equal(ids, want)


@pytest.mark.parametrize("exponent", [-99, -101, -119, -122, -128, -131])
def test_select_tiny_queries(cuda_device, exponent):
    """Queries whose largest magnitudes are so small that 127 over them overflows, down to
    subnormals of bf16: the ids are those of the formula with both scaled by 2^100."""
    g = np.random.default_rng(exponent + 500)
    n, H, k, P = 400, 8, 12, 16
    codes, scale = _summaries(g, n)
    table = g.permutation(n).astype(np.int32)[None]
    q = torch.from_numpy((g.standard_normal((1, 1, H, 128)) * 2.0 ** exponent).astype(np.float32)).bfloat16().float().numpy()
    w = (g.random((1, 1, H)) + 0.5).astype(np.float32) * np.float32(2.0 ** 100)  # w * sq a normal number
    ids, n_sel, status, qb = _select(q, w, codes, scale, table, P, [n * P], k, n_first=0, n_last=0)
    assert np.array_equal(qb, q)
    top = np.abs(q[0, 0]).max(1)
    up = np.where(top < 2.0 ** -100, np.float32(2.0 ** 100), np.float32(1))
    inv = np.float32(127) * (np.float32(1) / (top * up))
    qi = np.rint((q[0, 0] * up[:, None]) * inv[:, None])
    assert np.abs(qi).max() == 127
    weight = (w[0, 0] * (top * (np.float32(1) / np.float32(127)))).astype(np.float64)
    dot = np.maximum(qi @ codes[table[0]].astype(np.float64).T, 0)
    score = (dot * weight[:, None]).sum(0) * scale[table[0]].astype(np.float64)
    want = np.sort(np.argsort(-score, kind="stable")[:k])
    assert status == 0 and n_sel[0, 0] == k and np.array_equal(ids[0, 0], want)
