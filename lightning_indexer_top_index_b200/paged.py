"""Paged caches: rows appended with their position rotation (4-bit, 8-bit,
bf16 or fp32), block summaries of the index keys, block selection by a cheap
score, and MQA attention over the pages (the calls on lidx_pages in
include/lidx.h).

    cache = lidx.PagedKV(lidx.DeviceKV(lidx.E2M1, 512, codes, scales, rope), table, page_rows=64)
    lidx.paged_append(x, cache, seq, row, pos, inv_freq)
    lidx.block_pool(keys, length, codes, scale, first)
    ids, n_sel = lidx.block_select(q_idx, w, codes, scale, keys.table, 64, length, k=16)
    out, lse = lidx.paged_attn(q, cache, length, blocks=ids, n_sel=n_sel)

Every call has a prepared form (`*_call`): it checks its arguments and builds
the argument struct, the workspace and the outputs once, and returns a
PagedCall that enqueues the kernels each time it is called, on the current
stream or on the one it is given.  A prepared call reads and writes the same
tensors every time (as a CUDA graph does) and keeps them alive; one prepared
call, like its workspace, serves one stream at a time.  It stays with the
tensors that a PagedKV held when it was prepared: a cache whose pool or table is
replaced by another tensor needs its calls prepared again.  Preparing waits on the
host for the current stream (unless it is being captured), so that a workspace
and outputs made there are ready for every stream.  The memory of a call that
was given a raw stream handle is the caller's to keep (with the call) until that
stream's work is done; for torch's streams the allocator is told.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import dataclasses
import functools
from typing import Optional

import torch

from . import (BF16, E2M1, E4M3, F32, LAUNCH_PDL, OP_BLOCK_POOL, OP_BLOCK_SELECT, OP_PAGED_APPEND, OP_PAGED_ATTN,
               OP_PAGED_READ, ROPE_ADJACENT, BlockPoolArgs, BlockSelectArgs, DeviceKV, LidxError, PagedAppendArgs,
               PagedAttnArgs, PagedReadArgs, PagesArgs, launch_count, lib, read_device_status, workspace_size)


def _need(cond, msg):
    if not cond:
        raise ValueError(msg)


def _on(stream, device):
    """The torch stream of `stream` (a torch stream or a raw handle)."""
    return stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=device)


def _at(device):
    """Context in which `device` is current."""
    here = device.type == "cuda" and torch.cuda.current_device() == device.index
    return contextlib.nullcontext() if here else torch.cuda.device(device)


def _scope(device, stream):
    """Context in which a one-shot call allocates and enqueues: `device` is
    current and `stream`, when given, is its stream."""
    if stream is None:
        return _at(device)
    es = contextlib.ExitStack()
    es.enter_context(_at(device))
    es.enter_context(torch.cuda.stream(_on(stream, device)))
    return es


def _tensor(name, t, dtype, device, shape=None, contiguous=True):
    _need(isinstance(t, torch.Tensor) and t.is_cuda, f"{name} must be a CUDA tensor")
    _need(t.device == device, f"{name} is on {t.device}, the call on {device}")
    _need(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None:
        _need(tuple(t.shape) == tuple(shape), f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous:
        _need(t.is_contiguous(), f"{name} must be contiguous")
    return t


@dataclasses.dataclass
class PagedKV:
    """A paged cache: row r of sequence b is row table[b][r // page_rows] *
    page_rows + r % page_rows of `rows` (a pool of pages; page_rows a power of
    two, 16 to 256)."""
    rows: DeviceKV
    table: torch.Tensor
    page_rows: int

    @staticmethod
    def empty(dtype: int, dim: int, n_pages: int, page_rows: int, table: torch.Tensor) -> "PagedKV":
        """A zeroed pool of n_pages pages on the table's device."""
        rows, dev = n_pages * page_rows, table.device
        if dtype in (F32, BF16):
            data = torch.zeros((rows, dim), dtype=torch.float32 if dtype == F32 else torch.bfloat16, device=dev)
            return PagedKV(DeviceKV(dtype, dim, data), table, page_rows)
        _need(dtype in (E4M3, E2M1), f"storage format {dtype}")
        q = dim - 64
        data = torch.zeros((rows, q if dtype == E4M3 else q // 2), dtype=torch.uint8, device=dev)
        n_scale = q // 64 if dtype == E4M3 else q // 32
        scale = torch.zeros((rows, -(-n_scale // 8) * 8 if n_scale > 2 else n_scale), dtype=torch.uint8, device=dev)
        return PagedKV(DeviceKV(dtype, dim, data, scale, torch.zeros((rows, 64), dtype=torch.bfloat16, device=dev)),
                       table, page_rows)

    @property
    def device(self) -> torch.device:
        return self.rows.data.device

    @property
    def n_pages(self) -> int:
        return self.rows.rows // self.page_rows

    def tensors(self) -> tuple:
        """Those that the cache consists of now: what a prepared call keeps alive."""
        return tuple(t for t in (self.rows.data, self.rows.scale, self.rows.rope, self.table) if t is not None)

    def args(self) -> PagesArgs:
        r, dev = self.rows, self.device
        kinds = {F32: torch.float32, BF16: torch.bfloat16, E4M3: torch.uint8, E2M1: torch.uint8}
        _need(r.dtype in kinds, f"storage format {r.dtype}")
        width = {E4M3: r.dim - 64, E2M1: (r.dim - 64) // 2}.get(r.dtype, r.dim)
        planes = [("data", r.data, kinds[r.dtype], width)]
        if r.dtype in (E4M3, E2M1):
            planes += [("scale", r.scale, torch.uint8, (r.dim - 64) // (64 if r.dtype == E4M3 else 32)),
                       ("rope", r.rope, torch.bfloat16, 64)]
        for name, t, dtype, w in planes:
            _tensor(f"the cache's {name}", t, dtype, dev, contiguous=False)
            _need(t.dim() == 2 and t.shape[0] == r.data.shape[0] and t.shape[1] >= w and t.stride(1) == 1,
                  f"the cache's {name} must be [rows][>= {w}] with adjacent columns")
        _need(r.data.shape[0] % self.page_rows == 0, "the pool's rows must be whole pages")
        ld = table_stride(self.table, dev)
        return PagesArgs(r.args(), self.page_rows, self.n_pages, self.table.data_ptr(), ld, self.table.shape[1])


def table_stride(table, device) -> int:
    _tensor("table", table, torch.int32, device, contiguous=False)
    _need(table.dim() == 2 and table.shape[1] >= 1 and (table.stride(1) == 1 or table.shape[1] == 1),
          "table must be [B][blocks] with adjacent columns")
    return table.stride(0)


class PagedCall:
    """A prepared call: calling it enqueues the kernels on the current stream
    of its device (or on `stream`) and returns its outputs."""

    def __init__(self, name, op, args, device, out, keep, ws=None):
        self.name, self.op, self.args, self.device, self.out, self._keep = name, op, args, device, out, keep
        with _at(device):
            need = workspace_size(op, args)
            if ws is None:  # only the status word has to be clear
                ws = torch.empty(max(need, 256), dtype=torch.uint8, device=device)
                ws.narrow(0, 0, 256).zero_()
        _tensor("ws", ws, torch.uint8, device)
        self.ws = ws
        self._fn, self._ref = getattr(lib(), name), C.byref(args)
        self._ws, self._bytes, self._index = ws.data_ptr(), ws.numel(), device.index
        self._known = {torch._C._cuda_getCurrentRawStream(self._index)}  # streams that the memory made here is safe on

    @functools.cached_property
    def launches(self) -> int:
        """Kernels that one call launches."""
        with _at(self.device):
            return launch_count(self.op, self.args)

    def _settle(self) -> "PagedCall":
        """Wait for the stream that the workspace and the outputs were made on."""
        with _at(self.device):
            if not torch.cuda.is_current_stream_capturing():
                torch.cuda.current_stream().synchronize()
        return self

    def _meet(self, raw, stream):
        """First call on a stream: the memory made here is not to be given away before its work is done."""
        if stream is None:
            stream = torch.cuda.current_stream()
        if hasattr(stream, "cuda_stream"):
            for t in {id(t): t for t in (self.ws, *(self.out if isinstance(self.out, tuple) else (self.out,)))}.values():
                t.record_stream(stream)
            self._known.add(raw)

    def __call__(self, stream=None):
        if torch.cuda.current_device() != self._index:
            with torch.cuda.device(self.device):
                return self(stream)
        if stream is None:
            raw = torch._C._cuda_getCurrentRawStream(self._index)
        else:
            raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        if raw not in self._known:
            self._meet(raw, stream)
        rc = self._fn(self._ref, self._ws, self._bytes, raw)
        if rc:
            raise LidxError(rc, self.name)
        return self.out

    def status(self, stream=None) -> int:
        """Synchronise the stream, return and clear the call's device status word."""
        with torch.cuda.device(self.device):
            return read_device_status(self.ws, stream)


def _prepared(build):
    """`build` makes a PagedCall for the current stream; the prepared form, for any."""
    @functools.wraps(build)
    def call(*args, **kwargs) -> PagedCall:
        return build(*args, **kwargs)._settle()
    return call


def _rows_of(seq, row, n, device):
    _tensor("seq", seq, torch.int32, device, (n,))
    _tensor("row", row, torch.int32, device, (n,))


@_prepared
def paged_append_call(x: torch.Tensor, cache: PagedKV, seq: torch.Tensor, row: torch.Tensor, pos: torch.Tensor = None,
                      inv_freq: torch.Tensor = None, pairs: int = ROPE_ADJACENT, *, ws=None, flags=0) -> PagedCall:
    """Prepared form of paged_append; calling it returns the workspace."""
    dev = cache.device
    _need(x.dim() == 2 and x.dtype in (torch.float32, torch.bfloat16), "x must be [n][dim] float32 or bfloat16")
    n, dim = x.shape
    _need(n >= 1 and dim == cache.rows.dim, f"x must be [n >= 1][{cache.rows.dim}], got {tuple(x.shape)}")
    _tensor("x", x, x.dtype, dev, contiguous=False)
    _need(x.stride(1) == 1, "x must have adjacent columns")
    _rows_of(seq, row, n, dev)
    if pos is not None:
        _tensor("pos", pos, torch.int32, dev, (n,))
    if inv_freq is not None:
        _tensor("inv_freq", inv_freq, torch.float32, dev, (32,))
    a = PagedAppendArgs(n, cache.table.shape[0], F32 if x.dtype == torch.float32 else BF16, x.data_ptr(),
                        x.stride(0) if n > 1 else dim, cache.args(), seq.data_ptr(), row.data_ptr(),
                        None if pos is None else pos.data_ptr(), None if inv_freq is None else inv_freq.data_ptr(),
                        pairs, flags)
    call = PagedCall("lidx_paged_append", OP_PAGED_APPEND, a, dev, None, (x, *cache.tensors(), seq, row, pos, inv_freq),
                     ws)
    call.out = call.ws
    return call


def paged_append(x, cache: PagedKV, seq, row, pos=None, inv_freq=None, pairs: int = ROPE_ADJACENT, *, ws=None,
                 stream=None, flags=0):
    """Append the new rows x [n][dim] (float32 or bfloat16) to a paged cache:
    rotate the last 64 dims by pos[i] * inv_freq (pos defaults to `row`; no
    rotation without inv_freq), round to the cache's format and write entry i
    to row row[i] of sequence seq[i] (seq < 0: padding, left out).  Returns
    the workspace (see read_device_status)."""
    if x.shape[0] == 0:
        return ws
    with _scope(cache.device, stream):
        return paged_append_call.__wrapped__(x, cache, seq, row, pos, inv_freq, pairs, ws=ws, flags=flags)()


@_prepared
def paged_read_call(cache: PagedKV, seq: torch.Tensor, row: torch.Tensor, dtype=torch.float32, *, out=None, ws=None,
                    flags=0) -> PagedCall:
    """Prepared form of paged_read."""
    dev, n, dim = cache.device, seq.shape[0], cache.rows.dim
    _need(n >= 1, "no rows")
    _rows_of(seq, row, n, dev)
    if out is None:
        _need(dtype in (torch.float32, torch.bfloat16), "dtype must be float32 or bfloat16")
        out = torch.zeros((n, dim), dtype=dtype, device=dev)
    _need(out.dtype in (torch.float32, torch.bfloat16), "out must be float32 or bfloat16")
    _tensor("out", out, out.dtype, dev, (n, dim), contiguous=False)
    _need(out.stride(1) == 1 and (n == 1 or out.stride(0) >= dim), "out must have adjacent columns and rows apart")
    a = PagedReadArgs(n, cache.table.shape[0], cache.args(), seq.data_ptr(), row.data_ptr(),
                      F32 if out.dtype == torch.float32 else BF16, out.data_ptr(), out.stride(0) if n > 1 else dim, flags)
    return PagedCall("lidx_paged_read", OP_PAGED_READ, a, dev, out, (*cache.tensors(), seq, row), ws)


def paged_read(cache: PagedKV, seq, row, dtype=torch.float32, *, out=None, ws=None, stream=None):
    """Rows row[i] of sequences seq[i] as the values they stand for, [n][dim]
    (an entry with seq < 0 leaves its row of `out` as it was)."""
    with _scope(cache.device, stream):
        if seq.shape[0] == 0:
            return torch.zeros((0, cache.rows.dim), dtype=dtype, device=cache.device) if out is None else out
        return paged_read_call.__wrapped__(cache, seq, row, dtype, out=out, ws=ws)()


@_prepared
def block_pool_call(keys: PagedKV, length: torch.Tensor, codes: torch.Tensor, scale: torch.Tensor,
                    first: torch.Tensor = None, *, ws=None, flags=0) -> PagedCall:
    """Prepared form of block_pool."""
    dev, B = keys.device, keys.table.shape[0]
    _tensor("length", length, torch.int32, dev, (B,))
    if first is not None:
        _tensor("first", first, torch.int32, dev, (B,))
    _tensor("codes", codes, torch.int8, dev, (keys.n_pages, 128))
    _tensor("scale", scale, torch.float32, dev, (keys.n_pages,))
    a = BlockPoolArgs(B, keys.args(), length.data_ptr(), None if first is None else first.data_ptr(), codes.data_ptr(),
                      scale.data_ptr(), flags)
    return PagedCall("lidx_block_pool", OP_BLOCK_POOL, a, dev, (codes, scale), (*keys.tensors(), length, first), ws)


def block_pool(keys: PagedKV, length, codes, scale, first=None, *, ws=None, stream=None, flags=0):
    """Summaries of the blocks of a paged index-key cache, by page: codes int8
    [n_pages][128] and scale float32 [n_pages] of the mean key over the rows
    below length[b]; only blocks with a row >= first[b] when `first` is given
    (those an append touched).  Returns (codes, scale)."""
    with _scope(keys.device, stream):
        return block_pool_call.__wrapped__(keys, length, codes, scale, first, ws=ws, flags=flags)()


@_prepared
def block_select_call(q: torch.Tensor, w: torch.Tensor, codes: torch.Tensor, scale: torch.Tensor, table: torch.Tensor,
                      page_rows: int, length: torch.Tensor, k: int, *, n_first=1, n_last=2, ids=None, n_sel=None,
                      ws=None, flags=0) -> PagedCall:
    """Prepared form of block_select."""
    _need(q.dim() == 4 and q.shape[3] == 128, "q must be [B][T][H][128]")
    dev, (B, T, H, _) = q.device, q.shape
    _tensor("q", q, torch.bfloat16, dev)
    _tensor("w", w, torch.float32, dev, (B, T, H))
    _need(codes.dim() == 2, "codes must be [n_pages][128]")
    _tensor("codes", codes, torch.int8, dev, (codes.shape[0], 128))
    _tensor("scale", scale, torch.float32, dev, (codes.shape[0],))
    ld = table_stride(table, dev)
    _need(table.shape[0] == B, f"table has {table.shape[0]} sequences, q {B}")
    _tensor("length", length, torch.int32, dev, (B,))
    if ids is None:
        ids = torch.empty((B, T, k), dtype=torch.int32, device=dev)
    if n_sel is None:
        n_sel = torch.empty((B, T), dtype=torch.int32, device=dev)
    _tensor("ids", ids, torch.int32, dev, (B, T, k))
    _tensor("n_sel", n_sel, torch.int32, dev, (B, T))
    a = BlockSelectArgs(B, T, H, k, n_first, n_last, q.data_ptr(), w.data_ptr(), codes.data_ptr(), scale.data_ptr(),
                        page_rows, codes.shape[0], table.data_ptr(), ld, table.shape[1], length.data_ptr(),
                        ids.data_ptr(), n_sel.data_ptr(), flags)
    return PagedCall("lidx_block_select", OP_BLOCK_SELECT, a, dev, (ids, n_sel), (q, w, codes, scale, table, length), ws)


def block_select(q, w, codes, scale, table, page_rows: int, length, k: int, *, n_first=1, n_last=2, ids=None,
                 n_sel=None, ws=None, stream=None, flags=0):
    """The k blocks each query attends to: q [B][T][H][128] bfloat16 (the last
    T tokens of each sequence), w [B][T][H], summaries as block_pool writes
    them.  The first n_first and last n_last blocks a query sees are always
    taken.  Returns (ids int32 [B][T][k] ascending with -1 padding, n_sel
    int32 [B][T])."""
    with _scope(q.device, stream):
        return block_select_call.__wrapped__(q, w, codes, scale, table, page_rows, length, k, n_first=n_first, n_last=n_last,
                                 ids=ids, n_sel=n_sel, ws=ws, flags=flags)()


@_prepared
def paged_attn_call(q: torch.Tensor, cache: PagedKV, length: torch.Tensor, blocks: torch.Tensor = None,
                    n_sel: torch.Tensor = None, scale: float = None, *, out=None, lse=None, ws=None,
                    flags=0) -> PagedCall:
    """Prepared form of paged_attn."""
    _need(q.dim() == 4 and q.shape[3] == 512, "q must be [B][T][H][512]")
    dev, (B, T, H, D) = q.device, q.shape
    _tensor("q", q, torch.bfloat16, dev)
    _need(cache.table.shape[0] == B, f"the cache has {cache.table.shape[0]} sequences, q {B}")
    _tensor("length", length, torch.int32, dev, (B,))
    ld = 0
    if blocks is not None:
        _tensor("blocks", blocks, torch.int32, dev)
        _need(blocks.dim() == 3 and blocks.shape[:2] == (B, T), f"blocks must be [{B}][{T}][n]")
        ld = blocks.shape[2]
    if n_sel is not None:
        _need(blocks is not None, "n_sel needs blocks")
        _tensor("n_sel", n_sel, torch.int32, dev, (B, T))
    if out is None:
        out = torch.empty((B, T, H, D), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=dev)
    _tensor("out", out, torch.bfloat16, dev, (B, T, H, D))
    _tensor("lse", lse, torch.float32, dev, (B, T, H))
    a = PagedAttnArgs(B, T, H, q.data_ptr(), cache.args(), length.data_ptr(),
                      None if blocks is None else blocks.data_ptr(), ld, ld,
                      None if n_sel is None else n_sel.data_ptr(), float(D ** -0.5 if scale is None else scale),
                      out.data_ptr(), lse.data_ptr(), flags)
    return PagedCall("lidx_paged_attn", OP_PAGED_ATTN, a, dev, (out, lse),
                     (q, *cache.tensors(), length, blocks, n_sel), ws)


def paged_attn(q, cache: PagedKV, length, blocks=None, n_sel=None, scale: float = None, *, out=None, lse=None, ws=None,
               stream=None, flags=0):
    """MQA attention of q [B][T][H][512] (bfloat16; the last T tokens of each
    sequence) over rows r < length[b] - (T - 1 - t) of a paged cache, or over
    those in the blocks [B][T][n] (-1 skipped; the first n_sel[b][t] when
    given).  Returns (out bfloat16 [B][T][H][512], lse float32 [B][T][H])."""
    with _scope(q.device, stream):
        return paged_attn_call.__wrapped__(q, cache, length, blocks, n_sel, scale, out=out, lse=lse, ws=ws, flags=flags)()


class PagedLayer:
    """One layer's decode step over paged caches: the step's T new rows and
    index keys of each of B sequences are appended with their rotation, the
    blocks they fall in are summed up again, each query's blocks are chosen by
    their summaries, and attention reads the rows of those blocks.

    The step owns its inputs and outputs; `set_inputs` copies a step's data
    in, `enqueue` issues the five calls, `capture` records them as a CUDA
    graph that `replay` launches.  rows: PagedKV of dim 512; keys: PagedKV of
    dim 128 on the same table; H index heads and as many attention heads, up to
    64.  Every sequence takes part in a step: a batch with idle ones, or with
    other counts of heads, uses the calls themselves."""

    def __init__(self, rows: PagedKV, keys: PagedKV, H: int, k: int, T: int = 1, *, n_first: int = 1, n_last: int = 2,
                 inv_freq: torch.Tensor = None, pairs: int = ROPE_ADJACENT, scale: float = None, pdl: bool = True):
        a, b = rows.table, keys.table
        _need(rows.page_rows == keys.page_rows and rows.n_pages == keys.n_pages and a.device == b.device and
              a.data_ptr() == b.data_ptr() and a.shape == b.shape and a.stride() == b.stride(),
              "rows and keys must share pages and table")
        dev, B = rows.device, rows.table.shape[0]
        self.rows, self.keys, self.B, self.T = rows, keys, B, T
        flags = LAUNCH_PDL if pdl else 0  # every paged call waits for its predecessor before it reads anything

        def buf(*shape, dtype=torch.bfloat16):
            return torch.zeros(shape, dtype=dtype, device=dev)

        i32, f32 = torch.int32, torch.float32
        self.x_rows, self.x_keys = buf(B * T, 512), buf(B * T, 128)
        self.seq = torch.arange(B, dtype=i32, device=dev).repeat_interleave(T)
        self.row, self.pos = buf(B * T, dtype=i32), buf(B * T, dtype=i32)
        self.length, self.first = buf(B, dtype=i32), buf(B, dtype=i32)
        self.q_idx, self.w, self.q_attn = buf(B, T, H, 128), buf(B, T, H, dtype=f32), buf(B, T, H, 512)
        self.codes, self.scale = buf(keys.n_pages, 128, dtype=torch.int8), buf(keys.n_pages, dtype=f32)
        self._calls = [
            paged_append_call(self.x_rows, rows, self.seq, self.row, self.pos, inv_freq, pairs, flags=flags),
            paged_append_call(self.x_keys, keys, self.seq, self.row, self.pos, inv_freq, pairs, flags=flags),
            block_pool_call(keys, self.length, self.codes, self.scale, self.first, flags=flags),
            block_select_call(self.q_idx, self.w, self.codes, self.scale, keys.table, keys.page_rows, self.length, k,
                              n_first=n_first, n_last=n_last, flags=flags)]
        self.ids, self.n_sel = self._calls[3].out
        self._calls.append(paged_attn_call(self.q_attn, rows, self.length, self.ids, self.n_sel, scale, flags=flags))
        self.out, self.lse = self._calls[4].out
        self.graph: Optional[torch.cuda.CUDAGraph] = None

    def set_inputs(self, x_rows, x_keys, q_idx, w, q_attn, length, pos=None, non_blocking=True):
        """One step's data (host pinned or device): the new rows [B*T][512] and
        keys [B*T][128], the queries, the rows each sequence held before this
        step (length, int32 [B]) and the rotary positions (default: the rows)."""
        T, pos_in = self.T, () if pos is None else (("pos", self.pos, pos),)
        given = (("x_rows", self.x_rows, x_rows), ("x_keys", self.x_keys, x_keys), ("q_idx", self.q_idx, q_idx),
                 ("w", self.w, w), ("q_attn", self.q_attn, q_attn), ("length", self.first, length))
        for name, dst, src in (*given, *pos_in):  # a copy would spread a smaller one over the batch
            _need(src.shape == dst.shape, f"{name} must be {tuple(dst.shape)}, got {tuple(src.shape)}")
        for _, dst, src in given:
            dst.copy_(src, non_blocking=non_blocking)
        torch.add(self.first, T, out=self.length)
        at = self.first.unsqueeze(1) + torch.arange(T, dtype=torch.int32, device=self.first.device)
        self.row.copy_(at.reshape(-1))
        self.pos.copy_(self.row if pos is None else pos, non_blocking=non_blocking)

    def summarise(self, length):
        """Sum up every block of the rows already held (after a prefill that
        appended them by paged_append)."""
        return block_pool(self.keys, length, self.codes, self.scale)

    def enqueue(self, stream=None):
        for call in self._calls:
            call(stream)
        return self.out, self.lse

    def capture(self) -> torch.cuda.CUDAGraph:
        """Record one step into a CUDA graph (the library calls only).  The
        call enqueues one step outside capture first."""
        with torch.cuda.device(self.rows.device):
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                self.enqueue(s)
            torch.cuda.current_stream().wait_stream(s)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                self.enqueue()
        self.graph = g
        return g

    def replay(self):
        if self.graph is None:
            self.capture()
        self.graph.replay()
        return self.out, self.lse

    def kernel_launches(self) -> int:
        return sum(c.launches for c in self._calls)

    def status(self) -> int:
        """The OR of the calls' device status words (synchronises, clears them)."""
        s = 0
        for c in self._calls:
            s |= c.status()
        return s
