"""Cases of the paged-cache operators: appending rows with the position
rotation (and reading them back), block summaries of the index keys, block
selection by a cheap score, and attention over a paged cache in 4 bits.

`run` computes a case in plain torch operations, or, where `own` is true, by
the library's calls.  A cache is a pool of pages of `page` rows; block j of
sequence b lies in page table[b][j].  A 512-wide row holds 448 values in 4 or
8 bits (a power-of-two scale per 32 or 64 of them) and 64 bf16 RoPE values; a
128-wide index key holds 64 and 64.
"""
import random

import torch

own = False

ROPE = 64
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- the cases
def listed():
    return [
        # one decode step of 64 sequences: a new compressed row each, at far positions
        dict(name="append-decode-64", op="append", B=64, new=1, dim=512, fmt="e2m1", x="bf16", page=64, far=500000),
        # a chunk of prefill of five ragged sequences, projections in fp32
        dict(name="append-prefill-20k", op="append", B=5, new=4003, dim=512, fmt="e2m1", x="f32", page=64, far=65536),
        # index keys of a prefill chunk, in 8 bits
        dict(name="append-index-32k", op="append", B=8, new=4096, dim=128, fmt="e4m3", x="bf16", page=32, far=131072),
        # after a decode step: the last block of each of 64 sequences is summed up again
        dict(name="pool-decode-64", op="pool", B=64, rows=1954, tail=1, fmt="e4m3", page=64),
        # after prefill: every block of four sequences of 500K tokens (125000 entries each)
        dict(name="pool-500k-b4", op="pool", B=4, rows=125000, tail=0, fmt="e4m3", page=64),
        # block choice of one decode token at 500K tokens
        dict(name="select-500k", op="select", B=1, T=1, H=64, rows=125000, page=64, k=16),
        # block choice of 32 ragged sequences of up to 128K tokens
        dict(name="select-128k-b32", op="select", B=32, T=1, H=64, rows=32768, page=64, k=16),
        # block choice of every query of a prefill chunk, causal
        dict(name="select-prefill-512", op="select", B=1, T=512, H=64, rows=16384, page=64, k=16),
        # one decode token over every row of a 64K-token cache
        dict(name="attend-64k", op="attend", B=1, T=1, H=64, rows=16384, fmt="e2m1", page=64, k=0),
        # 32 ragged sequences, every row of up to 32K tokens
        dict(name="attend-32k-b32", op="attend", B=32, T=1, H=64, rows=8191, fmt="e2m1", page=64, k=0),
        # 32 ragged sequences of up to 128K tokens, 16 chosen blocks each
        dict(name="attend-blocks-b32", op="attend", B=32, T=1, H=64, rows=32768, fmt="e2m1", page=64, k=16),
        # a prefill chunk of 256 queries, each with its own 16 blocks
        dict(name="attend-blocks-prefill", op="attend", B=1, T=256, H=64, rows=16384, fmt="e2m1", page=64, k=16),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(("append", "pool", "select", "attend"))
    page = rng.choice((16, 32, 64, 128))
    if op == "append":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, new=max(1, _log(rng, 1, 20000) // B), dim=rng.choice((512, 512, 128)),
                    fmt=rng.choice(("e2m1", "e2m1", "e4m3", "bf16")), x=rng.choice(("bf16", "f32")), page=page,
                    far=_log(rng, 1000, 500000))
    if op == "pool":
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, rows=max(1, _log(rng, 64, 400000) // B), tail=rng.choice((0, 1)),
                    fmt=rng.choice(("e4m3", "bf16", "e2m1")), page=page)
    if op == "select":
        B = _log(rng, 1, 32)
        T = rng.choice((1, 1, 2, 4, _log(rng, 5, 256)))
        return dict(op=op, B=B, T=T, H=rng.choice((8, 24, 32, 64)), rows=max(T, _log(rng, 500, 1000000) // (B * T)), page=page,
                    k=_log(rng, 4, 48))
    B = _log(rng, 1, 32)
    H, fmt = rng.choice((16, 40, 64, 64)), rng.choice(("e2m1", "e2m1", "e2m1", "e4m3", "bf16"))
    if rng.random() < 0.5:
        T = rng.choice((1, 1, 2, 4))
        return dict(op=op, B=B, T=T, H=H, rows=max(T, _log(rng, 64, 120000) // (B * T)), fmt=fmt, page=page, k=0)
    T = rng.choice((1, 1, 3, max(1, _log(rng, 8, 128) // B)))
    return dict(op=op, B=B, T=T, H=H, rows=max(T, _log(rng, 500, 60000)), fmt=fmt, page=page,
                k=_log(rng, 2, max(2, 1024 // page)))


def _lens(c):
    """Cache rows of each sequence: ragged, the first one full, now and then an empty slot of the batch."""
    r = random.Random("%d %d %d" % (c["B"], c.get("rows", 0), c["page"]))
    got = [c["rows"]]
    for _ in range(c["B"] - 1):
        u = r.random()
        got.append(0 if u < 0.05 else max(c.get("T", 1), int(c["rows"] * (0.25 + 0.75 * r.random()))))
    return got


def _new_rows(c):
    """New rows of each sequence of an append (ragged where there are many)."""
    r = random.Random("%d %d" % (c["B"], c["new"]))
    return [c["new"] if c["new"] == 1 else max(1, int(c["new"] * (0.5 + r.random()))) for _ in range(c["B"])]


def _stored(fmt, dim):
    """Bytes of one stored row."""
    q = dim - ROPE
    return {"e2m1": q // 2 + q // 32 + 2 * ROPE, "e4m3": q + q // 64 + 2 * ROPE, "bf16": 2 * dim}[fmt]


# ----------------------------------------------------- the format, plain form
def _quantise(x, fmt):
    """fp32 [n][m] -> (codes uint8, scale bytes), in 64 bits where values lie next to a border."""
    n, m = x.shape
    blk = 32 if fmt == "e2m1" else 64
    v = x.double().reshape(n, m // blk, blk)
    amax = v.abs().amax(-1)
    f, ex = torch.frexp(amax)
    if fmt == "e2m1":  # smallest e with amax <= 6 * 2^e = 0.75 * 2^(e + 3)
        e = torch.where(f <= 0.75, ex - 3, ex - 2)
    else:  # smallest e with amax <= 448 * 2^e = 0.875 * 2^(e + 9)
        e = torch.where(f <= 0.875, ex - 9, ex - 8)
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))
    y = torch.ldexp(v, -e.unsqueeze(-1).double())
    scale = (e + 127).to(torch.uint8)
    if fmt == "e4m3":
        return y.float().to(torch.float8_e4m3fn).view(torch.uint8).reshape(n, m), scale
    a = y.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    code = (code | (torch.signbit(y).to(torch.uint8) << 3)).reshape(n, m // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), scale


def _dequantise(data, scale, rope, fmt):
    """Stored rows -> fp32 [n][dim]."""
    if fmt == "bf16":
        return data.float()
    n = data.shape[0]
    if fmt == "e2m1":
        table = torch.tensor(E2M1 + tuple(-t for t in E2M1), device=data.device)
        v = torch.stack((table[(data & 15).int()], table[(data >> 4).int()]), -1).reshape(n, -1, 32)
    else:
        v = data.view(torch.float8_e4m3fn).float().reshape(n, -1, 64)
    s = torch.exp2(scale[:, : v.shape[1]].float() - 127.0)
    return torch.cat(((v * s.unsqueeze(-1)).reshape(n, -1), rope.float()), 1)


def _rotate(x, pos, inv_freq):
    """Neighbouring pairs of the last 64 values turned by pos * inv_freq."""
    ang = pos.double().unsqueeze(1) * inv_freq.double()
    c, s = torch.cos(ang), torch.sin(ang)
    p = x[:, -ROPE:].double().reshape(-1, ROPE // 2, 2)
    return torch.stack((p[..., 0] * c - p[..., 1] * s, p[..., 0] * s + p[..., 1] * c), -1).reshape(-1, ROPE)


# ------------------------------------------------------------------- prepare
def _planes(rows, dim, fmt):
    """Empty planes of a pool of `rows` rows."""
    if fmt == "bf16":
        return dict(data=torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda"), scale=None, rope=None)
    q = dim - ROPE
    return dict(data=torch.zeros(rows, q // 2 if fmt == "e2m1" else q, dtype=torch.uint8, device="cuda"),
                scale=torch.zeros(rows, 16 if dim == 512 else 2, dtype=torch.uint8, device="cuda"),
                rope=torch.zeros(rows, ROPE, dtype=torch.bfloat16, device="cuda"))


def _filled(g, rows, dim, fmt):
    """A pool whose rows hold values of a few neighbouring scales, as projected and normalised keys do."""
    p = _planes(rows, dim, fmt)
    for at in range(0, rows, 65536):
        n = min(65536, rows - at)
        x = torch.randn(n, dim, generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(n, 1, generator=g, device="cuda"))
        if fmt == "bf16":
            p["data"][at:at + n] = x.bfloat16()
            continue
        code, scale = _quantise(x[:, :-ROPE], fmt)
        p["data"][at:at + n] = code
        p["scale"][at:at + n, : scale.shape[1]] = scale
        p["rope"][at:at + n] = x[:, -ROPE:].bfloat16()
    return p


def _table(seed, lens, page):
    """Pages of the sequences' blocks, scattered over the pool; -1 behind a sequence's last block."""
    need = [-(-n // page) for n in lens]
    pages = list(range(sum(need) + 3))
    random.Random(seed).shuffle(pages)
    table = torch.full((len(lens), max(max(need), 1)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = torch.tensor(pages[at:at + m], dtype=torch.int32)
        at += m
    return table.cuda(), len(pages)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "append":
        new = _new_rows(c)
        r = random.Random(seed)
        first = [r.randrange(0, 2 * c["page"]) for _ in new]  # rows that the sequence holds already
        s["table"], pages = _table(seed, [f + n for f, n in zip(first, new)], c["page"])
        s.update(_planes(pages * c["page"], c["dim"], c["fmt"]))
        seq = [b for b, n in enumerate(new) for _ in range(n)]
        row = [f + i for f, n in zip(first, new) for i in range(n)]
        at = [r.randrange(0, c["far"]) for _ in new]
        pos = [p + i for p, n in zip(at, new) for i in range(n)]
        s["seq"], s["row"], s["pos"] = (torch.tensor(v, dtype=torch.int32).cuda() for v in (seq, row, pos))
        x = torch.randn(len(seq), c["dim"], generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(len(seq), 1, generator=g, device="cuda"))
        s["x"] = x.bfloat16() if c["x"] == "bf16" else x
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64) / ROPE)).float().cuda()
        return s
    lens = _lens(c)
    s["len"] = torch.tensor(lens, dtype=torch.int32).cuda()
    s["table"], pages = _table(seed, lens, c["page"])
    if c["op"] == "pool":
        s.update(_filled(g, pages * c["page"], 128, c["fmt"]))
        s["first"] = (s["len"] - 1).clamp(min=0) if c["tail"] else None  # one row came in, or all of them
        s["codes"] = torch.zeros(pages, 128, dtype=torch.int8, device="cuda")
        s["code_scale"] = torch.zeros(pages, dtype=torch.float32, device="cuda")
        return s
    B, T, H = c["B"], c["T"], c["H"]
    if c["op"] == "select":
        s["q"] = torch.randn(B, T, H, 128, generator=g, device="cuda").bfloat16()
        s["w"] = torch.rand(B, T, H, generator=g, device="cuda") - 0.25
        mean = torch.randn(pages, 128, generator=g, device="cuda")
        top = mean.abs().amax(1)
        s["codes"] = torch.round(mean * (127.0 / top).unsqueeze(1)).to(torch.int8)
        s["code_scale"] = top / 127.0 * 0.125
        return s
    s.update(_filled(g, pages * c["page"], 512, c["fmt"]))
    s["q"] = (2.0 * torch.randn(B, T, H, 512, generator=g, device="cuda")).bfloat16()
    s["blocks"] = None
    if c["k"]:  # chosen blocks of each query, ascending, -1 behind them
        nb = -(-(s["len"].long().unsqueeze(1) - T + 1 + torch.arange(T, device="cuda")).clamp(min=0) // c["page"])
        width = s["table"].shape[1]
        u = torch.rand(B, T, width, generator=g, device="cuda")
        u[torch.arange(width, device="cuda") >= nb.unsqueeze(-1)] = 2.0
        u.scatter_(2, (nb - 1).clamp(min=0).unsqueeze(-1), 0.0)  # the last block is always chosen
        u.masked_fill_((nb == 0).unsqueeze(-1), 2.0)
        k = min(c["k"], width)
        v, i = torch.topk(u, k, dim=2, largest=False)
        i = torch.where(v < 2.0, i, torch.full_like(i, width)).sort(dim=2).values
        i = torch.where(i < width, i, torch.full_like(i, -1))
        s["blocks"] = torch.full((B, T, c["k"]), -1, dtype=torch.int32, device="cuda")
        s["blocks"][:, :, :k] = i.int()
    return s


# ----------------------------------------------------------------------- run
def run(s):
    return {"append": _append, "pool": _pool, "select": _select, "attend": _attend}[s["case"]["op"]](s)


def _paged(lidx, s, dim, fmt):
    kind = {"e2m1": lidx.E2M1, "e4m3": lidx.E4M3, "bf16": lidx.BF16}[fmt]
    return lidx.PagedKV(lidx.DeviceKV(kind, dim, s["data"], s["scale"], s["rope"]), s["table"], s["case"]["page"])


def _flat(s, seq, row):
    """Pool rows of rows `row` of sequences `seq`."""
    page = s["case"]["page"]
    return s["table"][seq.long(), (row // page).long()].long() * page + row % page


def _append(s):
    """New rows go into the cache, rotated and rounded, and are read back as the values that it then holds."""
    c = s["case"]
    if own:
        if "calls" not in s:
            import lightning_indexer_top_index_b200 as lidx
            cache = _paged(lidx, s, c["dim"], c["fmt"])
            s["calls"] = (lidx.paged_append_call(s["x"], cache, s["seq"], s["row"], s["pos"], s["inv_freq"]),
                          lidx.paged_read_call(cache, s["seq"], s["row"], dtype=torch.bfloat16))
        s["calls"][0]()
        return s["calls"][1]()
    at = _flat(s, s["seq"], s["row"])
    rot = _rotate(s["x"], s["pos"], s["inv_freq"]).bfloat16()
    if c["fmt"] == "bf16":
        s["data"][at] = torch.cat((s["x"][:, :-ROPE].bfloat16(), rot), 1)
        return s["data"][at]
    code, scale = _quantise(s["x"][:, :-ROPE].float(), c["fmt"])
    s["data"][at] = code
    s["scale"][at, : scale.shape[1]] = scale
    s["rope"][at] = rot
    return _dequantise(s["data"][at], s["scale"][at], s["rope"][at], c["fmt"]).bfloat16()


def _pool(s):
    """Summary of each block that holds new rows: the mean key as 8-bit codes and a scale, kept by page."""
    c = s["case"]
    page = c["page"]
    if own:
        if "call" not in s:
            import lightning_indexer_top_index_b200 as lidx
            s["call"] = lidx.block_pool_call(_paged(lidx, s, 128, c["fmt"]), s["len"], s["codes"], s["code_scale"], s["first"])
        return s["call"]()
    j = torch.arange(s["table"].shape[1], device="cuda")
    first = s["first"].unsqueeze(1) if s["first"] is not None else 0
    need = (j * page < s["len"].unsqueeze(1)) & ((j + 1) * page > first)
    b, j = need.nonzero(as_tuple=True)
    p = s["table"][b, j].long()
    count = (s["len"][b].long() - j * page).clamp(max=page)
    at = (p.unsqueeze(1) * page + torch.arange(page, device="cuda")).reshape(-1)
    some = [s[n][at] if s[n] is not None else None for n in ("data", "scale", "rope")]
    rows = _dequantise(*some, c["fmt"]).reshape(-1, page, 128).double()
    rows = torch.where((torch.arange(page, device="cuda") < count.unsqueeze(1)).unsqueeze(-1), rows, torch.zeros_like(rows))
    mean = rows.sum(1) / count.unsqueeze(1)
    scale = (mean.abs().amax(1) / 127.0).float()
    code = torch.round(mean / torch.where(scale > 0, scale, torch.ones_like(scale)).double().unsqueeze(1)).clamp(-127, 127)
    s["codes"][p] = code.to(torch.int8)
    s["code_scale"][p] = scale
    return s["codes"], s["code_scale"]


def _visible(s):
    """Rows that query t of each sequence sees: all that came before it, and its own."""
    T = s["case"]["T"]
    return (s["len"].long().unsqueeze(1) - (T - 1) + torch.arange(T, device="cuda")).clamp(min=0)


FIRST, LAST = 1, 2  # blocks at either end that are always chosen


def _select(s):
    """Ids of the k blocks with the largest score, the first one and the last two always among them."""
    c = s["case"]
    if own:
        if "call" not in s:
            import lightning_indexer_top_index_b200 as lidx
            s["call"] = lidx.block_select_call(s["q"], s["w"], s["codes"], s["code_scale"], s["table"], c["page"], s["len"], c["k"],
                                               n_first=FIRST, n_last=LAST)
        return s["call"]()
    B, T, H, k = c["B"], c["T"], c["H"], c["k"]
    width = s["table"].shape[1]
    q = s["q"].float()
    top = q.abs().amax(-1)
    sq = top / 127.0
    qi = torch.round(q * torch.where(top > 0, 127.0 / top, torch.zeros_like(top)).unsqueeze(-1))
    p = s["table"].clamp(min=0).long()
    dot = torch.matmul(qi.reshape(B, T * H, 128), s["codes"][p].float().transpose(1, 2))  # whole numbers below 2^24
    weight = (s["w"] * sq).double().unsqueeze(-1)
    score = (dot.clamp(min=0).reshape(B, T, H, width).double() * weight).sum(2) * s["code_scale"][p].double().unsqueeze(1)
    nb = ((_visible(s) + c["page"] - 1) // c["page"]).unsqueeze(-1)
    j = torch.arange(width, device="cuda")
    score = torch.where((j < FIRST) | (j >= nb - LAST), torch.full_like(score, float("inf")), score)
    score = torch.where(j < nb, score, torch.full_like(score, float("-inf")))
    n = nb.squeeze(-1).clamp(max=k)
    order = torch.sort(score, dim=2, descending=True, stable=True).indices[:, :, :k]
    keep = torch.arange(order.shape[2], device="cuda") < n.unsqueeze(-1)
    order = torch.where(keep, order, torch.full_like(order, width)).sort(dim=2).values
    ids = torch.full((B, T, k), -1, dtype=torch.int32, device="cuda")
    ids[:, :, : order.shape[2]] = torch.where(order < width, order, torch.full_like(order, -1)).int()
    return ids, n.int()


def _attend(s):
    """Attention of each query over the rows that it sees, or over those of its chosen blocks: out in bf16, and the log of the sums."""
    c = s["case"]
    B, T, H, page = c["B"], c["T"], c["H"], c["page"]
    if own:
        if "call" not in s:
            import lightning_indexer_top_index_b200 as lidx
            s["call"] = lidx.paged_attn_call(s["q"], _paged(lidx, s, 512, c["fmt"]), s["len"], blocks=s["blocks"], scale=512 ** -0.5)
        return s["call"]()
    seen = _visible(s).unsqueeze(-1)
    if s["blocks"] is None:
        j = torch.arange(s["table"].shape[1], device="cuda").expand(B, 1, -1)
    else:
        j = s["blocks"].long()
    row = (j.unsqueeze(-1) * page + torch.arange(page, device="cuda")).reshape(B, j.shape[1], -1)
    there = (row < seen) & (row >= 0)  # [B][T][rows]
    p = torch.gather(s["table"].long(), 1, j.clamp(min=0).reshape(B, -1)).clamp(min=0).reshape(j.shape)
    at = (p.unsqueeze(-1) * page + torch.arange(page, device="cuda")).reshape(-1)
    some = [s[n][at] if s[n] is not None else None for n in ("data", "scale", "rope")]
    x = _dequantise(*some, c["fmt"]).reshape(B, j.shape[1], -1, 512)
    q = s["q"].float()
    if x.shape[1] == T:
        q, x = q.reshape(B * T, H, 512), x.reshape(B * T, -1, 512)
    else:
        q, x = q.reshape(B, T * H, 512), x.reshape(B, -1, 512)
    logit = torch.matmul(q, x.transpose(1, 2)).reshape(B, T, H, -1) * 512 ** -0.5
    logit = torch.where(there.unsqueeze(2), logit, torch.full_like(logit, float("-inf")))
    top = logit.amax(-1, keepdim=True)
    top = torch.where(top > float("-inf"), top, torch.zeros_like(top))
    e = torch.exp(logit - top)
    total = e.sum(-1, keepdim=True)
    prob = e / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.matmul(prob.reshape(q.shape[0], q.shape[1], -1), x).reshape(B, T, H, 512)
    return out.bfloat16(), (torch.log(total) + top).squeeze(-1)


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "append":
        n = sum(_new_rows(c))
        per = c["dim"] * (2 if c["x"] == "bf16" else 4) + 2 * _stored(c["fmt"], c["dim"]) + 2 * c["dim"] + 16
        return {"bytes": n * per, "flops": n * (3 * ROPE + 4 * c["dim"])}
    lens, page = _lens(c), c["page"]
    if c["op"] == "pool":
        rows = sum(((n - 1) % page + 1 if n else 0) if c["tail"] else n for n in lens)
        blocks = sum((n > 0) if c["tail"] else -(-n // page) for n in lens)
        return {"bytes": rows * _stored(c["fmt"], 128) + blocks * 136, "flops": rows * 128 * 2}
    B, T, H = c["B"], c["T"], c["H"]
    blocks = sum(-(-n // page) for n in lens)
    if c["op"] == "select":
        seen = sum(-(-max(0, n - T + 1 + t) // page) for n in lens for t in range(T))
        return {"bytes": blocks * 136 + B * T * (H * 260 + 4 * c["k"]), "flops": 2.0 * seen * H * 128}
    seen = sum(max(0, n - T + 1 + t) if not c["k"] else min(c["k"] * page, max(0, n - T + 1 + t)) for n in lens for t in range(T))
    read = min(sum(lens), seen)
    return {"bytes": read * _stored(c["fmt"], 512) + B * T * H * (2 * 1024 + 4) + 4 * (B * T * c["k"] if c["k"] else blocks),
            "flops": 4.0 * seen * H * 512}


# --------------------------------------------------------------------- exact
def _grid(fmt):
    """The non-negative values of a format, in the order of their codes."""
    if fmt == "e2m1":
        return torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    codes = torch.arange(127, device="cuda")
    e, m = codes // 8, (codes % 8).double()
    return torch.where(e > 0, (8 + m) * torch.exp2(e.double() - 10), m * 2.0 ** -9)


def _stands_for(v, fmt):
    """64-bit [n][m] -> the nearest values that the format holds under its scales."""
    blk, top = (32, 6.0) if fmt == "e2m1" else (64, 448.0)
    y = v.reshape(v.shape[0], -1, blk)
    amax = y.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, top)) / top))
    e = torch.where(amax > top * torch.exp2(e), e + 1, e)
    e = torch.where(amax <= top * torch.exp2(e - 1), torch.where(amax > 0, e - 1, e), e).clamp(-127, 127)
    grid = _grid(fmt)
    a = (y * torch.exp2(-e)).abs()
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    near = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])
    return (torch.copysign(near, y) * torch.exp2(e)).reshape(v.shape)


def _held(s, at, fmt):
    """Pool rows `at` as 64-bit values."""
    if fmt == "bf16":
        return s["data"][at].double()
    data, grid = s["data"][at], _grid(fmt)
    if fmt == "e2m1":
        code = torch.empty(data.shape[0], 2 * data.shape[1], dtype=torch.int64, device="cuda")
        code[:, 0::2], code[:, 1::2] = (data % 16).long(), (data // 16).long()
        v, blk = torch.where(code >= 8, -grid[code % 8], grid[code % 8]), 32
    else:
        code = data.long()
        v, blk = torch.where(code >= 128, -grid[(code % 128).clamp(max=126)], grid[(code % 128).clamp(max=126)]), 64
    e = s["scale"][at][:, : v.shape[1] // blk].double() - 127
    return torch.cat((v * torch.exp2(e).repeat_interleave(blk, dim=1), s["rope"][at].double()), 1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    page = c["page"]
    if c["op"] == "append":
        x = s["x"].double()
        ang = torch.outer(s["pos"].double(), s["inv_freq"].double())
        z = torch.complex(x[:, -ROPE::2], x[:, -ROPE + 1::2]) * torch.polar(torch.ones_like(ang), ang)
        body = x[:, :-ROPE] if c["fmt"] == "bf16" else _stands_for(x[:, :-ROPE], c["fmt"])
        return torch.cat((body, torch.view_as_real(z).reshape(-1, ROPE)), 1)
    lens = s["len"].tolist()
    if c["op"] == "pool":
        codes, scales = torch.zeros_like(s["codes"]), torch.zeros(s["codes"].shape[0], dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            nb = -(-n // page)
            if nb == 0:
                continue
            j0 = nb - 1 if c["tail"] else 0
            p = s["table"][b, j0:nb].long()
            v = _held(s, (p.unsqueeze(1) * page + torch.arange(page, device="cuda")).reshape(-1), c["fmt"]).reshape(nb - j0, page, 128)
            ends = torch.full((nb - j0,), page, device="cuda")
            ends[-1] = n - (nb - 1) * page
            v[torch.arange(page, device="cuda") >= ends.unsqueeze(1)] = 0
            scales[p] = (v.sum(1) / ends.unsqueeze(1)).abs().amax(1) / 127
        return None, scales
    if c["op"] == "select":
        return None
    B, T, H = c["B"], c["T"], c["H"]
    out = torch.zeros(B, T, H, 512, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), float("-inf"), dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        held = None
        for t in range(T):
            seen = n - (T - 1 - t)
            if seen <= 0:
                continue
            if s["blocks"] is None:
                if held is None:
                    r = torch.arange(n, device="cuda")
                    held = _held(s, s["table"][b, r // page].long() * page + r % page, c["fmt"])
                x = held[:seen]
            else:
                j = s["blocks"][b, t]
                r = (j[j >= 0].long().unsqueeze(1) * page + torch.arange(page, device="cuda")).reshape(-1)
                r = r[r < seen]
                x = _held(s, s["table"][b, r // page].long() * page + r % page, c["fmt"])
            logit = s["q"][b, t].double() @ x.T / 512 ** 0.5
            lse[b, t] = torch.logsumexp(logit, -1)
            out[b, t] = torch.softmax(logit, -1) @ x
    return out, lse
