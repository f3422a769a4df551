"""Plain 64-bit forms of the paged-cache calls (numpy), from the formulas in
include/lidx.h.  A cache is decoded to float64 values [pool rows][dim]."""
import numpy as np

import oracle

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def bf16_value(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def decode(data, scale, rope, fmt, dim):
    """Planes (data: f32 | bf16 bits uint16 | uint8 codes) -> float64 [n][dim]."""
    if fmt == "f32":
        return np.asarray(data, np.float64)
    if fmt == "bf16":
        return bf16_value(data)
    q = dim - 64
    if fmt == "e4m3":
        table = np.array([oracle.decode_e4m3(c) for c in range(256)])
        v = table[data[:, :q]]
        blk = 64
    else:
        v = np.empty((data.shape[0], q))
        codes = data[:, : q // 2]
        for half in (0, 1):
            c = (codes >> (4 * half)) & 15
            v[:, half::2] = np.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])
        blk = 32
    e = scale[:, : q // blk].astype(np.float64)
    s = np.where(e == 255, np.nan, np.exp2(e - 127))
    return np.concatenate([v * np.repeat(s, blk, axis=1), bf16_value(rope[:, :64])], axis=1)


def encode_e2m1(x):
    """Finite-or-not float64 [n][m] -> (packed codes, scale bytes)."""
    n, m = x.shape
    codes, scale = np.zeros((n, m), np.uint8), np.zeros((n, m // 32), np.uint8)
    for i in range(n):
        for j in range(m // 32):
            v = x[i, 32 * j: 32 * j + 32]
            fin = np.abs(v[np.isfinite(v)])
            amax = fin.max() if fin.size else 0.0
            e = 0
            if amax > 0:
                e = -127
                while e < 127 and amax > 6.0 * 2.0 ** e:
                    e += 1
            scale[i, j] = e + 127
            for d in range(32):
                y = v[d] * 2.0 ** -e if not np.isnan(v[d]) else np.nan
                if np.isnan(y):
                    c = 7
                elif abs(y) >= 6:
                    c = 7
                else:
                    dist = np.abs(E2M1 - abs(y))
                    best = np.flatnonzero(dist == dist.min())
                    c = int(best[0]) if len(best) == 1 else int(best[best % 2 == 0][0])
                codes[i, 32 * j + d] = c | (8 if np.signbit(v[d]) and not np.isnan(v[d]) else 0)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scale


def rotate(x, pos, inv_freq, pairs):
    """Rotated last 64 dims of x (float64), pairs 0 = adjacent, 1 = halves."""
    p = x[:, -64:]
    a = np.outer(np.asarray(pos, np.float64), np.asarray(inv_freq, np.float64))
    c, s = np.cos(a), np.sin(a)
    u, v = (p[:, 0::2], p[:, 1::2]) if pairs == 0 else (p[:, :32], p[:, 32:])
    out = np.empty_like(p)
    ru, rv = u * c - v * s, u * s + v * c
    if pairs == 0:
        out[:, 0::2], out[:, 1::2] = ru, rv
    else:
        out[:, :32], out[:, 32:] = ru, rv
    mag = np.empty_like(p)
    if pairs == 0:
        mag[:, 0::2] = mag[:, 1::2] = np.abs(u) + np.abs(v)
    else:
        mag[:, :32] = mag[:, 32:] = np.abs(u) + np.abs(v)
    return out, mag


def pool(values, table, page_rows, n_pages, length, first=None):
    """{page: (codes int8 [128], scale float32)} of the blocks that are summed up."""
    got = {}
    for b, n in enumerate(length):
        n = min(max(int(n), 0), table.shape[1] * page_rows)
        f = 0 if first is None else max(int(first[b]), 0)
        if f >= n:
            continue
        for j in range(f // page_rows, -(-n // page_rows)):
            p = int(table[b, j])
            if p < 0 or p >= n_pages:
                continue
            rows = values[p * page_rows: p * page_rows + min(page_rows, n - j * page_rows)]
            with np.errstate(all="ignore"):
                mean = rows.sum(0) / rows.shape[0]
            if not np.isfinite(rows).all():
                got[p] = (np.zeros(128, np.int8), np.float32(np.nan))
                continue
            scale = np.float32(np.abs(mean).max() / 127.0)
            code = np.rint(mean / np.float64(scale)) if scale > 0 else np.zeros(128)
            got[p] = (np.clip(code, -127, 127).astype(np.int8), scale)
    return got


def seen_rows(length, b, t, T, max_pages, page_rows):
    return min(max(int(length[b]), 0), max_pages * page_rows) - (T - 1 - t)


def select(q, w, codes, scale, table, page_rows, n_pages, length, k, n_first, n_last):
    """ids [B][T][k], n_sel [B][T]; q float32 [B][T][H][128] (bf16 values)."""
    B, T, H, _ = q.shape
    ids, n_sel = np.full((B, T, k), -1, np.int32), np.zeros((B, T), np.int32)
    for b in range(B):
        for t in range(T):
            seen = seen_rows(length, b, t, T, table.shape[1], page_rows)
            nb = max(0, -(-seen // page_rows))
            if nb == 0:
                continue
            top = np.abs(q[b, t]).max(1).astype(np.float32)
            inv = np.where(top > 0, np.float32(127) * (np.float32(1) / np.where(top > 0, top, np.float32(1))), np.float32(0))
            qi = np.rint(q[b, t].astype(np.float32) * inv[:, None]).astype(np.int64)
            weight = (w[b, t].astype(np.float32) * (top * (np.float32(1) / np.float32(127)))).astype(np.float32).astype(np.float64)
            pages = table[b, :nb]
            ok = (pages >= 0) & (pages < n_pages)
            p = np.where(ok, pages, 0)
            dot = qi @ codes[p].astype(np.int64).T  # [H][nb]
            score = (np.maximum(dot, 0).astype(np.float64) * weight[:, None]).sum(0) * scale[p].astype(np.float64)
            j = np.arange(nb)
            forced = (j < n_first) | (j >= nb - n_last)
            eligible = forced | (ok & ~np.isnan(score))
            rank = np.where(forced, np.inf, score)
            order = sorted(j[eligible], key=lambda i: (not forced[i], -rank[i] if not forced[i] else 0, i))
            take = sorted(order[:k])
            ids[b, t, : len(take)] = take
            n_sel[b, t] = len(take)
    return ids, n_sel


def attend(q, values, table, page_rows, n_pages, length, scale, blocks=None, n_sel=None):
    """out, lse, and the two magnitudes the error bounds need: sum_r p |x| per
    element and the largest scale * sum_d |q_d x_d| per head."""
    B, T, H, D = q.shape
    out, lse = np.zeros((B, T, H, D)), np.full((B, T, H), -np.inf)
    mag, big = np.zeros((B, T, H, D)), np.zeros((B, T, H))
    for b in range(B):
        for t in range(T):
            seen = seen_rows(length, b, t, T, table.shape[1], page_rows)
            if blocks is None:
                js = range(max(0, -(-seen // page_rows)))
            else:
                js = blocks[b, t][: max(0, int(n_sel[b, t]))] if n_sel is not None else blocks[b, t]
            rows = []
            for j in js:
                if j < 0 or j >= table.shape[1]:
                    continue
                p = int(table[b, j])
                if p < 0 or p >= n_pages:
                    continue
                n = min(page_rows, seen - int(j) * page_rows)
                rows += list(range(p * page_rows, p * page_rows + max(0, n)))
            if not rows:
                continue
            x = values[rows]
            z = q[b, t].astype(np.float64) @ x.T * scale
            m = z.max(1, keepdims=True)
            e = np.exp(z - m)
            s = e.sum(1, keepdims=True)
            out[b, t] = (e / s) @ x
            lse[b, t] = (np.log(s) + m)[:, 0]
            mag[b, t] = (e / s) @ np.abs(x)
            big[b, t] = (np.abs(q[b, t]).astype(np.float64) @ np.abs(x).T * abs(scale)).max(1)
    return out, lse, mag, big
