"""Plain model of the key/value cache and its attention for the tests: numpy, one token at a time.

The cache's bytes are read by their documented layout, appends follow the fp32 rule operation by
operation (so codes and scales have to be equal bit for bit), attention is in 64 bits."""
import numpy as np

I8, BF16 = "i8", "bf16"


def to_bf16(x):
    """fp32 values rounded to bf16 (nearest even; NaN and infinity kept)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32)
    r = ((u.astype(np.uint64) + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    r = np.where((u & 0x7F800000) == 0x7F800000, u & 0xFFFF0000, r).astype(np.uint32)
    return r.view(np.float32)


def record_bytes(d, fmt, pt):
    return 2 * pt * d + 16 if fmt == I8 else 4 * pt * d


def page_bytes(H, d, fmt, pt):
    return -(-H * record_bytes(d, fmt, pt) // 256) * 256


def tile_index(d, fmt, pt):
    """Byte offset in a tile of (slot, byte of the row)."""
    row = d if fmt == I8 else 2 * d
    out = np.zeros((pt, row), np.int64)
    for t in range(pt):
        for b in range(row):
            if row == 64:
                out[t, b] = 64 * t + 16 * ((b // 16) ^ (t // 2 % 4)) + b % 16
            else:
                out[t, b] = b // 128 * pt * 128 + 128 * t + 16 * ((b // 16 % 8) ^ (t % 8)) + b % 16
    return out


def unpack(pool, H, d, fmt, pt):
    """pool bytes [pages, page_bytes] -> (stored [pages, H, 2, pt, d], scales [pages, H, 2] or None)."""
    rec, idx = record_bytes(d, fmt, pt), tile_index(d, fmt, pt)
    body = pool[:, :H * rec].reshape(len(pool), H, rec)
    size = idx.size
    rows = np.stack([body[:, :, :size][:, :, idx], body[:, :, size:2 * size][:, :, idx]], 2)
    if fmt == I8:
        return rows.view(np.int8), np.ascontiguousarray(body[:, :, 2 * size:2 * size + 8]).view(np.float32)
    return (np.ascontiguousarray(rows).view(np.uint16).astype(np.uint32) << 16).view(np.float32), None


def pack(stored, scales, fmt, size):
    """The inverse of unpack, into pages of `size` bytes."""
    P, H, _, pt, d = stored.shape
    rec, idx = record_bytes(d, fmt, pt), tile_index(d, fmt, pt)
    out = np.zeros((P, size), np.uint8)
    body = out[:, :H * rec].reshape(P, H, rec).copy()
    if fmt == I8:
        rows = stored.astype(np.int8).view(np.uint8)
    else:
        rows = np.ascontiguousarray((np.ascontiguousarray(stored, np.float32).view(np.uint32) >> 16).astype(np.uint16)).view(np.uint8)
    rows = rows.reshape(P, H, 2, pt, -1)
    n = idx.size
    for w in range(2):
        body[:, :, w * n + idx] = rows[:, :, w]
    if fmt == I8:
        body[:, :, 2 * n:2 * n + 8] = np.ascontiguousarray(scales, np.float32).view(np.uint8).reshape(P, H, 8)
    out[:, :H * rec] = body.reshape(P, -1)
    return out


def values(stored, scales):
    if scales is None:
        return stored.astype(np.float64)
    with np.errstate(invalid="ignore"):
        return (stored.astype(np.float32) * scales[..., None, None]).astype(np.float64)


def rotate(x, cs, pairs):
    """x fp32 [n, H, d], cs fp32 [n, rot]; every product and sum rounded to fp32 by itself."""
    if cs is None:
        return x.copy()
    r = cs.shape[1]
    c, s, y = cs[:, None, :r // 2], cs[:, None, r // 2:], x.copy()
    i = (slice(0, r, 2), slice(1, r, 2)) if pairs else (slice(0, r // 2), slice(r // 2, r))
    a, b = x[..., i[0]], x[..., i[1]]
    y[..., i[0]] = a * c - b * s
    y[..., i[1]] = b * c + a * s
    return y


def append(stored, scales, table, cu, kv_len, k, v, cs, pairs, pt):
    """Append in place.  k, v fp32 [T, H, d]; cs fp32 [positions, rot] or None."""
    for s in range(len(kv_len)):
        n = cu[s + 1] - cu[s]
        a = kv_len[s] - n
        ks = rotate(k[cu[s]:cu[s + 1]], None if cs is None else cs[a:a + n], pairs)
        new = np.stack([ks, v[cu[s]:cu[s + 1]]], 2)          # [n, H, 2, d]
        for b in range(a // pt, -(-(a + n) // pt) if n else a // pt):
            lo, hi = max(a - b * pt, 0), min(a + n - b * pt, pt)
            x = new[b * pt + lo - a:b * pt + hi - a].transpose(1, 2, 0, 3)     # [H, 2, rows, d]
            p = table[s][b]
            if scales is None:
                stored[p, :, :, lo:hi] = to_bf16(x)
                continue
            with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
                top = np.abs(x).max((2, 3))                  # a NaN wins, as the rule says
                sc = top / np.float32(127)
                old = np.abs(scales[p])
                if lo:
                    sc = np.where(np.isnan(old) | np.isnan(sc), np.float32(np.nan), np.maximum(sc, old)).astype(np.float32)
                def codes(z, q):
                    c = np.rint(z / q[..., None, None])
                    c = np.where(np.isfinite(c), np.clip(c, -127, 127), 0)
                    return np.where(q[..., None, None] == 0, 0, c)
                if lo:
                    was = stored[p, :, :, :lo].astype(np.float32) * old[..., None, None]
                    grown = ~((sc == old) | (np.isnan(sc) & np.isnan(old)))
                    stored[p, :, :, :lo] = np.where(grown[..., None, None], codes(was, sc), stored[p, :, :, :lo])
                stored[p, :, :, lo:hi] = codes(x, sc)
                scales[p] = sc


def sees(p, j, window, sinks):
    return j <= p and (not window or j > p - window or j < sinks)


def attend(vals, table, cu, kv_len, q, G, pt, scale, window, sinks):
    """o [T, Hq, d], lse [T, Hq] in 64 bits; what a query does not see is not touched at all."""
    T, Hq, d = q.shape
    o, lse = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf)
    for s in range(len(kv_len)):
        n, L = cu[s + 1] - cu[s], kv_len[s]
        if not n:
            continue
        for i in range(n):
            p = L - n + i
            at = np.array([j for j in range(max(p + 1, 0)) if sees(p, j, window, sinks)], np.int64)
            if not len(at):
                continue
            page, slot = np.asarray(table[s])[at // pt], at % pt
            for h in range(Hq):
                with np.errstate(invalid="ignore", over="ignore"):
                    x = scale * (vals[page, h // G, 0, slot] @ q[cu[s] + i, h].astype(np.float64))
                    m = x.max()
                    e = np.exp(x - m)
                    o[cu[s] + i, h] = e @ vals[page, h // G, 1, slot] / e.sum()
                    lse[cu[s] + i, h] = m + np.log(e.sum())
    return o, lse
