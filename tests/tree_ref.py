"""Plain model of speculation with trees of drafts for the tests: numpy, one draft at a time, in 64 bits where
values are computed and operation by operation where bits have to be equal."""
import numpy as np

import kv_ref as ref


def branch(parent, i):
    """Draft i and its ancestors, itself first."""
    out = []
    while i >= 0:
        out.append(i)
        i = int(parent[i])
    return out


def random_tree(r, n, chain=0.5):
    return [i - 1 if r.random() < chain else int(r.integers(-1, i)) if i else -1 for i in range(n)]


def random_path(r, parent, keep=0.9):
    path, at = [], -1
    while r.random() < keep:
        kids = [i for i in range(at + 1, len(parent)) if parent[i] == at]
        if not kids:
            break
        at = int(r.choice(kids))
        path.append(at)
    return path


def plan(parent, base):
    """(masks as Python ints, positions)."""
    ups = [branch(parent, i) for i in range(len(parent))]
    return [sum(1 << j for j in up) for up in ups], [base + len(up) - 1 for up in ups]


def as_int64(mask):
    return np.array([m - (1 << 64) if m >> 63 else m for m in mask], np.int64)


def draft_sees(mask, pos, base, n, j, window, sinks):
    if j < base:
        return not window or j > min(max(pos, base), base + n - 1) - window or j < sinks
    return j < base + n and bool(mask >> int(j - base) & 1)


def attend(vals, table, cu, kv_len, q, masks, pos, G, pt, scale, window, sinks):
    """o, lse in 64 bits; what a draft does not see is not touched at all.  A sequence with kv_len < n is skipped (None
    in the list of rows that come back)."""
    T, Hq, d = q.shape
    o, lse, rows = np.zeros((T, Hq, d)), np.full((T, Hq), -np.inf), []
    for s in range(len(kv_len)):
        n, L = cu[s + 1] - cu[s], kv_len[s]
        if L < n:
            continue
        for i in range(n):
            t = cu[s] + i
            rows.append(t)
            at = np.array([j for j in range(L) if draft_sees(masks[t], pos[t], L - n, n, j, window, sinks)], np.int64)
            if not len(at):
                continue
            page, slot = np.asarray(table[s])[at // pt], at % pt
            for h in range(Hq):
                with np.errstate(invalid="ignore", over="ignore"):
                    x = scale * (vals[page, h // G, 0, slot] @ q[t, h].astype(np.float64))
                    m = x.max()
                    e = np.exp(x - m)
                    o[t, h] = e @ vals[page, h // G, 1, slot] / e.sum()
                    lse[t, h] = m + np.log(e.sum())
    return o, lse, rows


def codes(x, s):
    """fp32 values [..., d] at scales s, broadcast: the 8-bit rule."""
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        c = np.rint((x / s).astype(np.float32))
    c = np.where(np.isfinite(c), np.clip(c, -127, 127), 0)
    return np.where(s == 0, 0, c)


def accept(stored, scales, table, base, path, pt):
    """Keep a branch, in place.  table: the sequence's pages; stored [pages, H, 2, pt, d]."""
    m = len(path)
    moved = [i for i in range(m) if path[i] != i]
    if not moved:
        return
    src = [(table[(base + p) // pt], (base + p) % pt, (base + p) // pt) for p in path]
    old_rows = np.stack([stored[p, :, :, slot].copy() for p, slot, _ in src])        # [m, H, 2, d]
    was = None if scales is None else np.abs(scales.copy())
    for b in sorted({(base + i) // pt for i in range(m)}):
        page = table[b]
        here = [i for i in range(m) if (base + i) // pt == b]
        if scales is None:
            for i in here:
                stored[page, :, :, (base + i) % pt] = old_rows[i]
            continue
        comes = [i for i in here if src[i][2] != b]
        kept = b * pt < base or len(comes) < len(here)
        if not comes:
            for i in here:
                stored[page, :, :, (base + i) % pt] = old_rows[i]
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            x = {i: (old_rows[i].astype(np.float32) * was[src[i][0]][..., None]).astype(np.float32) for i in here}
            top = np.abs(np.stack([x[i] for i in comes])).max((0, 3))
            top = np.where(np.isnan(np.stack([x[i] for i in comes])).any((0, 3)), np.nan, top).astype(np.float32)
            sc = (top / np.float32(127)).astype(np.float32)
            if kept:
                sc = np.where(np.isnan(sc) | np.isnan(was[page]), np.float32(np.nan), np.maximum(sc, was[page])).astype(np.float32)
            grown = ~((sc == was[page]) | (np.isnan(sc) & np.isnan(was[page])))[..., None]
            for t in range(max(base - b * pt, 0)):
                c = stored[page, :, :, t].astype(np.float32)
                v = (c * was[page][..., None]).astype(np.float32)
                stored[page, :, :, t] = np.where(grown, codes(v, sc[..., None]), c)
        for i in here:
            again = codes(x[i], sc[..., None])
            stored[page, :, :, (base + i) % pt] = again if i in comes else np.where(grown, again, old_rows[i])
        scales[page] = sc


def conv(raw, win, w, up):
    """Convolution of a draft whose branch is up (itself first): raw [n, H, 3d], win [H, 3, 3d], w [H, 3d, 4]."""
    return sum(w[..., 3 - j] * (raw[up[j]] if j < len(up) else win[:, 2 - (j - len(up))]) for j in range(4))


def step(S, x, alpha, beta):
    """One decode step of S [H, d, d] on a draft's convolved x [H, 3d]."""
    q, k, v = np.split(x, 3, -1)
    S = S * alpha[..., None]
    w = beta[:, None] * (v - np.einsum("hij,hi->hj", S, k))
    S = S + k[..., None] * w[:, None, :]
    return S, np.einsum("hij,hi->hj", S, q)


def verify(S0, win, w, raw, alpha, beta, parent):
    """(o [n, H, d], each draft's state) in 64 bits, every state from its parent's."""
    states, o = [], []
    for i, p in enumerate(parent):
        S, y = step(S0 if p < 0 else states[p], conv(raw, win, w, branch(parent, i)), alpha[i], beta[i])
        states.append(S)
        o.append(y)
    return np.array(o), states


def window_after(raw, win, path):
    rows = [win[:, i] for i in range(3)] + [raw[p] for p in path]
    return np.stack(rows[-3:], 1)


to_bf16 = ref.to_bf16
