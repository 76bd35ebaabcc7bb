"""Cases of the key/value-cache operators: appending rotated keys and values to a paged cache,
attention over an 8-bit cache with a scale for each block of tokens and head, and attention with
a sliding window and sinks.

A page of the pool is one block of `pt` tokens of all key/value heads of one layer.  Per head it
holds a record: the block's keys, its values and, for the 8-bit form, the two scales:

  tile   rows of one token each, cut into lines of 128 bytes (64 where a row has only 64): line
         block c holds bytes [128 c, 128 c + 128) of every token's row, token after token.  The
         16-byte unit u of token t's line lies at place u ^ (t % 8), or u ^ ((t / 2) % 4) in
         64-byte lines.
  record K tile | V tile | (8-bit only) float32 scale of K, float32 scale of V, 8 zero bytes
  page   one record a head, zero-padded to a multiple of 256 bytes

8-bit values are code * scale with code in [-127, 127] and scale = max|x| / 127 over the block and
head.  Sequence s has kv_len[s] tokens once the call's own n tokens are in, and those are its last.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2}

# ------------------------------------------------------------------ cases
# lens seeds the lengths of a ragged batch; [qmin, qmax] new tokens and [lmin, lmax] cached tokens
# (the new ones among them) a sequence.  Head counts and lengths: 16 and 32 heads of 64 or 128,
# 4 x 8192, 256 decoding requests, 32 sequences of 512 to 32768 tokens, 1,048,576 tokens and
# 4 draft tokens are this repository's own workloads; 4 and 8 key/value heads are generic.


def listed():
    A = dict(op="append", rot=128, pairs=False)
    T = dict(op="attend", window=0, sinks=0)
    return [
        # one user's next token: launch latency is all there is
        dict(A, name="append-1", fmt="i8", dtype="bf16", Hq=16, Hkv=4, d=128, pt=64, seqs=1, qmin=1, qmax=1,
             lmin=1000, lmax=1000, lens=1),
        # a decode step of 256 requests at odd positions, some of them opening a new block
        dict(A, name="append-decode-256", fmt="i8", dtype="bf16", Hq=32, Hkv=8, d=128, pt=64, seqs=256, qmin=1,
             qmax=1, lmin=1, lmax=8191, lens=2),
        # the batched prefill's four sequences into a 16-bit cache
        dict(A, name="append-prefill-bf16", fmt="bf16", dtype="bf16", Hq=16, Hkv=16, d=128, pt=64, seqs=4, qmin=8192,
             qmax=8192, lmin=8192, lmax=8192, lens=3),
        # ragged prompts behind cached prefixes, float32 tokens, half of each head rotated in pairs, 48-token blocks
        dict(A, name="append-ragged-f32", fmt="i8", dtype="f32", Hq=32, Hkv=8, d=64, rot=32, pairs=True, pt=48,
             seqs=32, qmin=1, qmax=2000, lmin=1, lmax=6000, lens=4),
        # one user's short conversation
        dict(T, name="i8-decode-1", fmt="i8", dtype="bf16", Hq=16, Hkv=4, d=128, pt=64, seqs=1, qmin=1, qmax=1,
             lmin=1000, lmax=1000, lens=5),
        # a decode step over 32 ragged contexts
        dict(T, name="i8-decode-32-ragged", fmt="i8", dtype="bf16", Hq=32, Hkv=8, d=128, pt=64, seqs=32, qmin=1,
             qmax=1, lmin=512, lmax=32768, lens=2),
        # one context of a million tokens
        dict(T, name="i8-decode-1m", fmt="i8", dtype="bf16", Hq=32, Hkv=4, d=128, pt=128, seqs=1, qmin=1, qmax=1,
             lmin=1048576, lmax=1048576, lens=6),
        # float32 tokens, small heads, 4 drafts a request, 48-token blocks
        dict(T, name="i8-verify-f32", fmt="i8", dtype="f32", Hq=16, Hkv=4, d=64, pt=48, seqs=24, qmin=4, qmax=4,
             lmin=4, lmax=5000, lens=7),
        # a prompt's chunk of 4096 tokens behind 12288 cached ones
        dict(T, name="i8-prefill-chunk", fmt="i8", dtype="bf16", Hq=32, Hkv=8, d=128, pt=64, seqs=1, qmin=4096,
             qmax=4096, lmin=16384, lmax=16384, lens=8),
        # one token behind a window that is hardly longer than the context's start
        dict(T, name="window-decode-1", fmt="bf16", dtype="bf16", Hq=16, Hkv=16, d=64, pt=16, seqs=1, qmin=1, qmax=1,
             lmin=700, lmax=700, lens=9, window=512, sinks=4),
        # a decode step of 256 requests through a window
        dict(T, name="window-decode-256", fmt="bf16", dtype="bf16", Hq=32, Hkv=8, d=128, pt=64, seqs=256, qmin=1,
             qmax=1, lmin=1, lmax=8192, lens=10, window=1024, sinks=4),
        # ragged prompts through a window
        dict(T, name="window-prefill", fmt="bf16", dtype="bf16", Hq=16, Hkv=4, d=128, pt=64, seqs=4, qmin=1,
             qmax=8192, lmin=1, lmax=8192, lens=11, window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: an append, a step over an 8-bit cache, or one through a window."""
    case = {"lens": rng.randrange(1 << 30), "dtype": rng.choice(["bf16", "bf16", "f32"]), "d": rng.choice([64, 128]),
            "pt": rng.choice([16, 32, 48, 64, 96, 128])}
    case["Hkv"] = rng.choice([1, 2, 3, 4, 8])
    case["Hq"] = case["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
    kind = rng.choice(["append", "i8", "window"])
    if kind == "append":
        case.update(op="append", fmt=rng.choice(["i8", "bf16"]), rot=rng.choice([0, 32, case["d"]]),
                    pairs=rng.random() < 0.5)
    else:
        case.update(op="attend", fmt="i8" if kind == "i8" else rng.choice(["bf16", "i8"]), window=0, sinks=0)
        if kind == "window":
            case.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 64, 200]))
    shape = rng.choice(["decode", "drafts", "prefill"])
    if shape == "decode":
        case.update(seqs=_log(rng, 1, 256), qmin=1, qmax=1)
        most = 4_000_000 // (case["seqs"] * case["Hkv"])
    elif shape == "drafts":
        k = rng.randint(2, 8)
        case.update(seqs=_log(rng, 1, 64), qmax=k)
        case.update(qmin=0 if case["seqs"] > 8 and rng.random() < 0.5 else k)
        most = 2_000_000 // (case["seqs"] * case["Hkv"])
    else:
        case.update(seqs=_log(rng, 1, 8))
        n = _log(rng, 16, 8192 // case["seqs"] if case["op"] == "append" else 4096 // case["seqs"])
        if case["dtype"] == "f32":
            n = min(n, 512)
        if case["Hq"] > 32:
            case["Hq"] = 2 * case["Hkv"]
        case.update(qmin=n if rng.random() < 0.5 else max(1, n // 7), qmax=n)
        most = 12000
    top = _log(rng, max(16, case["qmax"]), max(17, case["qmax"] + 1, min(most, 65536)))
    case.update(lmin=1 if rng.random() < 0.5 else max(1, top // 2), lmax=top)
    return case


def lengths(case):
    """[(new tokens, tokens in the cache once they are in)] of each sequence."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["seqs"]):
        n = r.randint(case["qmin"], case["qmax"])
        out.append((n, max(n, r.randint(case["lmin"], case["lmax"]))))
    return out


def _visible(case, n, L):
    """(pairs, tokens of the cache that some query sees) of a sequence."""
    w, s, pairs = case["window"], case["sinks"], 0
    if not n:
        return 0, 0
    if not w:
        return sum(range(L - n + 1, L + 1)), L
    for p in range(L - n, L):
        pairs += min(w, p + 1) + max(0, min(s, p + 1 - w))
    first = max(0, L - n - w + 1)
    return pairs, L - first + min(s, first)


def work(case):
    es, d, Hq, Hkv = ES[case["dtype"]], case["d"], case["Hq"], case["Hkv"]
    cs, scales = (1, 8) if case["fmt"] == "i8" else (2, 0)
    b = f = 0
    for n, L in lengths(case):
        b += 8
        if case["op"] == "append":
            if not n:
                continue
            first = (L - n) // case["pt"] * case["pt"]
            pages = (L - 1) // case["pt"] + 1 - first // case["pt"]
            b += n * (2 * Hq + 2 * Hkv) * d * es                    # q in and out, k and v in
            b += 2 * n * Hkv * d * cs + pages * (4 + Hkv * scales)  # the cache
            b += 2 * (L - n - first) * Hkv * d * cs                 # the older tokens of the first block
            b += 2 * (L - first) * Hkv * d * 2                      # the blocks' values
            f += n * (Hq + Hkv) * case["rot"] * 3 + (2 * (L - first) * Hkv * d * 3 if cs == 1 else 0)
        else:
            pairs, seen = _visible(case, n, L)
            b += n * Hq * (2 * d * es + 4) + 2 * seen * Hkv * d * cs + -(-seen // case["pt"]) * (4 + Hkv * scales)
            f += 4 * d * Hq * pairs
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------ inputs
def _record_bytes(case):
    return 2 * case["pt"] * case["d"] * (1 if case["fmt"] == "i8" else 2) + (16 if case["fmt"] == "i8" else 0)


def _lay_out(case, kv, scales, page_bytes):
    """The pages' bytes from kv [pages, Hkv, 2, pt, d] (codes or bf16) and scales [pages, Hkv, 2]."""
    P, Hkv, _, pt, _ = kv.shape
    out = torch.zeros(P, page_bytes, dtype=torch.uint8, device=kv.device)
    rows = kv.contiguous().view(torch.uint8)
    line = min(128, rows.shape[-1])
    units = line // 16
    tile = rows.view(P, Hkv, 2, pt, -1, units, 16).transpose(3, 4)  # [.., line block, token, unit, 16]
    t = torch.arange(pt, device=kv.device)
    flip = t % 8 if units == 8 else (t // 2) % 4
    at = torch.arange(units, device=kv.device)[None, :] ^ flip[:, None]
    tile = torch.take_along_dim(tile, at[None, None, None, None, :, :, None], 5)
    rec = _record_bytes(case)
    body = out[:, :Hkv * rec].view(P, Hkv, rec)
    body[:, :, :2 * pt * rows.shape[-1]] = tile.reshape(P, Hkv, -1)
    if case["fmt"] == "i8":
        body[:, :, rec - 16:rec - 8] = scales.contiguous().view(torch.uint8).view(P, Hkv, 8)
    return out


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rnd = random.Random(seed)
    dt, pt, Hq, Hkv, d = DT[case["dtype"]], case["pt"], case["Hq"], case["Hkv"], case["d"]
    lens = lengths(case)
    need = [-(-L // pt) for _, L in lens]
    pages = sum(need) + 3
    ids = list(range(pages))
    rnd.shuffle(ids)
    maxp = max(need)
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [-1] * (maxp - n))
        at += n
    cu, cu_out, begin = [0], [0], []
    for n, L in lens:
        cu.append(cu[-1] + n)
        first = (L - n) // pt * pt if n else L
        begin.append(first)
        cu_out.append(cu_out[-1] + L - first)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    T = cu[-1]
    # a cache as earlier steps left it, its blocks' free slots filled with what was there before
    store = torch.empty(pages, Hkv, 2, pt, d, dtype=torch.int8 if case["fmt"] == "i8" else torch.bfloat16, device=dev)
    scales = torch.empty(pages, Hkv, 2, device=dev) if case["fmt"] == "i8" else None
    step = max(1, (1 << 27) // (Hkv * 2 * pt * d))
    for a in range(0, pages, step):
        x = torch.randn(store[a:a + step].shape, generator=g, device=dev)
        if scales is None:
            store[a:a + step] = x
        else:
            x *= 0.5 + torch.rand(x.shape[0], Hkv, 2, 1, 1, generator=g, device=dev)
            sc = x.abs().amax((3, 4)) / 127
            scales[a:a + step] = sc
            store[a:a + step] = torch.round(x / sc[..., None, None])
    page_bytes = -(-Hkv * _record_bytes(case) // 256) * 256
    # queries, keys and values are parts of one projection's output
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=dev)
    x[:, :Hq] *= 2
    x = x.to(dt)
    st = {"case": dict(case), "lens": lens, "maxq": max(n for n, _ in lens), "store": store, "scales": scales,
          "bytes": _lay_out(case, store, scales, page_bytes), "table": i32(table).view(len(lens), maxp), "cu": i32(cu),
          "kv_len": i32([L for _, L in lens]), "cu_out": i32(cu_out), "begin": i32(begin), "rows": cu_out[-1],
          "spare": ids[-1],
          "q": x[:, :Hq], "k": x[:, Hq:Hq + Hkv], "v": x[:, Hq + Hkv:]}
    if case["op"] == "append":
        st["cos_sin"] = None
        if case["rot"]:
            top = max(L for _, L in lens)
            f = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev) / case["rot"])
            ang = torch.arange(top, dtype=torch.float64, device=dev)[:, None] * f
            st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["q_out"] = torch.empty(T, Hq, d, dtype=dt, device=dev)
        st["k_out"] = torch.empty(st["rows"], Hkv, d, dtype=torch.bfloat16, device=dev)
        st["v_out"] = torch.empty_like(st["k_out"])
    else:
        st["o"] = torch.empty(T, Hq, d, dtype=dt, device=dev)
        st["lse"] = torch.empty(T, Hq, device=dev)
    if own:  # the handles that a program keeps: the pool, a status word and a workspace
        import kda_state_chunked_gb300 as kda

        st["kda"] = kda
        st["pool"] = kda.Pool(page_bytes, pages)
        st["pool"].base = st["bytes"]
        st["fmt"] = kda.KDA_KV_I8 if case["fmt"] == "i8" else kda.KDA_KV_BF16
        st["status"] = torch.zeros(1, dtype=torch.int32, device=dev)
        if case["op"] == "attend":
            st["ws"] = kda.attn_workspace(st["q"], Hkv, len(lens), st["maxq"])
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    return _append(st) if st["case"]["op"] == "append" else _attend(st)


def _own(st):
    c, kda = st["case"], st["kda"]
    if c["op"] == "append":
        kda.kda_kv_append(st["pool"], st["fmt"], c["pt"], st["cu"], st["kv_len"], st["table"], st["maxq"], st["q"],
                          st["k"], st["v"], st["cos_sin"], st["q_out"], st["status"], interleaved=c["pairs"])
        kda.kda_kv_gather(st["pool"], st["fmt"], c["pt"], st["cu_out"], st["begin"], st["table"], st["k_out"],
                          st["v_out"], st["status"])
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    kda.kda_attn_paged(st["pool"], c["Hkv"], st["fmt"], c["pt"], st["cu"], st["kv_len"], st["table"], st["maxq"],
                       st["q"], st["o"], st["ws"], st["status"], window=c["window"], sinks=c["sinks"],
                       lse=st["lse"])
    return {"o": st["o"], "lse": st["lse"]}


def _where(cu, rows):
    """The sequence of each packed row, and the row's index in it."""
    at = torch.arange(rows, device=cu.device)
    s = torch.searchsorted(cu[1:].long(), at, right=True)
    return s, at - cu.long()[s]


def _rotate(x, cs, pairs):
    """x float32 [T, H, d], cs [T, rot]."""
    r = cs.shape[1]
    c, s = cs[:, None, :r // 2], cs[:, None, r // 2:]
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if pairs else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * c - b * s, b * c + a * s
    if pairs:
        y[..., 0:r:2], y[..., 1:r:2] = u, w
    else:
        y[..., :r // 2], y[..., r // 2:r] = u, w
    return y


def _append(st):
    c = st["case"]
    pt, Hkv, d, T = c["pt"], c["Hkv"], c["d"], st["q"].shape[0]
    nseq, maxp = st["table"].shape
    s, r = _where(st["cu"], T)
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    old = st["kv_len"].long() - n                     # tokens cached before the call
    pos = old[s] + r
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    if st["cos_sin"] is not None:
        cs = st["cos_sin"][pos]
        q, k = _rotate(q, cs, c["pairs"]), _rotate(k, cs, c["pairs"])
    # the blocks that the call touches, as rows of their own: [sequence, block, slot]
    p0 = old // pt
    J = (st["maxq"] + pt - 2) // pt + 1
    block = p0[:, None] + torch.arange(J, device=q.device)
    touched = (block * pt < st["kv_len"].long()[:, None]) & (n[:, None] > 0)
    page = torch.where(touched, st["table"].long().gather(1, block.clamp(max=maxp - 1)), st["spare"])
    new = torch.zeros(nseq, J * pt, Hkv, 2, d, device=q.device)
    new[s, pos - p0[s] * pt] = torch.stack([k, v], 2)
    new = new.view(nseq, J, pt, Hkv, 2, d).permute(0, 1, 3, 4, 2, 5)     # [seq, block, head, k/v, slot, d]
    at = (block[..., None] * pt + torch.arange(pt, device=q.device))
    is_new = ((at >= old[:, None, None]) & (at < st["kv_len"].long()[:, None, None]))[:, :, None, None, :, None]
    is_old = (at < old[:, None, None])[:, :, None, None, :, None]
    have = st["store"][page]
    if c["fmt"] == "i8":
        sc = st["scales"][page]
        seven = torch.full_like(sc, 127.0)
        grown = torch.where(is_new, new, 0).abs().amax((4, 5)) / seven
        kept = torch.where(is_old.any(4)[..., 0], sc, 0)
        scale = torch.maximum(grown, kept)
        val = torch.where(is_new, new, have.float() * sc[..., None, None])
        code = torch.where(scale[..., None, None] > 0, torch.round(val / scale[..., None, None]), 0)
        code = torch.where(is_new | is_old, code.to(torch.int8), have)
        value = code.float() * scale[..., None, None]
    else:
        code = torch.where(is_new, new.bfloat16(), have)
        scale, value = None, code
    # write the blocks back (those left out all go to the page that no sequence has)
    dest = page.reshape(-1)
    st["store"][dest] = code.reshape(-1, Hkv, 2, pt, d)
    if scale is not None:
        st["scales"][dest] = scale.reshape(-1, Hkv, 2)
    so, ro = _where(st["cu_out"], st["rows"])
    flat = value.permute(0, 1, 4, 2, 3, 5).reshape(nseq, J * pt, Hkv, 2, d)[so, ro].bfloat16()
    return {"q": q.to(st["q"].dtype), "k": flat[:, :, 0], "v": flat[:, :, 1]}


def _attend(st):
    c = st["case"]
    pt, Hq, Hkv, d, T = c["pt"], c["Hq"], c["Hkv"], c["d"], st["q"].shape[0]
    nseq, maxp = st["table"].shape
    G, M, L = Hq // Hkv, st["maxq"], maxp * pt
    page = st["table"].long().clamp(min=0)
    kv = st["store"][page].float()                    # [seq, block, head, k/v, slot, d]
    if c["fmt"] == "i8":
        kv *= st["scales"][page][..., None, None]
    kv = kv.permute(3, 0, 2, 1, 4, 5).reshape(2, nseq, Hkv, L, d)
    s, r = _where(st["cu"], T)
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    q = torch.zeros(nseq, M, Hq, d, device=kv.device)
    q[s, r] = st["q"].float()
    q = q.view(nseq, M, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(nseq, Hkv, G * M, d)
    score = torch.matmul(q, kv[0].transpose(-1, -2)).view(nseq, Hkv, G, M, L) * d ** -0.5
    p = (st["kv_len"].long() - n)[:, None] + torch.arange(M, device=q.device)        # [seq, row]
    j = torch.arange(L, device=q.device)
    see = (j <= p[..., None]) & (torch.arange(M, device=q.device) < n[:, None])[..., None]
    if c["window"]:
        see &= (j > p[..., None] - c["window"]) | (j < c["sinks"])
    see = see[:, None, None]
    score = score.masked_fill(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    e = torch.exp(score - top)
    total = e.sum(-1, keepdim=True)
    there = (j < st["kv_len"].long()[:, None])[:, None, :, None]
    o = torch.matmul(e.view(nseq, Hkv, G * M, L), torch.where(there, kv[1], 0)).view(nseq, Hkv, G, M, d)
    o = torch.where(total > 0, o / total, 0).permute(0, 3, 1, 2, 4).reshape(nseq, M, Hq, d)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(nseq, M, Hq)
    return {"o": o[s, r].to(st["q"].dtype), "lse": lse[s, r]}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    f = _exact_append if case["op"] == "append" else _exact_attend
    return f(case, st)


def _tokens(case, st, i, a, b):
    """Keys and values [b - a, Hkv, d] of the cache's tokens a .. b of sequence i."""
    pt = case["pt"]
    ids = st["table"][i, a // pt:-(-b // pt)].long()
    x = st["store"][ids].double()
    if case["fmt"] == "i8":
        x = x * st["scales"][ids].double()[..., None, None]
    x = x.permute(2, 0, 3, 1, 4).reshape(2, -1, case["Hkv"], case["d"])
    lo = a - a // pt * pt
    return x[0, lo:lo + b - a], x[1, lo:lo + b - a]


def _exact_turn(case, x, cs):
    """Rotation as a product of complex numbers."""
    if cs is None:
        return x
    h = case["rot"] // 2
    w = torch.complex(cs[:, :h], cs[:, h:])[:, None]
    x = x.clone()
    if case["pairs"]:
        z = torch.view_as_complex(x[..., :2 * h].reshape(*x.shape[:-1], h, 2).contiguous()) * w
        x[..., :2 * h] = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * h)
    else:
        z = torch.complex(x[..., :h], x[..., h:2 * h]) * w
        x[..., :h], x[..., h:2 * h] = z.real, z.imag
    return x


def _exact_append(case, st):
    pt, cu = case["pt"], st["cu"].tolist()
    qs, ks, vs = [], [], []
    for i, (n, L) in enumerate(st["lens"]):
        a, b = cu[i], cu[i + 1]
        if not n:
            continue
        cs = None if st["cos_sin"] is None else st["cos_sin"][L - n:L].double()
        qs.append(_exact_turn(case, st["q"][a:b].double(), cs))
        first = (L - n) // pt * pt
        k0, v0 = _tokens(case, st, i, first, L - n) if L - n > first else (None, None)
        for new, before, w, out in ((_exact_turn(case, st["k"][a:b].double(), cs), k0, 0, ks),
                                    (st["v"][a:b].double(), v0, 1, vs)):
            if case["fmt"] != "i8":
                out.append(new if before is None else torch.cat([before, new]))
                continue
            m = new.abs().amax(-1)                                        # [n, Hkv]
            low = torch.zeros(case["Hkv"], dtype=torch.float64, device=m.device)
            if before is not None:
                low = st["scales"][int(st["table"][i, first // pt]), :, w].double() * 127
                m = torch.cat([low.expand(before.shape[0], -1), m])
                new = torch.cat([before, new])
            pad = -m.shape[0] % pt
            m = torch.cat([m, m.new_zeros(pad, m.shape[1])]).view(-1, pt, case["Hkv"]).amax(1) / 127
            m = m.repeat_interleave(pt, 0)[:new.shape[0], :, None]
            out.append(torch.where(m > 0, torch.round(new / m) * m, 0))
    cat = lambda x, H: torch.cat(x) if x else torch.empty(0, H, case["d"], dtype=torch.float64)  # noqa: E731
    return {"q": cat(qs, case["Hq"]), "k": cat(ks, case["Hkv"]), "v": cat(vs, case["Hkv"])}


def _exact_attend(case, st):
    if work(case)["flops"] > 3e12:
        return None
    cu, G, d = st["cu"].tolist(), case["Hq"] // case["Hkv"], case["d"]
    o = torch.zeros(cu[-1], case["Hq"], d, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((cu[-1], case["Hq"]), -math.inf, dtype=torch.float64, device=o.device)
    for i, (n, L) in enumerate(st["lens"]):
        if not n:
            continue
        k, v = _tokens(case, st, i, 0, L)
        at = torch.arange(L, device=o.device)
        step = max(1, (1 << 27) // L)
        for a in range(0, n, step):
            b = min(n, a + step)
            p = torch.arange(L - n + a, L - n + b, device=o.device)[:, None]
            hide = at > p
            if case["window"]:
                hide |= (at <= p - case["window"]) & (at >= case["sinks"])
            for h in range(case["Hq"]):
                x = st["q"][cu[i] + a:cu[i] + b, h].double() @ k[:, h // G].T / math.sqrt(d)
                x[hide] = -math.inf
                z = torch.logsumexp(x, -1, keepdim=True)
                o[cu[i] + a:cu[i] + b, h] = torch.exp(x - z) @ v[:, h // G]
                lse[cu[i] + a:cu[i] + b, h] = z[:, 0]
    return {"o": o, "lse": lse}
