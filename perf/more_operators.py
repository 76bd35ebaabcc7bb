"""Cases of speculation with trees of drafted tokens: placing tokens in the cache at positions of their own
(a tree's depths; time, height and width of pictures), attention of a tree over the cache, keeping the
accepted branch in the cache, and verifying a tree against a recurrent state.

A tree: the n <= 64 drafts of a sequence, drafts parent[i] < i or -1 (a child of the last accepted token).
They stand in the cache as its last n tokens, and the accepted ones are a branch path[0] < path[1] < ...

Cache: a page of the pool is one block of `pt` tokens of all key/value heads of one layer.  Per head it
holds a record: the block's keys, its values and, for the 8-bit form, the two scales:

  tile   rows of one token each, cut into lines of 128 bytes (64 where a row has only 64): line
         block c holds bytes [128 c, 128 c + 128) of every token's row, token after token.  The
         16-byte unit u of token t's line lies at place u ^ (t % 8), or u ^ ((t / 2) % 4) in
         64-byte lines.
  record K tile | V tile | (8-bit only) float32 scale of K, float32 scale of V, 8 zero bytes
  page   one record a head, zero-padded to a multiple of 256 bytes

8-bit values are code * scale with code in [-127, 127].  Sequence s has kv_len[s] tokens once the call's own
n tokens are in, and those are its last.

States: a record a head, S float32 [d][d] | window [3][3d] (raw q | k | v of the last three tokens, oldest
first), padded to a multiple of 256 bytes; `hpp` heads to a page of the pool here.
"""
import math
import random

import torch

own = False
device = "cuda"

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ES = {"f32": 4, "bf16": 2}
MOST = 64  # drafts of a tree

# ------------------------------------------------------------------ cases
# lens seeds the lengths and trees of a ragged batch; [qmin, qmax] new tokens and [lmin, lmax] cached tokens (the
# new ones among them) a sequence; chain: the share of drafts that continue the one before.  Head counts and
# lengths: 16 and 32 heads of 64 or 128, 4 x 8192, 256 decoding requests, 32 sequences of 512 to 32768 tokens are
# this repository's own workloads; 4 and 8 key/value heads and trees of 8 to 64 drafts are generic.


def listed():
    P = dict(op="place", pairs=False, rot=128, sections="64")
    T = dict(op="attend", window=0, sinks=0)
    K = dict(op="keep")
    V = dict(op="verify")
    return [
        # one user's tree of 8 drafts enters the cache: launch latency is all there is
        dict(P, name="place-tree-1", fmt="i8", dtype="bf16", Hq=16, Hkv=4, d=128, pt=64, seqs=1, qmin=8, qmax=8,
             lmin=1000, lmax=1000, chain=0.5, lens=1),
        # 64 requests' trees of up to 32 drafts, at odd places
        dict(P, name="place-tree-64", fmt="i8", dtype="bf16", Hq=32, Hkv=8, d=128, pt=64, seqs=64, qmin=1, qmax=32,
             lmin=1, lmax=8191, chain=0.5, lens=2),
        # prompts of text and pictures, three coordinates a token
        dict(P, name="place-pictures", fmt="bf16", dtype="bf16", Hq=16, Hkv=16, d=128, sections="16,24,24", pt=64,
             seqs=4, qmin=4000, qmax=8192, lmin=4000, lmax=8192, chain=0.0, lens=3),
        # one user's tree over a short conversation
        dict(T, name="attend-tree-1", fmt="i8", dtype="bf16", Hq=16, Hkv=4, d=128, pt=64, seqs=1, qmin=8, qmax=8,
             lmin=1000, lmax=1000, chain=0.5, lens=4),
        # trees of 16 drafts over 32 ragged contexts
        dict(T, name="attend-tree-32-ragged", fmt="i8", dtype="bf16", Hq=32, Hkv=8, d=128, pt=64, seqs=32, qmin=16,
             qmax=16, lmin=512, lmax=32768, chain=0.5, lens=5),
        # large trees over a 16-bit cache
        dict(T, name="attend-tree-64-drafts", fmt="bf16", dtype="bf16", Hq=32, Hkv=8, d=128, pt=64, seqs=16, qmin=33,
             qmax=64, lmin=4096, lmax=16384, chain=0.6, lens=6),
        # float32 tokens, small heads, odd trees, 48-token blocks, through a window
        dict(T, name="attend-tree-f32", fmt="i8", dtype="f32", Hq=16, Hkv=4, d=64, pt=48, seqs=24, qmin=1, qmax=11,
             lmin=11, lmax=5000, window=2000, sinks=4, chain=0.4, lens=7),
        # one user's accepted branch
        dict(K, name="keep-1", fmt="i8", dtype="bf16", Hq=4, Hkv=4, d=128, pt=64, seqs=1, qmin=8, qmax=8, lmin=1000,
             lmax=1000, chain=0.5, lens=8),
        # the accepted branches of 256 requests, some across a block's end
        dict(K, name="keep-256", fmt="i8", dtype="bf16", Hq=8, Hkv=8, d=128, pt=64, seqs=256, qmin=1, qmax=64, lmin=64,
             lmax=8192, chain=0.6, lens=9),
        # one user's tree against a recurrent layer's states
        dict(V, name="verify-tree-1", dtype="bf16", H=16, d=128, hpp=1, seqs=1, qmin=8, qmax=8, chain=0.5, lens=10),
        # a decode batch's trees
        dict(V, name="verify-tree-256", dtype="bf16", H=32, d=128, hpp=4, seqs=256, qmin=16, qmax=16, chain=0.5, lens=11),
        # float32 tokens, small heads, large ragged trees
        dict(V, name="verify-tree-f32", dtype="f32", H=16, d=64, hpp=2, seqs=48, qmin=1, qmax=64, chain=0.5, lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: tokens placed, a tree attending, a branch kept, or a tree verified."""
    op = rng.choice(["place", "attend", "attend", "keep", "verify", "verify"])
    case = {"op": op, "lens": rng.randrange(1 << 30), "dtype": rng.choice(["bf16", "bf16", "f32"]),
            "d": rng.choice([64, 128]), "chain": rng.choice([0.0, 0.3, 0.6, 0.9, 1.0])}
    n = _log(rng, 1, MOST)
    case.update(qmax=n, qmin=n if rng.random() < 0.5 else rng.randint(1, n))
    if op == "verify":
        case["H"] = rng.choice([1, 2, 3, 4, 8, 16, 32])
        case["hpp"] = rng.choice([x for x in (1, 2, 4, 8) if case["H"] % x == 0])
        case["seqs"] = _log(rng, 1, max(1, min(256, 131072 // (case["H"] * n))))
        return case
    case["fmt"] = rng.choice(["i8", "i8", "bf16"])
    case["pt"] = rng.choice([16, 32, 48, 64, 96, 128])
    case["Hkv"] = rng.choice([1, 2, 3, 4, 8])
    case["Hq"] = case["Hkv"] * rng.choice([1, 2, 3, 4, 5, 8])
    top = 8192
    if op == "place":
        case["pairs"] = rng.random() < 0.5
        rot = rng.choice([r for r in (48, 64, 96, 128) if r <= case["d"]])
        case["rot"] = rot
        third = rot // 48 * 8
        case["sections"] = rng.choice([f"{rot // 2}", f"{rot // 2 - 2 * third},{third},{third}", f"16,{rot // 2 - 16}"])
        case["seqs"] = _log(rng, 1, 64)
        if rng.random() < 0.4:  # a prompt, not a tree
            case["seqs"] = _log(rng, 1, 8)
            n = _log(rng, 65, 8192 // case["seqs"])
            case.update(qmax=n, qmin=max(1, n // 3), chain=0.0)
    elif op == "keep":
        case["seqs"] = _log(rng, 1, 256)
    else:
        case.update(window=0, sinks=0)
        if rng.random() < 0.3:
            case.update(window=_log(rng, 64, 8192), sinks=rng.choice([0, 1, 4, 64]))
        case["seqs"] = _log(rng, 1, 64)
        G = case["Hq"] // case["Hkv"]
        most = min(4_000_000, 400_000_000 // (G * n)) if case["dtype"] == "bf16" else min(1_000_000, 30_000_000 // (G * n))
        top = min(65536, most // (case["seqs"] * case["Hkv"]))
    if n > 1 and case["seqs"] > 8 and rng.random() < 0.3:  # some sequences without drafts
        case["qmin"] = 0
    top = _log(rng, max(16, case["qmax"]), max(17, case["qmax"] + 1, top))
    case.update(lmin=1 if rng.random() < 0.5 else max(1, top // 2), lmax=top)
    return case


def lengths(case):
    """[(new tokens, tokens in the cache once they are in)] of each sequence."""
    r = random.Random(case["lens"])
    out = []
    for _ in range(case["seqs"]):
        n = r.randint(case["qmin"], case["qmax"])
        out.append((n, max(n, r.randint(case["lmin"], case["lmax"])) if "lmin" in case else n))
    return out


def sections(case):
    """How many of a head's angles go by each coordinate of a token's position."""
    return [int(x) for x in case["sections"].split(",")]


def trees(case):
    """[(parents, accepted branch)] of each sequence."""
    r = random.Random(case["lens"] + 1)
    out = []
    for n, _ in lengths(case):
        parent = [i - 1 if r.random() < case["chain"] else r.randint(max(-1, i - 12), i - 1) for i in range(n)]
        path, at = [], -1
        while r.random() < 0.85:
            kids = [i for i in range(at + 1, n) if parent[i] == at]
            if not kids:
                break
            at = r.choice(kids)
            path.append(at)
        out.append((parent, path))
    return out


def _branch(parent, i):
    """Draft i and its ancestors, itself first."""
    out = []
    while i >= 0:
        out.append(i)
        i = parent[i]
    return out


def _depths(parent):
    out = []
    for p in parent:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def work(case):
    es, d = ES[case["dtype"]], case["d"]
    b = f = 0
    if case["op"] == "verify":
        H, rec = case["H"], d * d * 4 + 9 * d * es
        for (n, _), (parent, path) in zip(lengths(case), trees(case)):
            pairs = sum(x + 1 for x in _depths(parent))
            b += n * H * (5 * d + 1) * es + 4 * n + 4 + H * rec       # tokens, outputs, the state
            b += (4 * len(path) + 4 + H * rec) if path else 4         # the state after the branch
            f += n * H * 4 * d * d + pairs * H * 8 * d + H * d * d * (1 + 2 * len(path)) * bool(path)
        return {"bytes": b + 3 * d * H * 16, "flops": f}
    Hq, Hkv, pt = case["Hq"], case["Hkv"], case["pt"]
    cs, scales = (1, 8) if case["fmt"] == "i8" else (2, 0)
    kept = trees(case) if case["op"] == "keep" else None
    marks = trees(case) if case["op"] == "attend" else None
    for i, (n, L) in enumerate(lengths(case)):
        b += 8
        if not n:
            continue
        first = (L - n) // pt * pt
        if case["op"] == "place":
            pages = (L - 1) // pt + 1 - first // pt
            b += n * (2 * Hq + 2 * Hkv) * d * es + 4 * n * len(sections(case))   # q in and out, k and v in, positions
            b += 2 * n * Hkv * d * cs + pages * (4 + Hkv * scales)                 # the cache
            b += 2 * (L - n - first) * Hkv * d * cs + 2 * (L - first) * Hkv * d * 2  # older tokens; the blocks' values
            f += n * (Hq + Hkv) * case["rot"] * 3 + (2 * (L - first) * Hkv * d * 3 if cs == 1 else 0)
        elif case["op"] == "keep":
            m = len(kept[i][1])
            moved = sum(a != j for j, a in enumerate(kept[i][1]))
            b += 4 * m + 4 * moved * Hkv * d * cs                                  # rows read and written
            b += 2 * (L - n + m - first) * Hkv * d * (cs + 2) if m else 0          # the blocks read back as values
            f += 2 * moved * Hkv * d * 3 if cs == 1 else 0
        else:
            base, w, s = L - n, case["window"], case["sinks"]
            deep = _depths(marks[i][0])
            pairs = sum(x + 1 for x in deep)
            seen = base
            if w:
                pairs += sum(min(base, max(0, w - 1 - x) + min(s, max(0, base + x + 1 - w))) for x in deep)
                seen = min(base, w - 1 + min(s, base))
            else:
                pairs += n * base
            seen += n
            b += n * Hq * (2 * d * es + 4) + 8 * n + 2 * seen * Hkv * d * cs + -(-seen // pt) * (4 + Hkv * scales)
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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=device)


def _tree_inputs(case, st):
    """Parents, the accepted branches (packed as the drafts are) and their lengths."""
    marks = trees(case)
    st["trees"] = marks
    st["parent"] = _i32([p for t in marks for p in t[0]])
    st["path"] = _i32([p for t in marks for p in t[1] + [0] * (len(t[0]) - len(t[1]))])
    st["accepted"] = _i32([len(t[1]) for t in marks])


def _coordinates(case, n, r):
    """Time, height and width of n tokens of text and pictures; text has its place in all three."""
    out, at = [], 0
    while len(out) < n:
        for _ in range(r.randint(1, 200)):
            out.append((at, at, at))
            at += 1
        h, w = r.randint(2, 24), r.randint(2, 24)
        out += [(at, at + y, at + x) for y in range(h) for x in range(w)]
        at += max(h, w)
    return out[:n]


def prepare(case, seed):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rnd = random.Random(seed)
    dt, d = DT[case["dtype"]], case["d"]
    lens = lengths(case)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    T = cu[-1]
    st = {"case": dict(case), "lens": lens, "maxq": max(1, max(n for n, _ in lens)), "cu": _i32(cu)}
    tree = st["maxq"] <= MOST
    if tree:
        _tree_inputs(case, st)
    if own:  # what a program keeps: the library, a status word
        import kda_state_chunked_gb300 as kda

        st["kda"] = kda
        st["status"] = torch.zeros(1, dtype=torch.int32, device=device)
    if case["op"] == "verify":
        return _prepare_states(case, st, g, rnd, T)
    pt, Hq, Hkv = case["pt"], case["Hq"], case["Hkv"]
    need = [-(-L // pt) for _, L in lens]
    pages = sum(need) + 3
    ids = list(range(pages))
    rnd.shuffle(ids)
    maxp = max(1, max(need))
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [-1] * (maxp - n))
        at += n
    # a cache as earlier steps left it, its blocks' free slots filled with what was there before
    store = torch.empty(pages, Hkv, 2, pt, d, dtype=torch.int8 if case["fmt"] == "i8" else torch.bfloat16, device=device)
    scales = torch.empty(pages, Hkv, 2, device=device) if case["fmt"] == "i8" else None
    step = max(1, (1 << 27) // (Hkv * 2 * pt * d))
    for a in range(0, pages, step):
        x = torch.randn(store[a:a + step].shape, generator=g, device=device)
        if scales is None:
            store[a:a + step] = x
        else:
            x *= 0.5 + torch.rand(x.shape[0], Hkv, 2, 1, 1, generator=g, device=device)
            sc = x.abs().amax((3, 4)) / 127
            scales[a:a + step] = sc
            store[a:a + step] = torch.round(x / sc[..., None, None])
    page_bytes = -(-Hkv * _record_bytes(case) // 256) * 256
    st.update(store=store, scales=scales, bytes=_lay_out(case, store, scales, page_bytes),
              table=_i32(table).view(len(lens), maxp), kv_len=_i32([L for _, L in lens]), spare=ids[-1])
    # what is read back of the cache: the blocks that a call touches, up to the tokens that it leaves there
    begin, cu_out = [], [0]
    for i, (n, L) in enumerate(lens):
        end = L - n + len(st["trees"][i][1]) if case["op"] == "keep" else L
        first = (L - n) // pt * pt if end > L - n else end
        begin.append(first)
        cu_out.append(cu_out[-1] + end - first)
    st.update(begin=_i32(begin), cu_out=_i32(cu_out), rows=cu_out[-1])
    if case["op"] != "attend":
        st["k_out"] = torch.empty(st["rows"], Hkv, d, dtype=torch.bfloat16, device=device)
        st["v_out"] = torch.empty_like(st["k_out"])
    if case["op"] == "keep":
        st["len_out"] = torch.zeros_like(st["kv_len"])
    else:
        # queries, keys and values are parts of one projection's output
        x = torch.randn(T, Hq + 2 * Hkv, d, generator=g, device=device)
        x[:, :Hq] *= 2
        x = x.to(dt)
        st.update(q=x[:, :Hq], k=x[:, Hq:Hq + Hkv], v=x[:, Hq + Hkv:])
    if tree and case["op"] != "keep":
        st["mask"] = torch.zeros(T, dtype=torch.int64, device=device)
        st["pos"] = torch.zeros(T, dtype=torch.int32, device=device)
        if case["op"] == "attend":
            # the plan of these trees, as the layers before this one used it
            st["mask"], st["pos"] = _plan(st)
    if case["op"] == "place":
        axes = len(sections(case))
        if not tree or axes > 1:
            r = random.Random(seed + 1)
            rows = []
            for n, L in lens:
                rows += _coordinates(case, L, r)[L - n:]
            st["coords"] = _i32([c[:axes] for c in rows]).view(T, axes)
        f = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=device) / case["rot"])
        ang = torch.arange(max(L for _, L in lens), dtype=torch.float64, device=device)[:, None] * f
        st["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float()
        st["q_out"] = torch.empty(T, Hq, d, dtype=dt, device=device)
    elif case["op"] == "attend":
        st["o"] = torch.empty(T, Hq, d, dtype=dt, device=device)
        st["lse"] = torch.empty(T, Hq, device=device)
    if own:
        st["pool"] = kda.Pool(page_bytes, pages)
        st["pool"].base = st["bytes"]
        st["fmt"] = kda.KDA_KV_I8 if case["fmt"] == "i8" else kda.KDA_KV_BF16
        if case["op"] == "attend":
            st["ws"] = kda.attn_tree_workspace(st["q"], Hkv, len(lens), st["maxq"])
    return st


def _state_record(case):
    es, d = ES[case["dtype"]], case["d"]
    return -(-(d * d * 4 + 9 * d * es) // 256) * 256


def _prepare_states(case, st, g, rnd, T):
    d, H, B, dt = case["d"], case["H"], case["seqs"], DT[case["dtype"]]
    rec, P = _state_record(case), H // case["hpp"]
    pages = B * P + 2
    ids = list(range(pages))
    rnd.shuffle(ids)
    unit = lambda x: x / x.square().sum(-1, keepdim=True).sqrt()  # noqa: E731
    rn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    st["q"], st["k"], st["v"] = unit(rn(T, H, d)).to(dt), unit(rn(T, H, d)).to(dt), rn(T, H, d).to(dt)
    st["alpha"], st["beta"] = torch.sigmoid(rn(T, H, d) + 3).to(dt), torch.sigmoid(rn(T, H)).to(dt)
    st["conv_w"] = rn(H, 3 * d, 4) * 0.5
    pool = torch.zeros(pages, case["hpp"], rec, dtype=torch.uint8, device=device)
    st["bytes"] = pool
    st["S"] = pool[..., :d * d * 4].view(torch.float32).view(pages, case["hpp"], d, d)
    for a in range(0, pages, 64):
        x = st["S"][a:a + 64]
        x.copy_(rn(*x.shape) * 0.3)
    st["win"] = pool[..., d * d * 4:d * d * 4 + 9 * d * ES[case["dtype"]]].view(dt).view(pages, case["hpp"], 3, 3 * d)
    st["win"].copy_(torch.cat([unit(rn(pages, case["hpp"], 3, d)), unit(rn(pages, case["hpp"], 3, d)),
                               rn(pages, case["hpp"], 3, d)], -1))
    st["pages"] = _i32(ids[:B * P]).view(B, P)
    st["o"] = torch.zeros(T, H, d, dtype=dt, device=device)
    if own:
        st["pool"] = st["kda"].Pool(rec * case["hpp"], pages)
        st["pool"].base = pool.view(-1)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    return {"place": _place, "attend": _attend, "keep": _keep, "verify": _verify}[st["case"]["op"]](st)


def _own(st):
    c, kda = st["case"], st["kda"]
    if c["op"] == "verify":
        kda.kda_verify_tree(st["pool"], st["cu"], st["parent"], st["maxq"], st["q"], st["k"], st["v"], st["alpha"],
                            st["beta"], st["conv_w"], st["o"], st["pages"], st["status"])
        kda.kda_verify_tree_accept(st["pool"], st["cu"], st["path"], st["accepted"], st["maxq"], st["q"], st["k"],
                                   st["v"], st["alpha"], st["beta"], st["conv_w"], st["pages"], st["status"])
        return {"o": st["o"], "S": st["S"], "win": st["win"]}
    where = (st["cu"], st["kv_len"], st["table"], st["maxq"])
    if c["op"] == "attend":
        kda.kda_attn_tree(st["pool"], c["Hkv"], st["fmt"], c["pt"], *where, st["mask"], st["q"], st["o"], st["ws"],
                          st["status"], window=c["window"], sinks=c["sinks"], pos=st["pos"], lse=st["lse"])
        return {"o": st["o"], "lse": st["lse"]}
    out = {}
    if c["op"] == "place":
        if "parent" in st:
            kda.kda_tree_plan(st["cu"], st["kv_len"], st["parent"], st["maxq"], st["mask"], st["pos"], st["status"])
            out = {"mask": st["mask"], "pos": st["pos"]}
        kda.kda_kv_append_at(st["pool"], st["fmt"], c["pt"], *where, st["q"], st["k"], st["v"], st["cos_sin"],
                             st["coords"] if "coords" in st else st["pos"], sections(c), st["q_out"], st["status"],
                             interleaved=c["pairs"])
        out["q"] = st["q_out"]
    else:
        kda.kda_kv_accept(st["pool"], c["Hkv"], c["d"], st["fmt"], c["pt"], *where, st["path"], st["accepted"],
                          st["len_out"], st["status"])
        out["kv_len"] = st["len_out"]
    kda.kda_kv_gather(st["pool"], st["fmt"], c["pt"], st["cu_out"], st["begin"], st["table"], st["k_out"], st["v_out"],
                      st["status"])
    out.update(k=st["k_out"], v=st["v_out"])
    return out


def _where(cu, rows):
    """The sequence of each packed row, and the row's index in it."""
    at = torch.arange(rows, device=cu.device)
    s = torch.searchsorted(cu[1:].long(), at, right=True)
    return s, at - cu.long()[s]


def _plan(st):
    """Bits of each draft's ancestors and itself, and its position."""
    T, M = st["parent"].shape[0], st["maxq"]
    s, r = _where(st["cu"], T)
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    parent = torch.full((n.shape[0], M), -1, dtype=torch.int64, device=s.device)
    parent[s, r] = st["parent"].long()
    mask = torch.zeros(n.shape[0], M + 1, dtype=torch.int64, device=s.device)   # the last for what has no parent
    depth = torch.full((n.shape[0], M + 1), -1, dtype=torch.int64, device=s.device)
    for i in range(M):
        up = torch.where(parent[:, i:i + 1] < 0, M, parent[:, i:i + 1])
        mask[:, i:i + 1] = mask.gather(1, up) | (1 << i if i < 63 else -1 << 63)
        depth[:, i:i + 1] = depth.gather(1, up) + 1
    base = st["kv_len"].long() - n
    return mask[s, r], (base[s] + depth[s, r]).int()


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


def _angles(st, coords):
    """The row of cosines and sines of each token: frequency i goes by its section's coordinate."""
    c = st["case"]
    axis = torch.repeat_interleave(torch.arange(len(sections(c))), torch.tensor(sections(c))).to(coords.device)
    h = c["rot"] // 2
    at = coords.long()[:, axis]
    i = torch.arange(h, device=coords.device)
    return torch.cat([st["cos_sin"][at, i], st["cos_sin"][at, h + i]], 1)


def _blocks(st):
    """The blocks from that of each sequence's first new token on: their pages (a spare one where the sequence has
    none), their slots' places in the sequence, and the first block's number.  [sequence, block(, slot)]"""
    pt, (nseq, maxp) = st["case"]["pt"], st["table"].shape
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    base = st["kv_len"].long() - n
    p0 = base // pt
    J = (st["maxq"] + pt - 2) // pt + 1
    block = p0[:, None] + torch.arange(J, device=p0.device)
    there = (block * pt < st["kv_len"].long()[:, None]) & (n[:, None] > 0)
    page = torch.where(there, st["table"].long().gather(1, block.clamp(max=maxp - 1)), st["spare"])
    return page, block[..., None] * pt + torch.arange(pt, device=p0.device), p0, base, n


def _place(st):
    c = st["case"]
    pt, Hkv, d, T = c["pt"], c["Hkv"], c["d"], st["q"].shape[0]
    nseq = st["table"].shape[0]
    out, coords = {}, st.get("coords")
    if "parent" in st:
        out["mask"], out["pos"] = _plan(st)
        coords = out["pos"][:, None] if coords is None else coords
    cs = _angles(st, coords)
    q, k, v = _rotate(st["q"].float(), cs, c["pairs"]), _rotate(st["k"].float(), cs, c["pairs"]), st["v"].float()
    page, at, p0, old, n = _blocks(st)
    s, r = _where(st["cu"], T)
    J = page.shape[1]
    new = torch.zeros(nseq, J * pt, Hkv, 2, d, device=q.device)
    new[s, old[s] + r - p0[s] * pt] = torch.stack([k, v], 2)
    new = new.view(nseq, J, pt, Hkv, 2, d).permute(0, 1, 3, 4, 2, 5)     # [seq, block, head, k/v, slot, d]
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
        st["scales"][page.reshape(-1)] = scale.reshape(-1, Hkv, 2)
    else:
        code = torch.where(is_new, new.bfloat16(), have)
    st["store"][page.reshape(-1)] = code.reshape(-1, Hkv, 2, pt, d)
    out["q"] = q.to(st["q"].dtype)
    out["k"], out["v"] = _read_back(st)
    return out


def _read_back(st):
    """Keys and values of the cached ranges, as bf16."""
    pt = st["case"]["pt"]
    s, r = _where(st["cu_out"], st["rows"])
    at = st["begin"].long()[s] + r
    page, slot = st["table"].long()[s, at // pt], at % pt
    x = st["store"][page, :, :, slot]                                    # [rows, head, k/v, d]
    if st["scales"] is not None:
        x = (x.float() * st["scales"][page][..., None]).bfloat16()
    return x[:, :, 0], x[:, :, 1]


def _keep(st):
    c = st["case"]
    pt, Hkv, d, M = c["pt"], c["Hkv"], c["d"], st["maxq"]
    nseq = st["table"].shape[0]
    page, at, p0, base, n = _blocks(st)
    J, m = page.shape[1], st["accepted"].long()
    s, r = _where(st["cu"], st["path"].shape[0])
    path = torch.zeros(nseq, M, dtype=torch.int64, device=s.device)
    path[s, r] = st["path"].long()
    i = at - base[:, None, None]                                         # a slot's place in the branch
    taken = (i >= 0) & (i < m[:, None, None])
    src = torch.where(taken, base[:, None, None] + path.gather(1, i.clamp(0, M - 1).view(nseq, -1)).view(i.shape), at)
    local = (src - p0[:, None, None] * pt).clamp(0, J * pt - 1)          # place among these blocks
    have = st["store"][page]                                             # [seq, block, head, k/v, slot, d]
    rows = have.permute(0, 1, 4, 2, 3, 5).reshape(nseq, J * pt, Hkv, 2, d)
    pick = torch.arange(nseq, device=s.device)[:, None], local.view(nseq, -1)
    code = rows[pick].view(nseq, J, pt, Hkv, 2, d).permute(0, 1, 3, 4, 2, 5)
    touched = taken.any(2)[..., None, None]
    mine = taken[:, :, None, None, :, None]
    if c["fmt"] == "i8":
        sc = st["scales"][page]                                          # [seq, block, head, k/v]
        home = torch.arange(J, device=s.device)[None, :, None]
        stays = (at < base[:, None, None]) | (taken & (local // pt == home))
        comes = (taken & ~stays)[:, :, None, None, :, None]
        per_slot = sc[torch.arange(nseq, device=s.device)[:, None, None], local // pt]
        per_slot = per_slot.permute(0, 1, 3, 4, 2)[..., None]            # the scale that a slot's row comes with
        val = code.float() * per_slot
        seven = torch.full_like(sc, 127.0)
        grown = torch.where(comes, val, 0).abs().amax((4, 5)) / seven
        kept = torch.where(stays.any(2)[..., None, None], sc, 0)
        scale = torch.where(touched, torch.maximum(grown, kept), sc)
        again = torch.where(scale[..., None, None] > 0, torch.round(val / scale[..., None, None]), 0).to(torch.int8)
        whole = (mine | (at < base[:, None, None])[:, :, None, None, :, None]) & touched[..., None, None]
        code = torch.where(whole, again, have)
        st["scales"][page.reshape(-1)] = scale.reshape(-1, Hkv, 2)
    else:
        code = torch.where(mine, code, have)
    st["store"][page.reshape(-1)] = code.reshape(-1, Hkv, 2, pt, d)
    k, v = _read_back(st)
    return {"kv_len": (base + m).int(), "k": k, "v": v}


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
    base = st["kv_len"].long() - n
    q = torch.zeros(nseq, M, Hq, d, device=kv.device)
    q[s, r] = st["q"].float()
    q = q.view(nseq, M, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(nseq, Hkv, G * M, d)
    score = torch.matmul(q, kv[0].transpose(-1, -2)).view(nseq, Hkv, G, M, L) * d ** -0.5
    mask = torch.zeros(nseq, M, dtype=torch.int64, device=q.device)
    pos = torch.zeros(nseq, M, dtype=torch.int64, device=q.device)
    mask[s, r], pos[s, r] = st["mask"], st["pos"].long()
    j = torch.arange(L, device=q.device)
    i = j - base[:, None]                             # a token's place among the drafts  [seq, token]
    old = (i < 0)[:, None, :].expand(-1, M, -1)
    if c["window"]:
        old = old & ((j > pos[..., None] - c["window"]) | (j < c["sinks"]))
    bit = (mask[..., None] >> i.clamp(0, 63)[:, None, :]) & 1
    see = old | ((i >= 0) & (i < n[:, None]))[:, None, :] & (bit == 1)
    see = (see & (torch.arange(M, device=q.device) < n[:, None])[..., None])[:, None, None]
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


def _padded(st, x):
    """[T, ...] as float32 [sequence, draft, ...], zeros behind a sequence's last."""
    s, r = _where(st["cu"], x.shape[0])
    y = torch.zeros(st["cu"].shape[0] - 1, st["maxq"], *x.shape[1:], device=x.device)
    y[s, r] = x.float()
    return y


def _step(S, q, k, v, alpha, beta):
    """Decay, delta-rule write, read.  S [B, H, d, d]; q, k, v, alpha [B, H, d]; beta [B, H]."""
    S = S * alpha[..., None]
    w = beta[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * w[..., None, :]
    return S, (S * q[..., None]).sum(-2)


def _verify(st):
    c = st["case"]
    d, H, B, M = c["d"], c["H"], c["seqs"], st["maxq"]
    pages = st["pages"].long()
    S0 = st["S"][pages].view(B, H, d, d)
    raw = torch.cat([st["q"], st["k"], st["v"]], -1)                     # [T, H, 3d]
    x, alpha, beta = _padded(st, raw), _padded(st, st["alpha"]), _padded(st, st["beta"])
    win = st["win"][pages].reshape(B, H, 3, 3 * d)
    s, r = _where(st["cu"], raw.shape[0])
    parent = torch.full((B, M), -1, dtype=torch.int64, device=raw.device)
    parent[s, r] = st["parent"].long()
    path = torch.zeros(B, M, dtype=torch.int64, device=raw.device)
    path[s, r] = st["path"].long()
    b = torch.arange(B, device=raw.device)
    # the raw tokens that a draft's convolution reads: itself and the three before it on its branch
    hist = torch.cat([x, win.float().transpose(1, 2).flip(1)], 1)        # drafts, then the window, newest first
    steps = torch.arange(M, device=raw.device)
    up = torch.cat([torch.where(parent < 0, M, parent), torch.tensor([M + 1, M + 2, M + 2], device=raw.device).expand(B, 3)], 1)
    at, y = steps.expand(B, M), torch.zeros_like(x)
    for j in range(4):
        y += st["conv_w"][..., 3 - j] * hist[b[:, None], at]
        at = up.gather(1, at)
    q, k, v = y.split(d, -1)
    states = torch.empty(M + 1, B, H, d, d, device=raw.device)
    states[M] = S0
    o = torch.empty(B, M, H, d, device=raw.device)
    for i in range(M):
        S, o[:, i] = _step(states[torch.where(parent[:, i] < 0, M, parent[:, i]), b], q[:, i], k[:, i], v[:, i], alpha[:, i],
                           beta[:, i])
        states[i] = S
    # the state and window after the accepted branch
    m = st["accepted"].long()
    last = torch.where(m > 0, path.gather(1, (m - 1).clamp(min=0)[:, None])[:, 0], M)
    st["S"][pages] = states[last, b].view(B, pages.shape[1], -1, d, d)
    at, new = last, []
    for _ in range(3):
        new.append(hist[b, at])
        at = up[b, at]
    win = torch.stack(new[::-1], 2).to(st["win"].dtype)                  # [B, H, 3, 3d]
    st["win"][pages] = win.view(B, pages.shape[1], -1, 3, 3 * d)
    return {"o": o[s, r].to(st["q"].dtype), "S": st["S"], "win": st["win"]}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    f = {"place": _exact_place, "attend": _exact_attend, "keep": _exact_keep, "verify": _exact_verify}[case["op"]]
    return f(case, prepare(case, seed))


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


def _exact_turn(case, x, w):
    """Rotation as a product of complex numbers, w [n, rot / 2]."""
    h, w = case["rot"] // 2, w[:, None]
    x = x.clone()
    if case["pairs"]:
        z = torch.view_as_complex(x[..., :2 * h].reshape(*x.shape[:-1], h, 2).contiguous()) * w
        x[..., :2 * h] = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * h)
    else:
        z = torch.complex(x[..., :h], x[..., h:2 * h]) * w
        x[..., :h], x[..., h:2 * h] = z.real, z.imag
    return x


def _marks(st):
    """The plan of each tree, by walking every draft's branch."""
    mask, pos = [], []
    for (n, L), (parent, _) in zip(st["lens"], st["trees"]):
        for i in range(n):
            up = _branch(parent, i)
            bits = sum(1 << j for j in up)
            mask.append(bits - (1 << 64) if bits >> 63 else bits)
            pos.append(L - n + len(up) - 1)
    return torch.tensor(mask, dtype=torch.int64, device=device), _i32(pos)


def _exact_place(case, st):
    pt, cu, h = case["pt"], st["cu"].tolist(), case["rot"] // 2
    out, coords = {}, st.get("coords")
    if "parent" in st:
        out["mask"], out["pos"] = _marks(st)
        coords = out["pos"][:, None] if coords is None else coords
    turn, at = [], 0
    for a, size in enumerate(sections(case)):
        row = st["cos_sin"][coords[:, a].long()].double()
        turn.append(torch.complex(row[:, at:at + size], row[:, h + at:h + at + size]))
        at += size
    turn = torch.cat(turn, 1)
    qs, ks, vs = [], [], []
    for i, (n, L) in enumerate(st["lens"]):
        a, b = cu[i], cu[i + 1]
        if not n:
            continue
        qs.append(_exact_turn(case, st["q"][a:b].double(), turn[a:b]))
        first = (L - n) // pt * pt
        k0, v0 = _tokens(case, st, i, first, L - n) if L - n > first else (None, None)
        for new, before, w, to in ((_exact_turn(case, st["k"][a:b].double(), turn[a:b]), k0, 0, ks),
                                   (st["v"][a:b].double(), v0, 1, vs)):
            if case["fmt"] != "i8":
                to.append(new if before is None else torch.cat([before, new]))
                continue
            m = new.abs().amax(-1)                                        # [n, Hkv]
            if before is not None:
                low = st["scales"][int(st["table"][i, first // pt]), :, w].double() * 127
                m = torch.cat([low.expand(before.shape[0], -1), m])
                new = torch.cat([before, new])
            to.append(_exact_codes(case, new, m))
    cat = lambda x, H: torch.cat(x) if x else torch.empty(0, H, case["d"], dtype=torch.float64)  # noqa: E731
    out.update(q=cat(qs, case["Hq"]), k=cat(ks, case["Hkv"]), v=cat(vs, case["Hkv"]))
    return out


def _exact_codes(case, x, m):
    """Values x [rows, Hkv, d] of whole blocks (the last one's end may lack) in codes of the blocks' largest m [rows, Hkv]."""
    pt = case["pt"]
    m = torch.cat([m, m.new_zeros(-m.shape[0] % pt, m.shape[1])]).view(-1, pt, case["Hkv"]).amax(1) / 127
    m = m.repeat_interleave(pt, 0)[:x.shape[0], :, None]
    return torch.where(m > 0, torch.round(x / m) * m, 0)


def _exact_keep(case, st):
    pt, ks, vs, lens = case["pt"], [], [], []
    for i, ((n, L), (_, path)) in enumerate(zip(st["lens"], st["trees"])):
        base, m = L - n, len(path)
        lens.append(base + m)
        if not m:
            continue
        first = base // pt * pt
        both = _tokens(case, st, i, first, L)
        rows = list(range(base - first)) + [base - first + p for p in path]   # the kept tokens' old places
        for w, to in ((0, ks), (1, vs)):
            x = both[w][rows]
            if case["fmt"] == "i8":
                # a token that stays in its block brings the block's scale, one that comes its own size
                sc = st["scales"][st["table"][i, first // pt:-(-L // pt)].long(), :, w].double() * 127
                old = torch.tensor([r // pt for r in rows], device=x.device)
                stays = old == torch.arange(len(rows), device=x.device) // pt
                x = _exact_codes(case, x, torch.where(stays[:, None], sc[old], x.abs().amax(-1)))
            to.append(x)
    cat = lambda x: torch.cat(x) if x else torch.empty(0, case["Hkv"], case["d"], dtype=torch.float64)  # noqa: E731
    return {"kv_len": _i32(lens), "k": cat(ks), "v": cat(vs)}


def _exact_attend(case, st):
    cu, G, d = st["cu"].tolist(), case["Hq"] // case["Hkv"], case["d"]
    o = torch.zeros(cu[-1], case["Hq"], d, dtype=torch.float64, device=st["q"].device)
    lse = torch.full((cu[-1], case["Hq"]), -math.inf, dtype=torch.float64, device=o.device)
    for i, ((n, L), (parent, _)) in enumerate(zip(st["lens"], st["trees"])):
        if not n:
            continue
        k, v = _tokens(case, st, i, 0, L)
        at = torch.arange(L, device=o.device)
        hide = torch.zeros(n, L, dtype=torch.bool, device=o.device)
        for r in range(n):
            up = _branch(parent, r)
            p = L - n + len(up) - 1
            if case["window"]:
                hide[r] = (at <= p - case["window"]) & (at >= case["sinks"])
            hide[r, L - n:] = True
            hide[r, torch.tensor(up, device=o.device) + L - n] = False
        for h in range(case["Hq"]):
            x = st["q"][cu[i]:cu[i + 1], h].double() @ k[:, h // G].T / math.sqrt(d)
            x[hide] = -math.inf
            z = torch.logsumexp(x, -1, keepdim=True)
            o[cu[i]:cu[i + 1], h] = torch.exp(x - z) @ v[:, h // G]
            lse[cu[i]:cu[i + 1], h] = z[:, 0]
    return {"o": o, "lse": lse}


def _exact_verify(case, st):
    """The closed form: every draft's write vector by substitution along its branch, no draft's state."""
    d, H, cu = case["d"], case["H"], st["cu"].tolist()
    o = torch.zeros(cu[-1], H, d, dtype=torch.float64, device=st["q"].device)
    S_out, win_out = st["S"].double().clone(), st["win"].double().clone()
    w4 = st["conv_w"].double()
    raw_all = torch.cat([st["q"], st["k"], st["v"]], -1).double()
    for b, ((n, _), (parent, path)) in enumerate(zip(st["lens"], st["trees"])):
        if not n:
            continue
        ids = st["pages"][b].long()
        S0 = st["S"][ids].double().view(H, d, d)
        win = st["win"][ids].double().view(H, 3, 3 * d)
        raw = raw_all[cu[b]:cu[b + 1]]
        al, be = st["alpha"][cu[b]:cu[b + 1]].double(), st["beta"][cu[b]:cu[b + 1]].double()
        x, ups = [], [_branch(parent, i) for i in range(n)]
        for i in range(n):
            up = ups[i]
            x.append(sum(w4[..., 3 - j] * (raw[up[j]] if j < len(up) else win[:, 2 - (j - len(up))]) for j in range(4)))
        x = torch.stack(x)
        q, k, v = x.split(d, -1)                                         # [n, H, d]
        A = torch.empty_like(al)                                         # decay from the state to each draft
        for i in range(n):
            A[i] = al[i] * (A[parent[i]] if parent[i] >= 0 else 1)
        yk = torch.einsum("nhi,hij->nhj", A * k, S0)
        yq = torch.einsum("nhi,hij->nhj", A * q, S0)
        u = torch.empty_like(v)
        for i in range(n):
            # keys of the branch, decayed from where they were written to this draft
            decay, rows = torch.ones_like(al[0]), []
            for j in ups[i]:
                rows.append(decay * k[j])
                decay = decay * al[j]
            rows = torch.stack(rows)                                     # [branch, H, d], itself first
            ck, cq = (rows * k[i]).sum(-1), (rows * q[i]).sum(-1)
            past = ups[i][1:]
            got = (ck[1:, :, None] * u[past]).sum(0) if past else 0
            u[i] = be[i][:, None] * (v[i] - yk[i] - got)
            o[cu[b] + i] = yq[i] + (cq[..., None] * u[ups[i]]).sum(0)
        if path:
            S, decay = torch.zeros_like(S0), torch.ones_like(al[0])
            for j in reversed(path):
                S += (decay * k[j])[..., None] * u[j][:, None, :]
                decay = decay * al[j]
            S += decay[..., None] * S0
            S_out[ids] = S.view(len(ids), -1, d, d)
            last = torch.cat([win, raw[path].transpose(0, 1)], 1)[:, -3:]
            win_out[ids] = last.reshape(len(ids), -1, 3, 3 * d)
    return {"o": o, "S": S_out, "win": win_out}
