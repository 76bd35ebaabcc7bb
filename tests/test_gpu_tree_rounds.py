"""Rounds on trees of drafts through all calls, a tree that is none among them, and the largest calls of single ones.

Attention has the tolerance of test_gpu_kv, states that of test_gpu_tree; everything else is equal."""
import numpy as np
import pytest
import torch

import kda_state_chunked_gb300 as kda
import kv_ref as ref
import tree_ref as tree
from kda_cases import write_object
from test_gpu_kv import DEV, TOL, i32
from test_gpu_tree import OK, Round, States

pytestmark = pytest.mark.gpu
FMTS = [kda.KDA_KV_BF16, kda.KDA_KV_I8]


def filled(fmt, starts, seed, kind=Round):
    """A round's tensors behind contexts of `starts` tokens."""
    c = kind(fmt, starts, seed=seed)
    cu = np.concatenate([[0], np.cumsum(starts)])
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((2, int(cu[-1]), c.Hkv, c.d)).astype(np.float32)).to(DEV, torch.bfloat16)
    kda.kda_kv_append(c.pool, fmt, c.pt, i32(cu), i32(starts), c.table, max(starts), None, x[0], x[1], c.cs, None, c.status)
    assert kda.kda_sync_status(c.status) == OK
    return c


def owned(c, s):
    """Bytes of a sequence's pages: its cache and its state."""
    return torch.cat([c.pool.page_view(int(p)) for p in list(c.table[s].cpu()) + list(c.pages[s])]).clone()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [0, 1, -2])          # draft 0's parent: itself, one behind it, none at all
@pytest.mark.parametrize("left", ["another round's", "nobody's"])
def test_a_tree_that_is_none_leaves_its_cache_and_state(fmt, bad, left):
    """The append and the attention see masks and positions alone: what an earlier round left in them, or a buffer that
    nobody wrote, must not pass for this tree's."""
    starts = [3, 21, 33]
    c, e = filled(fmt, starts, 53), filled(fmt, starts, 53)
    for x in (c, e):
        x.draft(74, starts)
        x.accepted[1] = 0
    if left == "nobody's":
        c.mask.fill_(-1)
        c.pos.fill_(5)
    else:
        base = c.pool.base.clone()
        c.calls()
        assert kda.kda_sync_status(c.status) == OK
        c.pool.base.copy_(base)
    first, end = int(c.cu_host[1]), int(c.cu_host[2])
    c.parent[first] = bad
    before = owned(c, 1)
    c.calls()
    e.calls()
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META) and kda.kda_sync_status(e.status) == OK
    assert torch.equal(owned(c, 1), before) and torch.equal(c.new_lens, e.new_lens) and int(c.new_lens[1]) == starts[1]
    assert (c.pos[first:end] == -1).all() and (c.mask[first:end] == 0).all()
    for s in (0, 2):
        rows = slice(int(c.cu_host[s]), int(c.cu_host[s + 1]))
        assert torch.equal(owned(c, s), owned(e, s))
        assert torch.equal(c.o[rows], e.o[rows]) and torch.equal(c.o_rec[rows], e.o_rec[rows])


class Seen(Round):
    """A round that also looks at the cache between the attention and the kept branch."""

    def calls(self):
        Hq, Hkv = self.Hq, self.Hkv
        x, meta = self.x, (self.cu, self.lens, self.table, self.max_q)
        kda.kda_tree_plan(self.cu, self.lens, self.parent, self.max_q, self.mask, self.pos, self.status)
        kda.kda_kv_append_at(self.pool, self.fmt, self.pt, *meta, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], self.cs, self.pos,
                             [self.d // 2], self.q, self.status)
        kda.kda_attn_tree(self.pool, Hkv, self.fmt, self.pt, *meta, self.mask, self.q, self.o, self.ws, self.status)
        lens = [int(n) for n in self.lens.cpu()]
        self.there = lens, *(t.double().cpu().numpy() for t in self.cached(lens))

    def check_answers(self):
        """o against a softmax in 64 bits over the values that the cache holds, by the branches of the trees themselves."""
        lens, k, v = self.there
        q, o = self.q.double().cpu().numpy(), self.o.double().cpu().numpy()
        G, off = self.Hq // self.Hkv, np.concatenate([[0], np.cumsum(lens)])
        worst = top = 0.0
        for s, parent in enumerate(self.trees):
            base = lens[s] - len(parent)
            for i in range(len(parent)):
                rows = off[s] + np.array(list(range(base)) + [base + j for j in sorted(tree.branch(parent, i))])
                for h in range(self.Hq):
                    x = k[rows, h // G] @ q[self.cu_host[s] + i, h] / self.d ** 0.5
                    e = np.exp(x - x.max())
                    want = e @ v[rows, h // G] / e.sum()
                    worst, top = max(worst, np.abs(o[self.cu_host[s] + i, h] - want).max()), max(top, np.abs(want).max())
        assert worst <= TOL["bf16"] * top, worst / top


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("max_q", [3, 24])           # 6 and 48 rows a head: either attention kernel
def test_answers_of_a_round(fmt, max_q, monkeypatch):
    monkeypatch.setattr(Seen, "max_q", max_q)
    starts = [0, 1, 15, 16, 40, 130]
    c = filled(fmt, starts, 57, Seen)
    for seed in (75, 76):
        c.draft(seed, starts)
        c.calls()
        assert kda.kda_sync_status(c.status) == OK
        c.check_answers()


def test_a_captured_round_over_the_8_bit_cache():
    starts = [3, 1, 33]
    c, e = filled(kda.KDA_KV_I8, starts, 58), filled(kda.KDA_KV_I8, starts, 58)
    c.draft(77, starts)
    side, base = torch.cuda.Stream(), c.pool.base.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.calls()
    torch.cuda.current_stream().wait_stream(side)
    c.pool.base.copy_(base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.calls()
    lens = starts
    for seed in (78, 79, 80):
        for x in (c, e):
            x.draft(seed, lens)
        graph.replay()
        e.calls()
        assert kda.kda_sync_status(c.status) == OK and kda.kda_sync_status(e.status) == OK
        T = c.cu_host[-1]
        assert torch.equal(c.pool.base, e.pool.base) and torch.equal(c.new_lens, e.new_lens)
        assert torch.equal(c.o[:T], e.o[:T]) and torch.equal(c.o_rec[:T], e.o_rec[:T])
        lens = c.new_lens.cpu().numpy()


@pytest.mark.parametrize("fmt", FMTS)
def test_drafts_on_three_axes_behind_pictures(fmt):
    """Coordinates formed from the plan's depths: the kept branch is the accepted tokens placed by themselves."""
    starts = [3, 16, 33]
    c, e = filled(fmt, starts, 60), filled(fmt, starts, 60)
    c.draft(81, starts)
    next_free = torch.tensor([[50, 50, 50], [9, 9, 9], [120, 120, 120]], device=DEV)     # behind pictures: not the places
    sections, x, Hq, Hkv = [c.d // 4, c.d // 8, c.d // 8], c.x, c.Hq, c.Hkv
    meta, T = (c.cu, c.lens, c.table, c.max_q), int(c.cu_host[-1])
    seq = torch.repeat_interleave(torch.arange(c.n, device=DEV), torch.tensor(np.diff(c.cu_host), device=DEV))
    kda.kda_tree_plan(c.cu, c.lens, c.parent, c.max_q, c.mask, c.pos, c.status)
    depth = c.pos[:T] - torch.tensor(starts, device=DEV)[seq]
    coords = torch.zeros(c.T, 3, dtype=torch.int32, device=DEV)
    coords[:T] = torch.where(c.pos[:T, None] < 0, -1, next_free[seq] + depth[:, None]).int()
    kda.kda_kv_append_at(c.pool, fmt, c.pt, *meta, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], c.cs, coords, sections, c.q, c.status)
    kda.kda_kv_accept(c.pool, Hkv, c.d, fmt, c.pt, *meta, c.path, c.accepted, c.new_lens, c.status)
    lens = [a + len(p) for a, p in zip(starts, c.paths)]
    rows = torch.tensor([c.cu_host[s] + i for s, p in enumerate(c.paths) for i in p], device=DEV)
    at = torch.tensor([[int(next_free[s, 0]) + i] * 3 for s, p in enumerate(c.paths) for i in range(len(p))], device=DEV)
    y, q = x[rows], torch.empty(len(rows), Hq, c.d, dtype=x.dtype, device=DEV)
    cu = i32(np.concatenate([[0], np.cumsum([len(p) for p in c.paths])]))
    kda.kda_kv_append_at(e.pool, fmt, e.pt, cu, i32(lens), e.table, e.max_q, y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], e.cs,
                         at.int(), sections, q, e.status)
    assert kda.kda_sync_status(c.status) == OK and kda.kda_sync_status(e.status) == OK
    assert c.new_lens.tolist() == lens and torch.equal(c.q[rows], q)
    for a, b in zip(c.cached(lens), e.cached(lens)):
        if fmt == kda.KDA_KV_BF16:
            assert torch.equal(a, b)
        else:                          # each side codes a block anew at most twice: steps of max / 127, rounded by half
            assert ((a - b).abs() <= 2 * b.abs().max() / 127).all()


# ------------------------------------------------------------------ the state after long branches
@pytest.mark.parametrize("page_bytes", [65536, 1 << 20])
def test_branches_of_every_length(page_bytes):
    """1 to 64 accepted tokens: those that come with a record, and those behind them."""
    c = States(list(range(1, 65)), H=4, d=128, chain=1.0, seed=55, page_bytes=page_bytes)
    paths = [list(range(n)) if b % 2 else tree.random_path(c.r, p, 1.0) for b, (n, p) in enumerate(zip(c.sizes, c.parents))]
    c.accept(paths)
    assert kda.kda_sync_status(c.status) == OK
    for b, path in enumerate(paths):
        c.check_state(b, path)


@pytest.mark.parametrize("B", [1 << 24, (1 << 24) + 1])
def test_millions_of_requests_of_which_two_accept(B):
    c = States([1, 2], H=1, d=128, chain=1.0, seed=56, page_bytes=1 << 20)
    one = dict(dtype=torch.int32, device=DEV)
    cu, accepted, pages = torch.ones(B + 1, **one), torch.zeros(B, **one), torch.zeros(B, 1, **one)
    cu[0], cu[-1] = 0, 3
    accepted[0], accepted[-1] = 1, 2
    pages[0], pages[-1] = i32(c.pages[0]), i32(c.pages[1])
    kda.kda_verify_tree_accept(c.pool, cu, i32([0, 0, 1]), accepted, 2, *c.tokens(), pages, c.status)
    assert kda.kda_sync_status(c.status) == OK
    c.check_state(0, [0])
    c.check_state(1, [0, 1])


# ------------------------------------------------------------------ products with a state that cancel
@pytest.mark.parametrize("d", [64, 128])
def test_a_state_that_cancels(d):
    """Keys and queries at right angles to what the state holds: the products with it are sums of large terms that come to
    little.  Element by element, with |.| products of absolute values: bf16 calls take either operand in two bf16 terms (2^-16
    of it each) and leave out the smallest product (2^-16), and their sums are cut at 2^-23 some 24 times: 4 x 2^-16 of
    |S|^T |A k| and |S|^T |A q|, the former times beta <q, k>; o's rounding is 2^-8 of it."""
    B, H, r = 6, 2, np.random.default_rng(59)
    c = States([1] * B, H=H, d=d, seed=59)
    c.w[:] = 0
    c.w[:, :, 3] = 1                                      # the convolution hands the token on
    bf = lambda x: ref.to_bf16(x.astype(np.float32)).astype(np.float64)  # noqa: E731
    o = np.zeros((B, H, d))
    room = np.zeros_like(o)
    for b in range(B):
        K, V = r.standard_normal((H, d // 2, d)), 8 * r.standard_normal((H, d // 2, d))
        S = np.einsum("hmi,hmj->hij", K, V).astype(np.float32)
        c.S[b][:] = S
        write_object(c.pool, c.pages[b], c.S[b], c.win[b], "bf16")
        for h in range(H):
            free = np.linalg.svd(K[h])[2][d // 2:]        # right angles to all keys
            c.q[b, h], c.k[b, h] = (bf(r.standard_normal(d // 2) @ free / d ** 0.5) for _ in range(2))
            q, k, v, a = (x[b, h].astype(np.float64) for x in (c.q, c.k, c.v, c.alpha))
            beta, S64 = float(c.beta[b, h]), S[h].astype(np.float64)
            u = beta * (v - S64.T @ (a * k))
            o[b, h] = S64.T @ (a * q) + (q @ k) * u
            room[b, h] = (np.abs(S64).T @ np.abs(a * q) + abs(q @ k) * beta * (np.abs(S64).T @ np.abs(a * k))) * 4 * 2.0 ** -16
    got = c.verify().double().cpu().numpy()
    assert kda.kda_sync_status(c.status) == OK
    assert np.abs(o - np.stack([c.expect(b)[0][0] for b in range(B)])).max() <= 1e-12 * np.abs(o).max()
    assert (np.abs(got - o) <= room + (np.abs(o) + room) * 2.0 ** -8).all()
