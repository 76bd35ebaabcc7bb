"""Speculation with trees of drafts on the GPU, against a plain model.

Plans, appended and kept bytes are equal bit for bit.  Attention has the tolerances of test_gpu_kv (the same kernels'
roundings).  States, on max |x - ref| / max |ref| of a (request, head):
  sums    192 products at most (128 channels, 64 drafts) of fp32 terms, each off by 2^-24 of its size: 1.2e-5 of the
          terms' sum, which in these inputs (unit keys, 0 < beta < 1) is within 8 times the largest result: 1e-4
  bf16 o  one rounding, 2^-9 of the value, and two-term products, 2^-16 of the terms' sum: 2^-9 + 8 x 2^-16 < 2^-8"""
import numpy as np
import pytest
import torch

import kda_state_chunked_gb300 as kda
import kv_ref as ref
import tree_ref as tree
from kda_cases import random_state, read_object, read_object_bytes, rel_err, write_object
from oracle import policy
from test_gpu_kv import DEV, DT, FMT, KINDS, Case, i32

pytestmark = pytest.mark.gpu
OK = (kda.KDA_OK, 0)
STATE_TOL = {"f32": 1e-4, "bf16": 2.0 ** -8}


def i64(mask):
    return torch.from_numpy(tree.as_int64(mask)).to(DEV)


def word():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ plans
def plan_call(parents, lens, max_q=64, cu=None):
    cu = np.concatenate([[0], np.cumsum([len(p) for p in parents])]) if cu is None else cu
    flat = [x for p in parents for x in p]
    mask = torch.full((len(flat),), -77, dtype=torch.int64, device=DEV)
    pos = torch.full((len(flat),), -77, dtype=torch.int32, device=DEV)
    st = word()
    kda.kda_tree_plan(i32(cu), i32(lens), i32(flat), max_q, mask, pos, st)
    return mask.cpu().numpy(), pos.cpu().numpy(), kda.kda_sync_status(st)


def test_plan_of_every_size_and_shape():
    r = np.random.default_rng(1)
    parents = [tree.random_tree(r, n, c) for n in (0, 1, 2, 3, 31, 32, 33, 63, 64) for c in (0.0, 0.5, 1.0)]
    parents += [[-1] * 64, list(range(-1, 63))]
    lens = [len(p) + int(r.integers(0, 5000)) for p in parents]
    mask, pos, st = plan_call(parents, lens)
    assert st == OK
    want = [tree.plan(p, L - len(p)) for p, L in zip(parents, lens)]
    assert np.array_equal(mask, tree.as_int64([m for w in want for m in w[0]]))
    assert np.array_equal(pos, np.array([p for w in want for p in w[1]]))


def test_plan_skips_trees_that_are_none():
    good = [-1, 0, 0, 1]
    parents = [good, [-1, 1, 0], [0], [-1, -2], [-1, 0, 1, 5], good, [-1] * 9]
    mask, pos, st = plan_call(parents, [4, 9, 9, 9, 9, 3, 99], max_q=8)
    assert st == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    assert list(mask[:4]) == [1, 3, 5, 11] and list(pos[:4]) == [0, 1, 1, 2]
    assert (mask[4:] == -77).all() and (pos[4:] == -77).all()
    mask, pos, st = plan_call([good, good], [4, 4], cu=[0, 4, 9])          # cu beyond the rows
    assert st == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META) and (mask[4:] == -77).all() and (mask[:4] > 0).all()


# ------------------------------------------------------------------ tokens at positions of their own
def angles(n, rot):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def gathered(cs, pos, sections):
    """Row t: angle f of its section's coordinate."""
    axis = np.repeat(np.arange(len(sections)), sections)
    f = np.arange(len(axis))
    return np.concatenate([cs[pos[:, axis], f], cs[pos[:, axis], len(axis) + f]], 1)


class Placed(Case):
    """A batch whose tokens have coordinates of their own, and the appended result as it has to be."""

    def __init__(self, lens, sections, pairs=False, **kw):
        super().__init__(lens, **kw)
        self.sections, self.pairs, self.rot = sections, pairs, 2 * sum(sections)
        self.cs = angles(300, self.rot)
        self.pos = self.r.integers(0, 300, (self.T, len(sections)))
        x = self.token(self.G * self.Hkv + 2 * self.Hkv)
        Hq = self.G * self.Hkv
        self.x, self.q, self.k, self.v = x, x[:, :Hq], x[:, Hq:Hq + self.Hkv], x[:, Hq + self.Hkv:]

    def append(self, pos=None, q_out=True):
        x = self.gpu(self.x)
        Hq, n = self.G * self.Hkv, self.Hkv
        out = torch.full((self.T, Hq, self.d), 7.0, dtype=DT[self.dtype], device=DEV)
        kda.kda_kv_append_at(self.pool, FMT[self.fmt], self.pt, *self.meta, self.max_q, x[:, :Hq] if q_out else None,
                             x[:, Hq:Hq + n], x[:, Hq + n:], torch.from_numpy(self.cs).to(DEV), i32(self.pos if pos is None else pos),
                             self.sections, out if q_out else None, self.status, interleaved=self.pairs)
        return out

    def expect(self, rows=None):
        turn = gathered(self.cs, self.pos, self.sections)
        q = ref.rotate(np.ascontiguousarray(self.q), turn, self.pairs)
        k = ref.rotate(np.ascontiguousarray(self.k), turn, self.pairs)
        ref.append(self.stored, self.scales, self.table, self.cu, self.kv_len, k, self.v, None, False, self.pt)
        return q if self.dtype == "f32" else ref.to_bf16(q)

    def bytes(self):
        return self.pool.base.cpu().numpy()

    def packed(self):
        return ref.pack(self.stored, self.scales, self.fmt, self.page_bytes)


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("sections,pairs", [([32], False), ([16, 8, 8], False), ([8, 24], True), ([8, 8, 8, 8], True)])
def test_append_at_matches_bit_for_bit(fmt, dtype, d, sections, pairs):
    c = Placed([(5, 5), (1, 64), (0, 30), (8, 70), (3, 131), (1, 1)], sections, pairs, fmt=fmt, dtype=dtype, d=d, pt=64, seed=3).on_gpu()
    q = c.append()
    assert kda.kda_sync_status(c.status) == OK
    want = c.expect()
    assert np.array_equal(q.float().cpu().numpy(), want)
    assert np.array_equal(c.bytes(), c.packed())


@pytest.mark.parametrize("lens,pt", [([(300, 300), (64, 500), (65, 130)], 48), ([(1, 9), (1, 16), (1, 17)], 16), ([(200, 333)], 128)])
@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
def test_append_at_of_prompts_and_single_tokens(lens, pt, fmt):
    c = Placed(lens, [16, 24, 24], fmt=fmt, d=128, pt=pt, seed=4).on_gpu()
    q = c.append()
    assert kda.kda_sync_status(c.status) == OK
    assert np.array_equal(q.float().cpu().numpy(), c.expect()) and np.array_equal(c.bytes(), c.packed())


def test_append_at_of_keys_alone():
    c = Placed([(6, 40), (2, 90)], [16, 16], d=64, seed=5).on_gpu()
    c.append(q_out=False)
    assert kda.kda_sync_status(c.status) == OK
    c.expect()
    assert np.array_equal(c.bytes(), c.packed())


def test_append_at_places_is_append():
    c = Placed([(6, 40), (9, 200), (1, 77)], [64], d=128, seed=6).on_gpu()
    c.pos = np.concatenate([np.arange(L - n, L) for n, L in c.lens])[:, None]
    before = c.pool.base.clone()
    q = c.append()
    at = c.pool.base.clone()
    c.pool.base.copy_(before)
    x, Hq, n = c.gpu(c.x), c.G * c.Hkv, c.Hkv
    plain = torch.empty_like(q)
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, x[:, :Hq], x[:, Hq:Hq + n], x[:, Hq + n:],
                      torch.from_numpy(c.cs).to(DEV), plain, c.status)
    assert kda.kda_sync_status(c.status) == OK
    assert torch.equal(q, plain) and torch.equal(at, c.pool.base)


@pytest.mark.parametrize("bad", [-1, 300, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
def test_append_at_skips_what_has_no_angle(bad, fmt):
    c = Placed([(20, 50), (4, 90)], [8, 24], fmt=fmt, d=64, pt=16, seed=7).on_gpu()   # the first: slots 30 .. 50, blocks 1 .. 3
    before = c.bytes().copy()
    pos = c.pos.copy()
    pos[5, 1] = bad                                                                   # slot 35: block 2
    q = c.append(pos).float().cpu().numpy()
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    want = c.expect()
    keep = [i for i in range(c.T) if i != 5]
    assert np.array_equal(q[keep], want[keep]) and (q[5] == 7).all()
    after, whole, page = c.bytes(), c.packed(), c.table[0][2]
    assert np.array_equal(after[page], before[page])
    others = [p for p in range(c.pages) if p != page]
    assert np.array_equal(after[others], whole[others])


# ------------------------------------------------------------------ attention
class Tree(Case):
    """A batch of trees behind their contexts."""

    def __init__(self, lens, chain=0.5, **kw):
        super().__init__(lens, **kw)
        self.parents = [tree.random_tree(self.r, n, chain) for n, _ in lens]
        plans = [tree.plan(p, L - len(p)) for p, (_, L) in zip(self.parents, lens)]
        self.mask, self.pos = [m for p in plans for m in p[0]], [x for p in plans for x in p[1]]

    def attend(self, window=0, sinks=0, q=None, stream=None, ws=None, scale=None):
        q = self.gpu(self.q) if q is None else q
        o = torch.full((self.T, self.G * self.Hkv, self.d), 7.0, dtype=DT[self.dtype], device=DEV)
        lse = torch.full((self.T, self.G * self.Hkv), 7.0, device=DEV)
        ws = kda.attn_tree_workspace(q, self.Hkv, len(self.lens), self.max_q).fill_(255) if ws is None else ws
        kda.kda_attn_tree(self.pool, self.Hkv, FMT[self.fmt], self.pt, *self.meta, self.max_q, i64(self.mask), q, o, ws, self.status,
                          scale=scale, window=window, sinks=sinks, pos=i32(self.pos) if window else None, lse=lse, stream=stream)
        return o, lse

    def expect(self, window=0, sinks=0, scale=None):
        o, lse, rows = tree.attend(ref.values(self.stored, self.scales), self.table, self.cu, self.kv_len, self.q, self.mask, self.pos,
                                   self.G, self.pt, self.d ** -0.5 if scale is None else scale, window, sinks)
        assert len(rows) == self.T
        return o, lse


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (100, 5), (64, 200)])
def test_small_trees(fmt, dtype, d, window, sinks):
    Tree([(1, 1), (4, 4), (8, 129), (0, 40), (3, 127), (5, 700), (7, 1000)], fmt=fmt, dtype=dtype, d=d, seed=11).on_gpu().check(window, sinks)


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (130, 7)])
def test_large_trees(fmt, dtype, d, window, sinks):
    Tree([(64, 64), (33, 300), (0, 10), (17, 129), (64, 700)], fmt=fmt, dtype=dtype, d=d, G=4 if dtype == "bf16" else 1,
         seed=12).on_gpu().check(window, sinks)


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("G,n", [(1, 16), (1, 17), (1, 32), (1, 33), (3, 43), (2, 64), (3, 64), (5, 60), (8, 64)])
def test_trees_of_any_number_of_rows(fmt, G, n):
    """Around 16, 32, 128 and 256 rows a head, with one unit, several, and more than a CTA's share."""
    Tree([(n, n + 3), (n, 1000), (1, 400), (n // 2, 130)], fmt=fmt, G=G, Hkv=1, seed=13 + G).on_gpu().check()


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("pt", [16, 48, 96, 128])
@pytest.mark.parametrize("chain", [0.0, 1.0])
def test_trees_over_pages_of_any_size(fmt, pt, chain):
    Tree([(30, 333), (12, 12), (5, 97)], chain=chain, fmt=fmt, pt=pt, G=2, seed=14).on_gpu().check()
    Tree([(3, 333), (2, 12), (5, 97)], chain=chain, fmt=fmt, pt=pt, G=2, seed=15).on_gpu().check(50, 3)


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("n", [4, 50])
def test_any_mask_will_do(fmt, dtype, d, n):
    """Masks that are no tree's: nothing at all, a draft without itself, later drafts, bits behind the last draft."""
    c = Tree([(n, n), (n, n + 200), (1, 1)], fmt=fmt, dtype=dtype, d=d, seed=16)
    c.mask = [int(c.r.integers(0, 1 << 62)) * 4 + int(c.r.integers(0, 4)) for _ in c.mask]
    c.mask[0] = 0                                   # nothing before the tree: sees nothing
    c.mask[1] = 1 << 63
    c.mask[n + 1] = 0                               # its context alone
    c.mask[2 * n] = (1 << 64) - 2                   # one token, not itself
    c.on_gpu()
    o, lse = c.attend()
    assert kda.kda_sync_status(c.status) == OK
    c.close(o, lse, *c.expect())
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all() and (o[2 * n] == 0).all()


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("n,G", [(6, 2), (40, 4)])
def test_unseen_infinities_and_nan(fmt, dtype, d, n, G):
    """Values and keys that a draft does not see, stale slots among them, never reach it."""
    c = Tree([(n, n + 90), (n, n)], chain=0.3, fmt=fmt, dtype=dtype, d=d, G=G if dtype == "bf16" else 1, seed=17)
    strange = [np.nan, np.inf, -np.inf]
    for s, (m, L) in enumerate(c.lens):
        page, slot = c.table[s][-1], L % c.pt
        if fmt == ref.BF16:
            if slot:
                c.stored[page, :, :, slot:] = np.nan                           # stale
            for i in (1, m - 1):                                               # drafts that some see
                j = L - m + i
                c.stored[c.table[s][j // c.pt], :, 1, j % c.pt, ::5] = strange[i % 3]
                c.stored[c.table[s][j // c.pt], 0, 0, j % c.pt, 3] = strange[(i + 1) % 3]
        c.mask[c.cu[s]] &= ~(1 << (m - 1))
    for p in c.free:
        c.stored[p] = 0 if fmt == ref.I8 else np.nan
        if fmt == ref.I8:
            c.scales[p] = np.nan
    c.on_gpu()
    o, lse = c.attend()
    assert kda.kda_sync_status(c.status) == OK
    # What does see an infinite value gets an infinity or NaN: with the probability in two terms, the lower one
    # is 0 or below it as often as not, and 0 or a negative number times infinity is no positive infinity.
    # The same goes for a float32 query's terms and an infinite key: a score of -infinity may come out as NaN.
    eo, el = c.expect()
    if fmt == ref.BF16:
        vals = ref.values(c.stored, None)
        for s, (m, L) in enumerate(c.lens):
            for t in range(c.cu[s], c.cu[s + 1]):
                for j in range(m):
                    key = vals[c.table[s][(L - m + j) // c.pt], :, 0, (L - m + j) % c.pt]
                    for h in np.flatnonzero(np.isinf(key).any(1)) if c.mask[t] >> j & 1 else []:
                        heads = slice(h * c.G, (h + 1) * c.G)
                        lost = torch.isnan(lse[t, heads]).cpu().numpy()
                        eo[t, heads][lost], el[t, heads][lost] = np.nan, np.nan
    c.close(torch.where(torch.isfinite(o), o, torch.nan), lse, np.where(np.isfinite(eo), eo, np.nan), el)


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("n", [4, 60])
def test_positions_outside_the_tree_count_as_its_ends(fmt, n):
    c = Tree([(n, n + 300)], fmt=fmt, seed=18)
    c.pos = [int(x) for x in c.r.choice([-2 ** 31, -1, 0, n + 299, n + 300, 2 ** 31 - 1], n)]
    c.on_gpu().check(90, 3)


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("n", [5, 48])
def test_a_chain_is_causal_attention(fmt, dtype, d, n):
    c = Tree([(n, n), (n, 600)], chain=1.0, fmt=fmt, dtype=dtype, d=d, seed=19).on_gpu()
    o, lse = c.attend()
    c.close(o, lse, *Case.expect(c))
    o2, lse2 = Case.attend(c)
    assert kda.kda_sync_status(c.status) == OK
    c.close(o2, lse2, o.double().cpu().numpy(), lse.double().cpu().numpy())


@pytest.mark.parametrize("n", [4, 40])
def test_sequences_that_do_not_fit_are_skipped(n):
    c = Tree([(n, n + 100), (n, n - 1), (n, n + 5)], seed=20).on_gpu()
    o, lse = c.attend()
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    assert (o[n:2 * n] == 7).all() and (lse[n:2 * n] == 7).all()
    eo, el, rows = tree.attend(ref.values(c.stored, c.scales), c.table, c.cu, c.kv_len, c.q, c.mask, c.pos, c.G, c.pt, c.d ** -0.5, 0, 0)
    assert rows == list(range(n)) + list(range(2 * n, 3 * n))
    c.close(o[rows], lse[rows], eo[rows], el[rows])


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("n,G,H", [(4, 2, 2), (16, 4, 2), (64, 4, 1)])
def test_long_contexts_are_joined(fmt, n, G, H):
    """Items that many CTAs share, beside short ones."""
    Tree([(n, 20000), (n, n + 1), (1, 3000)], fmt=fmt, G=G, Hkv=H, seed=21).on_gpu().check()


def test_many_trees_of_every_size():
    Tree([(i % 65, i % 65 + 37 * i % 1500) for i in range(90)], fmt=ref.I8, Hkv=1, G=2, seed=22).on_gpu().check()
    Tree([(i % 65, i % 65 + 37 * i % 1500) for i in range(90)], fmt=ref.BF16, Hkv=1, G=2, seed=23).on_gpu().check()


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("n", [4, 40])
def test_the_same_call_gives_the_same_bits(fmt, n):
    c = Tree([(n, 5000), (n, 77)], fmt=fmt, seed=24).on_gpu()
    a, b = c.attend(), c.attend()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_and_foreign_strides():
    c = Tree([(20, 3000), (9, 500)], seed=25).on_gpu()
    wide = torch.full((c.T, c.G * c.Hkv + 3, c.d), 9.0, dtype=DT[c.dtype], device=DEV)
    wide[:, 2:2 + c.G * c.Hkv] = c.gpu(c.q)
    q = wide[:, 2:2 + c.G * c.Hkv]
    torch.cuda.synchronize()
    outs = []
    for s in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            outs.append(c.attend(q=q, stream=s))
    torch.cuda.synchronize()
    for o, lse in outs:
        c.close(o, lse, *c.expect())


# ------------------------------------------------------------------ keeping a branch
class Kept(Case):
    def __init__(self, lens, chain=0.5, keep=0.9, paths=None, **kw):
        super().__init__(lens, **kw)
        self.paths = [tree.random_path(self.r, tree.random_tree(self.r, n, chain), keep) for n, _ in lens] if paths is None else paths

    def accept(self, path=None, accepted=None):
        flat = [x for p, (n, _) in zip(self.paths, self.lens) for x in list(p) + [-9] * (n - len(p))]
        self.out = torch.full((len(self.lens),), -5, dtype=torch.int32, device=DEV)
        kda.kda_kv_accept(self.pool, self.Hkv, self.d, FMT[self.fmt], self.pt, *self.meta, self.max_q, i32(flat if path is None else path),
                          i32([len(p) for p in self.paths] if accepted is None else accepted), self.out, self.status)
        return self.pool.base.cpu().numpy(), self.out.cpu().numpy()

    def expect(self, skipped=()):
        for s, (n, L) in enumerate(self.lens):
            if s not in skipped:
                tree.accept(self.stored, self.scales, self.table[s], L - n, self.paths[s], self.pt)
        lens = [-5 if s in skipped else L - n + len(self.paths[s]) for s, (n, L) in enumerate(self.lens)]
        return ref.pack(self.stored, self.scales, self.fmt, self.page_bytes), lens


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("d,pt", [(64, 16), (128, 64), (64, 128), (128, 48)])
@pytest.mark.parametrize("chain,keep", [(0.2, 1.0), (0.9, 0.95), (0.5, 0.0)])
def test_kept_branches_match_bit_for_bit(fmt, d, pt, chain, keep):
    lens = [(n, n + off) for n in (1, 2, 5, 31, 64) for off in (0, 1, 15, 16, 40, 63, 64, 127)] + [(0, 33), (0, 0)]
    c = Kept(lens, chain, keep, fmt=fmt, d=d, pt=pt, Hkv=3, seed=31).on_gpu()
    got, out = c.accept()
    assert kda.kda_sync_status(c.status) == OK
    want, lens = c.expect()
    assert list(out) == lens
    assert np.array_equal(got, want)


@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_kept_rows_of_blocks_of_other_scales(spread):
    """Scales far apart both ways, scales of 0, infinity and no number, a branch that leaves a block's first rows out."""
    paths = [[3, 20, 40, 41, 63], [16, 17, 33], [0, 1, 17, 48], [5], [63], list(range(1, 64)), list(range(0, 64, 3))]
    for seed in (32, 33):
        c = Kept([(64, 64 + o) for o in (0, 3, 15, 16, 30, 31, 60)], paths=paths, d=64, pt=16, spread=spread, seed=seed)
        if spread:
            for k, x in enumerate([0.0, np.inf, np.nan, 1e-42, 3e38]):
                c.scales[c.table[k][(c.kv_len[k] - 1) // 16 - k % 2], 0] = x
                c.scales[c.table[k][(c.kv_len[k] - 64) // 16], 1, 1] = x
        c.on_gpu()
        got, out = c.accept()
        assert kda.kda_sync_status(c.status) == OK
        want, lens = c.expect()
        assert list(out) == lens
        a, b = ref.unpack(got, c.Hkv, c.d, c.fmt, c.pt), ref.unpack(want, c.Hkv, c.d, c.fmt, c.pt)
        assert np.array_equal(a[1], b[1], equal_nan=True)
        fine = np.isfinite(b[1])[..., None, None]           # a block that reads as NaN may hold any codes
        assert np.array_equal(np.where(fine, a[0], 0), np.where(fine, b[0], 0))


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
def test_branches_that_are_none_change_nothing(fmt):
    n = 8
    paths = [[0, 2, 3], [3, 2], [0, 0], [1, 8], [-1, 2], [2, 5], [1, 4]]
    c = Kept([(n, 50)] * len(paths), paths=paths, fmt=fmt, d=64, pt=16, seed=34).on_gpu()
    got, out = c.accept()
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    want, lens = c.expect(skipped=(1, 2, 3, 4))
    assert list(out) == lens and np.array_equal(got, want)
    for accepted in ([-1] * len(paths), [n + 1] * len(paths)):
        before = got
        got, out = c.accept(accepted=accepted)
        assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
        assert (out == -5).all() and np.array_equal(got, before)


def test_a_lost_page_skips_its_sequence_alone():
    c = Kept([(20, 60), (20, 60), (20, 60)], paths=[[0, 5, 19], [0, 5, 19], [0, 5, 6]], d=64, pt=16, seed=35)
    c.on_gpu()
    c.table[1][3] = c.pages                               # slots 48 .. 63: the branch's last draft
    c.table[2][3] = -1                                    # behind the branch: not looked at
    c.meta = (i32(c.cu), i32(c.kv_len), i32(c.table))
    got, out = c.accept()
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_PAGE)
    want, lens = c.expect(skipped=(1,))
    assert list(out) == lens and np.array_equal(got, want)


# ------------------------------------------------------------------ recurrent states
class States:
    """Requests with states, and trees of drafts for them."""

    def __init__(self, sizes, H=2, d=128, dtype="bf16", page_bytes=65536, chain=0.5, seed=0, parents=None):
        r = self.r = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.H, self.d, self.dtype, self.sizes, self.B = H, d, dtype, sizes, len(sizes)
        self.parents = [tree.random_tree(r, n, chain) for n in sizes] if parents is None else parents
        self.cu = np.concatenate([[0], np.cumsum(sizes)])
        T = self.T = int(self.cu[-1])
        unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
        rn = lambda *s: r.standard_normal(s)  # noqa: E731
        form = (lambda x: ref.to_bf16(x.astype(np.float32))) if dtype == "bf16" else (lambda x: x.astype(np.float32))
        self.q, self.k, self.v = form(unit(rn(T, H, d))), form(unit(rn(T, H, d))), form(rn(T, H, d))
        self.alpha, self.beta = form(1 / (1 + np.exp(-rn(T, H, d) - 3))), form(1 / (1 + np.exp(-rn(T, H))))
        self.w = (rn(H, 3 * d, 4) * 0.5).astype(np.float32)
        self.P = policy.object_pages(H, d, dtype, page_bytes)
        self.pool = kda.Pool(page_bytes, self.B * self.P + 3, DEV)
        ids = r.permutation(self.pool.num_pages)[:self.B * self.P]
        self.pages = ids.reshape(self.B, self.P)
        self.S, self.win = zip(*[random_state(H, d, dtype, g) for _ in range(self.B)])
        for b in range(self.B):
            write_object(self.pool, self.pages[b], self.S[b], self.win[b], dtype)
        self.bytes = policy.object_bytes(H, d, dtype)
        self.status = word()
        self.max_q = max(max(sizes), 1)

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(DEV, DT[self.dtype])

    def tokens(self):
        return [self.dev(x) for x in (self.q, self.k, self.v, self.alpha, self.beta)] + [torch.from_numpy(self.w).to(DEV)]

    def raw(self, b):
        a, e = self.cu[b], self.cu[b + 1]
        return np.concatenate([self.q[a:e], self.k[a:e], self.v[a:e]], -1).astype(np.float64)

    def verify(self, parents=None, pages=None, tokens=None):
        flat = [x for p in (self.parents if parents is None else parents) for x in p]
        o = torch.full((self.T, self.H, self.d), 7.0, dtype=DT[self.dtype], device=DEV)
        kda.kda_verify_tree(self.pool, i32(self.cu), i32(flat), self.max_q, *(self.tokens() if tokens is None else tokens), o,
                            i32(self.pages if pages is None else pages), self.status)
        return o

    def expect(self, b):
        a, e = self.cu[b], self.cu[b + 1]
        return tree.verify(self.S[b], self.win[b], self.w.astype(np.float64), self.raw(b), self.alpha[a:e].astype(np.float64),
                           self.beta[a:e].astype(np.float64), self.parents[b])

    def check(self, o, skipped=()):
        o = o.double().cpu().numpy()
        for b in range(self.B):
            a, e = self.cu[b], self.cu[b + 1]
            if b in skipped:
                assert (o[a:e] == 7).all()
                continue
            if e == a:
                continue
            want = self.expect(b)[0]
            for t in range(e - a):
                for h in range(self.H):
                    err = rel_err(o[a + t, h], want[t, h])
                    assert err <= STATE_TOL[self.dtype], (b, t, h, err)

    def accept(self, paths, accepted=None, pages=None):
        flat = [x for p, n in zip(paths, self.sizes) for x in (list(p) + [-9] * n)[:n]]
        kda.kda_verify_tree_accept(self.pool, i32(self.cu), i32(flat), i32([len(p) for p in paths] if accepted is None else accepted),
                                   self.max_q, *self.tokens(), i32(self.pages if pages is None else pages), self.status)

    def objects(self):
        return [read_object_bytes(self.pool, p, self.bytes) for p in self.pages]

    def check_state(self, b, path):
        S, win = read_object(self.pool, self.pages[b], self.H, self.d, self.dtype)
        want = self.expect(b)[1][path[-1]]
        for h in range(self.H):
            assert rel_err(S[h], want[h]) <= STATE_TOL["f32"], (b, h, rel_err(S[h], want[h]))
        assert np.array_equal(win, tree.window_after(self.raw(b), self.win[b], path))


SHAPES = [(t, d, p) for t in ("bf16", "f32") for d in (64, 128) for p in (65536, 4096)] + [("bf16", 128, 256), ("bf16", 128, 260 * 256)]


@pytest.mark.parametrize("dtype,d,page_bytes", SHAPES)
@pytest.mark.parametrize("chain", [0.0, 0.6, 1.0])
def test_verify_matches_every_draft(dtype, d, page_bytes, chain):
    c = States([1, 2, 0, 5, 16, 17], d=d, dtype=dtype, page_bytes=page_bytes, chain=chain, seed=41)
    before = c.pool.base.clone()
    o = c.verify()
    assert kda.kda_sync_status(c.status) == OK
    c.check(o)
    assert torch.equal(before, c.pool.base)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("sizes", [[64, 33], [64, 1], [32, 31], [24], [8, 7, 9], [48, 41]])
def test_verify_of_large_trees(dtype, d, sizes):
    for chain in (0.3, 1.0):
        c = States(sizes, H=1, d=d, dtype=dtype, chain=chain, seed=42)
        o = c.verify()
        assert kda.kda_sync_status(c.status) == OK
        c.check(o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alpha_of_zero_and_one(dtype):
    c = States([12, 40], dtype=dtype, seed=43)
    c.alpha[c.r.random(c.alpha.shape) < 0.3] = 0
    c.alpha[c.r.random(c.alpha.shape) < 0.3] = 1
    c.alpha[3] = 0
    c.beta[5], c.beta[7] = 0, 1
    o = c.verify()
    assert kda.kda_sync_status(c.status) == OK
    c.check(o)
    paths = [[0], tree.random_path(c.r, c.parents[1], 1.0)]
    c.accept(paths)
    assert kda.kda_sync_status(c.status) == OK
    for b in range(2):
        c.check_state(b, paths[b])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_strange_draft_reaches_its_descendants_alone(dtype):
    c = States([30, 6], dtype=dtype, chain=0.3, seed=44)
    clean = c.verify()
    c.v[4, 0, 5] = np.nan
    c.k[9, 1, 7] = np.inf
    o = c.verify()
    assert kda.kda_sync_status(c.status) == OK
    same = [t for t in range(c.T) if t >= 30 or not {4, 9} & set(tree.branch(c.parents[0], t))]
    assert 30 > len([t for t in same if t < 30]) > 5
    assert torch.equal(o[same], clean[same])
    for t in set(range(30)) - set(same):
        up = tree.branch(c.parents[0], t)
        assert (4 not in up or torch.isnan(o[t, 0, 5])) and (9 not in up or not torch.isfinite(o[t, 1]).all())


def test_verify_skips_what_does_not_fit():
    c = States([4, 4, 4, 4], H=2, d=64, seed=45)
    parents = [list(p) for p in c.parents]
    parents[1] = [-1, 1, 0, 0]
    parents[2] = [-1, -2, 0, 0]
    o = c.verify(parents=parents)
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    c.check(o, skipped=(1, 2))
    pages = c.pages.copy()
    pages[0, -1] = c.pool.num_pages
    pages[3, 0] = -1
    before = c.objects()
    o = c.verify(pages=pages)
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_PAGE)
    c.check(o, skipped=(0, 3))
    c.accept([[0], [], [], [0]], pages=pages)
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_PAGE)
    for paths, accepted in (([[1, 0], [0, 0], [0, 4], [-1]], None), ([[0, 1, 2, 3]] * 4, [-1, 5, 65, -2 ** 31])):
        c.accept(paths, accepted)
        assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    assert c.objects() == before


@pytest.mark.parametrize("dtype,d,page_bytes", SHAPES)
def test_accepted_branches_advance_the_state(dtype, d, page_bytes):
    c = States([1, 3, 0, 6, 16, 64, 5], d=d, dtype=dtype, page_bytes=page_bytes, chain=0.8, seed=46)
    paths = [tree.random_path(c.r, p, 1.0) for p in c.parents]
    paths[3], paths[6] = paths[3][:1], []
    before = c.objects()
    c.accept(paths)
    assert kda.kda_sync_status(c.status) == OK
    after = c.objects()
    for b, path in enumerate(paths):
        if path:
            c.check_state(b, path)
        else:
            assert after[b] == before[b]


def test_many_requests_and_heads():
    c = States([(7 * b) % 19 for b in range(60)], H=5, d=128, chain=0.5, seed=47)
    o = c.verify()
    paths = [tree.random_path(c.r, p, 0.9) for p in c.parents]
    c.accept(paths)
    assert kda.kda_sync_status(c.status) == OK
    c.check(o)
    for b, path in enumerate(paths):
        if path:
            c.check_state(b, path)


@pytest.mark.parametrize("page_bytes", [65536, 260 * 256, 1 << 20])
def test_many_branches_beside_bad_ones(page_bytes):
    """More (request, head) pairs than SMs: long and empty branches, requests without drafts, branches that are none and lost pages."""
    c = States([(5 * b) % 23 + (40 if b == 7 else 0) for b in range(80)], H=4, d=128, chain=0.9, seed=49, page_bytes=page_bytes)
    paths = [tree.random_path(c.r, p, 0.95) if b % 3 else [] for b, p in enumerate(c.parents)]
    bad = [b for b in range(80) if c.sizes[b] > 3][4:8]
    paths[bad[0]], paths[bad[1]] = [1, 0], [0, c.sizes[bad[1]]]
    paths[bad[2]] = paths[bad[3]] = [0]
    pages = c.pages.copy()
    pages[bad[2], -1], pages[bad[3], 0] = c.pool.num_pages, -1
    before = c.objects()
    c.accept(paths, pages=pages)
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META | kda.KDA_DEV_BAD_PAGE)
    after = c.objects()
    assert max(len(p) for p in paths) > 8
    for b, path in enumerate(paths):
        if path and b not in bad:
            c.check_state(b, path)
        else:
            assert after[b] == before[b], b


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_a_chain_is_the_verify_step(dtype, d):
    K = 5
    c = States([K] * 3, d=d, dtype=dtype, chain=1.0, seed=48, page_bytes=65536)
    o = c.verify()
    pool2 = kda.Pool(65536, (K + 1) * 3 * c.P, DEV)
    src = kda.kda_page_alloc(pool2, 3 * c.P).reshape(3, c.P)
    for b in range(3):
        write_object(pool2, src[b], c.S[b], c.win[b], dtype)
    inter = kda.kda_verify_plan(pool2, c.H, d, kda.DTYPES[dtype], 3, K)
    major = [x.reshape(3, K, *x.shape[1:]).transpose(0, 1).contiguous() for x in c.tokens()[:5]]
    o2 = torch.empty_like(major[0])
    kda.kda_verify_step(pool2, *major, torch.from_numpy(c.w).to(DEV), o2, i32(src), i32(inter), c.status)
    paths = [[0, 1, 2], list(range(K)), [0]]
    c.accept(paths)
    assert kda.kda_sync_status(c.status) == OK
    a, b = o.double().cpu().numpy(), o2.transpose(0, 1).reshape(o.shape).double().cpu().numpy()
    assert rel_err(a, b) <= 2 * STATE_TOL[dtype]
    for r, path in enumerate(paths):
        S, win = read_object(c.pool, c.pages[r], c.H, d, dtype)
        S2, win2 = read_object(pool2, inter[len(path) - 1, r], c.H, d, dtype)
        assert rel_err(S, S2) <= 1e-4 and np.array_equal(win, win2)


# ------------------------------------------------------------------ a round of all of them
def ragged(trees):
    return [x for t in trees for x in t]


class Round:
    """One layer of each kind over one pool: a tree is placed, answered for, and a branch of it kept."""

    Hq, Hkv, H, d, pt, max_q = 4, 2, 2, 128, 16, 24

    def __init__(self, fmt, starts, seed=51):
        r = self.r = np.random.default_rng(seed)
        self.fmt, self.n = fmt, len(starts)
        self.blocks = 12
        page = max(kda.kda_kv_page_bytes(self.Hkv, self.d, fmt, self.pt), 16384)
        self.P = -(-kda.kda_object_bytes(self.H, self.d, kda.KDA_BF16) // page)
        self.pool = kda.Pool(page, self.n * (self.P + self.blocks) + 2, DEV)
        self.table = i32(kda.kda_page_alloc(self.pool, self.n * self.blocks).reshape(self.n, self.blocks))
        self.pages = kda.kda_page_alloc(self.pool, self.n * self.P).reshape(self.n, self.P)
        g = torch.Generator().manual_seed(seed)
        for b in range(self.n):
            write_object(self.pool, self.pages[b], *random_state(self.H, self.d, "bf16", g), "bf16")
        self.pages_dev = i32(self.pages)
        self.cs = torch.from_numpy(angles(400, self.d)).to(DEV)
        self.conv_w = torch.from_numpy((r.standard_normal((self.H, 3 * self.d, 4)) * 0.5).astype(np.float32)).to(DEV)
        self.status = word()
        # what a round's tensors hold; T rows at most
        self.T = self.n * self.max_q
        self.cu, self.lens = i32(np.zeros(self.n + 1)), i32(starts)
        self.parent, self.path = i32(np.zeros(self.T)), i32(np.zeros(self.T))
        self.accepted, self.new_lens = i32(np.zeros(self.n)), i32(np.zeros(self.n))
        bf = dict(dtype=torch.bfloat16, device=DEV)
        self.x = torch.zeros(self.T, self.Hq + 2 * self.Hkv, self.d, **bf)
        self.q, self.o = (torch.zeros(self.T, self.Hq, self.d, **bf) for _ in range(2))
        self.tok = [torch.zeros(self.T, self.H, self.d, **bf) for _ in range(4)] + [torch.zeros(self.T, self.H, **bf)]
        self.o_rec = torch.zeros(self.T, self.H, self.d, **bf)
        self.mask = torch.zeros(self.T, dtype=torch.int64, device=DEV)
        self.pos = i32(np.zeros(self.T))
        self.ws = kda.attn_tree_workspace(self.q, self.Hkv, self.n, self.max_q)

    def draft(self, seed, starts):
        """New drafts behind `starts` tokens, into the tensors."""
        r = np.random.default_rng(seed)
        sizes = [int(x) for x in r.integers(1, self.max_q + 1, self.n)]
        self.trees = [tree.random_tree(r, n, 0.6) for n in sizes]
        self.paths = [tree.random_path(r, t, 0.9) for t in self.trees]
        cu = np.concatenate([[0], np.cumsum(sizes)])
        self.cu_host, self.starts = cu, np.asarray(starts)
        self.cu.copy_(i32(cu))
        self.lens.copy_(i32(self.starts + sizes))
        pad = lambda x: i32(list(x) + [0] * (self.T - len(x)))  # noqa: E731
        self.parent.copy_(pad(ragged(self.trees)))
        self.path.copy_(pad(ragged([list(p) + [0] * (n - len(p)) for p, n in zip(self.paths, sizes)])))
        self.accepted.copy_(i32([len(p) for p in self.paths]))
        put = lambda t, x: t.copy_(torch.from_numpy(x.astype(np.float32)).to(DEV, torch.bfloat16))  # noqa: E731
        rn = lambda *s: r.standard_normal(s)  # noqa: E731
        unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
        put(self.x, rn(*self.x.shape))
        for i in range(3):
            put(self.tok[i], unit(rn(*self.tok[i].shape)) if i < 2 else rn(*self.tok[i].shape))
        put(self.tok[3], 1 / (1 + np.exp(-rn(*self.tok[3].shape) - 3)))
        put(self.tok[4], 1 / (1 + np.exp(-rn(*self.tok[4].shape))))

    def calls(self):
        Hq, Hkv = self.Hq, self.Hkv
        x, meta = self.x, (self.cu, self.lens, self.table, self.max_q)
        kda.kda_tree_plan(self.cu, self.lens, self.parent, self.max_q, self.mask, self.pos, self.status)
        kda.kda_kv_append_at(self.pool, self.fmt, self.pt, *meta, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], self.cs, self.pos,
                             [self.d // 2], self.q, self.status)
        kda.kda_attn_tree(self.pool, Hkv, self.fmt, self.pt, *meta, self.mask, self.q, self.o, self.ws, self.status)
        kda.kda_verify_tree(self.pool, self.cu, self.parent, self.max_q, *self.tok, self.conv_w, self.o_rec, self.pages_dev, self.status)
        kda.kda_kv_accept(self.pool, Hkv, self.d, self.fmt, self.pt, *meta, self.path, self.accepted, self.new_lens, self.status)
        kda.kda_verify_tree_accept(self.pool, self.cu, self.path, self.accepted, self.max_q, *self.tok, self.conv_w, self.pages_dev,
                                   self.status)

    def one_by_one(self):
        """The accepted tokens alone, a token at a time through the calls without trees, over the same pool; their answers."""
        Hq, Hkv = self.Hq, self.Hkv
        lens, outs = self.starts.copy(), {}
        for step in range(max(len(p) for p in self.paths)):
            go = [s for s in range(self.n) if step < len(self.paths[s])]
            rows = torch.tensor([self.cu_host[s] + self.paths[s][step] for s in go], device=DEV)
            lens[go] += 1
            x = self.x[rows]
            cu, kl = i32(range(len(go) + 1)), i32(lens[go])
            meta = cu, kl, self.table[go].contiguous(), 1
            q = torch.empty_like(x[:, :Hq])
            kda.kda_kv_append(self.pool, self.fmt, self.pt, *meta, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], self.cs, q, self.status)
            o = torch.empty_like(q)
            kda.kda_attn_paged(self.pool, Hkv, self.fmt, self.pt, *meta, q, o, kda.attn_workspace(q, Hkv, len(go), 1), self.status)
            t = [y[rows].contiguous() for y in self.tok]
            o_rec = torch.empty_like(t[0])
            kda.kda_decode_step(self.pool, *t, self.conv_w, o_rec, i32(self.pages[go]), self.status)
            for i, s in enumerate(go):
                outs[s, step] = o[i], o_rec[i]
        return lens, outs

    def cached(self, lens):
        total = int(sum(lens))
        k, v = (torch.zeros(total, self.Hkv, self.d, device=DEV) for _ in range(2))
        kda.kda_kv_gather(self.pool, self.fmt, self.pt, i32(np.concatenate([[0], np.cumsum(lens)])), i32([0] * self.n), self.table, k, v,
                          self.status)
        return k, v

    def compare(self, before):
        """After calls(): the pool, the lengths and the branch's answers against the tokens one by one from `before`."""
        assert kda.kda_sync_status(self.status) == OK
        after, lens = self.pool.base.clone(), self.new_lens.cpu().numpy().copy()
        k, v = self.cached(lens)
        S = [read_object(self.pool, p, self.H, self.d, "bf16") for p in self.pages]
        self.pool.base.copy_(before)
        want, outs = self.one_by_one()
        assert list(want) == list(lens)
        k2, v2 = self.cached(lens)
        if self.fmt == kda.KDA_KV_BF16:
            assert torch.equal(k, k2) and torch.equal(v, v2)
        else:                          # each side codes a block anew a few times: steps of max / 127, rounded by half
            for a, b in ((k, k2), (v, v2)):
                assert ((a - b).abs() <= 4 * b.abs().max() / 127).all()
        for p, (S1, w1) in zip(self.pages, S):
            S2, w2 = read_object(self.pool, p, self.H, self.d, "bf16")
            assert rel_err(S1, S2) <= 1e-4 and np.array_equal(w1, w2)
        for (s, step), (o, o_rec) in outs.items():
            row = self.cu_host[s] + self.paths[s][step]
            assert rel_err(self.o_rec[row].double().cpu(), o_rec.double().cpu()) <= 2 * STATE_TOL["bf16"]
            if self.fmt == kda.KDA_KV_BF16:
                assert rel_err(self.o[row].double().cpu(), o.double().cpu()) <= 2 * 4 * 2.0 ** -9
        self.pool.base.copy_(after)
        return lens


@pytest.mark.parametrize("fmt", [kda.KDA_KV_BF16, kda.KDA_KV_I8])
def test_rounds_leave_what_the_accepted_tokens_alone_leave(fmt):
    c = Round(fmt, [0, 1, 15, 16, 40])
    lens = [0, 1, 15, 16, 40]
    fill = torch.randn(c.n * 40, c.Hkv, c.d, device=DEV).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(lens)])
    kda.kda_kv_append(c.pool, fmt, c.pt, i32(cu), i32(lens), c.table, 40, None, fill[:cu[-1]], fill[:cu[-1]], c.cs, None, c.status)
    for seed in (61, 62, 63):
        c.draft(seed, lens)
        before = c.pool.base.clone()
        c.calls()
        lens = c.compare(before)


def test_a_captured_round_replays_on_other_trees():
    starts = [3, 0, 33]
    c, e = Round(kda.KDA_KV_BF16, starts, seed=52), Round(kda.KDA_KV_BF16, starts, seed=52)
    c.draft(71, starts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    base = c.pool.base.clone()
    with torch.cuda.stream(side):
        c.calls()
    torch.cuda.current_stream().wait_stream(side)
    c.pool.base.copy_(base)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.calls()
    lens = starts
    for seed in (72, 73):
        for x in (c, e):
            x.draft(seed, lens)
        graph.replay()
        e.calls()
        assert kda.kda_sync_status(c.status) == OK and kda.kda_sync_status(e.status) == OK
        T = c.cu_host[-1]
        assert torch.equal(c.pool.base, e.pool.base) and torch.equal(c.new_lens, e.new_lens)
        assert torch.equal(c.o[:T], e.o[:T]) and torch.equal(c.o_rec[:T], e.o_rec[:T])
        lens = c.new_lens.cpu().numpy()
