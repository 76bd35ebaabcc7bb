"""The paged key/value cache and its attention on the GPU, against a plain model.

Appends: codes, scales and stored bytes are equal bit for bit (the rule is fp32 operation by
operation).  Attention tolerances, on max |o - ref| / max |ref| of a call:
  bf16   2^-9 for the output's rounding, 2^-9 for the probabilities' over the 16-bit cache (the
         8-bit one keeps 2^-11), and as much again for sums of either:  4 x 2^-9 = 8e-3
  f32    scores are sums of up to 128 products in fp32 with |score| up to about 40 here: an error
         of 40 x 2^-24 x 4 in the exponent, 1e-5 in all
log-sum-exp: 1e-5 (1 + |lse|) for either, as its inputs are exact in both."""
import numpy as np
import pytest
import torch

import kda_state_chunked_gb300 as kda
import kv_ref as ref

pytestmark = pytest.mark.gpu

FMT = {ref.I8: kda.KDA_KV_I8, ref.BF16: kda.KDA_KV_BF16}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = {"f32": 1e-5, "bf16": 4 * 2.0 ** -9}
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Case:
    """A cache of random contents with a batch of [(new tokens, tokens in the cache)]."""

    def __init__(self, lens, Hkv=2, G=2, d=128, dtype="bf16", fmt=ref.I8, pt=64, seed=0, spread=1.0, qscale=2.0):
        r = self.r = np.random.default_rng(seed)
        self.lens, self.Hkv, self.G, self.d, self.dtype, self.fmt, self.pt = lens, Hkv, G, d, dtype, fmt, pt
        need = [max(1, -(-L // pt)) for _, L in lens]
        self.maxp = max(need)
        ids = list(r.permutation(sum(need) + 4))
        self.pages = len(ids)
        self.table = np.full((len(lens), self.maxp), -7, np.int64)     # entries past the end are not ids at all
        for s, n in enumerate(need):
            self.table[s, :n] = [ids.pop() for _ in range(n)]
        self.free = ids
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
        self.kv_len = np.array([L for _, L in lens])
        self.T, self.max_q = int(self.cu[-1]), max(max(n for n, _ in lens), 1)
        x = r.standard_normal((self.pages, Hkv, 2, pt, d)).astype(np.float32)
        x *= np.exp(spread * r.standard_normal((self.pages, Hkv, 2, 1, 1))).astype(np.float32)
        if fmt == ref.I8:
            self.scales = (np.abs(x).max((3, 4)) / np.float32(127)).astype(np.float32)
            self.stored = np.rint(x / self.scales[..., None, None]).astype(np.float32)
        else:
            self.scales, self.stored = None, ref.to_bf16(x)
        self.q = self.token(G * Hkv) * qscale if dtype == "f32" else ref.to_bf16(self.token(G * Hkv) * qscale)
        self.page_bytes = ref.page_bytes(Hkv, d, fmt, pt)

    def token(self, H):
        x = self.r.standard_normal((self.T, H, self.d)).astype(np.float32)
        return x if self.dtype == "f32" else ref.to_bf16(x)

    def on_gpu(self, extra=0):
        self.pool = kda.Pool(self.page_bytes + extra, self.pages, DEV)
        self.pool.base = torch.from_numpy(ref.pack(self.stored, self.scales, self.fmt, self.page_bytes + extra)).to(DEV)
        self.status = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.meta = (i32(self.cu), i32(self.kv_len), i32(self.table))
        return self

    def gpu(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(DEV, DT[self.dtype])

    def attend(self, window=0, sinks=0, q=None, stream=None, ws=None, scale=None):
        q = self.gpu(self.q) if q is None else q
        o = torch.full((self.T, self.G * self.Hkv, self.d), 7.0, dtype=DT[self.dtype], device=DEV)
        lse = torch.full((self.T, self.G * self.Hkv), 7.0, device=DEV)
        ws = kda.attn_workspace(q, self.Hkv, len(self.lens), self.max_q).fill_(255) if ws is None else ws
        kda.kda_attn_paged(self.pool, self.Hkv, FMT[self.fmt], self.pt, *self.meta, self.max_q, q, o, ws, self.status,
                           scale=scale, window=window, sinks=sinks, lse=lse, stream=stream)
        return o, lse

    def expect(self, window=0, sinks=0, scale=None):
        return ref.attend(ref.values(self.stored, self.scales), self.table, self.cu, self.kv_len, self.q, self.G, self.pt,
                          self.d ** -0.5 if scale is None else scale, window, sinks)

    def check(self, window=0, sinks=0, **kw):
        o, lse = self.attend(window, sinks, **kw)
        assert kda.kda_sync_status(self.status) == (kda.KDA_OK, 0)
        self.close(o, lse, *self.expect(window, sinks, kw.get("scale")))

    def close(self, o, lse, eo, el):
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.array_equal(np.isnan(o), np.isnan(eo))
        assert np.array_equal(np.isneginf(lse), np.isneginf(el)) and np.array_equal(np.isnan(lse), np.isnan(el))
        fine = np.isfinite(eo)
        if fine.any():
            err = np.abs(o - eo)[fine].max() / max(np.abs(eo[fine]).max(), 1e-30)
            assert err <= TOL[self.dtype], err
        fine = np.isfinite(el)
        if fine.any():
            assert (np.abs(lse - el)[fine] <= 1e-5 * (1 + np.abs(el[fine]))).all()


KINDS = [(f, t, d) for f in (ref.I8, ref.BF16) for t in ("bf16", "f32") for d in (64, 128)]


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 0), (130, 5), (64, 200)])
def test_decode_matches(fmt, dtype, d, window, sinks):
    Case([(1, 1), (1, 17), (0, 40), (1, 127), (1, 128), (1, 129), (1, 700), (1, 1000)], fmt=fmt, dtype=dtype, d=d,
         seed=1).on_gpu().check(window, sinks)


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (3, 0), (70, 4)])
def test_drafts_and_empty_rows_match(fmt, dtype, d, window, sinks):
    # kv_len < n leaves the first rows nothing to see; a sequence may have no tokens at all
    Case([(4, 300), (7, 7), (5, 2), (3, 0), (0, 0), (1, 260), (8, 129)], fmt=fmt, dtype=dtype, d=d,
         seed=2).on_gpu().check(window, sinks)


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("pt", [16, 32, 48, 64, 80, 112, 128])
def test_block_sizes_match(fmt, pt):
    Case([(1, 1), (2, pt), (1, pt + 1), (3, 3 * pt - 1), (1, 5 * pt + 7)], fmt=fmt, pt=pt, seed=3).on_gpu().check(90, 3)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (3, 1), (2, 3), (1, 5), (4, 8), (1, 16), (1, 20), (2, 40)])
@pytest.mark.parametrize("fmt,dtype", [(ref.I8, "bf16"), (ref.BF16, "bf16"), (ref.I8, "f32")])
def test_head_layouts_match(Hkv, G, fmt, dtype):
    Case([(1, 200), (3, 77), (1, 1)], Hkv=Hkv, G=G, fmt=fmt, dtype=dtype, seed=4).on_gpu().check()


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 6)])
def test_prompts_match(fmt, dtype, d, window, sinks):
    Case([(150, 150), (97, 333), (1, 90), (40, 12), (0, 5)], Hkv=2, G=4, fmt=fmt, dtype=dtype, d=d,
         seed=5).on_gpu().check(window, sinks)


def test_many_sequences_match():
    r = np.random.default_rng(6)
    lens = [(int(r.integers(0, 3)), int(r.integers(0, 150))) for _ in range(600)]     # more than one scan's worth
    Case(lens, Hkv=1, G=2, d=64, seed=6).on_gpu().check()


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
def test_long_context_is_joined_from_many_parts(fmt):
    Case([(1, 40000)], Hkv=1, G=8, fmt=fmt, seed=7).on_gpu().check()


@pytest.mark.parametrize("fmt,d", [(f, d) for f in (ref.I8, ref.BF16) for d in (64, 128)])
@pytest.mark.parametrize("n", [4, 5, 8, 9])
def test_rows_around_a_tile(fmt, d, n):
    # 16, 20, 32 and 36 rows a head: either side of where the kernels change over
    Case([(n, 300), (n, n), (1, 77), (0, 5), (n, 1500)], fmt=fmt, d=d, Hkv=2, G=4, seed=31 + n).on_gpu().check(120, 3)


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
def test_short_items_beside_a_long_one(fmt):
    # items of one unit, several to a share, and a long one that many shares take
    lens = [(1 + 7 * i % 40, 41 + 5 * i) for i in range(60)]
    Case(lens + [(40, 6000)] + lens[:20], fmt=fmt, Hkv=4, G=2, seed=41).on_gpu().check()


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("tokens", [383, 385, 640, 767, 769])
def test_lengths_around_unsplit_items(fmt, tokens):
    Case([(1, tokens), (1, 5), (2, tokens - 1)], fmt=fmt, Hkv=2, G=4, seed=51).on_gpu().check()


# A score of up to 8 kept to 23 bits is off by 5e-7 at most, and so is its probability; the exponential
# adds 2 ulp (2.4e-7), and sums of some 50 rounded terms a warp 2e-7: under 1e-6 of the result's size,
# taken one and a half times.
@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
def test_float32_sums_over_long_contexts_keep_their_bits(fmt):
    nseq, L, G, d, pt = 40, 40000, 8, 64, 64
    g = torch.Generator(device=DEV).manual_seed(61)
    blocks = L // pt
    pool = kda.Pool(kda.kda_kv_page_bytes(1, d, FMT[fmt], pt), nseq * blocks, DEV)
    table = torch.randperm(nseq * blocks, generator=g, device=DEV).to(torch.int32).reshape(nseq, blocks)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    k, v = (torch.randn(nseq * L, 1, d, generator=g, device=DEV) for _ in range(2))
    lens, begin = i32([L] * nseq), i32([0] * nseq)
    kda.kda_kv_append(pool, FMT[fmt], pt, i32(np.arange(nseq + 1) * L), lens, table, L, None, k, v, None, None, status)
    kda.kda_kv_gather(pool, FMT[fmt], pt, i32(np.arange(nseq + 1) * L), begin, table, k, v, status)
    q = torch.randn(nseq, G, d, generator=g, device=DEV)
    o = torch.empty_like(q)
    kda.kda_attn_paged(pool, 1, FMT[fmt], pt, i32(np.arange(nseq + 1)), lens, table, 1, q, o, kda.attn_workspace(q, 1, nseq, 1),
                       status)
    assert kda.kda_sync_status(status) == (kda.KDA_OK, 0)
    wrong = size = 0.0
    for s in range(nseq):
        ks, vs = k[s * L:(s + 1) * L, 0].double(), v[s * L:(s + 1) * L, 0].double()
        e = torch.softmax(q[s].double() @ ks.T * d ** -0.5, dim=1) @ vs
        wrong, size = wrong + float((o[s].double() - e).pow(2).sum()), size + float(e.pow(2).sum())
    assert (wrong / size) ** 0.5 <= 1.5e-6


def test_wide_value_scales():
    """Blocks whose scales lie many powers of ten apart keep their precision."""
    Case([(1, 900), (2, 500)], fmt=ref.I8, dtype="f32", spread=6.0, qscale=1e-3, seed=8).on_gpu().check()


@pytest.mark.parametrize("qscale", [1e-30, 1e-6, 1e6])
def test_query_range(qscale):
    c = Case([(1, 300), (3, 200)], dtype="f32", qscale=qscale, seed=9).on_gpu()
    c.check(scale=0.05 / qscale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_unseen_values_never_matter(dtype, n, bad):
    """Stale slots behind the end, later drafts and tokens outside the window hold NaN and infinity."""
    c = Case([(n, 200), (n, 131), (n, 64)], fmt=ref.BF16, dtype=dtype, seed=10)
    for s, (_, L) in enumerate(c.lens):
        for j in range(L, -(-L // c.pt) * c.pt):
            c.stored[c.table[s, j // c.pt], :, :, j % c.pt] = bad
    c.on_gpu().check()
    # the last token's key and value: only its own query may see them
    for s, (_, L) in enumerate(c.lens):
        c.stored[c.table[s, (L - 1) // c.pt], :, 1, (L - 1) % c.pt, ::3] = bad
    c.on_gpu()
    o, lse = c.attend()
    eo, el = c.expect()
    o = o.double().cpu().numpy()
    for s in range(len(c.lens)):
        rows = slice(int(c.cu[s]), int(c.cu[s + 1]) - 1)
        assert np.isfinite(o[rows]).all() and np.abs(o[rows] - eo[rows]).max(initial=0) <= TOL[dtype] * np.abs(eo[rows]).max(initial=1e-30)
        last = int(c.cu[s + 1]) - 1
        assert not np.isfinite(o[last, :, ::3]).any()
    # the first tokens, outside the window
    c = Case([(n, 400), (1, 300)], fmt=ref.BF16, dtype=dtype, seed=11)
    for s in range(2):
        c.stored[c.table[s, 1], :, :, 10:40] = bad
    c.on_gpu().check(window=150, sinks=20)


def test_scales_that_are_not_numbers_stay_in_their_block():
    c = Case([(1, 300), (4, 200)], fmt=ref.I8, seed=12)
    c.scales[c.table[0, 1]] = np.nan            # outside the window below
    c.scales[c.free[0]] = np.inf
    c.on_gpu().check(window=120, sinks=30)
    c.on_gpu()
    o, _ = c.attend()
    assert torch.isnan(o[0]).all() and torch.isfinite(o[1:]).all()


def test_zero_and_equal_scores():
    c = Case([(1, 500), (3, 129)], fmt=ref.I8, seed=13)
    c.stored[:] = 0
    c.scales[:] = 0
    o, lse = c.on_gpu().attend()
    assert (o == 0).all()
    want = np.log(np.array([500.0, 127, 128, 129]))[:, None]
    assert np.abs(lse.cpu().numpy() - want).max() < 1e-5


def test_strided_queries_other_stream_and_page_padding():
    c = Case([(1, 300), (5, 200)], fmt=ref.I8, seed=14).on_gpu(extra=768)
    wide = torch.randn(c.T, 9, c.d, device=DEV).to(torch.bfloat16)
    wide[:, 2:6] = c.gpu(c.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = c.attend(q=wide[:, 2:6], stream=s)
    s.synchronize()
    c.close(o, lse, *c.expect())


def test_graph_replays_on_new_lengths():
    c = Case([(1, 300), (1, 200), (1, 64)], fmt=ref.I8, seed=15).on_gpu()
    q = c.gpu(c.q)
    ws = kda.attn_workspace(q, c.Hkv, 3, 1)
    c.attend(q=q, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = c.attend(q=q, ws=ws)
    for lens in ([300, 200, 64], [1, 33, 64], [299, 0, 17]):
        c.kv_len = np.array(lens)
        c.meta[1].copy_(i32(lens))
        g.replay()
        torch.cuda.synchronize()
        c.close(o, lse, *c.expect())


def test_same_call_same_bits():
    c = Case([(2, 5000), (1, 3001), (3, 70)], fmt=ref.I8, Hkv=2, G=4, seed=16).on_gpu()
    a = c.attend()
    for _ in range(3):
        b = c.attend()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n", [1, 40])
def test_bad_pages_and_lengths_are_reported(n):
    c = Case([(n, 300), (n, 200)], seed=17).on_gpu()
    good, _ = c.attend()
    c.meta[2][0, 1] = c.pages
    o, _ = c.attend()
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_PAGE)
    assert torch.equal(o[n:], good[n:]) and torch.isfinite(o).all()
    c.on_gpu()
    c.meta[1][0] = c.maxp * c.pt + 1
    o, _ = c.attend()
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    assert torch.equal(o[n:], good[n:])


# ------------------------------------------------------------------ append and gather
def table_of(rot, top, r):
    if not rot:
        return None
    a = r.standard_normal((top, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def run_append(c, rot, pairs, q=True, extra=0, strided=False):
    cs = table_of(rot, int(c.kv_len.max()) + 3, c.r)
    k, v = c.token(c.Hkv), c.token(c.Hkv)
    c.on_gpu(extra)
    Hq = c.G * c.Hkv
    if strided:
        x = c.gpu(np.concatenate([c.q, k, v], 1))
        qg, kg, vg = x[:, :Hq], x[:, Hq:Hq + c.Hkv], x[:, Hq + c.Hkv:]
    else:
        qg, kg, vg = c.gpu(c.q), c.gpu(k), c.gpu(v)
    qo = torch.empty(c.T, Hq, c.d, dtype=DT[c.dtype], device=DEV) if q else None
    csg = None if cs is None else torch.from_numpy(cs).to(DEV)
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, qg if q else None, kg, vg, csg, qo, c.status,
                      interleaved=pairs)
    assert kda.kda_sync_status(c.status) == (kda.KDA_OK, 0)
    ref.append(c.stored, c.scales, c.table, c.cu, c.kv_len, k, v, cs, pairs, c.pt)
    want = ref.pack(c.stored, c.scales, c.fmt, c.page_bytes + extra)
    assert np.array_equal(c.pool.base.cpu().numpy(), want)
    if q:
        for s, (n, L) in enumerate(c.lens):
            a, b = int(c.cu[s]), int(c.cu[s + 1])
            x = ref.rotate(c.q[a:b], None if cs is None else cs[L - n:L], pairs)
            x = x if c.dtype == "f32" else ref.to_bf16(x)
            assert np.array_equal(qo[a:b].float().cpu().numpy(), x)
    return kg, vg


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("rot,pairs", [(0, False), (32, False), (32, True), (64, False)])
def test_append_bytes(fmt, dtype, d, rot, pairs):
    run_append(Case([(1, 1), (1, 64), (1, 65), (3, 130), (0, 9), (64, 64), (200, 333), (129, 190)], fmt=fmt, dtype=dtype,
                    d=d, seed=20), rot, pairs)


@pytest.mark.parametrize("fmt,dtype,d", KINDS)
def test_append_single_tokens_bytes(fmt, dtype, d):
    run_append(Case([(1, L) for L in (1, 2, 17, 63, 64, 65, 128, 700)] + [(0, 3)], fmt=fmt, dtype=dtype, d=d, seed=21), d, False,
               strided=True)


@pytest.mark.parametrize("pt", [16, 48, 128])
@pytest.mark.parametrize("n", [1, 5, 8, 9, 300])
def test_append_block_sizes_bytes(pt, n):
    lens = [(n, n), (n, n + pt - 1), (max(n - 1, 0), n + 3 * pt + 5), (n, n + 7)]
    run_append(Case(lens, pt=pt, Hkv=3, seed=22), 16, True, extra=512, strided=True)


def test_append_keys_and_values_only():
    run_append(Case([(5, 40), (1, 9)], seed=23), 64, False, q=False)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_append_of_what_is_no_number_poisons_its_block(bad):
    c = Case([(70, 200), (1, 30)], dtype="f32", seed=24)
    cs, k, v = None, c.token(c.Hkv), c.token(c.Hkv)
    k[3, 0, 5] = bad
    v[70, 1, 0] = bad
    c.on_gpu()
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, None, c.gpu(k), c.gpu(v), cs, None, c.status)
    stored, scales = ref.unpack(c.pool.base.cpu().numpy(), c.Hkv, c.d, c.fmt, c.pt)
    p0, p1 = c.table[0, 133 // c.pt], c.table[1, 0]
    assert not np.isfinite(scales[p0, 0, 0]) and not np.isfinite(scales[p1, 1, 1])
    assert np.isfinite(scales[p0, 0, 1]) and np.isfinite(scales[p0, 1]).all() and np.isfinite(scales[p1, 0]).all()


@pytest.mark.parametrize("size", [0.0, 1e-45, 1e-43, 1e-38, 3e38])
def test_append_at_the_ends_of_the_range(size):
    c = Case([(20, 20), (3, 30)], dtype="f32", seed=25)
    c.stored[:] = 0
    c.scales[:] = 0
    token = c.token
    c.token = lambda H: np.clip(token(H), -1, 1) * np.float32(size)
    run_append(c, 0, False, q=False)


def test_append_refuses_what_does_not_fit():
    c = Case([(4, 70), (2, 20)], seed=26).on_gpu()
    before = c.pool.base.clone()
    k = torch.ones(c.T, c.Hkv, c.d, dtype=torch.bfloat16, device=DEV)
    cs = torch.ones(69, 32, device=DEV)           # one position short for the first sequence
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, None, k, k, cs, None, c.status)
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    first = torch.from_numpy(c.table[0, :2]).to(DEV)
    assert torch.equal(c.pool.base[first], before[first]) and not torch.equal(c.pool.base, before)
    for lens in ([3, 20], [c.maxp * c.pt + 1, 20]):     # fewer cached than new; more than the table has
        c.on_gpu()
        c.meta[1].copy_(i32(lens))
        kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, None, k, k, None, None, c.status)
        assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
        assert torch.equal(c.pool.base[first], before[first])
    c.on_gpu()
    c.meta[2][0, 1] = -1
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, None, k, k, None, None, c.status)
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_PAGE)


@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_gather_values(fmt, d, out):
    c = Case([(0, 200), (0, 5), (0, 0), (0, 333)], fmt=fmt, d=d, pt=48, Hkv=3, seed=27).on_gpu()
    begin, n = [37, 0, 0, 100], [163, 5, 0, 200]
    cu = np.concatenate([[0], np.cumsum(n)])
    k = torch.full((int(cu[-1]) + 2, 3, d), 9.0, dtype=DT[out], device=DEV)
    v = k.clone()
    kda.kda_kv_gather(c.pool, FMT[fmt], c.pt, i32(cu), i32(begin), c.meta[2], k, v, c.status)
    assert kda.kda_sync_status(c.status) == (kda.KDA_OK, 0)
    vals = ref.values(c.stored, c.scales).astype(np.float32)
    for s in range(4):
        at = begin[s] + np.arange(n[s])
        for w, x in ((0, k), (1, v)):
            want = vals[c.table[s][at // c.pt], :, w, at % c.pt]
            want = want if out == "f32" else ref.to_bf16(want)
            assert np.array_equal(x[cu[s]:cu[s + 1]].float().cpu().numpy(), want)
    assert (k[cu[-1]:] == 9).all() and (v[cu[-1]:] == 9).all()       # rows that no sequence owns


@pytest.mark.parametrize("fmt,dtype", [(ref.I8, "bf16"), (ref.BF16, "bf16"), (ref.I8, "f32")])
def test_append_token_by_token_then_attend(fmt, dtype):
    """A prompt in two pieces, then single tokens: the cache that the steps build is the one that
    the attention reads."""
    c = Case([(0, 60), (0, 21)], fmt=fmt, dtype=dtype, pt=32, seed=28)
    c.kv_len = np.array([0, 0])
    need = [ -(-60 // 32), 1]
    c.on_gpu()
    cs = table_of(64, 64, c.r)
    csg = torch.from_numpy(cs).to(DEV)
    for step in [(30, 11), (17, 5), (1, 1), (1, 0), (1, 1), (1, 1)]:
        c.lens = [(n, L + n) for n, L in zip(step, c.kv_len)]
        c.kv_len = np.array([L for _, L in c.lens])
        c.cu = np.concatenate([[0], np.cumsum(step)])
        c.T, c.max_q = int(c.cu[-1]), max(step)
        c.q = c.token(c.Hkv * c.G)
        k, v = c.token(c.Hkv), c.token(c.Hkv)
        c.meta = (i32(c.cu), i32(c.kv_len), c.meta[2])
        qo = torch.empty(c.T, c.Hkv * c.G, c.d, dtype=DT[dtype], device=DEV)
        kda.kda_kv_append(c.pool, FMT[fmt], c.pt, *c.meta, c.max_q, c.gpu(c.q), c.gpu(k), c.gpu(v), csg, qo, c.status)
        o, lse = c.attend(q=qo)
        ref.append(c.stored, c.scales, c.table, c.cu, c.kv_len, k, v, cs, False, c.pt)
        c.q = qo.float().cpu().numpy()
        c.close(o, lse, *c.expect())
    assert kda.kda_sync_status(c.status) == (kda.KDA_OK, 0)
    del need
