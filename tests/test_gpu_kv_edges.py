"""Edges of the paged attention and the append, each query row by itself.

A row's error is taken over its own columns (root mean square) and held against that row's own
answer e = sum_j p_j v_j, not against the largest of the call:

    rms(o - e) <= u_o rms(e) + u_p sqrt(sum_j p_j^2 mean_c v_jc^2)

u_o: the output's rounding, 2^-8 of bf16 (8 bits); u_p: the probabilities', 2^-8 where they enter
the product as bf16 (16-bit cache), 2^-11 as fp16 (8-bit cache), independent from token to token.
Either gets 1e-5 for fp32 scores: sums of |scale q k log2 e| up to 30 in eight steps, each cut at
2^-24 of that, times ln 2; float32 calls have nothing else.  A log-sum-exp is held to
1e-5 (1 + |lse|)."""
import numpy as np
import pytest
import torch

import kda_state_chunked_gb300 as kda
import kv_ref as ref
from test_gpu_kv import DEV, FMT, KINDS, Case, i32

pytestmark = pytest.mark.gpu

U_O = {"bf16": 2.0 ** -8 + 1e-5, "f32": 1e-5}


def u_p(c):
    return 1e-5 + (0 if c.dtype == "f32" else 2.0 ** -11 if c.fmt == ref.I8 else 2.0 ** -8)


def exact(c, window=0, sinks=0, scale=None, lose=None):
    """o, lse and the probabilities' root sum of squares of every row in 64 bits.  A token whose key
    or value is no number makes the rows that see it NaN and reaches no other.  lose: positions to
    leave out (a planted mistake)."""
    vals, G, d = ref.values(c.stored, c.scales), c.G, c.d
    scale = d ** -0.5 if scale is None else scale
    o = np.zeros((c.T, G * c.Hkv, d))
    lse, noise = np.full(o.shape[:2], -np.inf), np.zeros(o.shape[:2])
    for s, (n, L) in enumerate(zip(np.diff(c.cu), c.kv_len)):
        if not n or not L:
            continue
        j, p = np.arange(L), L - n + np.arange(n)[:, None]
        see = j <= p
        if window:
            see &= (j > p - window) | (j < sinks)
        if lose is not None:
            see &= ~np.isin(j, lose)
        page, slot = np.asarray(c.table[s])[j // c.pt], j % c.pt
        for h in range(G * c.Hkv):
            k, v = vals[page, h // G, 0, slot], vals[page, h // G, 1, slot]
            bad_k, bad_v = ~np.isfinite(k).all(1), ~np.isfinite(v).all(1)
            k, v = np.where(bad_k[:, None], 0, k), np.where(bad_v[:, None], 0, v)
            x = np.where(see, scale * (c.q[c.cu[s]:c.cu[s] + n, h].astype(np.float64) @ k.T), -np.inf)
            m = x.max(1, keepdims=True)
            e = np.exp(x - np.where(np.isfinite(m), m, 0))
            l = e.sum(1, keepdims=True)
            w = e / np.where(l > 0, l, 1)
            rows = slice(c.cu[s], c.cu[s] + n)
            with np.errstate(divide="ignore"):
                z = m + np.log(l)
            poisoned = (see & bad_k).any(1, keepdims=True)
            lse[rows, h] = np.where(poisoned, np.nan, np.where(l > 0, z, -np.inf))[:, 0]
            o[rows, h] = np.where(poisoned | (see & bad_v).any(1, keepdims=True), np.nan, w @ v)
            noise[rows, h] = np.sqrt(w ** 2 @ (v ** 2).mean(1))
    return o, lse, noise


def hold(c, o, lse, want):
    e, el, noise = want
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(o), np.isnan(e)) and np.array_equal(np.isnan(lse), np.isnan(el))
    assert np.array_equal(np.isneginf(lse), np.isneginf(el))
    fine = ~np.isnan(e).any(-1)
    rms = lambda x: np.sqrt((x[fine] ** 2).mean(-1))  # noqa: E731
    over = rms(o - e) / np.maximum(U_O[c.dtype] * rms(e) + u_p(c) * noise[fine], 1e-300)
    assert over.size == 0 or over.max() <= 1, over.max()
    fine = np.isfinite(el)
    assert (np.abs(lse - el)[fine] <= 1e-5 * (1 + np.abs(el[fine]))).all()


def check(c, window=0, sinks=0, **kw):
    o, lse = c.on_gpu().attend(window, sinks, **kw)
    assert kda.kda_sync_status(c.status) == (kda.KDA_OK, 0)
    hold(c, o, lse, exact(c, window, sinks, kw.get("scale")))
    return o, lse


# ------------------------------------------------------------------ every group of tokens counts in its row
@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("n", [1, 4, 40])
def test_every_group_of_tokens_is_felt_by_its_rows(fmt, dtype, d, n):
    """One short context beside long ones, each row against its own answer; the same check has to
    notice a group of 16 tokens left out anywhere."""
    c = Case([(n, n), (n, 700), (n, 1000)], fmt=fmt, dtype=dtype, d=d, Hkv=1, seed=111, qscale=0.5, spread=0.2)
    o, lse = check(c)
    _, el, noise = exact(c)
    for first in range(0, 688, 48):
        with pytest.raises(AssertionError):
            hold(c, o, lse, (exact(c, lose=np.arange(first, first + 16))[0], el, noise))


# ------------------------------------------------------------------ scales that are no numbers
@pytest.mark.parametrize("which,bad", [(0, np.nan), (1, np.nan), (1, np.inf)])
@pytest.mark.parametrize("G,n,pt", [(1, 40, 16), (1, 150, 48), (5, 40, 16), (2, 3, 16)])
def test_rows_before_a_block_that_is_no_number_keep_their_results(which, bad, G, n, pt):
    # block 12 begins in the middle of a warp's rows: those before it do not see it
    c = Case([(n, 12 * pt + n // 2 + 1), (n, n + 7)], fmt=ref.I8, Hkv=2, G=G, pt=pt, seed=101)
    c.scales[c.table[0, 12], :, which] = bad
    c.scales[c.table[1, (n + 6) // pt], :, which] = bad
    o, _ = check(c)
    assert torch.isfinite(o).any() and torch.isnan(o).any()
    # and the rows whose window has left it
    c = Case([(n, 200), (n, n + 90)], fmt=ref.I8, Hkv=2, G=G, pt=pt, seed=102)
    for s, (_, L) in enumerate(c.lens):
        c.scales[c.table[s, (L - n // 2 - 40) // pt], :, which] = bad
    check(c, window=41)


# ------------------------------------------------------------------ blocks of zero keys, scale 0
@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("qscale,scale", [(5e-12, None), (1e-30, None), (2.0, 0.0), (1e30, 0.0)])
def test_equal_scores_at_the_ends_of_the_range(fmt, dtype, d, n, qscale, scale):
    c = Case([(n, 300), (n, 45)], fmt=fmt, dtype=dtype, d=d, qscale=qscale, seed=103)
    c.stored[:, :, 0] = 0
    if fmt == ref.I8:
        c.scales[:, :, 0] = 0
    check(c, scale=scale)
    check(c, window=50, sinks=3, scale=scale)


# ------------------------------------------------------------------ factors beyond the usual range
@pytest.mark.parametrize("fmt,dtype,d", KINDS)
@pytest.mark.parametrize("n", [1, 40])
def test_small_scale_over_large_queries(fmt, dtype, d, n):
    c = Case([(n, 200)], fmt=fmt, dtype=dtype, d=d, qscale=1e32, seed=109, spread=0.1)
    check(c, scale=0.5e-33)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 40])
def test_large_keys_under_small_queries(dtype, n):
    c = Case([(n, 200)], fmt=ref.I8, dtype=dtype, qscale=1e-35, seed=110, spread=0.1)
    c.scales[:, :, 0] *= np.float32(1e35)
    check(c)


# ------------------------------------------------------------------ key scales of 0 and infinity over other codes
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_key_scales_read_as_they_stand(dtype, n):
    c = Case([(n, 300), (n, 45)], fmt=ref.I8, dtype=dtype, G=1, pt=16, qscale=1e30, seed=115)
    c.scales[:, :, 0] = 0
    check(c)                                  # zeros, however large the queries
    c = Case([(n, 300), (n, 45)], fmt=ref.I8, dtype=dtype, G=1, pt=16, seed=116)
    c.scales[c.table[0, 3], :, 0] = np.inf
    c.scales[c.table[1, 2], :, 0] = np.inf    # some of whose rows see it
    check(c)
    check(c, window=40)


# ------------------------------------------------------------------ value scales far apart
def far_apart(c, block, bits, quiet):
    """Blocks `block(s)` get values 2^bits times larger; quiet: and keys that give them 2^-41 of the others'
    weights (a query's first element is 32, and a key's -10 there and 0 elsewhere)."""
    for s in range(len(c.lens)):
        for b in block(s):
            p = c.table[s, b]
            c.scales[p, :, 1] *= 2.0 ** bits
            if quiet:
                c.scales[p, :, 0] = 10 / 127
                c.stored[p, :, 0] = 0
    if quiet:
        c.q[..., 0] = 32
        c.stored[:, :, 0, :, 0] = 0
        for s in range(len(c.lens)):
            for b in block(s):
                c.stored[c.table[s, b], :, 0, :, 0] = -127
    return c


@pytest.mark.parametrize("dtype,bits", [("bf16", 28), ("bf16", 40), ("f32", 16), ("f32", 28), ("f32", 60)])
@pytest.mark.parametrize("n,many", [(1, 1), (4, 1), (40, 1), (2, 40), (40, 40)])
def test_large_values_without_weight_cost_the_others_nothing(dtype, bits, n, many):
    # first in each sequence, and behind others; `many` sequences: a share takes several units
    lens = [(n, 700 - 13 * (i % 7)) for i in range(many)]
    c = Case(lens, fmt=ref.I8, dtype=dtype, Hkv=2, G=2, pt=16, seed=104, qscale=0.5)
    check(far_apart(c, lambda s: [0, 9], bits, True))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [28, 60])
@pytest.mark.parametrize("n,L", [(4, 50), (4, 402), (40, 300), (40, 55)])
def test_large_values_that_a_row_does_not_see_cost_it_nothing(dtype, bits, n, L):
    c = Case([(n, L), (n, L + 32)], fmt=ref.I8, dtype=dtype, Hkv=2, G=2, pt=16, seed=105, qscale=0.5)
    far_apart(c, lambda s: [(int(c.kv_len[s]) - 1) // 16], bits, False)
    check(c)
    c = Case([(n, 300), (n, 340)], fmt=ref.I8, dtype=dtype, Hkv=2, G=2, pt=16, seed=106, qscale=0.5)
    check(far_apart(c, lambda s: [0, 12], bits, False), window=100)


@pytest.mark.parametrize("n", [1, 4])
def test_float32_weights_far_below_the_largest_count(n):
    """A first token with 2^30 times the others' weight and a value of 0: all that comes out is theirs."""
    c = Case([(n, 700)], fmt=ref.I8, dtype="f32", Hkv=2, G=4, pt=16, seed=107, qscale=0.25)
    c.q[..., 0] = 32
    c.stored[:, :, 0, :, 0] = 0
    p = c.table[0, 0]
    c.stored[p, :, :, 0] = 0
    c.scales[p, :, 0] = 7.35 / 127
    c.stored[p, :, 0, 1:] = 0
    c.stored[p, :, 0, 0, 0] = 127
    check(c)


# ------------------------------------------------------------------ scales of 0 over codes that are not
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 40])
def test_codes_under_a_scale_of_zero_read_as_zeros(dtype, n):
    c = Case([(n, 300), (n, 77)], fmt=ref.I8, dtype=dtype, G=2, pt=16, seed=108)
    for s, (_, L) in enumerate(c.lens):
        c.scales[c.table[s, 0]] = 0
        c.scales[c.table[s, 2], :, 0] = 0
        c.scales[c.table[s, 3], :, 1] = 0
    check(c)
    c.scales[:, :, 1] = 0
    o, _ = check(c)
    assert (o == 0).all()


# ------------------------------------------------------------------ append: queries in place, refused sequences
def angles(top, rot, r):
    a = r.standard_normal((top, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rot,pairs", [(32, False), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("lens", [[(1, 30), (1, 1), (1, 64)], [(70, 200), (0, 9), (3, 3)]])
def test_queries_rotate_in_place(dtype, rot, pairs, lens):
    c = Case(lens, fmt=ref.I8, dtype=dtype, G=3, seed=112).on_gpu()
    cs = angles(300, rot, c.r)
    k = c.gpu(c.token(c.Hkv))
    q = c.gpu(c.q)
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, q, k, k, torch.from_numpy(cs).to(DEV), q, c.status,
                      interleaved=pairs)
    assert kda.kda_sync_status(c.status) == (kda.KDA_OK, 0)
    for s, (n, L) in enumerate(c.lens):
        a, b = int(c.cu[s]), int(c.cu[s + 1])
        x = ref.rotate(c.q[a:b], cs[L - n:L], pairs)
        assert np.array_equal(q[a:b].float().cpu().numpy(), x if dtype == "f32" else ref.to_bf16(x))


@pytest.mark.parametrize("rot,what", [(r, w) for r in (0, 32, 128) for w in ("angles", "length", "table") if r or w != "angles"])
@pytest.mark.parametrize("in_place", [False, True])
def test_queries_of_a_refused_sequence_stay(rot, what, in_place):
    c = Case([(4, 70), (2, 20), (3, 70)], G=2, seed=113).on_gpu()
    if what == "angles":
        c.meta[1][2] = 40                      # only the first sequence reaches past the table
    cs = torch.from_numpy(angles(69 if what == "angles" else 100, rot, c.r)).to(DEV) if rot else None
    if what == "length":
        c.meta[1][0] = 3
    if what == "table":
        c.meta[1][0] = c.maxp * c.pt + 1
    k, q = c.gpu(c.token(c.Hkv)), c.gpu(c.q)
    before = q.clone()
    out = q if in_place else torch.full_like(q, 7.0)
    stays = out[:4].clone()
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, q, k, k, cs, out, c.status)
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    assert torch.equal(out[:4], stays)
    assert (rot == 0 and torch.equal(out[4:], before[4:])) or (rot and not torch.equal(out[4:], before[4:]) and (out[4:] != 7).any())


@pytest.mark.parametrize("rot", [0, 32])
def test_query_rows_that_no_sequence_owns_stay(rot):
    c = Case([(2, 20), (9, 70)], G=2, seed=117).on_gpu()
    q = torch.cat([c.gpu(c.q), c.gpu(c.q)])
    k = q[:, :c.Hkv].contiguous()
    out = torch.full_like(q, 7.0)
    cs = torch.from_numpy(angles(100, rot, c.r)).to(DEV) if rot else None
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, q, k, k, cs, out, c.status)
    assert kda.kda_sync_status(c.status) == (kda.KDA_OK, 0)
    assert (out[c.T:] == 7).all() and not (out[:c.T] == 7).all(-1).any()


@pytest.mark.parametrize("n", [1, 3, 20, 200])
@pytest.mark.parametrize("rot", [0, 32])
def test_new_tokens_of_a_sequence_without_length_are_reported(n, rot):
    c = Case([(n, n), (2, 20)], seed=114).on_gpu()
    c.meta[1][0] = 0
    before = c.pool.base.clone()
    k = c.gpu(c.token(c.Hkv))
    cs = torch.from_numpy(angles(300, rot, c.r)).to(DEV) if rot else None
    kda.kda_kv_append(c.pool, FMT[c.fmt], c.pt, *c.meta, c.max_q, None, k, k, cs, None, c.status)
    assert kda.kda_sync_status(c.status) == (kda.KDA_EDEVICE, kda.KDA_DEV_BAD_META)
    mine = torch.from_numpy(c.table[0][c.table[0] >= 0]).to(DEV)
    assert torch.equal(c.pool.base[mine], before[mine]) and not torch.equal(c.pool.base, before)


# ------------------------------------------------------------------ sums over long contexts
def shared_context(L, Hkv, d, fmt, seed):
    """One context of L tokens whose values lie around a mean of 1 to 2 a column: pool, its pages, and the
    keys and values that the cache stands for."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pt = 64
    blocks = -(-L // pt)
    pool = kda.Pool(kda.kda_kv_page_bytes(Hkv, d, FMT[fmt], pt), blocks, DEV)
    pages = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32).view(1, blocks)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    mean = 1 + torch.rand(Hkv, d, generator=g, device=DEV)
    for a in range(0, L, 1 << 17):
        b = min(L, a + (1 << 17))
        k = 0.1 * torch.randn(b - a, Hkv, d, generator=g, device=DEV)
        v = mean + 0.1 * torch.randn(b - a, Hkv, d, generator=g, device=DEV)
        kda.kda_kv_append(pool, FMT[fmt], pt, i32([0, b - a]), i32([b]), pages, b - a, None, k, v, None, None, status)
    k, v = (torch.empty(L, Hkv, d, device=DEV) for _ in range(2))
    kda.kda_kv_gather(pool, FMT[fmt], pt, i32([0, L]), i32([0]), pages, k, v, status)
    assert kda.kda_sync_status(status) == (kda.KDA_OK, 0)
    return pool, pages, k, v, g


# The mean error of a row set's 512 columns: a bf16's rounding, 1.7e-3 in each, leaves 3e-4 at four times its
# deviation, and sums cut no more than 2,048 times 1e-4; of a single column, half a bf16's step and that.
@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("n,nseq,L", [(1, 512, 524288), (4, 160, 70001), (1024, 1, 524288), (300, 24, 70001)])
def test_sums_over_long_contexts_are_not_cut(fmt, n, nseq, L):
    Hkv, G, d = 4, 4, 128
    pool, pages, k, v, g = shared_context(L, Hkv, d, fmt, 118)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.randn(nseq * n, Hkv * G, d, generator=g, device=DEV).to(torch.bfloat16)
    o, lse = torch.empty_like(q), torch.empty(nseq * n, Hkv * G, device=DEV)
    kda.kda_attn_paged(pool, Hkv, FMT[fmt], 64, i32(np.arange(nseq + 1) * n), i32([L] * nseq),
                       pages.expand(nseq, -1).contiguous(), n, q, o, kda.attn_workspace(q, Hkv, nseq, n), status, lse=lse)
    assert kda.kda_sync_status(status) == (kda.KDA_OK, 0)
    off = []
    for t in np.linspace(0, nseq * n - 1, 6).astype(int):
        for h in range(Hkv):
            seen = L - n + t % n + 1
            s = d ** -0.5 * (k[:seen, h].double() @ q[t, h * G].double())
            e = torch.softmax(s, 0) @ v[:seen, h].double()
            off.append((o[t, h * G].double() - e) / e)
            assert abs(float(lse[t, h * G]) - float(torch.logsumexp(s, 0))) <= 1e-5 * (1 + 14)
    off = torch.stack(off)
    assert float(off.abs().max()) <= 2.0 ** -8 + 1e-4 and abs(float(off.mean())) <= 4e-4
    pool.close()


# ------------------------------------------------------------------ few rows over the 16-bit cache round only the output
# Probabilities of 16 bits and fp32 scores leave an answer off by some 3e-5 of the row's size.  A bf16's step is
# 3.9e-3 and more of a value, so that moves 2% of the typical outputs to another bf16, and as many again of
# the small ones; probabilities of 8 bits (1.4e-3) move a third and more.
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 1), (1, 8), (4, 4)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 4)])
def test_few_rows_over_the_16_bit_cache_round_only_the_output(d, n, G, window, sinks):
    c = Case([(n, 700), (n, 1000), (n, 350)], fmt=ref.BF16, d=d, Hkv=3, G=G, seed=119)
    o, _ = check(c, window, sinks)
    nearest = ref.to_bf16(exact(c, window, sinks)[0].astype(np.float32))
    assert (o.float().cpu().numpy() != nearest).mean() <= 0.05


# Contexts a little longer than the pieces that sums are taken in, so that some rows see nothing of the last one;
# with a window, rows that see nothing of the first.  (Half a bf16's step, and 1e-4 as above.)
@pytest.mark.parametrize("fmt", [ref.I8, ref.BF16])
@pytest.mark.parametrize("n,nseq,L,window", [(200, 64, 32868, 0), (200, 64, 40000, 33000), (4, 160, 32770, 0), (4, 160, 16386, 0),
                                             (1, 200, 33001, 33000)])
def test_pieces_that_not_every_row_sees(fmt, n, nseq, L, window):
    Hkv, G, d, sinks = 4, 1, 64, 3
    pool, pages, k, v, g = shared_context(L, Hkv, d, fmt, 120)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.randn(nseq * n, Hkv * G, d, generator=g, device=DEV).to(torch.bfloat16)
    o, lse = torch.empty_like(q), torch.empty(nseq * n, Hkv * G, device=DEV)
    kda.kda_attn_paged(pool, Hkv, FMT[fmt], 64, i32(np.arange(nseq + 1) * n), i32([L] * nseq),
                       pages.expand(nseq, -1).contiguous(), n, q, o, kda.attn_workspace(q, Hkv, nseq, n), status, window=window,
                       sinks=sinks, lse=lse)
    assert kda.kda_sync_status(status) == (kda.KDA_OK, 0)
    p, j = L - n + torch.arange(n, device=DEV)[:, None], torch.arange(L, device=DEV)
    hide = j > p
    if window:
        hide |= (j <= p - window) & (j >= sinks)
    for s in range(0, nseq, 3):
        for h in range(Hkv):
            x = d ** -0.5 * (q[s * n:s * n + n, h].double() @ k[:, h].double().T)
            x.masked_fill_(hide, -np.inf)
            e = torch.softmax(x, 1) @ v[:, h].double()
            assert float(((o[s * n:s * n + n, h].double() - e) / e).abs().max()) <= 2.0 ** -8 + 1e-4
            assert float((lse[s * n:s * n + n, h] - torch.logsumexp(x, 1)).abs().max()) <= 1e-5 * (1 + 11)
    pool.close()
