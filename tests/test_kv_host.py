"""Key/value cache calls on the CPU: sizes, and refusals before anything is enqueued."""
import ctypes

import pytest

import kda_state_chunked_gb300 as kda
import kv_ref as ref
from kda_state_chunked_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


@pytest.mark.parametrize("H,d,pt", [(1, 64, 16), (8, 128, 64), (3, 64, 48), (4, 128, 128)])
def test_page_bytes(H, d, pt):
    for name, fmt in (("i8", kda.KDA_KV_I8), ("bf16", kda.KDA_KV_BF16)):
        assert kda.kda_kv_page_bytes(H, d, fmt, pt) == ref.page_bytes(H, d, name, pt)


@pytest.mark.parametrize("bad", [(0, 64, 0, 64), (1, 96, 0, 64), (1, 64, 2, 64), (1, 64, 1, 8), (1, 64, 1, 40), (1, 64, 1, 144)])
def test_page_bytes_refuses(bad):
    assert kda.lib().kda_kv_page_bytes(*bad) == kda.KDA_EINVAL


A = 1 << 20          # an aligned address that no refused call touches


def append_args(**kw):
    pool = kda.Pool(kda.kda_kv_page_bytes(2, 64, kda.KDA_KV_I8, 32), 4)
    a = dict(pool=pool.handle, Hq=4, Hkv=2, d=64, dtype=kda.KDA_BF16, fmt=kda.KDA_KV_I8, pt=32, nseq=1, T=3, max_q=3,
             cu=A, kv_len=A, table=A, max_pages=2, q=A, q_stride=256, k=A, k_stride=128, v=A, v_stride=128, cs=A,
             max_pos=64, rot=32, il=0, q_out=A, base=A, status=A, stream=None)
    a.update(kw)
    return pool, list(a.values())


APPEND_BAD = [dict(pool=None), dict(Hkv=0), dict(d=96), dict(dtype=2), dict(fmt=5), dict(pt=24), dict(pt=48), dict(nseq=0),
              dict(T=-1), dict(max_q=-1), dict(cu=None), dict(kv_len=None), dict(table=None), dict(max_pages=0),
              dict(max_pages=-1), dict(q=None), dict(q_out=None), dict(q=A + 2), dict(q_stride=255), dict(q_stride=260),
              dict(k=None), dict(k_stride=64), dict(k=A + 8), dict(v=None), dict(v_stride=132), dict(rot=24), dict(rot=80),
              dict(rot=0), dict(max_pos=0), dict(cs=None), dict(cs=A + 4), dict(base=None), dict(base=A + 8),
              dict(status=None), dict(Hq=0), dict(max_pages=1 << 30)]


@pytest.mark.parametrize("bad", APPEND_BAD, ids=lambda b: "-".join("%s=%s" % i for i in b.items()))
def test_append_refuses(bad):
    pool, args = append_args(**bad)
    assert kda.lib().kda_kv_append(*args) == kda.KDA_EINVAL


def test_nothing_to_append_is_no_error():
    for kw in (dict(T=0), dict(max_q=0)):
        pool, args = append_args(**kw)
        assert kda.lib().kda_kv_append(*args) == kda.KDA_OK


def gather_args(**kw):
    pool = kda.Pool(kda.kda_kv_page_bytes(2, 64, kda.KDA_KV_I8, 32), 4)
    a = dict(pool=pool.handle, Hkv=2, d=64, dtype=kda.KDA_BF16, fmt=kda.KDA_KV_I8, pt=32, nseq=1, T=3, cu=A, begin=A,
             table=A, max_pages=2, k=A, v=A, base=A, status=A, stream=None)
    a.update(kw)
    return pool, list(a.values())


@pytest.mark.parametrize("bad", [dict(pool=None), dict(Hkv=3), dict(dtype=7), dict(nseq=0), dict(T=-1), dict(cu=None),
                                 dict(begin=None), dict(table=None), dict(max_pages=0), dict(k=None), dict(v=A + 2),
                                 dict(status=None)], ids=str)
def test_gather_refuses(bad):
    pool, args = gather_args(**bad)
    assert kda.lib().kda_kv_gather(*args) == kda.KDA_EINVAL


def attn_args(**kw):
    pool = kda.Pool(kda.kda_kv_page_bytes(2, 64, kda.KDA_KV_I8, 32), 4)
    a = dict(pool=pool.handle, Hq=4, Hkv=2, d=64, dtype=kda.KDA_BF16, fmt=kda.KDA_KV_I8, pt=32, nseq=1, T=3, max_q=3, cu=A,
             kv_len=A, table=A, max_pages=2, q=A, q_stride=256, scale=0.1, window=0, sinks=0, o=A, lse=None, base=A, ws=A,
             ws_bytes=kda.kda_attn_workspace_bytes(4, 2, 64, kda.KDA_BF16, 1, 3, 3), status=A, stream=None)
    a.update(kw)
    return pool, list(a.values())


@pytest.mark.parametrize("bad", [dict(pool=None), dict(Hq=3), dict(Hq=0), dict(d=80), dict(dtype=-1), dict(fmt=2), dict(pt=0),
                                 dict(nseq=0), dict(T=-2), dict(max_q=-1), dict(cu=None), dict(kv_len=None), dict(table=None),
                                 dict(q=None), dict(q=A + 4), dict(q_stride=128), dict(window=-1), dict(sinks=-1),
                                 dict(o=None), dict(o=A + 8), dict(base=None), dict(ws=None), dict(ws=A + 8), dict(ws_bytes=64),
                                 dict(status=None)], ids=str)
def test_attention_refuses(bad):
    pool, args = attn_args(**bad)
    assert kda.lib().kda_attn_paged(*args) == kda.KDA_EINVAL


def test_no_queries_is_no_error():
    for kw in (dict(T=0), dict(max_q=0)):
        pool, args = attn_args(**kw)
        assert kda.lib().kda_attn_paged(*args) == kda.KDA_OK


def test_workspace_bytes_refuses():
    f = kda.lib().kda_attn_workspace_bytes
    for bad in ((3, 2, 64, 1, 1, 1, 1), (4, 0, 64, 1, 1, 1, 1), (4, 2, 32, 1, 1, 1, 1), (4, 2, 64, 3, 1, 1, 1),
                (4, 2, 64, 1, 0, 1, 1), (4, 2, 64, 1, 1, -1, 1), (4, 2, 64, 1, 1, 1, -1)):
        assert f(*bad) == kda.KDA_EINVAL


def test_binding_refuses_shapes_that_do_not_fit():
    torch = pytest.importorskip("torch")
    pool = kda.Pool(kda.kda_kv_page_bytes(2, 64, kda.KDA_KV_I8, 32), 4)
    x = torch.zeros(3, 2, 64)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):          # not on a GPU
        kda.kda_kv_append(pool, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, None, x, x, None, None, i)
    with pytest.raises(ValueError):          # q without q_out
        kda.kda_kv_append(pool, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, x, x, x, None, None, i)
    with pytest.raises(ValueError):          # int64 lengths
        kda.kda_attn_paged(pool, 2, kda.KDA_KV_I8, 32, i.long(), i[:1], i.view(1, 2), 3, x, x, i, i)
    assert isinstance(pool.handle, ctypes.c_void_p)
