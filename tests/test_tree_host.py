"""Calls on trees of drafts on the CPU: refusals before anything is enqueued."""
import numpy as np
import pytest

import kda_state_chunked_gb300 as kda
from kda_state_chunked_gb300 import build as kbuild
from test_kv_host import A, append_args, attn_args


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


def named(bad):
    return "-".join("%s=%s" % i for i in bad.items())


def plan_args(**kw):
    a = dict(nseq=2, T=5, max_q=3, cu=A, kv_len=A, parent=A, mask=A, pos=A, status=A, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("bad", [dict(nseq=0), dict(T=-1), dict(max_q=-1), dict(max_q=65), dict(cu=None), dict(kv_len=None),
                                 dict(parent=None), dict(mask=None), dict(pos=None), dict(status=None)], ids=named)
def test_plan_refuses(bad):
    assert kda.lib().kda_tree_plan(*plan_args(**bad)) == kda.KDA_EINVAL


SECTIONS = np.array([8, 8], np.int32)


def append_at_args(sections=SECTIONS, pos=A, axes=2, **kw):
    pool, args = append_args(**kw)
    at = list(append_args()[1]).__len__() - 4     # before q_out, base, status, stream
    sec = None if sections is None else sections.ctypes.data
    return pool, args[:at] + [pos, axes, sec] + args[at:]


@pytest.mark.parametrize("bad", [dict(pos=None), dict(axes=0), dict(axes=5), dict(axes=1), dict(sections=None), dict(cs=None),
                                 dict(sections=np.array([8, 16], np.int32)), dict(sections=np.array([16, 0], np.int32)),
                                 dict(sections=np.array([24, -8], np.int32)), dict(sections=np.array([12, 4], np.int32)),
                                 dict(rot=64), dict(max_pos=0), dict(q=None), dict(k=A + 8), dict(v_stride=132), dict(status=None),
                                 dict(pool=None), dict(pt=24)],
                         ids=lambda b: "-".join("%s=%s" % (k, list(v) if isinstance(v, np.ndarray) else v) for k, v in b.items()))
def test_append_at_refuses(bad):
    pool, args = append_at_args(**bad)
    assert kda.lib().kda_kv_append_at(*args) == kda.KDA_EINVAL


def tree_attn_args(mask=A, pos=A, **kw):
    pool, args = attn_args(**kw)
    at = 14                                       # behind max_pages
    return pool, args[:at] + [mask, pos] + args[at:]


@pytest.mark.parametrize("bad", [dict(mask=None), dict(pos=None, window=5), dict(max_q=65), dict(pool=None), dict(Hq=3), dict(d=80),
                                 dict(q=A + 4), dict(window=-1), dict(sinks=-1), dict(o=A + 8), dict(ws=None), dict(ws_bytes=64),
                                 dict(status=None), dict(scale=float("nan")), dict(cu=None), dict(table=None)], ids=named)
def test_tree_attention_refuses(bad):
    pool, args = tree_attn_args(**bad)
    assert kda.lib().kda_attn_tree(*args) == kda.KDA_EINVAL


def test_tree_attention_workspace():
    f = kda.lib().kda_attn_tree_workspace_bytes
    assert f(4, 2, 64, 1, 1, 64, 64) >= kda.kda_attn_workspace_bytes(4, 2, 64, 1, 1, 64, 64) > 0
    assert f(4, 2, 64, 1, 1, 65, 65) == kda.KDA_EINVAL and f(3, 2, 64, 1, 1, 1, 1) == kda.KDA_EINVAL


def accept_args(**kw):
    pool = kda.Pool(kda.kda_kv_page_bytes(2, 64, kda.KDA_KV_I8, 32), 4)
    a = dict(pool=pool.handle, Hkv=2, d=64, fmt=kda.KDA_KV_I8, pt=32, nseq=2, T=3, max_q=3, cu=A, kv_len=A, table=A, max_pages=2,
             path=A, accepted=A, out=A + 4096, base=A, status=A, stream=None)
    a.update(kw)
    return pool, list(a.values())


@pytest.mark.parametrize("bad", [dict(pool=None), dict(Hkv=3), dict(d=96), dict(fmt=2), dict(pt=40), dict(nseq=0), dict(T=-1),
                                 dict(max_q=65), dict(cu=None), dict(kv_len=None), dict(table=None), dict(path=None),
                                 dict(accepted=None), dict(out=None), dict(out=A), dict(out=A + 4), dict(kv_len=A + 4100), dict(accepted=A + 4092),
                                 dict(base=None), dict(base=A + 8), dict(status=None), dict(max_pages=-1)], ids=named)
def test_accept_refuses(bad):
    pool, args = accept_args(**bad)
    assert kda.lib().kda_kv_accept(*args) == kda.KDA_EINVAL


def verify_args(accept=False, **kw):
    pool = kda.Pool(4096, 64)
    a = dict(pool=pool.handle, H=2, d=64, dtype=kda.KDA_BF16, B=2, T=3, max_q=3, cu=A, tree=A)
    if accept:
        a["accepted"] = A
    a.update(q=A, k=A, v=A, alpha=A, beta=A, conv_w=A)
    if not accept:
        a["o"] = A
    a.update(base=A, pages=A, status=A, stream=None)
    a.update(kw)
    return pool, list(a.values())


BAD = [dict(pool=None), dict(H=0), dict(d=96), dict(dtype=2), dict(B=0), dict(T=-1), dict(max_q=65), dict(max_q=-1), dict(cu=None),
       dict(tree=None), dict(q=None), dict(k=A + 8), dict(v=None), dict(alpha=A + 4), dict(beta=None), dict(conv_w=A + 8),
       dict(base=None), dict(base=A + 8), dict(pages=None), dict(status=None), dict(H=4096, B=1 << 20)]


@pytest.mark.parametrize("bad", BAD + [dict(o=None), dict(o=A + 2)], ids=named)
def test_verify_refuses(bad):
    pool, args = verify_args(**bad)
    assert kda.lib().kda_verify_tree(*args) == kda.KDA_EINVAL


@pytest.mark.parametrize("bad", BAD + [dict(accepted=None)], ids=named)
def test_verify_accept_refuses(bad):
    pool, args = verify_args(accept=True, **bad)
    assert kda.lib().kda_verify_tree_accept(*args) == kda.KDA_EINVAL


def test_no_drafts_is_no_error():
    for kw in (dict(T=0), dict(max_q=0)):
        assert kda.lib().kda_tree_plan(*plan_args(**kw)) == kda.KDA_OK
        for f, (pool, args) in ((kda.lib().kda_kv_append_at, append_at_args(**kw)), (kda.lib().kda_attn_tree, tree_attn_args(**kw)),
                                (kda.lib().kda_verify_tree, verify_args(**kw)),
                                (kda.lib().kda_verify_tree_accept, verify_args(accept=True, **kw))):
            assert f(*args) == kda.KDA_OK


# ------------------------------------------------------------------ the binding
def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    pool = kda.Pool(kda.kda_kv_page_bytes(2, 64, kda.KDA_KV_I8, 32), 4)
    x, i, m = torch.zeros(3, 2, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    j = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="mask"):
        kda.kda_tree_plan(i, i[:1], j, 3, j, j, i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_tree_plan(i, i[:1], j, 3, m, j, i[:1])
    with pytest.raises(ValueError, match="mask"):
        kda.kda_attn_tree(pool, 2, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, j, x, x, i, i[:1])
    with pytest.raises(ValueError, match="cos_sin"):
        kda.kda_kv_append_at(pool, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, None, x, x, None, j, [8], None, i[:1])
    with pytest.raises(ValueError, match="pos"):
        kda.kda_kv_append_at(pool, kda.KDA_KV_I8, 32, i, i[:1], i.view(1, 2), 3, None, x, x, x.view(6, 64), j, [8, 8], None, i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_verify_tree(pool, i, j, 3, x, x, x, x, x[..., 0], x, x, i.view(1, 2), i[:1])
