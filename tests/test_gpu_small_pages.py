"""States in pages smaller than what a thread reads of them, in an order whose ends look contiguous and whose middle is not."""
import numpy as np
import pytest
import torch

import kda_state_chunked_gb300 as kda
from kda_state_chunked_gb300 import workloads
from kda_cases import random_state, read_object_bytes, write_object
from oracle import policy

pytestmark = pytest.mark.gpu
DEV, H, D, PAGE = "cuda", 1, 128, 4096      # 32 rows of a state, 16 KiB, go over four pages


def orders(P, first):
    """Page lists of one object: in order, and with the two middle ones of every four exchanged."""
    whole = np.arange(first, first + P, dtype=np.int32)
    mixed = whole.copy()
    mixed[1:P - 2:4], mixed[2:P - 1:4] = whole[2:P - 1:4], whole[1:P - 2:4]
    return whole, mixed


def test_resumed_prefill_reads_and_writes_every_page_in_its_place():
    P = policy.object_pages(H, D, "bf16", PAGE)
    pool = kda.Pool(PAGE, 8 * P, DEV)
    T = 640
    tok = {k: v.to(DEV) for k, v in workloads.make_tokens(T, H, D, "bf16", 9, "cpu").items()}
    S, win = random_state(H, D, "bf16", torch.Generator().manual_seed(9))
    got = []
    for at, act in enumerate(orders(P, 0)):
        kda.kda_page_claim(pool, act)
        ck = orders(P, 2 * P)[at]
        kda.kda_page_claim(pool, ck)
        write_object(pool, act, S, win, "bf16")
        ws = kda.prefill_workspace(tok["q"], [0, T], [512], 1, P)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o = torch.empty_like(tok["q"])
        kda.kda_prefill_varlen(pool, [0, T], [512], [1], tok["q"], tok["k"], tok["v"], tok["alpha"], tok["beta"], tok["conv_w"], o, act,
                               [0], [1024], ck, ws, st)
        assert kda.kda_sync_status(st) == (kda.KDA_OK, 0)
        nb = policy.object_bytes(H, D, "bf16")
        got.append((o, read_object_bytes(pool, act, nb), read_object_bytes(pool, ck, nb)))
        kda.kda_page_decref(pool, act)
        kda.kda_page_decref(pool, ck)
    assert torch.equal(got[0][0], got[1][0]) and got[0][1:] == got[1][1:]


def shuffles(P, first, rng):
    """Page lists of one object: in order, back to front, any order, and in order but for one page in the middle of every
    three, four and seven, which is another's of those."""
    whole = np.arange(first, first + P, dtype=np.int32)
    out = [whole, whole[::-1].copy(), rng.permutation(whole)]
    for step in (3, 4, 7):
        at = np.arange(step // 2, P, step)
        some = whole.copy()
        some[at] = np.roll(whole[at], 1)
        out.append(some)
    return out


@pytest.mark.parametrize("page", [256, 768, 1024, 2560, 8192, 16384, 20480])
def test_any_order_of_pages_of_any_size(page):
    P = policy.object_pages(H, D, "bf16", page)
    pool = kda.Pool(page, 2 * P, DEV)
    T = 200
    tok = {k: v.to(DEV) for k, v in workloads.make_tokens(T, H, D, "bf16", 10, "cpu").items()}
    S, win = random_state(H, D, "bf16", torch.Generator().manual_seed(10))
    nb, want = policy.object_bytes(H, D, "bf16"), None
    rng = np.random.default_rng(page)
    for act, ck in zip(shuffles(P, 0, rng), shuffles(P, P, rng)):
        kda.kda_page_claim(pool, act)
        kda.kda_page_claim(pool, ck)
        write_object(pool, act, S, win, "bf16")
        ws = kda.prefill_workspace(tok["q"], [0, T], [512], 1, P)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        o = torch.empty_like(tok["q"])
        kda.kda_prefill_varlen(pool, [0, T], [512], [1], tok["q"], tok["k"], tok["v"], tok["alpha"], tok["beta"], tok["conv_w"], o, act,
                               [0], [640], ck, ws, st)
        assert kda.kda_sync_status(st) == (kda.KDA_OK, 0)
        got = o, read_object_bytes(pool, act, nb), read_object_bytes(pool, ck, nb)
        want = want or got
        assert torch.equal(got[0], want[0]) and got[1:] == want[1:]
        kda.kda_page_decref(pool, act)
        kda.kda_page_decref(pool, ck)
