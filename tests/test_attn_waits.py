"""Waits of the attention kernels that run out let every warp leave.

A warp's wait on an mbarrier is bounded, but one that stands at a named barrier stands there until
its whole group has come.  Two rules keep that bounded too: in the register kernel a warp that leaves
sets the error and arrives once more, and every meeting is followed by a look at the error; in the
tensor-core kernel one warp of a group looks at mbarriers and all get its answer at the barrier.
Here every order of steps is tried on a model of the first rule, and the sources are held to both."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "kda_state_chunked_gb300", "csrc", "kernels")
PROGRAM = "wMMwMw"      # w: a wait, which may run out; M: a meeting of the group


def stuck(warps, arrives, looks):
    """Whether some order of steps leaves a warp at a meeting for good."""
    # a warp: place in the program, whether it stands at a meeting; len(PROGRAM): gone
    start = (tuple((0, False) for _ in range(warps)), 0, False)      # warps, arrivals of this phase, error
    seen, todo = {start}, [start]
    while todo:
        state = todo.pop()
        ws, count, err = state
        nexts = []

        def step(i, w, count=count, err=err, ws=ws):
            new = list(ws)
            new[i] = w
            if count == warps:           # the phase is over: all who stand go on, and look at the error
                count = 0
                for j, (at, standing) in enumerate(new):
                    if standing:
                        new[j] = (at, None)
            nexts.append((tuple(new), count, err))

        gone = len(PROGRAM)
        for i, (at, standing) in enumerate(ws):
            if at == gone or standing is True:
                continue
            if standing is None:                                   # behind a meeting, before the look
                if looks and err:
                    step(i, (gone, False), count + arrives)
                else:
                    step(i, (at + 1, False))
            elif PROGRAM[at] == "M":
                step(i, (at, True), count + 1)
            else:
                step(i, (at + 1, False))                           # what it waits for has come
                step(i, (gone, False), count + arrives, True)      # or the wait runs out
        if not nexts and any(at != gone for at, _ in ws):
            return True
        for n in nexts:
            if n not in seen:
                seen.add(n)
                todo.append(n)
    return False


@pytest.mark.parametrize("warps", [2, 3, 4])
def test_leaving_warps_hold_nobody(warps):
    assert not stuck(warps, arrives=1, looks=True)


def test_either_half_of_the_rule_alone_does():
    assert stuck(3, arrives=0, looks=True) and stuck(3, arrives=1, looks=False) and stuck(3, arrives=0, looks=False)


def source(name):
    return open(os.path.join(SRC, name)).read()


def test_register_kernel_looks_after_every_meeting():
    t = source("attn_decode.cu")
    calls, looked = re.findall(r"\bmeet\(\)", t), re.findall(r"\bok = meet\(\);", t)
    assert len(calls) == len(looked) > 0
    assert len(re.findall(r"bar\.sync", t)) == len(re.findall(r"bar\.arrive", t)) == 1
    body = t[t.index("auto meet = "):]
    assert re.search(r"if \(!ok\) \{[^}]*flag_status[^}]*bar\.arrive", body, re.S)


def test_tensor_core_kernel_waits_in_groups_where_it_meets_in_groups():
    t = source("attn_prefill.cu")
    soft = t[t.index("softmax and output"):t.index("queries, and keys and values")]
    load = t[t.index("queries, and keys and values"):t.index("// ================================================== products")]
    for role in (soft, load):
        # no warp decides by itself to leave: each wait is a group's
        assert not re.search(r"\bwait_job\(|\bwait\(|\bwait_slow\(|mbar_", role)
        alone = [line for line in role.splitlines() if "wait1(" in line and "together" not in line and "return wait1" not in line]
        assert not alone, alone
