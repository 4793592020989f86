"""Host-side refusals of a step's tables and of keeping a path (no GPU), and their
oracle: every call here is refused before any launch, or launches nothing."""

import ctypes

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import paged_oracle as O
from tests.test_attn_abi_host import A, INV, L, MIS, OK, UNS   # noqa: F401


@pytest.mark.parametrize("bad,status", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(width=-1), INV), (dict(cap=-1), INV), (dict(page=0), INV),
    (dict(B=8193), UNS), (dict(T=(1 << 30) + 1), UNS), (dict(cap=(1 << 30) + 1), UNS), (dict(page=(1 << 20) + 1), UNS),
    (dict(width=1 << 30, stride=1 << 30), UNS), (dict(stride=7), INV), (dict(stride=(1 << 36) + 1), UNS),
    (dict(new=None), INV), (dict(lens=None), INV), (dict(table=None), INV), (dict(held=None), INV),
    (dict(free=None), INV), (dict(count=None), INV), (dict(cu=None), INV), (dict(kv=None), INV), (dict(pos=None), INV),
    (dict(slots=None), INV), (dict(tree=None), INV), (dict(parents=None), INV), (dict(words=0), INV),
    (dict(words=33), UNS), (dict(new=A + 2), MIS), (dict(slots=A + 4), MIS), (dict(tree=A + 1), MIS),
    (dict(held=A + 3), MIS), (dict(count=A + 2), MIS), (dict(parents=A + 2), MIS)])
def test_step_refusals(L, bad, status):                   # noqa: F811
    a = dict(new=A, lens=A, B=4, table=A, stride=8, width=8, held=A, free=A, cap=10, count=A, page=16, T=9, parents=A,
             words=1, cu=A, kv=A, pos=A, slots=A, tree=A)
    a.update(bad)
    assert L.mhc_paged_step(*a.values(), None) == status


STEP_INPUTS, STEP_OUTPUTS = ("new", "lens", "parents"), ("table", "held", "free", "count", "cu", "kv", "pos", "slots", "tree")


def _step_apart(**o):
    """Arguments of a step whose tensors lie 64 KB apart: 4 sequences, a table of 4 rows
    of 8 entries 12 apart, 9 tokens, 10 free pages."""
    a = dict(new=0, lens=0, B=4, table=0, stride=12, width=8, held=0, free=0, cap=10, count=0, page=16, T=9, parents=0,
             words=2, cu=0, kv=0, pos=0, slots=0, tree=0)
    for i, k in enumerate(STEP_INPUTS + STEP_OUTPUTS):
        a[k] = A + 65536 * i
    a.update(o)
    return a


@pytest.mark.parametrize("out", STEP_OUTPUTS)
def test_step_refuses_outputs_in_the_memory_of_others(L, out):        # noqa: F811
    """Blocks read the inputs while outputs are written (lengths that are to advance in
    place, kv_lens = lens, among them)."""
    size = dict(new=16, lens=16, parents=36, table=4 * (3 * 12 + 8), held=16, free=40, count=4, cu=20, kv=16, pos=36,
                slots=72, tree=72)
    a = _step_apart()
    for other in STEP_INPUTS + STEP_OUTPUTS:
        if other == out:
            continue
        last = size[other] - 4 if out != "slots" else (size[other] - 1) // 8 * 8
        for at in (a[other], a[other] + last):                         # its first and its last entry
            assert L.mhc_paged_step(*_step_apart(**{out: at}).values(), None) == INV, (other, at - a[other])


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory: nothing may be launched")
def test_step_takes_outputs_beside_and_between_others(L):             # noqa: F811
    """Behind an input's last entry, in the gaps of a table's rows, and inputs that are
    one tensor: past the checks, at the launch (which needs a GPU)."""
    a = _step_apart()
    for o in ({}, dict(kv=a["lens"] + 16), dict(kv=a["lens"] - 16), dict(new=a["lens"]), dict(held=a["table"] + 32),
              dict(held=a["table"] + 4 * 44), dict(table=a["held"] - 32), dict(count=a["table"] + 4 * (12 + 11)),
              dict(slots=a["pos"] + 40), dict(parents=None, tree=None, words=0)):
        assert L.mhc_paged_step(*_step_apart(**o).values(), None) == B.MHC_ERR_CUDA, o


def _pointers(*p):
    return (ctypes.c_void_p * len(p))(*p)


def _keep(L, **o):                                        # noqa: F811
    a = dict(dt=B.MHC_BF16, k=_pointers(A, A), kp=2048, ks=128, kh=64, v=_pointers(A, A), vp=2048, vs=128, vh=64,
             layers=2, pages=4, page=16, table=A, ts=4, cu=A, kv=A, max_kv=64, B=2, Hk=2, Dh=64, path=A, ps=3, most=3,
             keep=A, lens=A)
    a.update(o)
    return L.mhc_cache_keep(*a.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(dt=5), INV), (dict(Hk=0), INV), (dict(Dh=60), UNS), (dict(Dh=264), UNS), (dict(B=-1), INV),
    (dict(layers=-1), INV), (dict(most=-1), INV), (dict(max_kv=-1), INV), (dict(max_kv=65), INV),
    (dict(max_kv=1 << 31), UNS), (dict(k=None), INV), (dict(v=_pointers(A, None)), INV), (dict(k=_pointers(A, A + 8)), MIS),
    (dict(ps=2), INV), (dict(kp=2052), MIS), (dict(vh=60), INV), (dict(page=0), INV), (dict(table=None), INV),
    (dict(cu=None), INV), (dict(kv=A + 2), MIS), (dict(path=None), INV), (dict(keep=None), INV), (dict(lens=A + 2), MIS),
    (dict(ts=3), INV), (dict(B=(1 << 24) + 1), UNS)])
def test_keep_refusals(L, bad, status):                   # noqa: F811
    assert _keep(L, **bad) == status


def test_keep_refuses_lengths_that_it_reads(L):           # noqa: F811
    """Blocks read kv_lens (and the others) while lens is written."""
    far = {k: A + 4096 * i for i, k in enumerate(("table", "cu", "kv", "path", "keep"), 1)}
    for k, at in far.items():
        for lens in (at, at - 4):
            assert _keep(L, **{**far, "lens": lens}) == INV, k
    assert _keep(L, **far, lens=far["table"] + 4 * 7) == INV     # its second row's last page
    assert _keep(L, **far, lens=far["path"] + 4 * 5) == INV


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are not memory: nothing may be launched")
def test_keep_takes_lengths_beside_and_between_what_it_reads(L):      # noqa: F811
    """In the gaps of a table's or a path's rows, and behind their last entries."""
    far = {k: A + 4096 * i for i, k in enumerate(("table", "cu", "kv", "path", "keep"), 1)}
    for lens in (far["table"] + 16, far["table"] + 48, far["path"] + 12, far["cu"] + 12, far["kv"] - 8, far["keep"] + 8):
        assert _keep(L, **far, ts=8, ps=6, lens=lens) == B.MHC_ERR_CUDA, lens
    for lens in (far["table"] + 12, far["table"] + 28, far["table"] + 44, far["path"] + 20, far["path"] + 32):
        assert _keep(L, **far, ts=8, ps=6, lens=lens) == INV, lens


def test_keep_of_nothing(L):                              # noqa: F811
    for none in (dict(B=0, cu=None), dict(layers=0, k=None), dict(most=0, path=None)):
        assert _keep(L, **none) == OK


def test_binding_refuses_what_it_cannot_pass_on(L):       # noqa: F811
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)       # noqa: E731
    with pytest.raises(ValueError):
        B.mhc_paged_step(i(2), i(2), i(2, 3), i(2), i(4), i(1), 16, 2)        # host tensors
    with pytest.raises(TypeError):
        B.mhc_paged_step(i(2), i(2), i(2, 3).long(), i(2), i(4), i(1), 16, 2)
    c = torch.zeros(2, 16, 2, 64)
    with pytest.raises(ValueError):
        B.mhc_cache_keep(c, c, i(2, 3), i(3), i(2), i(2, 2), i(2))
    with pytest.raises(TypeError):
        B.mhc_cache_keep(c.half(), c, i(2, 3), i(3), i(2), i(2, 2), i(2))


def test_oracle_pages_are_each_in_one_place():
    """Random steps: every page is free or held by one sequence, and covers it."""
    rng = np.random.default_rng(0)
    table, held, lens, free = [[-1] * 8 for _ in range(5)], [0] * 5, [0] * 5, list(range(20))
    starved = 0
    for _ in range(200):
        new = [-1 if rng.random() < 0.1 else min(int(rng.integers(0, 7)), 32 - m) for m in lens]
        r = O.step(new, lens, table, held, free, 4, sum(max(0, n) for n in new))
        mine = [p for t, h in zip(table, held) for p in t[:h]]
        assert sorted(mine + free) == list(range(20))
        starved += sum(k == m and n > 0 for k, m, n in zip(r["kv_lens"], lens, new))
        lens = r["kv_lens"]
        assert all(h * 4 >= m for h, m in zip(held, lens))
        used = [s for s in r["slots"] if s >= 0]
        assert len(set(used)) == len(used)
    assert starved > 0


def test_oracle_of_a_tree():
    r = O.step([3, 4], [5, 0], [[3, 1], [2, 0]], [2, 1], [], 4, 8, [-1, 0, 0, -1, 0, 1, 0], 1)
    assert r["tree"][:, 0].tolist() == [1, 3, 5, 1, 3, 7, 9, 0]
    assert r["positions"] == [5, 6, 6, 0, 1, 2, 1, 0]
    assert r["slots"] == [5, 6, 7, 8, 9, 10, 11, -1] and r["kv_lens"] == [8, 4] and r["cu_q"] == [0, 3, 7]
