"""Host-side refusals of the drafted trees' attention (no GPU), and its oracle:
every call here is refused before any launch, or launches nothing."""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import attn_oracle as O
from tests.test_attn_abi_host import A, BAD_HEADS, INV, L, MIS, OK, UNS   # noqa: F401


def _call(L, **o):                                        # noqa: F811
    a = dict(dt=B.MHC_BF16, q=A, qs=512, kc=A, kp=2048, ksl=128, kh=64, vc=A, vp=2048, vsl=128, vh=64, pages=4,
             ps=16, pt=A, ts=4, tree=A, trs=1, cu=A, kv=A, T=4, B=2, Hq=8, Hk=2, Dh=64, mq=4, mkv=64, window=0,
             scale=0.125, cap=0.0, o=A, lse=A, ws=A, n=1 << 30)
    a.update(o)
    return L.mhc_tree_attn(*a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_HEADS + [
    (dict(q=None), INV), (dict(tree=None), INV), (dict(tree=A + 2), MIS), (dict(trs=0), INV), (dict(mq=33), INV),
    (dict(mq=1025, trs=33), UNS), (dict(trs=(1 << 36) + 1), UNS), (dict(pt=None), INV), (dict(o=None), INV),
    (dict(ws=None), INV), (dict(n=100), INV), (dict(cu=None), INV), (dict(kv=None), INV),
    (dict(cu=None, kv=None), INV), (dict(kv=A + 2), MIS), (dict(scale=0.0), INV),
    (dict(cap=float("nan")), INV), (dict(window=-1), INV), (dict(mkv=65), INV), (dict(mkv=1 << 31), UNS)])
def test_refusals(L, bad, status):                        # noqa: F811
    assert _call(L, **bad) == status


def test_of_nothing(L):                                   # noqa: F811
    assert _call(L, T=0, q=None, tree=None) == OK
    assert _call(L, B=0, pt=None) == OK


def test_binding_refuses_what_it_cannot_pass_on(L):       # noqa: F811
    q, k = torch.zeros(2, 4, 64), torch.zeros(1, 2, 2, 64)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)       # noqa: E731
    with pytest.raises(ValueError):
        B.mhc_tree_attn(q, k, k, i(1, 1), i(2, 1), i(2), i(1))        # host tensors
    with pytest.raises(TypeError):
        B.mhc_tree_attn(q, k, k, i(1, 1), i(2, 1).bool(), i(2), i(1))
    with pytest.raises(TypeError):
        B.mhc_tree_attn(q, k, k, i(1, 1), None, i(2), i(1))


def test_oracle_of_a_chain_is_causal():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(5, 4, 8)), rng.normal(size=(9, 2, 8)), rng.normal(size=(9, 2, 8))
    for window in (0, 1, 3, 7):
        a = O.attention(q, k, v, 0.3, window, 2.0)
        chain = np.tril(np.ones((5, 5), bool))
        if window:       # a causal window hides the chain's own early tokens too
            chain &= np.arange(5)[None, :] > np.arange(5)[:, None] - window
        b = O.tree_attention(q, k, v, 0.3, chain, window, 2.0)
        for x, y in zip(a, b):
            assert np.allclose(x, y, atol=1e-13)


def test_oracle_of_a_tree_is_its_paths():
    """Every node's row is that of the last token of its path alone."""
    rng = np.random.default_rng(1)
    parents = [-1, 0, 0, 1, 2, 2, -1]
    q, k, v = rng.normal(size=(7, 2, 8)), rng.normal(size=(11, 1, 8)), rng.normal(size=(11, 1, 8))
    mask = np.zeros((7, 7), bool)
    for i, p in enumerate(parents):
        mask[i] = mask[p] if p >= 0 else False
        mask[i, i] = True
    for window in (0, 3, 5):
        o, lse, *_ = O.tree_attention(q, k, v, 0.3, mask, window)
        for i in range(7):
            keys = list(range(4)) + [4 + j for j in range(7) if mask[i, j]]
            po, pl, *_ = O.attention(q[i:i + 1], k[keys], v[keys], 0.3, window)
            assert np.allclose(o[i], po[0]) and np.allclose(lse[i], pl[0])
