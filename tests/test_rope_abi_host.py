"""Host-side refusals of the rotation's entry points (no GPU): every call here is
refused before any launch, or launches nothing."""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import attn_oracle as O
from tests.test_attn_abi_host import A, BAD_HEADS, BAD_ROPE, INV, L, MIS, OK, UNS   # noqa: F401

NO_EPS = [b for b in BAD_ROPE if "eps" not in b[0]] + [(dict(rot=0), INV)]


def _rope(fn, **o):
    a = dict(dt=B.MHC_BF16, q=A, qs=512, k=A, ks=128, pos=A, cs=A, mp=10, T=4, Hq=8, Hk=2, Dh=64, rot=64, flags=0,
             qo=A, qos=512, ko=A, kos=128)
    a.update(o)
    return fn(*a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_HEADS + NO_EPS + [
    (dict(q=None), INV), (dict(ko=None), INV), (dict(q=A + 8), MIS), (dict(ko=A + 4), MIS), (dict(qs=504), INV),
    (dict(qs=516), MIS), (dict(kos=120), INV), (dict(ks=132), MIS), (dict(mp=(1 << 30) + 1), UNS)])
def test_rotation_refusals(L, bad, status):              # noqa: F811
    for fn in (L.mhc_rope, L.mhc_rope_bwd):
        assert _rope(fn, **bad) == status


def test_rotation_of_nothing(L):                          # noqa: F811
    assert _rope(L.mhc_rope, T=0, q=None, pos=None) == OK and _rope(L.mhc_rope_bwd, T=0, k=None) == OK


@pytest.mark.parametrize("bad,status", BAD_HEADS + NO_EPS + [
    (dict(v=None), INV), (dict(slots=None), INV), (dict(slots=A + 4), MIS), (dict(vs=100), INV), (dict(ps=0), INV),
    (dict(pages=0), INV), (dict(kp=2052), MIS), (dict(vh=60), INV), (dict(vh=68), MIS), (dict(vc=A + 2), MIS)])
def test_append_refusals(L, bad, status):                 # noqa: F811
    a = dict(dt=B.MHC_BF16, q=A, qs=512, k=A, ks=128, v=A, vs=128, pos=A, cs=A, mp=10, slots=A, T=4, Hq=8, Hk=2,
             Dh=64, rot=64, flags=0, qo=A, qos=512, kc=A, kp=2048, ksl=128, kh=64, vc=A, vp=2048, vsl=128, vh=64,
             pages=4, ps=16)
    a.update(bad)
    assert L.mhc_rope_append(*a.values(), None) == status


@pytest.mark.parametrize("bad,status", [
    (dict(n=-1), INV), (dict(rot=0), INV), (dict(rot=24), UNS), (dict(rot=272), UNS), (dict(n=(1 << 30) + 1), UNS),
    (dict(base=0.5), INV), (dict(base=float("inf")), INV), (dict(factor=0.0), INV), (dict(factor=-1.0), INV),
    (dict(factor=float("nan")), INV), (dict(original=-1.0), INV), (dict(low=4.0, high=4.0), INV),
    (dict(low=float("nan")), INV), (dict(high=float("inf")), INV), (dict(amplitude=float("inf")), INV),
    (dict(out=None), INV), (dict(out=A + 4), MIS)])
def test_table_refusals(L, bad, status):                  # noqa: F811
    a = dict(n=10, rot=64, base=1e4, factor=2.0, original=100.0, low=1.0, high=32.0, amplitude=1.0, out=A)
    a.update(bad)
    assert L.mhc_rope_table(*a.values(), None) == status
    if status == INV and "n" not in bad:
        a["n"] = 0
        assert L.mhc_rope_table(*a.values(), None) == (OK if "out" in bad else INV)


def test_binding_refuses_what_it_cannot_pass_on(L):       # noqa: F811
    q, k, pos, cs = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(9, 64)
    with pytest.raises(ValueError):
        B.mhc_rope(q, k, pos, cs)                            # host tensors
    with pytest.raises(ValueError):
        B.mhc_rope(q, torch.zeros(3, 2, 64), pos, cs)
    with pytest.raises(TypeError):
        B.mhc_rope(q.half(), k.half(), pos, cs)
    with pytest.raises(ValueError):
        B.mhc_rope_table(4, 64, device="cpu")
    with pytest.raises(ValueError):
        B.mhc_rope_table(-4, 64)


def test_oracle_table():
    """A table's rows turn one into the next by their frequencies; scaling by parts
    is plain for fast pairs, linear for slow ones."""
    plain, a = O.rope_table(50, 32)
    z = plain[:, :16] + 1j * plain[:, 16:]
    assert np.allclose(z[1:], z[:-1] * z[1], atol=1e-14) and np.allclose(a[1], 10000.0 ** (-np.arange(16) / 16.0))
    _, b = O.rope_table(50, 32, factor=8.0, original=512.0, low=1.0, high=32.0)
    turns = 512.0 * a[1] / (2 * np.pi)
    assert np.allclose(b[1][turns > 32], a[1][turns > 32]) and np.allclose(b[1][turns < 1], a[1][turns < 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all((b[1][mid] < a[1][mid]) & (b[1][mid] > a[1][mid] / 8))
    _, c = O.rope_table(50, 32, factor=8.0)
    assert np.allclose(c, a / 8)
