"""Host-side refusals of the attention sublayer's entry points (no GPU): every
call here is refused before any launch, or launches nothing."""

import pytest
import torch

from mhc_pre_gb300 import binding as B
from mhc_pre_gb300 import build as mbuild

A = 0x7F0000000000          # never dereferenced, 16-byte aligned
OK, INV, UNS, MIS = B.MHC_OK, B.MHC_ERR_INVALID_ARG, B.MHC_ERR_UNSUPPORTED, B.MHC_ERR_MISALIGNED


@pytest.fixture(scope="module")
def L():
    mbuild.build()
    return B.lib()


def _fwd(L, **o):
    a = dict(dt=B.MHC_BF16, q=A, qs=512, k=A, ks=128, wq=A, wk=A, pos=A, cs=A, mp=10, T=4, Hq=8, Hk=2, Dh=64,
             rot=64, flags=0, eps=1e-6, qo=A, qos=512, ko=A, kos=128)
    a.update(o)
    return L.mhc_qk_norm_rope(*a.values(), None)


BAD_HEADS = [(dict(dt=3), INV), (dict(T=-1), INV), (dict(Hq=0), INV), (dict(Hk=0), INV), (dict(Hk=3), UNS),
             (dict(Dh=60), UNS), (dict(Dh=264), UNS), (dict(Hq=2048, Hk=2), UNS)]
BAD_ROPE = [(dict(rot=-16), INV), (dict(rot=80), INV), (dict(rot=24), UNS), (dict(flags=2), INV),
            (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(pos=None), INV), (dict(cs=None), INV),
            (dict(mp=0), INV), (dict(cs=A + 4), MIS), (dict(pos=A + 2), MIS)]


@pytest.mark.parametrize("bad,status", BAD_HEADS + BAD_ROPE + [
    (dict(q=None), INV), (dict(wk=None), INV), (dict(ko=None), INV), (dict(q=A + 8), MIS), (dict(ko=A + 4), MIS),
    (dict(qs=504), INV), (dict(qs=516), MIS), (dict(kos=120), INV), (dict(ks=132), MIS)])
def test_forward_refusals(L, bad, status):
    assert _fwd(L, **bad) == status


def test_forward_of_nothing(L):
    assert _fwd(L, T=0, q=None, k=None, pos=None) == OK


def _bwd(L, **o):
    a = dict(dt=B.MHC_F32, gq=A, gqs=512, gk=A, gks=128, q=A, qs=512, k=A, ks=128, wq=A, wk=A, pos=A, cs=A, mp=10,
             T=4, Hq=8, Hk=2, Dh=64, rot=64, flags=0, eps=1e-6, dq=A, dqs=512, dk=A, dks=128, dwq=A, dwk=A, ws=A,
             n=1 << 20)
    a.update(o)
    return L.mhc_qk_norm_rope_bwd(*a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_HEADS + BAD_ROPE + [
    (dict(gq=None), INV), (dict(dwk=None), INV), (dict(ws=None), INV), (dict(ws=A + 8), MIS), (dict(n=100), INV),
    (dict(dqs=500), INV), (dict(gks=130), MIS), (dict(T=0, dwq=None), INV)])
def test_backward_refusals(L, bad, status):
    assert _bwd(L, **bad) == status


def _append(L, **o):
    a = dict(dt=B.MHC_BF16, q=A, qs=512, k=A, ks=128, v=A, vs=128, wq=A, wk=A, pos=A, cs=A, mp=10, slots=A, T=4,
             Hq=8, Hk=2, Dh=64, rot=64, flags=0, eps=1e-6, qo=A, qos=512, kc=A, kp=2048, ksl=128, kh=64, vc=A,
             vp=2048, vsl=128, vh=64, pages=4, ps=16)
    a.update(o)
    return L.mhc_qk_norm_rope_append(*a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_HEADS + BAD_ROPE + [
    (dict(v=None), INV), (dict(slots=None), INV), (dict(slots=A + 4), MIS), (dict(vs=100), INV), (dict(ps=0), INV),
    (dict(pages=0), INV), (dict(kp=2052), MIS), (dict(vh=60), INV), (dict(vh=68), MIS), (dict(vc=A + 2), MIS)])
def test_append_refusals(L, bad, status):
    assert _append(L, **bad) == status


def _attn(L, **o):
    a = dict(dt=B.MHC_BF16, q=A, qs=512, kc=A, kp=2048, ksl=128, kh=64, vc=A, vp=2048, vsl=128, vh=64, pages=4,
             ps=16, pt=A, ts=4, cu=A, kv=A, T=4, B=2, Hq=8, Hk=2, Dh=64, mq=4, mkv=64, window=0, scale=0.125,
             cap=0.0, o=A, lse=A, ws=A, n=1 << 30)
    a.update(o)
    return L.mhc_paged_attn(*a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_HEADS + [
    (dict(q=None), INV), (dict(pt=None), INV), (dict(o=None), INV), (dict(ws=None), INV), (dict(n=100), INV),
    (dict(cu=None), INV), (dict(kv=None), INV), (dict(q=A + 8), MIS), (dict(pt=A + 2), MIS), (dict(lse=A + 2), MIS),
    (dict(cu=A + 1), MIS), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("inf")), INV),
    (dict(cap=-1.0), INV), (dict(cap=float("nan")), INV), (dict(window=-1), INV), (dict(ps=0), INV),
    (dict(B=-1), INV), (dict(mq=-1), INV), (dict(mkv=-1), INV), (dict(mkv=65), INV), (dict(mkv=1 << 31), UNS),
    (dict(mq=1 << 30), UNS), (dict(ksl=60), INV), (dict(vp=2052), MIS), (dict(qs=511), INV)])
def test_attention_refusals(L, bad, status):
    assert _attn(L, **bad) == status


def test_attention_of_nothing(L):
    assert _attn(L, T=0, q=None, o=None) == OK
    assert _attn(L, B=0, pt=None) == OK


def test_plan_refusals(L):
    def plan(**o):
        a = dict(dt=B.MHC_BF16, cu=A, kv=A, T=4, B=2, Hq=8, Hk=2, Dh=64, ps=16, mq=4, mkv=64, window=0, ws=A,
                 n=1 << 30)
        a.update(o)
        return L.mhc_paged_attn_plan(*a.values(), None)
    for bad, status in BAD_HEADS + [(dict(cu=None), INV), (dict(kv=None), INV), (dict(ws=None), INV),
                                    (dict(n=10), INV), (dict(ws=A + 4), MIS), (dict(kv=A + 2), MIS)]:
        assert plan(**bad) == status, bad
    assert plan(T=0, cu=None) == OK


def test_workspace_sizes(L):
    assert L.mhc_paged_attn_workspace_bytes(B.MHC_BF16, 0, 1, 8, 2, 64, 16, 1) == 0
    assert L.mhc_paged_attn_workspace_bytes(B.MHC_BF16, 4, 1, 7, 2, 64, 16, 1) == 0
    small = L.mhc_paged_attn_workspace_bytes(B.MHC_BF16, 4, 4, 8, 2, 64, 16, 1)
    large = L.mhc_paged_attn_workspace_bytes(B.MHC_BF16, 4096, 4, 8, 2, 64, 16, 4096)
    assert 0 < small < large < 1 << 28
    assert L.mhc_qk_norm_rope_bwd_workspace_bytes(0, 64) == 0


def test_binding_refuses_what_it_cannot_pass_on(L):
    q, k, w = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64), torch.ones(64)
    with pytest.raises(ValueError):
        B.mhc_qk_norm_rope(q, k, w, w)                       # host tensors
    with pytest.raises(ValueError):
        B.mhc_qk_norm_rope(q, torch.zeros(3, 2, 64), w, w)
    with pytest.raises(TypeError):
        B.mhc_qk_norm_rope(q, k, w.double(), w)
    with pytest.raises(ValueError):
        B.mhc_qk_norm_rope(q, k, w[:32], w)
    with pytest.raises(TypeError):
        B.mhc_paged_attn(q.half(), k[None], k[None], torch.zeros(1, 1, dtype=torch.int32), w, w)
