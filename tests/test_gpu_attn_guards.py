"""The attention sublayer's kernels write nothing outside their outputs and
workspaces, and its bounded waits report when they run out (GPU)."""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import attn_oracle as A
from tests.test_gpu_guard_bands import GuardedAllocator
from tests.test_gpu_paged_attn import Case
from tests.test_gpu_qk_norm_rope import _inputs

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,dh,rot", [(1, 40, 8, 128, 128), (131, 6, 2, 96, 32), (1700, 12, 4, 64, 64),
                                            (6500, 2, 1, 64, 64)])
def test_norm_and_rotation_stay_inside(T, Hq, Hk, dh, rot, dtype, monkeypatch):
    q, k, v, w, pos, cs, g = _inputs(T, Hq, Hk, dh, rot, dtype, _dev())
    kw = dict(positions=pos, cos_sin=cs)

    def run():
        pages = -(-T // 16) + 1
        slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(0))[:T].to(q.device)
        caches = [B._empty((pages, 16, Hk, dh), dtype=q.dtype, device=q.device).zero_() for _ in range(2)]
        a = B.mhc_qk_norm_rope(q, k, *w, **kw)
        b = B.mhc_qk_norm_rope_bwd(*g, q, k, *w, **kw)
        c = B.mhc_qk_norm_rope_append(q, k, v, *w, *caches, slots, **kw)
        return [*a, *b, c, *caches]

    plain = run()
    guarded = GuardedAllocator()
    monkeypatch.setattr(B, "_empty", guarded)
    got = run()
    monkeypatch.undo()
    guarded.check(f"T={T} {dtype}")
    assert all(torch.equal(a, b) for a, b in zip(plain, got))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hk,dh,page", [
    ([(1, 5000), (3, 17)], 10, 2, 128, 64), ([(300, 700), (1, 3), (0, 0), (129, 129)], 5, 1, 80, 16),
    ([(33, 400)], 4, 4, 64, 3)])
def test_attention_stays_inside(lens, Hq, Hk, dh, page, dtype, monkeypatch):
    c = Case(lens, Hq, Hk, dh, page, dtype)
    plain = c.run()
    guarded = GuardedAllocator()
    monkeypatch.setattr(B, "_empty", guarded)
    got = c.run()
    monkeypatch.undo()
    guarded.check(f"{lens} {dtype}")
    assert len(guarded.bufs) == 3
    assert torch.equal(plain.o, got.o) and torch.equal(plain.lse, got.lse)


@pytest.mark.parametrize("T,Hq,Hk,dh,rot,dtype,adjacent", [
    (1700, 40, 8, 128, 128, "bf16", False),    # four warps a token
    (1650, 10, 2, 128, 64, "f32", True),
    (400, 64, 8, 256, 256, "f32", False),      # stages of 72 KB, one block an SM
    (6200, 2, 1, 64, 64, "bf16", True),        # two warps a token
    (6300, 4, 4, 40, 32, "f32", False),
    (24500, 2, 1, 64, 32, "bf16", False),      # a warp a token
])
def test_many_tokens(T, Hq, Hk, dh, rot, dtype, adjacent):
    """Batches that the staged kernels take: every 37th token and the last ones
    against the oracle (the weight gradients whole), tolerances as for few tokens."""
    from tests.test_gpu_qk_norm_rope import U, _close, f64
    q, k, v, w, pos, cs, g = _inputs(T, Hq, Hk, dh, rot, dtype, _dev(), seed=5)
    kw = dict(positions=pos, cos_sin=cs, eps=1e-5, interleaved=adjacent)
    r = B.mhc_qk_norm_rope(q, k, *w, **kw)
    b = B.mhc_qk_norm_rope_bwd(*g, q, k, *w, **kw)
    pages = -(-T // 16) + 1
    slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(0))[:T].to(q.device)
    slots[7] = -1
    caches = [torch.zeros(pages, 16, Hk, dh, dtype=q.dtype, device=q.device) for _ in range(2)]
    qa = B.mhc_qk_norm_rope_append(q, k, v, *w, *caches, slots, **kw)
    keep = slots >= 0
    assert torch.equal(qa, r.q)
    for c, src in zip(caches, (r.k, v)):
        want = torch.zeros_like(c).flatten(0, 1)
        want[slots[keep]] = src[keep]
        assert torch.equal(c.flatten(0, 1), want)
    at = np.unique(np.r_[np.arange(0, T, 37), np.arange(T - 3, T)])
    R = A.rotation(f64(cs), pos.cpu().numpy()[at], rot, dh, adjacent)
    flat = R * 0 + np.eye(dh)
    for got, x, wt in ((r.q, q, w[0]), (r.k, k, w[1])):
        z = np.abs(A.norm_rope(f64(x)[at], f64(wt), flat, 1e-5)).max(-1, keepdims=True)
        _close(got[at], A.norm_rope(f64(x)[at], f64(wt), R, 1e-5), 2 * z, dtype, dh)
    for dx, gg, x, wt in ((b.dq, g[0], q, w[0]), (b.dk, g[1], k, w[1])):
        X, G, W = f64(x)[at], f64(gg)[at], f64(wt)
        ref, _ = A.norm_rope_bwd(G, X, W, R, 1e-5)
        rr = 1 / np.sqrt((X ** 2).mean(-1, keepdims=True) + 1e-5)
        h = np.einsum("tji,thj->thi", R, G)
        size = rr * (np.abs(G).max(-1, keepdims=True) * 2 * np.abs(W).max()
                     + np.abs(X) * rr ** 2 * np.abs(h * W * X).mean(-1, keepdims=True))
        _close(dx[at], ref, 2 * size, dtype, dh)
    # the weight gradients: all tokens, a part of the heads' rotation matrices at a time
    for dw, gg, x in ((b.dw_q, g[0], q), (b.dw_k, g[1], k)):
        total, square, size = np.zeros(dh), np.zeros(dh), np.zeros(dh)
        for t0 in range(0, T, 500):
            s = slice(t0, t0 + 500)
            Rs = A.rotation(f64(cs), pos.cpu().numpy()[s], rot, dh, adjacent)
            X = f64(x)[s]
            rr = 1 / np.sqrt((X ** 2).mean(-1, keepdims=True) + 1e-5)
            terms = np.einsum("tji,thj->thi", Rs, f64(gg)[s]) * X * rr
            total += terms.sum((0, 1))
            square += (terms ** 2).sum((0, 1))
            size += np.abs(terms).sum((0, 1))
        n = T * x.shape[1]
        assert np.all(np.abs(f64(dw) - total) <= 8 * np.sqrt(n) * U * np.sqrt(square) + 2 * (dh + 8) * U * size)
    assert B.get_last_device_error() == B.MHC_OK


def test_numbers_outside_their_tensors_among_many_tokens():
    q, k, v, w, pos, cs, g = _inputs(1700, 40, 8, 128, 128, "bf16", _dev())
    good = B.mhc_qk_norm_rope(q, k, *w, positions=pos, cos_sin=cs)
    bad = pos.clone()
    bad[3], bad[1600] = 300, -7
    r = B.mhc_qk_norm_rope(q, k, *w, positions=bad, cos_sin=cs)
    assert B.get_last_device_error() == B.MHC_ERR_RANGE
    rows = torch.tensor([3, 1600], device=q.device)
    assert not r.q[rows].any() and not r.k[rows].any()
    keep = torch.ones(1700, dtype=torch.bool, device=q.device)
    keep[rows] = False
    assert torch.equal(r.q[keep], good.q[keep]) and torch.equal(r.k[keep], good.k[keep])
    b = B.mhc_qk_norm_rope_bwd(*g, q, k, *w, positions=bad, cos_sin=cs)
    assert B.get_last_device_error() == B.MHC_ERR_RANGE
    assert not b.dq[rows].any() and not b.dk[rows].any() and bool(b.dw_q.isfinite().all())


def test_forced_timeout_of_the_attention_is_reported():
    c = Case([(1, 300), (20, 40)], 4, 2, 64, 64, "bf16")
    want = c.run()
    assert B.get_last_device_error() == B.MHC_OK
    L = B.lib()
    try:
        assert L.mhc_test_force_timeout(1) == B.MHC_OK
        c.run()
        assert B.get_last_device_error() == B.MHC_ERR_TIMEOUT
    finally:
        assert L.mhc_test_force_timeout(0) == B.MHC_OK
    got = c.run()
    assert B.get_last_device_error() == B.MHC_OK
    assert torch.equal(got.o, want.o)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_a_plan_of_other_sizes_is_reported(dtype):
    """The C entry point, for which the workspace's plan is the only witness."""
    c = Case([(8, 300), (2, 40)], 4, 2, 64, 64, dtype)
    want = c.run(max_q=8, max_kv=300)
    L, code = B.lib(), B.MHC_BF16 if dtype == "bf16" else B.MHC_F32
    s = torch.cuda.current_stream().cuda_stream
    sizes = (10, 2, 4, 2, 64)                         # T, B, Hq, Hk, Dh
    n = L.mhc_paged_attn_workspace_bytes(code, *sizes, 64, 8)
    ws = torch.empty(n, dtype=torch.uint8, device=c.q.device)
    o = torch.full(c.q.shape, 7.0, dtype=c.q.dtype, device=c.q.device)

    def call(max_q, max_kv, window):
        assert L.mhc_paged_attn(code, c.q.data_ptr(), c.q.stride(0), c.k.data_ptr(), *c.k.stride()[:3],
                                c.v.data_ptr(), *c.v.stride()[:3], c.k.shape[0], 64, c.table.data_ptr(),
                                c.table.stride(0), None, None, *sizes, max_q, max_kv, window, 0.125, 0.0,
                                o.data_ptr(), None, ws.data_ptr(), n, s) == B.MHC_OK
        return B.get_last_device_error()

    assert L.mhc_paged_attn_plan(code, c.cu.data_ptr(), c.kv.data_ptr(), *sizes, 64, 8, 300, 0, ws.data_ptr(), n,
                                 s) == B.MHC_OK
    assert B.get_last_device_error() == B.MHC_OK
    for other in ((1, 300, 0), (7, 300, 0), (8, 64, 0), (8, 300, 100)):
        assert call(*other) == B.MHC_ERR_RANGE, other
        assert bool((o == 7.0).all()), other
    assert call(8, 300, 0) == B.MHC_OK
    assert torch.equal(o, want.o)
