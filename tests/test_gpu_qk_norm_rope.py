"""GPU parity of the per-head normalisation with rotation (forward, backward,
cache append) against the float64 oracle.

Tolerances.  u = 2^-24.  The sum of dh squares and the products give each
result a relative error of at most (dh + 8) u before the last rounding, and a
rotated value is a sum of two products, so the error is held to (dh + 8) u times
the size of the head's largest normalised value; bf16 adds its half unit in the
last place, 2^-8 of the value.  A weight gradient sums N terms: sqrt(N) u times
8, times the root of the sum of the terms' squares, and the terms' own error.
"""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SHAPES = [  # T, Hq, Hk, dh, rot
    (1, 40, 8, 128, 128), (3, 5, 1, 128, 64), (130, 6, 2, 64, 64), (17, 4, 4, 8, 0), (9, 3, 3, 16, 16),
    (33, 12, 4, 96, 96), (5, 2, 1, 256, 256), (1025, 2, 1, 40, 32), (700, 16, 8, 64, 32),
]


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().cpu().double().numpy()


def _inputs(T, Hq, Hk, dh, rot, dtype, dev, seed=0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)            # noqa: E731
    qkv = n(T, (Hq + 2 * Hk) * dh).to(DT[dtype]).to(dev)
    q, k, v = (t.view(T, -1, dh) for t in qkv.split([Hq * dh, Hk * dh, Hk * dh], 1))
    ang = torch.rand(300, max(rot // 2, 1), generator=gen) * 6 - 3
    cs = torch.cat([ang.cos(), ang.sin()], 1).to(dev) if rot else None
    pos = torch.randint(0, 300, (T,), generator=gen, dtype=torch.int32).to(dev)
    w = [(1 + 0.3 * n(dh)).to(dev) for _ in range(2)]
    g = [n(T, h, dh).to(DT[dtype]).to(dev) for h in (Hq, Hk)]
    return q, k, v, w, pos, cs, g


def _R(pos, cs, rot, dh, adjacent):
    cs = np.zeros((300, 0)) if cs is None else f64(cs)
    return A.rotation(cs, pos.cpu().numpy(), rot, dh, adjacent)


def _close(got, ref, size, dtype, dh):
    tol = (dh + 8) * U * size + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0.0)
    bad = np.abs(f64(got) - ref) - tol
    assert np.all(np.isfinite(f64(got))) and bad.max() <= 0, f"over by {bad.max()}"


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,dh,rot", SHAPES)
def test_forward_and_append(T, Hq, Hk, dh, rot, dtype, adjacent):
    dev = _dev()
    q, k, v, w, pos, cs, _ = _inputs(T, Hq, Hk, dh, rot, dtype, dev)
    kw = dict(positions=pos, cos_sin=cs, eps=1e-5, interleaved=adjacent)
    r = B.mhc_qk_norm_rope(q, k, *w, **kw)
    R = _R(pos, cs, rot, dh, adjacent)
    for got, x, wt in ((r.q, q, w[0]), (r.k, k, w[1])):
        ref = A.norm_rope(f64(x), f64(wt), R, 1e-5)
        z = np.abs(A.norm_rope(f64(x), f64(wt), R * 0 + np.eye(dh), 1e-5)).max(-1, keepdims=True)
        _close(got, ref, 2 * z, dtype, dh)
    # the same values in the cache, both memory orders, other slots untouched
    ps, pages = 7, -(-T // 7) + 2
    slots = torch.randperm(ps * pages, generator=torch.Generator().manual_seed(1))[:T].to(dev)
    if T > 2:
        slots[1] = -1
    for order in ("place", "head"):
        shape = (pages, ps, Hk, dh) if order == "place" else (pages, Hk, ps, dh)
        caches = [torch.full(shape, 7.0, dtype=q.dtype, device=dev) for _ in range(2)]
        views = [c if order == "place" else c.transpose(1, 2) for c in caches]
        qa = B.mhc_qk_norm_rope_append(q, k, v, *w, *views, slots, **kw)
        assert torch.equal(qa, r.q)
        for c, src in zip(views, (r.k, v)):
            want = torch.full((pages, ps, Hk, dh), 7.0, dtype=q.dtype, device=dev)
            keep = slots >= 0
            want[slots[keep] // ps, slots[keep] % ps] = src[keep]
            assert torch.equal(c, want)
    assert B.get_last_device_error() == B.MHC_OK


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,dh,rot", SHAPES)
def test_backward(T, Hq, Hk, dh, rot, dtype, adjacent):
    dev = _dev()
    q, k, _, w, pos, cs, g = _inputs(T, Hq, Hk, dh, rot, dtype, dev, seed=1)
    kw = dict(positions=pos, cos_sin=cs, eps=1e-5, interleaved=adjacent)
    r = B.mhc_qk_norm_rope_bwd(*g, q, k, *w, **kw)
    R = _R(pos, cs, rot, dh, adjacent)
    for dx, dw, gg, x, wt in ((r.dq, r.dw_q, g[0], q, w[0]), (r.dk, r.dw_k, g[1], k, w[1])):
        ref, ref_w = A.norm_rope_bwd(f64(gg), f64(x), f64(wt), R, 1e-5)
        X, W = f64(x), f64(wt)
        rr = 1 / np.sqrt((X ** 2).mean(-1, keepdims=True) + 1e-5)
        h = np.einsum("tji,thj->thi", R, f64(gg))
        # r (u - x m) with m a mean of dh products: its error goes with sum |u x|
        size = rr * (np.abs(f64(gg)).max(-1, keepdims=True) * 2 * np.abs(W).max()
                     + np.abs(X) * rr ** 2 * (np.abs(h * W * X)).mean(-1, keepdims=True))
        _close(dx, ref, 2 * size, dtype, dh)
        terms = h * X * rr
        n = terms.shape[0] * terms.shape[1]
        tol = 8 * np.sqrt(n) * U * np.sqrt((terms ** 2).sum((0, 1))) + 2 * (dh + 8) * U * np.abs(terms).sum((0, 1)) + 1e-30
        assert np.all(np.abs(f64(dw) - ref_w) <= tol)
    # the same bits again, and into parts of a packed gradient
    packed = torch.zeros(T, (Hq + 2 * Hk) * dh, dtype=q.dtype, device=dev)
    dq, dk, rest = (t.view(T, -1, dh) for t in packed.split([Hq * dh, Hk * dh, Hk * dh], 1))
    r2 = B.mhc_qk_norm_rope_bwd(*g, q, k, *w, dq=dq, dk=dk, **kw)
    assert all(torch.equal(a, b) for a, b in zip(r, r2)) and not rest.any()
    assert B.get_last_device_error() == B.MHC_OK


def test_backward_against_differences_of_the_forward():
    """<g, out> of the float32 forward moved by +-h along random directions.  The
    forward's rounding, about 2^-22 of sum |g out| over 2 h, and the third
    derivative's h^2 bound what can be asked: 2e-3 of the derivative's scale."""
    dev = _dev()
    T, Hq, Hk, dh, rot = 6, 3, 1, 32, 32
    q, k, _, w, pos, cs, g = _inputs(T, Hq, Hk, dh, rot, "f32", dev, seed=3)
    kw = dict(positions=pos, cos_sin=cs)
    r = B.mhc_qk_norm_rope_bwd(*g, q, k, *w, **kw)

    def f(q, k, wq, wk):
        o = B.mhc_qk_norm_rope(q, k, wq, wk, **kw)
        return float((g[0].double() * o.q.double()).sum() + (g[1].double() * o.k.double()).sum())

    base, h = [q.contiguous(), k.contiguous(), *w], 1e-2
    for i, grad in enumerate(r):
        d = torch.randn(base[i].shape, generator=torch.Generator().manual_seed(i)).to(dev)
        up, dn = list(base), list(base)
        up[i], dn[i] = base[i] + h * d, base[i] - h * d
        slope = (f(*up) - f(*dn)) / (2 * h)
        scale = float(grad.double().norm() * d.double().norm()) / np.sqrt(d.numel())
        assert abs(slope - float((grad.double() * d.double()).sum())) <= 2e-3 * max(scale, 1.0)


def test_values_outside_float32_comfort():
    """Zero heads (eps decides), tiny and large values, no NaN from any of them."""
    dev = _dev()
    q = torch.zeros(4, 2, 64, device=dev)
    q[1] = 1e-18
    q[2] = 1e15
    k = q[:, :1].clone()
    w = torch.ones(64, device=dev)
    r = B.mhc_qk_norm_rope(q, k, w, w, eps=1e-6)
    ref = A.norm_rope(f64(q), np.ones(64), np.eye(64)[None].repeat(4, 0), 1e-6)
    assert np.allclose(f64(r.q), ref, rtol=1e-5, atol=0)


def test_numbers_outside_their_tensors_are_reported_and_skipped():
    dev = _dev()
    T, Hq, Hk, dh, rot = 6, 2, 1, 64, 64
    q, k, v, w, pos, cs, g = _inputs(T, Hq, Hk, dh, rot, "bf16", dev)
    good = B.mhc_qk_norm_rope(q, k, *w, positions=pos, cos_sin=cs)
    bad = pos.clone()
    bad[2], bad[4] = 300, -1
    r = B.mhc_qk_norm_rope(q, k, *w, positions=bad, cos_sin=cs)
    assert B.get_last_device_error() == B.MHC_ERR_RANGE
    assert B.get_last_device_error() == B.MHC_OK
    keep = torch.tensor([0, 1, 3, 5], device=dev)
    assert torch.equal(r.q[keep], good.q[keep]) and not r.q[[2, 4]].any() and not r.k[[2, 4]].any()
    rb = B.mhc_qk_norm_rope_bwd(*g, q, k, *w, positions=bad, cos_sin=cs)
    assert B.get_last_device_error() == B.MHC_ERR_RANGE and not rb.dq[[2, 4]].any()
    caches = [torch.zeros(3, 4, Hk, dh, dtype=q.dtype, device=dev) for _ in range(2)]
    slots = torch.tensor([0, 12, 5, -2, 2, 11], device=dev)
    B.mhc_qk_norm_rope_append(q, k, v, *w, *caches, slots, positions=pos, cos_sin=cs)
    assert B.get_last_device_error() == B.MHC_ERR_RANGE
    flat = caches[1].flatten(0, 1)
    assert torch.equal(flat[[0, 5, 2, 11]], v[[0, 2, 4, 5]]) and int(flat.abs().sum((1, 2)).ne(0).sum()) == 4


def test_in_place_and_on_another_stream():
    dev = _dev()
    q, k, v, w, pos, cs, _ = _inputs(64, 8, 2, 64, 64, "bf16", dev)
    want = B.mhc_qk_norm_rope(q, k, *w, positions=pos, cos_sin=cs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = B.mhc_qk_norm_rope(q, k, *w, positions=pos, cos_sin=cs)
    s.synchronize()
    assert torch.equal(got.q, want.q) and torch.equal(got.k, want.k)
    L = B.lib()
    st = L.mhc_qk_norm_rope(B.MHC_BF16, q.data_ptr(), q.stride(0), k.data_ptr(), k.stride(0), w[0].data_ptr(),
                            w[1].data_ptr(), pos.data_ptr(), cs.data_ptr(), 300, 64, 8, 2, 64, 64, 0, 1e-6,
                            q.data_ptr(), q.stride(0), k.data_ptr(), k.stride(0),
                            torch.cuda.current_stream().cuda_stream)
    assert st == B.MHC_OK
    assert torch.equal(q, want.q) and torch.equal(k, want.k)


def test_empty_batch():
    dev = _dev()
    q, k = torch.zeros(0, 4, 64, device=dev), torch.zeros(0, 2, 64, device=dev)
    w = torch.ones(64, device=dev)
    r = B.mhc_qk_norm_rope(q, k, w, w)
    assert r.q.shape == q.shape
    b = B.mhc_qk_norm_rope_bwd(q, k, q, k, w, w)
    assert not b.dw_q.any() and not b.dw_k.any() and b.dw_q.shape == (64,)
