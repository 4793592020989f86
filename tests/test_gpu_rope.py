"""GPU parity of the rotation without normalisation, and of its table, against
the float64 oracle.

Tolerances.  u = 2^-24.  A turned value is a product and a fused product: at most
2 u (|a c| + |b s|) of it, in bf16 its rounding 2^-8 |y| more.  A table's value:
its angle, at most an eighth of a turn after the quarter turns, is rounded to 24
bits (2 pi 2^-28 radians, 0.4 u), the sine or cosine of at most 0.71 is right to
a unit in the last place (u), the product with the amplitude to u, so 3 u of the
amplitude with what the fractions of a turn leave out; frequencies in double
move the angle by 2^-51 of it.
"""

import math
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import attn_oracle as A
from tests.test_gpu_guard_bands import GuardedAllocator

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().cpu().double().numpy()


def _inputs(T, Hq, Hk, dh, rot, dtype, seed=0, max_pos=300):
    dev, gen = _dev(), torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)            # noqa: E731
    packed = n(T, (Hq + 2 * Hk) * dh).to(DT[dtype]).to(dev)
    q, k, v = (t.view(T, -1, dh) for t in packed.split([Hq * dh, Hk * dh, Hk * dh], 1))
    pos = torch.randint(0, max_pos, (T,), generator=gen).to(torch.int32).to(dev)
    ang = n(max_pos, rot // 2) * 3
    return q, k, v, pos, (1.25 * torch.cat([ang.cos(), ang.sin()], 1)).float().to(dev)


def _check(got, x, R, dtype):
    """`got` is R x, at the module's tolerances."""
    x, got = f64(x), f64(got)
    ref = np.einsum("tij,thj->thi", R, x)
    tol = 2 * U * np.einsum("tij,thj->thi", np.abs(R), np.abs(x)) + (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0)
    assert np.all(np.abs(got - ref) <= tol)


SHAPES = [(1, 40, 8, 128, 128), (5, 4, 4, 64, 32), (131, 6, 2, 96, 48), (33, 3, 1, 256, 256), (64, 1, 1, 24, 16),
          (1700, 40, 8, 128, 64), (6500, 2, 1, 64, 64), (400, 64, 8, 256, 256), (24500, 2, 1, 64, 32),
          (5000, 40, 8, 128, 128), (5000, 12, 4, 96, 96), (4900, 6, 3, 96, 48), (5100, 2, 2, 256, 256),
          (9001, 3, 3, 24, 16), (5000, 33, 3, 40, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,dh,rot", SHAPES)
def test_forward_backward_append(T, Hq, Hk, dh, rot, adjacent, dtype):
    q, k, v, pos, cs = _inputs(T, Hq, Hk, dh, rot, dtype)
    kw = dict(positions=pos, cos_sin=cs, interleaved=adjacent)
    r, b = B.mhc_rope(q, k, **kw), B.mhc_rope_bwd(q, k, **kw)
    at = np.unique(np.r_[np.arange(0, T, max(1, T // 40)), np.arange(max(0, T - 3), T)])
    R = A.rotation(f64(cs), f64(pos).astype(int)[at], rot, dh, adjacent)
    _check(r.q[at], q[at], R, dtype)
    _check(r.k[at], k[at], R, dtype)
    _check(b.q[at], q[at], R.transpose(0, 2, 1), dtype)
    _check(b.k[at], k[at], R.transpose(0, 2, 1), dtype)
    pages = -(-T // 16) + 1
    slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(0))[:T].to(q.device)
    slots[T // 2] = -1
    caches = [torch.zeros(pages, 16, Hk, dh, dtype=q.dtype, device=q.device) for _ in range(2)]
    qa = B.mhc_rope_append(q, k, v, *caches, slots, **kw)
    assert torch.equal(qa, r.q)
    keep = slots >= 0
    for c, src in zip(caches, (r.k, v)):
        want = torch.zeros_like(c).flatten(0, 1)
        want[slots[keep]] = src[keep]
        assert torch.equal(c.flatten(0, 1), want)
    # caches with the heads outside
    outside = [torch.zeros(pages, Hk, 16, dh, dtype=q.dtype, device=q.device).transpose(1, 2) for _ in range(2)]
    B.mhc_rope_append(q, k, v, *outside, slots, **kw)
    assert all(torch.equal(a, b) for a, b in zip(outside, caches))
    assert B.get_last_device_error() == B.MHC_OK


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T", [3, 1700, 5000])
def test_the_backward_is_the_transpose(T, adjacent):
    """<g, R x> = <R^T g, x>, and its change with x: the operator is linear, so a
    difference of any step is the gradient.  Sums of N products of size 1.6 in
    float64 of float32 results: N^0.5 4 u 1.6 at most in the mean, 8 times that held."""
    q, k, v, pos, cs = _inputs(T, 6, 2, 64, 32, "f32", seed=1)
    g, h, *_ = _inputs(T, 6, 2, 64, 32, "f32", seed=2)
    kw = dict(positions=pos, cos_sin=cs, interleaved=adjacent)
    y0, y1, b = B.mhc_rope(q, k, **kw), B.mhc_rope(q + g, k + h, **kw), B.mhc_rope_bwd(g, h, **kw)
    left = (g.double() * y0.q.double()).sum() + (h.double() * y0.k.double()).sum()
    right = (b.q.double() * q.double()).sum() + (b.k.double() * k.double()).sum()
    tol = 8 * 4 * 1.6 * U * (T * 8 * 64) ** 0.5
    assert abs(float(left - right)) <= tol
    rise = (g.double() * (y1.q.double() - y0.q.double())).sum() + (h.double() * (y1.k.double() - y0.k.double())).sum()
    along = (b.q.double() * g.double()).sum() + (b.k.double() * h.double()).sum()
    assert abs(float(rise - along)) <= 4 * tol       # differences of values twice as large, and q + g is rounded


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_do_not_turn_are_copied(dtype):
    """Whatever they are: infinities and NaN among them reach nothing else."""
    for T in (4, 6500):
        q, k, v, pos, cs = _inputs(T, 2, 1, 64, 32, dtype)
        q[0, 0, 40], q[1, 1, 63], k[2, 0, 32], q[3, 0, 50] = float("inf"), float("nan"), -float("inf"), -0.0
        for adjacent in (False, True):
            r = B.mhc_rope(q, k, pos, cs, interleaved=adjacent)
            assert torch.equal(r.q[..., 32:].contiguous().view(torch.uint8), q[..., 32:].contiguous().view(torch.uint8))
            assert torch.equal(r.k[..., 32:].contiguous().view(torch.uint8), k[..., 32:].contiguous().view(torch.uint8))
            assert bool(r.q[..., :32].isfinite().all()) and bool(r.k[..., :32].isfinite().all())


@pytest.mark.parametrize("T", [7, 6500])
def test_gradients_into_a_packed_tensor_and_in_place(T):
    q, k, v, pos, cs = _inputs(T, 6, 2, 64, 64, "bf16")
    kw = dict(positions=pos, cos_sin=cs)
    want = B.mhc_rope_bwd(q, k, **kw)
    packed = torch.full((T, 10 * 64), 7.0, dtype=torch.bfloat16, device=q.device)
    dq, dk, dv = (t.view(T, -1, 64) for t in packed.split([6 * 64, 2 * 64, 2 * 64], 1))
    r = B.mhc_rope_bwd(q, k, **kw, dq=dq, dk=dk)
    assert r.q is dq and torch.equal(dq, want.q) and torch.equal(dk, want.k) and bool((dv == 7.0).all())
    B.mhc_rope_bwd(q, k, **kw, dq=q, dk=k)
    assert torch.equal(q, want.q) and torch.equal(k, want.k)


@pytest.mark.parametrize("T", [9, 6500])
def test_numbers_outside_their_tensors(T):
    q, k, v, pos, cs = _inputs(T, 2, 1, 64, 64, "bf16")
    good = B.mhc_rope(q, k, pos, cs)
    bad = pos.clone()
    bad[3], bad[T - 1] = 300, -7
    keep = torch.ones(T, dtype=torch.bool, device=q.device)
    keep[torch.tensor([3, T - 1], device=q.device)] = False
    for call in (B.mhc_rope, B.mhc_rope_bwd):
        r = call(q, k, bad, cs)
        assert B.get_last_device_error() == B.MHC_ERR_RANGE
        assert not r.q[~keep].any() and not r.k[~keep].any()
    assert torch.equal(B.mhc_rope(q, k, bad, cs).q[keep], good.q[keep])
    B.get_last_device_error()
    slots = torch.arange(T, device=q.device)
    slots[1], slots[2] = -2, 10 ** 12
    pages = -(-T // 16)
    caches = [torch.full((pages, 16, 1, 64), 5.0, dtype=q.dtype, device=q.device) for _ in range(2)]
    B.mhc_rope_append(q, k, v, *caches, slots, bad, cs)
    assert B.get_last_device_error() == B.MHC_ERR_RANGE
    keep[1] = keep[2] = False
    rows = caches[0].flatten(0, 1)[:T]
    assert torch.equal(rows[keep], good.k[keep]) and bool((rows[~keep] == 5.0).all())
    assert bool((caches[1].flatten(0, 1)[:T][~keep] == 5.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hq,Hk,dh,rot", [(1, 40, 8, 128, 128), (131, 6, 2, 96, 32), (6500, 2, 1, 64, 64)])
def test_nothing_is_written_outside(T, Hq, Hk, dh, rot, dtype, monkeypatch):
    q, k, v, pos, cs = _inputs(T, Hq, Hk, dh, rot, dtype)

    def run():
        return [*B.mhc_rope(q, k, pos, cs), *B.mhc_rope_bwd(q, k, pos, cs), B.mhc_rope_table(T, rot, factor=4.0)]

    plain = run()
    guarded = GuardedAllocator()
    monkeypatch.setattr(B, "_empty", guarded)
    got = run()
    monkeypatch.undo()
    guarded.check(f"T={T} {dtype}")
    assert all(torch.equal(a, b) for a, b in zip(plain, got))


@pytest.mark.parametrize("T,Hq,Hk", [(420000, 40, 8), (66000, 256, 8)])
def test_tensors_past_32_bits(T, Hq, Hk):
    """More than 2^31 values: the last tokens as in a call of their own."""
    q, k, v, pos, cs = _inputs(5, Hq, Hk, 128, 64, "bf16")
    Q, K = (torch.zeros(T, h, 128, dtype=torch.bfloat16, device=q.device) for h in (Hq, Hk))
    P = torch.zeros(T, dtype=torch.int32, device=q.device)
    Q[-5:], K[-5:], P[-5:] = q, k, pos
    for f in (B.mhc_rope, B.mhc_rope_bwd):
        r, want = f(Q, K, P, cs), f(q, k, pos, cs)
        assert torch.equal(r.q[-5:], want.q) and torch.equal(r.k[-5:], want.k)
        assert not bool(r.q[:1000].any()) and not bool(r.q[T // 2:T // 2 + 1000].any())
    cache = torch.zeros(2, 16, Hk, 128, dtype=torch.bfloat16, device=q.device)
    slots = torch.full((T,), -1, dtype=torch.int64, device=q.device)
    slots[-5:] = torch.arange(5)
    got = B.mhc_rope_append(Q, K, K, cache, cache.clone(), slots, P, cs)
    want = B.mhc_rope(q, k, pos, cs)
    assert torch.equal(got[-5:], want.q) and torch.equal(cache[0, :5], want.k)
    assert B.get_last_device_error() == B.MHC_OK


def test_another_stream_and_a_graph():
    q, k, v, pos, cs = _inputs(50, 6, 2, 64, 64, "bf16")
    want = B.mhc_rope(q, k, pos, cs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = B.mhc_rope(q, k, pos, cs)
    s.synchronize()
    assert torch.equal(got.q, want.q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tab = B.mhc_rope_table(300, 64)
        r = B.mhc_rope(q, k, pos, tab)
        b = B.mhc_rope_bwd(r.q, r.k, pos, tab)
    q.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.q, B.mhc_rope(q, k, pos, tab).q) and torch.equal(b.k, B.mhc_rope_bwd(r.q, r.k, pos, tab).k)


TABLES = [dict(), dict(factor=4.0), dict(factor=16.0, original=8192, amplitude=1.25), dict(base=500000.0, factor=8.0,
          original=8192, low=1.0, high=4.0), dict(factor=0.25), dict(base=1.0, factor=3.0, amplitude=-2.0)]


@pytest.mark.parametrize("rot", [16, 64, 96, 128, 256])
@pytest.mark.parametrize("scaling", TABLES)
def test_table(rot, scaling):
    _dev()
    for n in (1, 17, 4000):
        got = f64(B.mhc_rope_table(n, rot, **scaling))
        ref, angles = A.rope_table(n, rot, **scaling)
        a = abs(scaling.get("amplitude", 1.0))
        assert np.all(np.abs(got - ref) <= a * (3 * U + np.tile(np.abs(angles), 2) * 2.0 ** -51))


def test_far_positions():
    """Where an angle in float32 has lost its fraction."""
    _dev()
    n = (1 << 24) + 3000
    got = B.mhc_rope_table(n, 16, base=3.0, factor=1.5)
    for first in (0, 1 << 20, (1 << 24) - 5, n - 100):
        ref, angles = A.rope_table(100, 16, base=3.0, factor=1.5, first=first)
        assert np.all(np.abs(f64(got[first:first + 100]) - ref) <= 3 * U + np.tile(angles, 2) * 2.0 ** -51)


PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def _table_row(p, rot, base, factor=1.0, original=0.0, low=1.0, high=32.0):
    """Row p in 60 digits."""
    with localcontext() as digits:
        digits.prec = 60
        c, s = [], []
        for j in range(rot // 2):
            e = Decimal(base) ** (Decimal(-2 * j) / rot)
            g = min(Decimal(1), max(Decimal(0), (Decimal(original) * e / (2 * PI) - Decimal(low)) /
                                    (Decimal(high) - Decimal(low))))
            a = float(p * e * (g + (1 - g) / Decimal(factor)) % (2 * PI))
            c.append(math.cos(a))
            s.append(math.sin(a))
    return np.array(c + s)


@pytest.mark.parametrize("rot,scaling", [
    (16, dict(base=1e6, factor=16.0, original=8192.0)), (16, dict(base=1e4)), (96, dict(base=1e6, factor=16.0, original=8192.0)),
    (32, dict(base=5e5, factor=8.0, original=8192.0, low=1.0, high=4.0)), (16, dict(base=1e9, factor=0.25)),
    (64, dict(base=1e4, factor=40.0, original=4096.0, low=3.0, high=3.5))])
def test_slow_pairs_at_far_positions(rot, scaling):
    """The angles' bound as include/mhc.h states it, and 2^-50 for the rows themselves,
    whose angles below 8 are rounded to double."""
    _dev()
    n = (1 << 24) * 16 // rot + 77
    got = B.mhc_rope_table(n, rot, **scaling)
    low, high = scaling.get("low", 1.0), scaling.get("high", 32.0)
    per = max(1.0, 1.0 / scaling.get("factor", 1.0)) * (2.0 ** -49 + 2.0 ** -50 * high / (high - low))
    for p in (1, 4097, 131071, n // 3, n // 2 + 1, n - 2, n - 1):
        assert np.all(np.abs(f64(got[p]) - _table_row(p, rot, **scaling)) <= 3 * U + p * per + 2.0 ** -50)


def test_scaled_table_serves_the_normalising_rotation():
    q, k, v, pos, _ = _inputs(20, 4, 2, 64, 64, "f32")
    cs = B.mhc_rope_table(300, 64, factor=4.0, original=128.0)
    w = torch.ones(64, device=q.device)
    r, s = B.mhc_qk_norm_rope(q, k, w, w, pos, cs, eps=0.0), B.mhc_rope(q, k, pos, cs)
    scale = (q.double() ** 2).mean(-1, keepdim=True) ** -0.5
    want = s.q.double() * scale
    # two roundings of the same sums, and the inverse root's
    assert bool(((r.q.double() - want).abs() <= 16 * U * (scale * q.double().norm(dim=-1, keepdim=True))).all())


def test_empty_calls():
    dev = _dev()
    q, k = torch.zeros(0, 4, 64, device=dev), torch.zeros(0, 2, 64, device=dev)
    pos, cs = torch.zeros(0, dtype=torch.int32, device=dev), torch.zeros(8, 64, device=dev)
    assert B.mhc_rope(q, k, pos, cs).q.shape == (0, 4, 64)
    assert B.mhc_rope_table(0, 64).shape == (0, 64)
