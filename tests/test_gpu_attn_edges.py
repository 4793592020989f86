"""Attention over a paged cache where its numbers are at their limits, against
the float64 oracle: caps far above the scores, page numbers outside the cache.

Tolerances.  u = 2^-24; a score's products and sums are held to 32 sqrt(dh) u
times the row's largest scale * sum |q k| ("size").  The cap: a relative 2^-18
of the score, whatever the cap is (where the tanh is formed from a quotient, two
approximations and five roundings come to 2^-20.5 of the cap, of which the
score is then at least 0.3).  The rest is as in test_gpu_paged_attn.py: 2 e sum
p |v| of an error e of the scores, 8 sqrt(n) u of the sums, 2^-20 of the
exponentials, and for bf16 2^-8 of sum p |v| and of |o|.
"""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import attn_oracle as A
from tests.test_gpu_paged_attn import LENS, U, Case, f64

pytestmark = pytest.mark.gpu


def check(c, r, softcap):
    q, at = f64(c.q), 0
    dh = q.shape[-1]
    o, lse = f64(r.o), f64(r.lse)
    for b, (n, m) in enumerate(c.lens):
        assert np.all(np.isfinite(o[at:at + n]))
        ro, rl, pabs, size = A.attention(q[at:at + n], f64(c.kd[b]), f64(c.vd[b]), dh ** -0.5, c.window, softcap)
        e = (32 * np.sqrt(dh) * U + 2.0 ** -18) * size
        tol = (2 * e + 8 * np.sqrt(max(m, 1)) * U + 2.0 ** -20)[..., None] * pabs
        if c.dtype == "bf16":
            tol = tol + 2.0 ** -8 * (pabs + np.abs(ro))
        assert np.all(np.abs(o[at:at + n] - ro) <= tol), b
        empty = ~np.isfinite(rl)
        assert np.array_equal(empty, lse[at:at + n] == -np.inf)
        ref = np.where(empty, 0, rl)
        d = np.abs(np.where(empty, 0, lse[at:at + n]) - ref)
        assert np.all(d <= e + 8 * np.sqrt(max(m, 1)) * U + 2.0 ** -20 * (1 + np.abs(ref))), (b, d.max())
        at += n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [60.0, 400.0, 1e3, 1e4, 1e5, 1e6, 1e7, 1e30])
@pytest.mark.parametrize("std", [1.5, 4.0])
def test_a_caps_error_does_not_grow_with_it(std, softcap, dtype):
    for dh, window in ((128, 0), (64, 60)):
        c = Case(LENS["chunks"], 10, 2, dh, 64, dtype, std=std, window=window)
        check(c, c.run(softcap=softcap), softcap)
        assert B.get_last_device_error() == B.MHC_OK


@pytest.mark.parametrize("softcap", [60.0, 1e5])
def test_scores_on_both_sides_of_a_high_cap(softcap):
    """Keys whose scores lie far below, near and above the cap, in every 32 of them."""
    c = Case([(130, 300), (1, 200)], 4, 2, 64, 64, "bf16")
    for b, (_, m) in enumerate(c.lens):
        grow = (softcap ** (torch.arange(m) % 7 / 5.0 - 0.2))[:, None, None]
        c.kd[b] = (c.kd[b].float() * grow).bfloat16()
        for j in range(-(-m // 64)):
            n = min(64, m - j * 64)
            c.k[int(c.table[b, j]), :n] = c.kd[b][j * 64:j * 64 + n].to(c.k.device)
    check(c, c.run(softcap=softcap), softcap)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [51.9, 51.97, 52.1])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_every_score_at_a_cap_near_52(sign, softcap, dtype):
    """tanh is +-1 for every key on both sides of the cap from which a maximum is kept."""
    c = Case([(3, 300), (1, 70)], 4, 2, 64, 64, dtype)
    c.q.fill_(16.0)
    c.k = torch.where(c.k.isnan(), c.k, torch.full_like(c.k, 16.0 * sign))
    c.kd = [torch.full_like(k, 16.0 * sign) for k in c.kd]
    check(c, c.run(softcap=softcap), softcap)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("number", [10 ** 6, -5])
@pytest.mark.parametrize("dh,lens", [(64, [(2, 200), (3, 90), (1, 300)]), (128, [(130, 700), (40, 200), (1, 64)])])
def test_a_page_outside_the_cache_counts_as_zeros(dh, lens, number, dtype):
    """Its keys score 0 and its values are 0, whatever ran on the GPU before."""
    c = Case(lens, 4, 2, dh, 64, dtype)
    want = c.run()
    table = c.table.clone()
    table[1, 1] = number
    c.kd[1][64:128], c.vd[1][64:128] = 0.0, 0.0
    results = []
    for fill in (3.0, float("nan")):
        other = Case([(5, 2000)] * 40, 4, 2, dh, 64, dtype)      # leaves its keys in every SM's shared memory
        other.k.fill_(fill)
        other.v.fill_(fill)
        other.run()
        r = B.mhc_paged_attn(c.q, c.k, c.v, table, c.cu, c.kv)
        c.check(r, error=B.MHC_ERR_RANGE)
        results.append(r)
    n, m = lens[0][0], lens[0][0] + lens[1][0]
    assert torch.equal(results[0].o, results[1].o) and torch.equal(results[0].lse, results[1].lse)
    assert torch.equal(r.o[:n], want.o[:n]) and torch.equal(r.o[m:], want.o[m:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [64, 128])
def test_buffers_at_16_bytes(dh, dtype, monkeypatch):
    """Workspace and outputs at odd multiples of 16 bytes, which is all that the
    library asks for; the long sequence's parts go through the workspace."""
    c = Case([(1, 5000), (40, 900), (3, 3)], 10, 2, dh, 64, dtype)
    want = c.run()

    def empty(shape, dtype=None, device=None):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        t = torch.empty(n + 32, dtype=torch.uint8, device=device)
        at = (16 - t.data_ptr()) % 32
        t = t[at:at + n].view(dtype).view(tuple(shape))
        assert t.data_ptr() % 32 == 16
        return t

    monkeypatch.setattr(B, "_empty", empty)
    got = c.run()
    assert torch.equal(got.o, want.o) and torch.equal(got.lse, want.lse)
    assert B.get_last_device_error() == B.MHC_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 7, 2 ** 30])
@pytest.mark.parametrize("dh", [64, 128])
def test_a_window_of_any_size(dh, window, dtype):
    """Also where a tile's first rows see nothing: their bounds stay in 32 bits."""
    for lens in (LENS["empty"], [(40, 30), (1010, 1000), (1, 0), (3, 500)]):
        c = Case(lens, 4, 2, dh, 16, dtype, window=window)
        c.check(c.run())


def test_a_plan_is_spent_by_a_timeout():
    """Parts that never came would leave a plan's counters in mid-join: after a
    timeout calls with it compute nothing and say so, and a new plan works."""
    c = Case([(1, 3000), (20, 40)], 4, 2, 64, 64, "bf16")
    sizes = (torch.bfloat16, c.T, 4, 2, 64, 64, c.T, c.table.shape[1] * 64)
    plan = B.mhc_paged_attn_plan(c.cu, c.kv, *sizes)
    want = B.mhc_paged_attn(c.q, c.k, c.v, c.table, plan=plan)
    assert B.get_last_device_error() == B.MHC_OK
    L = B.lib()
    try:
        assert L.mhc_test_force_timeout(1) == B.MHC_OK
        B.mhc_paged_attn(c.q, c.k, c.v, c.table, plan=plan)
        assert B.get_last_device_error() == B.MHC_ERR_TIMEOUT
    finally:
        assert L.mhc_test_force_timeout(0) == B.MHC_OK
    out = torch.full_like(want.o, 7.0)
    for _ in range(2):
        B.mhc_paged_attn(c.q, c.k, c.v, c.table, plan=plan, out=out)
        assert B.get_last_device_error() == B.MHC_ERR_RANGE
        assert bool((out == 7.0).all())
    plan = B.mhc_paged_attn_plan(c.cu, c.kv, *sizes)
    got = B.mhc_paged_attn(c.q, c.k, c.v, c.table, plan=plan, out=out)
    assert B.get_last_device_error() == B.MHC_OK
    assert torch.equal(got.o, want.o) and torch.equal(got.lse, want.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_that_overlap_have_no_more_tiles_than_fit(dtype):
    """cu_q that goes back and forth: more tiles than any batch of these rows has."""
    c = Case([(1024, 1100)], 4, 2, 64, 64, dtype)
    n = 1400
    cu = torch.tensor([0, 1024] * (n // 2) + [0], dtype=torch.int32, device=c.q.device)
    kv = torch.full((n,), 1100, dtype=torch.int32, device=c.q.device)
    r = B.mhc_paged_attn(c.q, c.k, c.v, c.table.expand(n, -1).contiguous(), cu, kv)
    c.check(r, error=B.MHC_ERR_RANGE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [136, 256])
def test_wide_heads(dh, dtype):
    """Heads above 128: windows, caps, both, and contexts that are split and joined."""
    for lens in (LENS["chunks"], [(1, 6000), (2, 1500)]):
        for window, softcap in ((100, 0.0), (0, 30.0), (100, 60.0), (0, 0.0)):
            c = Case(lens, 4, 2, dh, 16, dtype, window=window)
            check(c, c.run(softcap=softcap), softcap)
    assert B.get_last_device_error() == B.MHC_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [24, 64])
def test_long_contexts_with_the_heads_outside(page, dtype):
    for softcap in (0.0, 30.0, 60.0, 1e4):
        c = Case([(1, 7000), (2, 3001), (1, 5)], 10, 2, 128, page, dtype, order="head")
        check(c, c.run(softcap=softcap), softcap)
    assert B.get_last_device_error() == B.MHC_OK
