"""GPU parity of attention over a paged cache against the float64 oracle.

Tolerances.  u = 2^-24.  A score sums dh products: its error is held to
32 sqrt(dh) u times the largest scale * sum |q k| of the row (a tensor core's
float32 accumulation included), capped scores to 2^-20 of the cap more.  An
error e of the scores moves a weighted mean by at most 2 e sum p |v|; the sums
over n keys add 8 sqrt(n) u, the exponentials 2^-20.  With bf16 the
exponentials' rounding adds 2^-8 sum p |v| and the result's own 2^-8 |o|.
"""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


def f64(t):
    return t.detach().cpu().double().numpy()


class Case:
    """A cache whose unused places are NaN, with pages in random order."""

    def __init__(self, lens, Hq, Hk, dh, page, dtype, order="place", std=1.5, seed=0, extra=3, window=0):
        dev, gen = _dev(), torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=gen)            # noqa: E731
        self.lens, self.page, self.dtype, self.window = lens, page, dtype, window
        self.T = sum(a for a, _ in lens)
        # q is a part of a packed projection
        self.q = (n(self.T, (Hq + 2 * Hk) * dh) * std).to(DT[dtype]).to(dev)[:, :Hq * dh].view(self.T, Hq, dh)
        need = [-(-m // page) for _, m in lens]
        pages = sum(need) + extra
        shape = (pages, page, Hk, dh) if order == "place" else (pages, Hk, page, dh)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=DT[dtype], device=dev) for _ in range(2))
        if order == "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        ids = torch.randperm(pages, generator=gen)
        self.table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
        self.kd, self.vd, at = [], [], 0
        for b, (m_q, m) in enumerate(lens):
            mine = ids[at:at + need[b]]
            at += need[b]
            kk, vv = (n(m, Hk, dh) * std).to(DT[dtype]), n(m, Hk, dh).to(DT[dtype])
            self.kd.append(kk)
            self.vd.append(vv)
            # pages that no query sees may be gone
            gone = max(0, m - m_q + 1 - window) // page if window else 0
            for j, pg in enumerate(mine.tolist()):
                if j < gone:
                    continue
                c = min(page, m - j * page)
                self.k[pg, :c] = kk[j * page:j * page + c].to(dev)
                self.v[pg, :c] = vv[j * page:j * page + c].to(dev)
                self.table[b, j] = pg
        self.table = self.table.to(dev)
        self.cu = torch.tensor(np.cumsum([0] + [a for a, _ in lens]), dtype=torch.int32, device=dev)
        self.kv = torch.tensor([m for _, m in lens], dtype=torch.int32, device=dev)

    def run(self, **kw):
        kw = dict(window=self.window, **kw)
        return B.mhc_paged_attn(self.q, self.k, self.v, self.table, self.cu, self.kv, **kw)

    def check(self, r, softcap=0.0, scale=None, only=None, error=B.MHC_OK):
        """``only``: the sequences to look at; ``error``: what the device reports."""
        q, at = f64(self.q), 0
        dh = q.shape[-1]
        scale = dh ** -0.5 if scale is None else scale
        o, lse = f64(r.o), f64(r.lse)
        for b, (n, m) in enumerate(self.lens):
            if only is not None and b not in only:
                at += n
                continue
            assert np.all(np.isfinite(o[at:at + n]))
            ro, rl, pabs, size = A.attention(q[at:at + n], f64(self.kd[b]), f64(self.vd[b]), scale, self.window,
                                             softcap)
            e = 32 * np.sqrt(dh) * U * size + softcap * 2.0 ** -20
            rel = 2 * e + 8 * np.sqrt(max(m, 1)) * U + 2.0 ** -20
            tol = rel[..., None] * pabs
            if self.dtype == "bf16":
                tol = tol + 2.0 ** -8 * (pabs + np.abs(ro))
            over = np.abs(o[at:at + n] - ro) - tol
            assert over.size == 0 or over.max() <= 0, (b, over.max())
            empty = ~np.isfinite(rl)
            assert np.array_equal(empty, lse[at:at + n] == -np.inf)
            d = np.abs(np.where(empty, 0, lse[at:at + n]) - np.where(empty, 0, rl))
            assert np.all(d <= e + 8 * np.sqrt(max(m, 1)) * U + 2.0 ** -20 * (1 + np.abs(np.where(empty, 0, rl))))
            at += n
        assert B.get_last_device_error() == error


LENS = {
    "one": [(1, 1)],
    "decode": [(1, 200), (1, 1), (1, 129), (1, 64), (1, 1000)],
    "drafts": [(3, 300), (2, 2), (4, 127)],
    "prompts": [(5, 5), (128, 128), (77, 77), (1, 1)],
    "chunks": [(40, 300), (1, 513), (130, 131), (64, 64)],
    "empty": [(0, 0), (3, 0), (0, 50), (6, 2), (5, 5), (0, 0)],
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk,dh,page", [(10, 2, 128, 64), (4, 4, 64, 16), (8, 1, 128, 128), (6, 2, 96, 32)])
def test_lengths(lens, dtype, Hq, Hk, dh, page):
    c = Case(LENS[lens], Hq, Hk, dh, page, dtype)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 3, 8, 16, 48, 128, 256, 384])
def test_page_sizes(page, dtype):
    c = Case([(9, 300), (1, 255), (130, 400)], 4, 2, 64, page, dtype)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [8, 24, 40, 64, 72, 80, 112, 128, 136, 192, 256])
def test_head_sizes(dh, dtype):
    c = Case([(9, 200), (1, 33), (60, 60)], 4, 2, dh, 16, dtype)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (7, 7), (20, 4), (40, 2), (64, 1)])
def test_groups_of_heads(Hq, Hk, dtype):
    c = Case([(1, 260), (3, 70), (50, 50)], Hq, Hk, 64, 32, dtype)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 17, 128, 200, 5000])
@pytest.mark.parametrize("lens", ["decode", "prompts", "chunks", "empty"])
def test_window(window, lens, dtype):
    c = Case(LENS[lens], 10, 2, 128, 16, dtype, window=window)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap,std", [(30.0, 1.5), (5.0, 4.0), (50.0, 0.2)])
def test_capped_scores(softcap, std, dtype):
    c = Case(LENS["chunks"], 10, 2, 128, 64, dtype, std=std)
    c.check(c.run(softcap=softcap), softcap=softcap)
    c = Case(LENS["decode"], 10, 2, 64, 64, dtype, std=std, window=100)
    c.check(c.run(softcap=softcap), softcap=softcap)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [0.25, 51.9, 52.1, 400.0])
def test_caps_of_any_size(softcap, dtype):
    """Scores on both sides of the cap, which they reach where it is small."""
    for dh, window in ((128, 0), (64, 60)):
        c = Case(LENS["chunks"], 10, 2, dh, 64, dtype, std=4.0, window=window)
        c.check(c.run(softcap=softcap), softcap=softcap)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap", [30.0, 52.0, 60.0])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_every_score_at_the_cap(sign, softcap, dtype):
    """tanh is +-1 for every key: o is the mean of the values, lse +-cap + log m."""
    c = Case([(3, 300), (1, 70)], 4, 2, 64, 64, dtype)
    c.q.fill_(16.0)
    c.k = torch.where(c.k.isnan(), c.k, torch.full_like(c.k, 16.0 * sign))
    c.kd = [torch.full_like(k, 16.0 * sign) for k in c.kd]
    c.check(c.run(softcap=softcap), softcap=softcap)


def test_a_capped_rows_own_nan_is_seen():
    """A key that a row sees is not hidden by the cap."""
    c = Case([(70, 200)], 4, 2, 64, 64, "bf16")
    c.k[int(c.table[0, 3]), 2] = float("nan")     # token 194: the last 6 rows see it
    r = c.run(softcap=30.0)
    bad = r.o.isnan().flatten(1).all(1)
    assert bad[-6:].all()
    B.get_last_device_error()



@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_peaked_and_flat_scores(dtype):
    """Scores of hundreds (one key takes the row) and of almost zero."""
    for std, scale in ((6.0, 1.0), (0.01, None)):
        c = Case([(3, 500), (130, 200)], 4, 2, 64, 64, dtype, std=std)
        c.check(c.run(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_growing_scores(dtype):
    """Each block of keys scores higher than the one before: every step raises
    the running maximum."""
    c = Case([(4, 700), (140, 400)], 4, 2, 64, 64, dtype)
    for b, (_, m) in enumerate(c.lens):
        up = torch.linspace(0.0, 8.0, m)[:, None, None]
        c.kd[b] = (torch.ones(m, 2, 64) * up).to(DT[dtype])
        for j in range(-(-m // 64)):
            n = min(64, m - j * 64)
            c.k[int(c.table[b, j]), :n] = c.kd[b][j * 64:j * 64 + n].to(c.k.device)
    c.q.abs_()
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cache_with_the_heads_outside(dtype):
    c = Case(LENS["chunks"], 10, 2, 128, 64, dtype, order="head")
    c.check(c.run())


def test_later_rows_do_not_touch_earlier_ones():
    """A NaN among the keys that a row does not see leaves it alone."""
    c = Case([(100, 300)], 4, 2, 64, 64, "bf16")
    want = c.run()
    last = int(c.table[0, 299 // 64])
    c.k[last, 299 % 64] = float("nan")
    got = c.run()
    assert torch.equal(got.o[:99], want.o[:99]) and torch.equal(got.lse[:99], want.lse[:99])
    assert bool(got.o[99].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_context_is_split_and_repeats(dtype):
    """Few rows over many keys: the pieces are joined in the same order each time."""
    c = Case([(1, 9000), (2, 4097)], 5, 1, 128, 64, dtype)
    r = c.run()
    c.check(r)
    for _ in range(3):
        s = c.run()
        assert torch.equal(r.o, s.o) and torch.equal(r.lse, s.lse)


def test_large_chunk_matches_rows_of_the_oracle():
    """A chunk of many tiles: every 97th row against the oracle."""
    c = Case([(700, 1500)], 8, 2, 128, 64, "bf16")
    r = c.run()
    q, rows = f64(c.q), list(range(0, 700, 97)) + [699]
    for i in rows:
        m = 1500 - 700 + i + 1
        ro, rl, pabs, size = A.attention(q[i:i + 1], f64(c.kd[0])[:m], f64(c.vd[0])[:m], 128 ** -0.5)
        e = 32 * np.sqrt(128) * U * size
        tol = (2 * e + 8 * np.sqrt(m) * U + 2.0 ** -20)[..., None] * pabs + 2.0 ** -8 * (pabs + np.abs(ro))
        assert np.all(np.abs(f64(r.o[i:i + 1]) - ro) <= tol)
        assert np.all(np.abs(f64(r.lse[i:i + 1]) - rl) <= e + 1e-5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_plan_serves_many_calls(dtype):
    c = Case([(1, 3000), (40, 900), (0, 5), (1, 1)], 10, 2, 64, 64, dtype)
    want = c.run()
    plan = B.mhc_paged_attn_plan(c.cu, c.kv, DT[dtype], c.T, 10, 2, 64, 64, c.T, c.table.shape[1] * 64)
    for _ in range(4):
        r = B.mhc_paged_attn(c.q, c.k, c.v, c.table, plan=plan)
        assert torch.equal(r.o, want.o) and torch.equal(r.lse, want.lse)
    with pytest.raises(ValueError):
        B.mhc_paged_attn(c.q, c.k, c.v, c.table, plan=plan, window=64)
    with pytest.raises(ValueError):
        B.mhc_paged_attn(c.q[:10], c.k, c.v, c.table, plan=plan)


def test_padding_rows_stay_and_out_is_taken():
    c = Case([(2, 50), (3, 90)], 4, 2, 64, 16, "bf16")
    q = torch.cat([c.q, c.q[:4]])
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=q.device)
    want = c.run()
    r = B.mhc_paged_attn(q, c.k, c.v, c.table, c.cu, c.kv, out=out)
    assert r.o is out and torch.equal(out[:5], want.o) and torch.all(out[5:] == 9.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_numbers_outside_their_tensors_are_reported(dtype):
    c = Case([(2, 200), (3, 90), (1, 300)], 4, 2, 64, 64, dtype)
    want = c.run()
    for at, value in (((1, 0), 10 ** 6), ((1, 1), -5)):
        table = c.table.clone()
        table[at] = value
        r = B.mhc_paged_attn(c.q, c.k, c.v, table, c.cu, c.kv)
        assert B.get_last_device_error() == B.MHC_ERR_RANGE
        assert torch.equal(r.o[:2], want.o[:2]) and torch.equal(r.o[5:], want.o[5:])
    # a sequence whose numbers do not fit is left out; the others come out as ever
    # (not bit for bit: the batch is split over the GPU in other pieces)
    for cu, kv, kept in (([0, 2, 50, 6], None, [0]), ([0, 2, -3, 6], None, [0]),
                         (None, [200, 10 ** 6, 300], [0, 2]), (None, [200, -1, 300], [0, 2])):
        cu = c.cu if cu is None else torch.tensor(cu, dtype=torch.int32, device=c.q.device)
        kv = c.kv if kv is None else torch.tensor(kv, dtype=torch.int32, device=c.q.device)
        c.check(B.mhc_paged_attn(c.q, c.k, c.v, c.table, cu, kv), only=kept, error=B.MHC_ERR_RANGE)
    c.check(c.run(max_q=2), only=[0, 2], error=B.MHC_ERR_RANGE)
    assert torch.equal(c.run().o, want.o) and B.get_last_device_error() == B.MHC_OK


def test_cache_past_32_bits():
    """Pages whose elements lie past 2^31 in the cache."""
    dev = _dev()
    page, Hk, dh = 128, 8, 128
    pages = (2 ** 31) // (page * Hk * dh) + 40
    k = torch.empty(pages, page, Hk, dh, dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    c = Case([(1, 1000), (70, 600)], 8, Hk, dh, page, "bf16", extra=0)
    n = c.k.shape[0]
    k[-n:], v[-n:] = c.k, c.v
    table = torch.where(c.table >= 0, c.table + (pages - n), c.table)
    r = B.mhc_paged_attn(c.q, k, v, table, c.cu, c.kv)
    c.check(r)


def test_many_sequences():
    """More sequences than the plan kernel has threads."""
    rng = np.random.default_rng(0)
    lens = [(1, int(m)) for m in rng.integers(1, 40, 700)]
    c = Case(lens, 2, 1, 64, 16, "bf16")
    c.check(c.run(max_q=1))


def test_another_stream_and_a_graph():
    c = Case([(1, 700), (20, 300)], 10, 2, 128, 64, "bf16")
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run()
    s.synchronize()
    assert torch.equal(got.o, want.o)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = c.run()
    r.o.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.o, want.o)
    # the graph reads the lengths on the device: new ones, no new capture
    c.kv.copy_(torch.tensor([500, 290], dtype=torch.int32))
    g.replay()
    c.lens = [(1, 500), (20, 290)]
    c.kd, c.vd = [k[:m] for k, (_, m) in zip(c.kd, c.lens)], [v[:m] for v, (_, m) in zip(c.vd, c.lens)]
    c.check(r)


def test_empty_calls():
    dev = _dev()
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)       # noqa: E731
    assert B.mhc_paged_attn(q, k, k, i(1, 1), i(2), i(1)).o.shape == (0, 4, 64)
    assert B.mhc_paged_attn(q, k, k, i(0, 1), i(1), i(0)).lse.shape == (0, 4)
