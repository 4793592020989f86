"""GPU parity of attention of drafted trees over a paged cache against the
float64 oracle.  The tolerances are those of tests/test_gpu_paged_attn.py: the
sums, exponentials and roundings are the same, only the keys differ.
"""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import attn_oracle as A
from tests.test_gpu_guard_bands import GuardedAllocator
from tests.test_gpu_paged_attn import DT, U, Case, f64

pytestmark = pytest.mark.gpu


def tree_mask(kind, n, rng):
    """[n, n] bool: which of n drafted tokens each one sees."""
    if kind == "chain":
        return np.tril(np.ones((n, n), bool))
    if kind == "any":                                   # not a tree: a third of all pairs, some rows with nothing
        m = rng.random((n, n)) < 0.33
        m[rng.random(n) < 0.2] = False
        return m
    order = rng.permutation(n) if kind == "shuffled" else np.arange(n)
    m = np.zeros((n, n), bool)
    for i in range(n):
        p = -1 if i == 0 or kind == "star" or rng.random() < 0.1 else rng.integers(max(0, i - 6), i)
        if p >= 0:
            m[order[i]] = m[order[p]]
        m[order[i], order[i]] = True
    if kind == "padded":                                # the last quarter is padding: it sees nothing and nobody sees it
        m[n - n // 4:] = False
        m[:, n - n // 4:] = False
    return m


def pack(masks, width, stray):
    """Rows of all sequences as int32 words; `stray` sets the bits past a sequence's tokens."""
    rows = []
    for m in masks:
        bits = np.full((len(m), 32 * width), stray, bool)
        bits[:, :len(m)] = m
        rows.append(np.packbits(bits, axis=1, bitorder="little").view("<i4"))
    return torch.from_numpy(np.concatenate(rows) if rows else np.zeros((0, width), "<i4"))


class Trees(Case):
    """A cache whose unused places are NaN; so are the drafted tokens that nobody sees."""

    def __init__(self, lens, Hq, Hk, dh, page, dtype, kind="tree", words=None, stray=True, **kw):
        super().__init__(lens, Hq, Hk, dh, page, dtype, **kw)
        rng = np.random.default_rng(kw.get("seed", 0))
        self.masks = [tree_mask(kind, n, rng) for n, _ in lens]
        self.most = max([n for n, _ in lens])
        self.tree = pack(self.masks, words or max(1, -(-self.most // 32)), stray).to(self.q.device)
        for b, (n, m) in enumerate(lens):
            for j in range(n):
                if m >= n and not self.masks[b][:, j].any():
                    key = m - n + j
                    pg = int(self.table[b, key // page])
                    if pg >= 0:
                        self.k[pg, key % page] = float("nan")
                        self.v[pg, key % page] = float("nan")

    def run(self, **kw):
        kw = dict(window=self.window, max_q=self.most, **kw)
        return B.mhc_tree_attn(self.q, self.k, self.v, self.table, self.tree, self.cu, self.kv, **kw)

    def check(self, r, softcap=0.0, scale=None, only=None, error=B.MHC_OK):
        q, at = f64(self.q), 0
        dh = q.shape[-1]
        scale = dh ** -0.5 if scale is None else scale
        o, lse = f64(r.o), f64(r.lse)
        for b, (n, m) in enumerate(self.lens):
            if only is None or b in only:
                assert np.all(np.isfinite(o[at:at + n]))
                ro, rl, pabs, size = A.tree_attention(q[at:at + n], f64(self.kd[b]), f64(self.vd[b]), scale,
                                                      self.masks[b], self.window, softcap)
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
    "drafts": [(13, 300), (1, 200), (7, 7), (32, 160), (33, 129), (2, 1000)],
    "wide": [(64, 300), (65, 65), (128, 128), (100, 513)],
    "large": [(300, 700), (1, 129)],
    "empty": [(0, 0), (3, 0), (0, 50), (6, 2), (5, 5), (0, 0)],
}
KINDS = ["tree", "shuffled", "any", "padded", "chain", "star"]


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,Hk,dh,page", [(10, 2, 128, 64), (4, 4, 64, 16)])
def test_trees(lens, dtype, kind, Hq, Hk, dh, page):
    c = Trees(LENS[lens], Hq, Hk, dh, page, dtype, kind)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,m", [(1000, 1100), (1024, 1024), (513, 2000)])
def test_the_largest_trees(n, m, dtype):
    c = Trees([(n, m), (1, 40)], 2, 1, 64, 64, dtype, "tree")
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 3, 8, 48, 128, 256])
def test_page_sizes(page, dtype):
    c = Trees([(9, 300), (21, 255), (70, 400)], 4, 2, 64, page, dtype, "padded")
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [8, 40, 72, 96, 136, 256])
def test_head_sizes(dh, dtype):
    c = Trees([(9, 200), (33, 33), (60, 190)], 4, 2, dh, 16, dtype, "any")
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (20, 4), (40, 2), (64, 1)])
def test_groups_of_heads(Hq, Hk, dtype):
    c = Trees([(12, 260), (3, 70), (50, 50)], Hq, Hk, 64, 32, dtype, "shuffled")
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 5, 30, 128, 200, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("kind", ["tree", "any", "padded"])
def test_window(window, kind, dtype):
    c = Trees(LENS["drafts"] + [(64, 300), (6, 2)], 10, 2, 128, 16, dtype, kind, window=window)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("softcap,std", [(5.0, 4.0), (30.0, 1.5), (60.0, 4.0), (400.0, 4.0)])
@pytest.mark.parametrize("kind", ["tree", "any"])
def test_capped_scores(softcap, std, kind, dtype):
    for dh, window in ((128, 0), (64, 60)):
        c = Trees(LENS["drafts"] + [(100, 260)], 10, 2, dh, 64, dtype, kind, std=std, window=window)
        c.check(c.run(softcap=softcap), softcap=softcap)
    # no context: rows of the mask may leave nothing at all
    c = Trees([(40, 40), (6, 2), (1, 1), (130, 131)], 10, 2, 64, 16, dtype, kind, std=std)
    c.check(c.run(softcap=softcap), softcap=softcap)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("edge", range(120, 137, 4))
def test_trees_across_the_borders_of_blocks(edge, dtype):
    """The drafted tokens begin before, at and behind a block of 128 keys."""
    for n in (1, 31, 40, 150):
        c = Trees([(n, edge + n), (n, edge + 256 + n)], 4, 2, 64, 64, dtype, "padded")
        c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chains_are_causal(dtype):
    """A chain is a chunk: the same keys for every row."""
    c = Trees([(20, 300), (1, 129), (70, 70)], 10, 2, 64, 16, dtype, "chain")
    r = c.run()
    s = B.mhc_paged_attn(c.q, c.k, c.v, c.table, c.cu, c.kv, max_q=c.most)
    c.check(r)
    c.check(s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 7, 20, 45, 130])
def test_chains_with_a_window_are_causal(window, dtype):
    """A chain longer than the window, with the ancestors that it hides taken out of the
    mask: the same keys as a chunk's."""
    c = Trees([(20, 300), (1, 129), (70, 70), (90, 400)], 10, 2, 64, 16, dtype, "chain", window=window)
    c.masks = [m & np.triu(np.ones_like(m), 1 - window) for m in c.masks]
    c.tree = pack(c.masks, c.tree.shape[1], False).to(c.q.device)
    s = B.mhc_paged_attn(c.q, c.k, c.v, c.table, c.cu, c.kv, max_q=c.most, window=window)
    c.check(c.run())
    c.check(s)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_contexts_are_split_and_repeat(dtype):
    c = Trees([(21, 9000), (40, 4097)], 5, 1, 128, 64, dtype, "tree")
    r = c.run()
    c.check(r)
    for _ in range(3):
        s = c.run()
        assert torch.equal(r.o, s.o) and torch.equal(r.lse, s.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_that_are_parts_of_wider_ones(dtype):
    """Words that no bit of the call needs, and a mask with a distance between its rows."""
    c = Trees([(13, 300), (33, 129)], 4, 2, 64, 64, dtype, "tree")
    want = c.run()
    wide = torch.full((c.T, 9), -1, dtype=torch.int32, device=c.q.device)
    wide[:, 3:5] = c.tree
    c.tree = wide[:, 3:]
    r = c.run()
    assert torch.equal(r.o, want.o) and torch.equal(r.lse, want.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(70, 6000), (10, 5000), (30, 3000), (1, 7000), (0, 9)], [(101, 900), (26, 2500)],
                                  [(51, 4000), (25, 60), (25, 70), (26, 80)] * 3, [(120, 5000)]])
def test_tiles_of_all_kinds_split_at_any_block(lens, dtype):
    """Tiles of one lane's rows, of both and several of a sequence, whose blocks weigh
    differently in the CTAs' shares."""
    for dh in (64, 128):
        c = Trees(lens, 5, 1, dh, 64, dtype, "any")
        c.check(c.run())


def test_many_sequences():
    """More sequences than a CTA has threads, which each find their share: some
    with nothing, some with numbers that do not fit."""
    rng = np.random.default_rng(0)
    lens = [(int(n), int(n + m)) for n, m in zip(rng.integers(0, 4, 1500), rng.integers(0, 40, 1500))]
    for dtype in ("bf16", "f32"):
        c = Trees(lens, 2, 1, 64, 16, dtype, "tree")
        c.check(c.run())
        c.kv[700] = -3
        c.check(c.run(), only=[0, 1, 2, 699, 701, 1498, 1499], error=B.MHC_ERR_RANGE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("at", [[0, 1, 2], [0, 17, 18, 146, 147, 400, 1183], [1999], [127, 128, 129, 255, 256, 385], [],
                                list(range(3, 2000, 97)), [0, 1, 33, 1998]])
def test_sequences_far_apart_among_idle_ones(at, dtype):
    """Most of a large batch has no new tokens in this step; the same with the idle
    ones taken out."""
    rng = np.random.default_rng(len(at))
    lens = [(0, int(m)) for m in rng.integers(0, 30, 2000)]
    for b in at:
        n = int(rng.integers(1, 30))
        lens[b] = (n, n + int(rng.integers(0, 900)))
    c = Trees(lens, 5, 1, 64, 16, dtype, "tree") if at else Trees([(0, 9)] * 2000, 5, 1, 64, 16, dtype)
    kw = dict(max_q=30, max_kv=c.table.shape[1] * 16)
    if not at:
        c.tree = c.tree[:0].reshape(0, 1)
    r = B.mhc_tree_attn(c.q, c.k, c.v, c.table, c.tree, c.cu, c.kv, **kw)
    c.check(r)
    here = torch.tensor(at, dtype=torch.long, device=c.q.device)
    cu = torch.cat([c.cu[:1], c.cu[1:][here]])
    s = B.mhc_tree_attn(c.q, c.k, c.v, c.table[here], c.tree, cu, c.kv[here], **kw)
    assert torch.equal(r.o, s.o) and torch.equal(r.lse, s.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("first,idle,last", [(598, 7400, 20), (229, 7400, 20), (598, 1, 20), (200, 7900, 1)])
def test_shares_that_begin_behind_idle_sequences(first, idle, last, dtype):
    """Short trees, then a run of sequences without new tokens, then more trees.  With 152
    SMs a share of 598 (bf16) or 229 (float32) of them begins behind the run.  The same
    with the idle ones taken out."""
    rng = np.random.default_rng(0)
    new = np.concatenate([rng.integers(1, 9, first), np.zeros(idle, int), rng.integers(1, 9, last)])
    context = np.where(new > 0, rng.integers(0, 200, len(new)), 5)
    c = Trees([(int(n), int(n + m)) for n, m in zip(new, context)], 10, 2, 128, 64, dtype, "tree")
    r = B.mhc_tree_attn(c.q, c.k, c.v, c.table, c.tree, c.cu, c.kv, max_q=9)
    here = torch.tensor(np.flatnonzero(new), device=c.q.device)
    cu = torch.cat([c.cu[:1], c.cu[1:][here]])
    s = B.mhc_tree_attn(c.q, c.k, c.v, c.table[here], c.tree, cu, c.kv[here], max_q=9)
    assert torch.equal(r.o, s.o) and torch.equal(r.lse, s.lse)
    if first < 300:
        c.check(r)
    assert B.get_last_device_error() == B.MHC_OK


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 12, 25, 26, 50, 51, 90])
def test_short_contexts_in_great_number(n, dtype):
    """Tiles far smaller than a CTA's share, whole and with borders moved."""
    c = Trees([(n, n + 3 * (i % 50)) for i in range(120)], 5, 1, 64, 16, dtype, "tree")
    c.check(c.run())


def _without_max_q(c):
    return B.mhc_tree_attn(c.q, c.k, c.v, c.table, c.tree, c.cu, c.kv, window=c.window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,words", [([(20, 120)] * 32, 1), ([(20, 60)] * 60, 2), ([(20, 60)] * 60, 60),
                                        ([(1024, 1100), (1024, 1024), (9, 40)], 32), ([(3, 30)], 4), ([(32, 32)], 1)])
def test_the_default_most_new_tokens(lens, words, dtype):
    """Without max_q a sequence may have as many as the mask has bits for, at most
    1024, whatever the batch's rows are."""
    c = Trees(lens, 2, 1, 64, 64, dtype, "tree", words=words)
    c.check(_without_max_q(c))


def test_the_default_most_new_tokens_is_held_to():
    """A sequence with more of them than the mask's bits is left out and reported."""
    c = Trees([(9, 40), (33, 100), (32, 50)], 2, 1, 64, 64, "bf16", "tree", words=2)
    c.tree = c.tree[:, :1].contiguous()
    c.check(_without_max_q(c), only=[0, 2], error=B.MHC_ERR_RANGE)
    c.tree = c.tree[:, :0]
    with pytest.raises(ValueError):
        _without_max_q(c)


def test_padding_rows_stay_and_out_is_taken():
    c = Trees([(2, 50), (3, 90)], 4, 2, 64, 16, "bf16")
    q, tree = torch.cat([c.q, c.q[:4]]), torch.cat([c.tree, c.tree[:4]])
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device=q.device)
    want = c.run()
    r = B.mhc_tree_attn(q, c.k, c.v, c.table, tree, c.cu, c.kv, out=out)
    assert r.o is out and torch.equal(out[:5], want.o) and torch.all(out[5:] == 9.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_numbers_outside_their_tensors_are_reported(dtype):
    c = Trees([(12, 200), (3, 90), (1, 300)], 4, 2, 64, 64, dtype)
    want = c.run()
    for at, value in (((1, 0), 10 ** 6), ((1, 1), -5)):
        table = c.table.clone()
        table[at] = value
        r = B.mhc_tree_attn(c.q, c.k, c.v, table, c.tree, c.cu, c.kv, max_q=12)
        assert B.get_last_device_error() == B.MHC_ERR_RANGE
        assert torch.equal(r.o[:12], want.o[:12]) and torch.equal(r.o[15:], want.o[15:])
    for cu, kv, kept in (([0, 12, 50, 16], None, [0]), (None, [200, 10 ** 6, 300], [0, 2]),
                         (None, [200, -1, 300], [0, 2])):
        cu = c.cu if cu is None else torch.tensor(cu, dtype=torch.int32, device=c.q.device)
        kv = c.kv if kv is None else torch.tensor(kv, dtype=torch.int32, device=c.q.device)
        c.check(B.mhc_tree_attn(c.q, c.k, c.v, c.table, c.tree, cu, kv, max_q=12), only=kept, error=B.MHC_ERR_RANGE)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hk,dh,page", [([(1, 5000), (13, 170)], 10, 2, 128, 64),
                                                ([(300, 700), (0, 0), (129, 129)], 5, 1, 80, 16)])
def test_nothing_is_written_outside(lens, Hq, Hk, dh, page, dtype, monkeypatch):
    c = Trees(lens, Hq, Hk, dh, page, dtype)
    plain = c.run()
    guarded = GuardedAllocator()
    monkeypatch.setattr(B, "_empty", guarded)
    got = c.run()
    monkeypatch.undo()
    guarded.check(f"{lens} {dtype}")
    assert len(guarded.bufs) == 3
    assert torch.equal(plain.o, got.o) and torch.equal(plain.lse, got.lse)


def test_forced_timeout_is_reported():
    c = Trees([(1, 300), (20, 40)], 4, 2, 64, 64, "bf16")
    want = c.run()
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


@pytest.mark.parametrize("dtype,dh,page", [("f32", 64, 64), ("bf16", 136, 64), ("bf16", 64, 48)])
def test_the_timeout_hook_leaves_kernels_without_waits_alone(dtype, dh, page):
    """On the CUDA cores nothing waits, so nothing runs out: whole tiles and split
    ones get their rows, and there is nothing to report."""
    c = Trees([(20, 3000), (3, 40)], 4, 2, dh, page, dtype)
    want = c.run()
    L = B.lib()
    try:
        assert L.mhc_test_force_timeout(1) == B.MHC_OK
        got = c.run(out=torch.full_like(c.q, float("nan")))
        assert B.get_last_device_error() == B.MHC_OK
    finally:
        assert L.mhc_test_force_timeout(0) == B.MHC_OK
    assert torch.equal(got.o, want.o) and torch.equal(got.lse, want.lse)


def test_another_stream_and_a_graph():
    c = Trees([(7, 700), (20, 300)], 10, 2, 128, 64, "bf16")
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
    # another mask, no new capture
    c.masks = [np.eye(n, dtype=bool) for n, _ in c.lens]
    c.tree.copy_(pack(c.masks, c.tree.shape[1], False))
    g.replay()
    c.check(r)


def test_two_streams_at_once():
    """Calls that overlap have a workspace each."""
    cases = [Trees([(13, 3000), (40, 900)], 10, 2, 128, 64, "bf16", "tree", seed=i) for i in range(2)]
    cases.append(Trees([(20, 700)], 10, 2, 64, 64, "f32", "any"))
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(c.run())
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a.o, b.o) and torch.equal(a.lse, b.lse)
    assert B.get_last_device_error() == B.MHC_OK


def test_cache_past_32_bits():
    dev = torch.device("cuda", 0)
    page, Hk, dh = 128, 8, 128
    pages = (2 ** 31) // (page * Hk * dh) + 40
    k = torch.empty(pages, page, Hk, dh, dtype=torch.bfloat16, device=dev)
    v = torch.empty_like(k)
    c = Trees([(13, 1000), (70, 600)], 8, Hk, dh, page, "bf16", extra=0)
    n = c.k.shape[0]
    k[-n:], v[-n:] = c.k, c.v
    table = torch.where(c.table >= 0, c.table + (pages - n), c.table)
    c.check(B.mhc_tree_attn(c.q, k, v, table, c.tree, c.cu, c.kv, max_q=c.most))


def test_empty_calls():
    dev = torch.device("cuda", 0)
    q = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev)
    k = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)       # noqa: E731
    assert B.mhc_tree_attn(q, k, k, i(1, 1), i(0, 1), i(2), i(1)).o.shape == (0, 4, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hk,dh", [([(13, 777)], 10, 2, 128), ([(21, 3000), (60, 900), (1, 5000)], 5, 1, 64)])
def test_nothing_depends_on_what_the_memory_held(lens, Hq, Hk, dh, dtype, monkeypatch):
    """Workspace and outputs of any contents: the same bits."""
    c = Trees(lens, Hq, Hk, dh, 64, dtype, "tree")
    got = []
    for value in (0, 255, 127):
        def filled(shape, dtype, device, value=value):
            t = torch.empty(shape, dtype=dtype, device=device)
            t.view(-1).view(torch.uint8).fill_(value)
            return t
        monkeypatch.setattr(B, "_empty", filled)
        got.append(c.run())
    monkeypatch.undo()
    for r in got[1:]:
        assert torch.equal(got[0].o, r.o) and torch.equal(got[0].lse, r.lse)
    c.check(got[0])
