"""The integer tables of a step (mhc_paged_step) against the oracle, entry by
entry (GPU)."""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import paged_oracle as O
from tests.test_gpu_guard_bands import GuardedAllocator

pytestmark = pytest.mark.gpu


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


class Server:
    """The state of some sequences and their free pages, on both sides."""

    def __init__(self, B_, page, width, spare, rng, most=None, capacity=None):
        self.page, self.width = page, width
        self.lens = [int(rng.integers(0, (most or width * page) + 1)) for _ in range(B_)]
        self.held = [min(width, -(-m // page) + int(rng.integers(0, 2))) for m in self.lens]
        ids = rng.permutation(sum(self.held) + spare).tolist()
        self.table = [[-7] * width for _ in range(B_)]
        for b, h in enumerate(self.held):
            for j in range(h):
                self.table[b][j] = ids.pop()
        self.free = ids
        dev, i32 = _dev(), torch.int32
        cap = capacity or sum(self.held) + spare
        self.d_table = torch.tensor(self.table, dtype=i32, device=dev).view(B_, width)
        self.d_held = torch.tensor(self.held, dtype=i32, device=dev)
        self.d_free = torch.full((cap,), -9, dtype=i32, device=dev)
        self.d_free[:spare] = torch.tensor(self.free, dtype=i32)
        self.d_count = torch.tensor([spare], dtype=i32, device=dev)

    def step(self, new, T=None, parents=None, words=None, check=True):
        dev = self.d_table.device
        rows = sum(max(0, n) for n in new)
        T = rows if T is None else T
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)     # noqa: E731
        r = B.mhc_paged_step(i32(new), i32(self.lens), self.d_table, self.d_held, self.d_free, self.d_count,
                             self.page, T, None if parents is None else i32(parents + [-1] * (T - rows))[:T], words)
        if check:
            self.check(r, new, T, parents, words)
        return r

    def check(self, r, new, T, parents=None, words=None):
        want = O.step(new, self.lens, self.table, self.held, self.free, self.page, T, parents, words or 1)
        for name in ("cu_q", "kv_lens", "positions", "slots"):
            assert getattr(r, name).tolist() == want[name], name
        assert (r.tree is None) == (parents is None)
        if parents is not None:
            assert np.array_equal(r.tree.cpu().numpy(), want["tree"])
        assert self.d_held.tolist() == self.held
        assert int(self.d_count) == len(self.free)
        assert self.d_free[:len(self.free)].tolist() == self.free
        table = self.d_table.tolist()
        for b, h in enumerate(self.held):
            assert table[b][:h] == self.table[b][:h]


def random_parents(rng, n, deep=False):
    return [-1 if i == 0 or rng.random() < 0.05 else i - 1 if deep else int(rng.integers(max(0, i - 6), i))
            for i in range(n)]


def random_new(rng, server, most):
    out = []
    for m in server.lens:
        room = server.width * server.page - m
        kind = rng.integers(0, 8)
        out.append(-1 if kind == 0 else min(room, 0 if kind == 1 else 1 if kind < 4 else int(rng.integers(1, most + 1))))
    return out


@pytest.mark.parametrize("page", [1, 3, 16, 48, 64, 128])
@pytest.mark.parametrize("B_,most", [(1, 1), (1, 700), (5, 40), (64, 3), (513, 9), (2100, 2)])
def test_steps_one_after_the_other(B_, most, page):
    """Growing, ending and starting sequences; now and then too few pages are free."""
    rng = np.random.default_rng(B_ * 1000 + page)
    width = max(2, 900 // page)
    s = Server(B_, page, width, B_ + most // page, rng, most=width * page // 2)
    assert B.get_last_device_error() == B.MHC_OK
    for _ in range(5):
        new = random_new(rng, s, most)
        r = s.step(new)
        # a server goes on from there: some of the new tokens are dropped again
        kv = r.kv_lens.tolist()
        s.lens = [0 if n == -1 else m + int(rng.integers(0, k - m + 1)) for n, m, k in zip(new, s.lens, kv)]
    assert B.get_last_device_error() == B.MHC_OK


@pytest.mark.parametrize("B_,n,words", [(1, 1, 1), (1, 1000, 32), (3, 33, 2), (40, 64, 2), (600, 20, 1), (7, 300, 10)])
@pytest.mark.parametrize("deep", [False, True])
def test_trees(B_, n, words, deep):
    rng = np.random.default_rng(B_ + n)
    s = Server(B_, 16, 100 + n // 16, B_ * (n // 16 + 1), rng, most=1500)
    new = [int(rng.integers(1, n + 1)) if B_ > 1 else n for _ in range(B_)]
    parents = [p for k in new for p in random_parents(rng, k, deep)]
    s.step(new, parents=parents, words=words)
    assert B.get_last_device_error() == B.MHC_OK


def test_paths_longer_than_any_tree_are_cut_off():
    """A chain of thousands of rows: each climbs at most 1024 nodes."""
    n, m = 5000, 37
    dev = _dev()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)       # noqa: E731
    r = B.mhc_paged_step(i32([n]), i32([m]), torch.zeros(1, 400, dtype=torch.int32, device=dev), i32([400]), i32([0]),
                         i32([0]), 16, n, parents=torch.arange(-1, n - 1, dtype=torch.int32, device=dev))
    assert B.get_last_device_error() == B.MHC_ERR_RANGE
    assert r.positions.tolist() == [m + min(i, 1023) for i in range(n)]
    got = r.tree.cpu().numpy().view(np.uint32)
    bits = (got[:, :, None] >> np.arange(32, dtype=np.uint32) & 1).reshape(n, 1024).astype(bool)
    i, j = np.arange(n)[:, None], np.arange(1024)[None]
    assert (bits == ((j <= i) & (j > i - 1024))).all()


def test_pages_given_back_are_used_in_the_same_step():
    """The list alone would not do: the top of the list is what has come back."""
    rng = np.random.default_rng(3)
    s = Server(6, 16, 10, 1, rng, most=100)
    s.lens[0], s.lens[2] = 160, 150
    for b in (0, 2):
        while s.held[b] < 10:       # full rows
            s.table[b][s.held[b]] = 100 + 10 * b + s.held[b]
            s.d_table[b, s.held[b]] = s.table[b][s.held[b]]
            s.held[b] += 1
    s.d_held.copy_(torch.tensor(s.held, dtype=torch.int32))
    s.d_free = torch.cat([s.d_free, torch.full((30,), -9, dtype=torch.int32, device=s.d_free.device)])
    s.step([-1, 60, -1, 40, 0, 33])
    s.lens = [0, s.lens[1], 0, s.lens[3], s.lens[4], s.lens[5]]
    s.step([100, 1, 100, 1, 1, -1])
    assert B.get_last_device_error() == B.MHC_OK


def test_rows_past_the_new_tokens():
    rng = np.random.default_rng(4)
    s = Server(3, 16, 20, 9, rng, most=200)
    parents = random_parents(rng, 5) + random_parents(rng, 9) + [-1]
    s.step([5, 9, 1], T=40, parents=parents, words=3)
    assert B.get_last_device_error() == B.MHC_OK


def test_empty_steps():
    rng = np.random.default_rng(5)
    s = Server(4, 16, 20, 9, rng, most=200)
    s.step([0, 0, -1, 0])
    s.step([0, 0, -1, 0], T=7)
    dev = s.d_table.device
    z = lambda *n: torch.zeros(*n, dtype=torch.int32, device=dev)       # noqa: E731
    r = B.mhc_paged_step(z(0), z(0), z(0, 4), z(0), z(3), z(1), 16, 2)
    assert r.cu_q.tolist() == [0] and r.slots.tolist() == [-1, -1] and r.positions.tolist() == [0, 0]
    r = B.mhc_paged_step(z(2), z(2), z(2, 0), z(2), z(0), z(1), 16, 0)
    assert r.cu_q.tolist() == [0, 0, 0] and r.kv_lens.tolist() == [0, 0]
    assert B.get_last_device_error() == B.MHC_OK


def test_the_most_sequences():
    rng = np.random.default_rng(6)
    s = Server(8192, 64, 4, 3000, rng, most=200)
    s.step([1] * 8192)
    s = Server(8192, 64, 4, 3000, rng, most=200)
    new = [int(n) for n in rng.integers(0, 5, 8192)]
    s.step(new, parents=[p for n in new for p in random_parents(rng, n)], words=1)
    assert B.get_last_device_error() == B.MHC_OK
    with pytest.raises(B.MhcError):
        Server(8193, 64, 4, 10, rng, most=200).step([1] * 8193)


def _numbers(rng):
    return Server(4, 16, 20, 30, rng, most=200)


@pytest.mark.parametrize("what", ["new", "len", "held", "past held", "past table", "rows", "parents", "nodes", "count",
                                  "room", "page"])
def test_numbers_that_do_not_fit_are_reported(what):
    """Sequence 1 has the number; the others come out as without it."""
    rng = np.random.default_rng(7)
    s = _numbers(rng)
    s.lens = [40, 50, 60, 70]
    s.held = [3, 4, 4, 5]
    for b, h in enumerate(s.held):
        for j in range(h):
            s.table[b][j] = 200 + 10 * b + j
    s.d_held.copy_(torch.tensor(s.held, dtype=torch.int32))
    s.d_table.copy_(torch.tensor([[t if t >= 0 else -1 for t in row] for row in s.table], dtype=torch.int32))
    new, parents, words, T = [3, 4, 5, 6], None, None, None
    bad_rows, free0 = slice(3, 7), list(s.free)
    if what == "new":
        new[1] = -2
        bad_rows = slice(0, 0)
    elif what == "len":
        s.lens[1] = -1
    elif what == "held":
        s.d_held[1] = 21
    elif what == "past held":
        s.lens[1] = 65
    elif what == "past table":
        new[1] = 271
        bad_rows = slice(3, 274)
    elif what == "rows":
        T, bad_rows = 11, slice(0, 0)
    elif what in ("parents", "nodes"):
        parents = [-1, 0, 0, -1, 0, 1, 2, -1, 0, 1, 2, 3, -1, 0, 1, 2, 3, 4]
        words = 1
        if what == "parents":
            parents[4], parents[6] = 1, -5
        else:
            new, parents, bad_rows = [3, 40, 5, 6], [-1, 0, 0] + list(range(-1, 39)) + parents[7:], slice(3, 43)
    elif what == "count":
        s.d_count.fill_(10 ** 6)
    elif what == "room":
        new[1], bad_rows = -1, slice(0, 0)
        s.d_free, s.d_count = s.d_free[:2].clone(), torch.tensor([2], dtype=torch.int32, device=s.d_free.device)
        new = [0, -1, 0, 0]
    elif what == "page":
        s.d_table[1, 3] = -3
    r = s.step(new, T=T, parents=parents, words=words, check=False)
    assert B.get_last_device_error() == B.MHC_ERR_RANGE
    cu, kv, pos, slots = (x.tolist() for x in r[:4])
    if what == "rows":
        assert cu == [0, 3, 7, 7, 7] and kv[2:] == [60, 70] and slots[7:] == [-1] * 4
        return
    if what == "room":
        assert kv == [40, 0, 60, 70] and int(s.d_count) == 2 and s.d_free.tolist() == free0[:2] and int(s.d_held[1]) == 0
        return
    if what == "count":        # the whole list counts
        assert kv == [43, 54, 65, 76] and int(s.d_count) < s.d_free.numel()
        return
    for b in (0, 2, 3):
        assert kv[b] == s.lens[b] + new[b]
        for i in range(new[b]):
            at = s.lens[b] + i
            assert slots[cu[b] + i] == int(s.d_table[b, at // 16]) * 16 + at % 16
    if what in ("new", "len", "held", "past held", "past table"):
        assert kv[1] == 0 and all(x == -1 for x in slots[bad_rows]) and not any(pos[bad_rows])
    if what == "parents":      # as nodes that follow the context
        assert r.tree[3:7, 0].tolist() == [1, 2, 6, 8] and pos[3:7] == [50, 50, 51, 50]
    if what == "nodes":        # those past the words have no bit
        assert r.tree[3:43, 0].tolist() == [(1 << i + 1) - 1 for i in range(31)] + [-1] * 9
    if what == "page":
        assert slots[bad_rows] == [-1, -1, -1, -1]


def test_nothing_is_written_outside(monkeypatch):
    rng = np.random.default_rng(8)
    for B_, n in ((1, 1), (5, 33), (700, 6)):
        s = Server(B_, 16, 40, 3 * B_, rng, most=500)
        new = [n] * B_
        parents = [p for k in new for p in random_parents(rng, k)]
        dev = s.d_table.device
        guarded = GuardedAllocator()
        # the state in guarded buffers too, the table's rows apart
        wide = torch.full((B_, 48), 12345, dtype=torch.int32, device=dev)
        wide[:, 3:43] = s.d_table
        s.d_table = wide[:, 3:43]
        for name in ("d_held", "d_free", "d_count"):
            t = getattr(s, name)
            buf = guarded(tuple(t.shape), dtype=t.dtype, device=dev)
            setattr(s, name, buf.copy_(t))
        monkeypatch.setattr(B, "_empty", guarded)
        s.step(new, parents=parents, words=2)
        monkeypatch.undo()
        guarded.check(f"{B_} {n}")
        assert bool((wide[:, :3] == 12345).all()) and bool((wide[:, 43:] == 12345).all())


def test_a_captured_step_serves_any_lengths():
    rng = np.random.default_rng(9)
    s = Server(9, 16, 40, 200, rng, most=300)
    dev = s.d_table.device
    new, lens = torch.zeros(9, dtype=torch.int32, device=dev), torch.zeros(9, dtype=torch.int32, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):           # nothing to do: the state stays
        B.mhc_paged_step(new, lens, s.d_table, s.d_held, s.d_free, s.d_count, 16, 50)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = B.mhc_paged_step(new, lens, s.d_table, s.d_held, s.d_free, s.d_count, 16, 50)
    for k in range(4):
        fresh = [int(rng.integers(-1, 6)) for _ in range(9)]
        new.copy_(torch.tensor(fresh, dtype=torch.int32))
        lens.copy_(torch.tensor(s.lens, dtype=torch.int32))
        g.replay()
        s.check(r, fresh, 50)
        s.lens = r.kv_lens.tolist()
    assert B.get_last_device_error() == B.MHC_OK
