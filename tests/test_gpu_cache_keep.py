"""Keeping an accepted path in the caches (mhc_cache_keep) against the oracle, bit
for bit (GPU)."""

import numpy as np
import pytest
import torch

from mhc_pre_gb300 import binding as B
from oracle import paged_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda", 0)


class Case:
    def __init__(self, lens, Hk, dh, page, dtype, layers=1, order="place", seed=0, paths=None, most=None):
        dev, rng = _dev(), np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.lens, self.page = lens, page
        need = [-(-m // page) for _, m in lens]
        pages = sum(need) + 3
        ids = rng.permutation(pages).tolist()
        self.table = torch.full((len(lens), max(need + [1])), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for j in range(n):
                self.table[b, j] = ids.pop()
        self.paths = paths or [sorted(rng.permutation(n)[:rng.integers(0, min(n, most or n) + 1)].tolist()) for n, _ in lens]
        width = max([len(p) for p in self.paths] + [1])
        self.path = torch.full((len(lens), width), -5, dtype=torch.int32)
        for b, p in enumerate(self.paths):
            self.path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        self.caches = [torch.randn(pages, page, Hk, dh, generator=gen).to(DT[dtype]) for _ in range(2 * layers)]
        self.want = [c.view(torch.int16 if dtype == "bf16" else torch.int32).numpy().copy() for c in self.caches]
        for (n, m), p, t in zip(lens, self.paths, self.table.tolist()):
            for c in self.want:
                O.keep(c, t, page, n, m, p)
        put = (lambda c: c.to(dev)) if order == "place" else (lambda c: c.transpose(1, 2).contiguous().to(dev).transpose(1, 2))
        self.caches = [put(c) for c in self.caches]
        self.k, self.v = self.caches[:layers], self.caches[layers:]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)     # noqa: E731
        self.table, self.path = self.table.to(dev), self.path.to(dev)
        self.cu, self.kv = i32(np.cumsum([0] + [n for n, _ in lens]).tolist()), i32([m for _, m in lens])
        self.keep, self.after = i32([len(p) for p in self.paths]), i32([77] * len(lens))

    def run(self, **kw):
        B.mhc_cache_keep(self.k, self.v, self.table, self.cu, self.kv, self.path, self.keep, lens=self.after, **kw)

    def check(self, error=B.MHC_OK, but=()):
        assert B.get_last_device_error() == error
        for c, w in zip(self.caches, self.want):
            got = c.contiguous().cpu()
            assert np.array_equal(got.view(torch.int16 if got.dtype == torch.bfloat16 else torch.int32).numpy(), w)
        for b, ((n, m), p, a) in enumerate(zip(self.lens, self.paths, self.after.tolist())):
            assert a == (77 if not p or b in but else m - n + len(p))


LENS = {"one": [(1, 1)], "two": [(2, 2)], "batch": [(13, 300), (1, 200), (7, 7), (32, 160), (33, 129), (0, 50), (5, 5)],
        "large": [(1000, 1300), (300, 300)]}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("Hk,dh,page", [(8, 128, 64), (1, 8, 3), (4, 96, 16), (2, 256, 128), (40, 256, 48)])
def test_paths(lens, Hk, dh, page, dtype):
    for seed in range(3):
        c = Case(LENS[lens], Hk, dh, page, dtype, seed=seed)
        c.run()
        c.check()


@pytest.mark.parametrize("path", [[0], [5], [0, 1, 2], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9], [1, 2, 3, 4, 5, 6, 7, 8, 9],
                                  [0, 2, 3, 4, 5, 6, 7, 8, 9], [0, 1, 9], [2, 4, 6, 8]])
@pytest.mark.parametrize("Hk,dh", [(1, 8), (8, 128), (64, 128)])
def test_rows_that_are_sources_and_goals(path, Hk, dh):
    """Shifts by one and two, where a goal is a later row's source; rows of one
    piece of 16 bytes and of more than a block holds."""
    c = Case([(10, 37)], Hk, dh, 16, "bf16", paths=[path])
    c.run()
    c.check()


@pytest.mark.parametrize("layers", [1, 2, 64, 65, 130])
def test_layers(layers):
    c = Case([(9, 30), (4, 20)], 2, 64, 16, "bf16", layers=layers)
    c.run()
    c.check()


@pytest.mark.parametrize("sequences,layers", [(3000, 3), (4097, 1), (9000, 7), (700, 67), (8192, 9)])
def test_many_sequences_of_which_few_keep_something(sequences, layers):
    """Blocks that take several caches, the last one fewer."""
    lens = [(0, 2)] * sequences
    for b in range(5, sequences, 397):
        lens[b] = (20, 30 + b % 40)
    c = Case(lens, 2, 8, 16, "bf16", layers=layers)
    c.run()
    c.check()


@pytest.mark.parametrize("sequences,layers", [(8191, 1), (8192, 1), (8193, 1), (4096, 2), (8191, 2), (8192, 2)])
def test_either_side_of_a_second_and_a_fourth_cache_of_a_block(sequences, layers):
    lens = [(0, 2)] * sequences
    for b in range(0, sequences, 511):
        lens[b] = (20, 30 + b % 40)
    c = Case(lens, 2, 8, 16, "bf16", layers=layers)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_caches_with_the_heads_outside(dtype):
    c = Case(LENS["batch"], 4, 64, 16, dtype, layers=2, order="head")
    c.run()
    c.check()


def test_numbers_that_do_not_fit_are_reported():
    lens = [(8, 40), (8, 40), (8, 40)]
    for path, change in (([3, 3], None), ([4, 2], None), ([2, 8], None), ([-1, 2], None), ([1, 2], "keep"),
                         ([1, 2], "negative"), ([1, 2], "m"), ([1, 2], "max_kv")):
        c = Case(lens, 2, 64, 16, "bf16", paths=[[2, 5, 6], [], [0, 7]])
        c.paths[1] = path
        c.path[1, :2] = torch.tensor(path, dtype=torch.int32)
        c.keep[1] = {"keep": 4, "negative": -1}.get(change, 2)
        kw = {}
        if change == "m":
            c.kv[1] = 7
        if change == "max_kv":
            c.kv[1] = 41
            kw = dict(max_kv=40)
        c.run(**kw)
        c.check(B.MHC_ERR_RANGE, but=(1,))


def test_pages_outside_the_cache_are_reported():
    c = Case([(8, 40), (8, 40)], 2, 64, 16, "bf16", paths=[[], [0, 7]])
    c.table[1, 2] = 10 ** 6          # tokens 32 to 39: all of the drafted ones
    c.want = [x.contiguous().cpu().view(torch.int16).numpy().copy() for x in c.caches]
    c.run()
    c.check(B.MHC_ERR_RANGE)


def test_bad_rows_of_the_host():
    c = Case(LENS["batch"], 2, 64, 16, "bf16", layers=2)
    with pytest.raises(ValueError):
        B.mhc_cache_keep(c.k, c.v[:1], c.table, c.cu, c.kv, c.path, c.keep)
    with pytest.raises(ValueError):
        B.mhc_cache_keep([c.k[0], c.k[1].transpose(1, 2).contiguous().transpose(1, 2)], c.v, c.table, c.cu, c.kv, c.path,
                         c.keep)
    with pytest.raises(ValueError):
        B.mhc_cache_keep(c.k, c.v, c.table, c.cu, c.kv, c.path[:2], c.keep)
    with pytest.raises(TypeError):
        B.mhc_cache_keep(c.k, [x.float() for x in c.v], c.table, c.cu, c.kv, c.path, c.keep)
    with pytest.raises(ValueError):
        B.mhc_cache_keep(c.k, c.v, c.table, c.cu, c.kv, c.path, c.keep, max_kv=10 ** 6)


def test_one_tensor_another_stream_and_a_graph():
    c = Case([(13, 300), (7, 7)], 2, 64, 16, "bf16", paths=[[0, 5, 6, 12], [3]])
    first = [x.clone() for x in c.caches]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        B.mhc_cache_keep(c.k[0], c.v[0], c.table, c.cu, c.kv, c.path, c.keep, lens=c.after)
    s.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for x, y in zip(c.caches, first):
        x.copy_(y)
    g.replay()
    c.check()


def test_cache_past_32_bits():
    dev = _dev()
    page, Hk, dh = 128, 8, 128
    pages = (2 ** 31) // (page * Hk * dh) + 40
    c = Case([(13, 1000), (40, 600)], Hk, dh, page, "bf16")
    n = c.k[0].shape[0]
    big = []
    for x in c.caches:
        y = torch.empty(pages, page, Hk, dh, dtype=torch.bfloat16, device=dev)
        y[-n:] = x
        big.append(y)
    table = torch.where(c.table >= 0, c.table + (pages - n), c.table)
    B.mhc_cache_keep(big[0], big[1], table, c.cu, c.kv, c.path, c.keep, lens=c.after)
    c.caches = [y[-n:] for y in big]
    c.check()
