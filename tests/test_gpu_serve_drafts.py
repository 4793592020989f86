"""Layers served by drafted trees, all operators of such a step together, against
the whole streams at once (GPU).

As in tests/test_gpu_serve_layer.py: both paths round to bf16 at the same places,
but a row's keys come in other pieces (and places of its tree), so the sublayer's
output differs by up to one unit in the last place, and four units in the last
place of the state's largest values bound what follows of it in a layer.  Two
layers: the second one's inputs differ by that too, so eight.
"""

import importlib

import pytest
import torch

from mhc_pre_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def drafts():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return importlib.import_module("examples.serve_drafts")


@pytest.mark.parametrize("Hq,Hk,Dh,window,page,most", [(20, 4, 128, 0, 64, 24), (8, 8, 64, 100, 16, 40),
                                                       (6, 1, 96, 0, 48, 9)])
def test_kept_paths_match_whole_streams(drafts, Hq, Hk, Dh, window, page, most):
    layers = [drafts.ServedLayer(D=1024, Hq=Hq, Hk=Hk, Dh=Dh, window=window, max_pos=1024, seed=i) for i in range(2)]
    g = torch.Generator(device="cuda").manual_seed(2)
    lens, steps = (300, 1, 129, 63), 30
    streams = [torch.randn(n + steps, 4, 1024, generator=g, device="cuda").bfloat16() for n in lens]
    new = torch.stack([s[n:] for s, n in zip(streams, lens)])
    server = drafts.DraftServer(layers, 4, 400, page)
    kept = drafts.serve(server, [s[:n] for s, n in zip(streams, lens)], new, most)
    assert server.lens.tolist() == [n + steps for n in lens]
    # the kept tokens' pages: held once, and none lost
    used = [p for row, h in zip(server.table.tolist(), server.held.tolist()) for p in row[:h]]
    assert sorted(used + server.free[:int(server.count)].tolist()) == list(range(server.free.numel()))
    whole = drafts.serve(drafts.DraftServer(layers, 4, 400, page), streams, new[:, :0], most)
    assert B.get_last_device_error() == B.MHC_OK
    for a, b in zip(kept, whole):
        assert a.shape == b.shape and bool(a.isfinite().all())
        assert float((a.float() - b.float()).abs().max()) <= 8 * 2.0 ** -8 * float(b.float().abs().max())


@pytest.mark.parametrize("windows", [(0, 3), (5, 0, 5), (40, 2)])
def test_layers_of_different_windows(drafts, windows):
    """Prompts through several layers at once and through each of them alone: the same bits."""
    layers = [drafts.ServedLayer(D=1024, Hq=8, Hk=2, Dh=64, window=w, max_pos=64, seed=i) for i, w in enumerate(windows)]
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(33, 4, 1024, generator=g, device="cuda").bfloat16()
    y = drafts.DraftServer(layers, 2, 64, 16).step(x, [24, 9])
    for layer in layers:
        x = drafts.DraftServer([layer], 2, 64, 16).step(x, [24, 9])
    assert torch.equal(x, y)
    assert B.get_last_device_error() == B.MHC_OK


def test_paths_longer_than_a_window_are_refused(drafts):
    """The step's masks have all ancestors of a node, also those that the window hides;
    a path as long as the window is served."""
    assert drafts.depths([-1, 0, 1, -1, -1, 0, 0, 2], [3, 1, 4]) == [1, 2, 3, 1, 1, 2, 2, 3]
    layers = [drafts.ServedLayer(D=1024, Hq=8, Hk=2, Dh=64, window=w, max_pos=64) for w in (0, 3)]
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(24, 4, 1024, generator=g, device="cuda").bfloat16()
    whole = drafts.DraftServer(layers, 1, 64, 16).step(x, [24])
    server = drafts.DraftServer(layers, 1, 64, 16)
    server.step(x[:20], [20])
    lens = server.lens.clone()
    with pytest.raises(ValueError):
        server.step(x[20:], [4], [-1, 0, 1, 2], [[0, 1, 2, 3]])
    assert torch.equal(server.lens, lens)
    y = server.step(x[20:23], [3], [-1, 0, 1], [[0, 1, 2]])
    assert B.get_last_device_error() == B.MHC_OK
    assert float((y.float() - whole[20:23].float()).abs().max()) <= 8 * 2.0 ** -8 * float(whole.float().abs().max())


def test_keys_of_kept_paths_are_those_of_whole_streams(drafts):
    """The caches, token by token: in one layer keys and values depend on the token
    and its position alone.  The projections of other batch sizes may round
    differently, which the bound above covers."""
    layers = [drafts.ServedLayer(D=1024, Hq=8, Hk=2, Dh=64, max_pos=512)]
    g = torch.Generator(device="cuda").manual_seed(3)
    lens, steps = (60, 64), 20
    streams = [torch.randn(n + steps, 4, 1024, generator=g, device="cuda").bfloat16() for n in lens]
    new = torch.stack([s[n:] for s, n in zip(streams, lens)])
    a, b = drafts.DraftServer(layers, 2, 200, 16), drafts.DraftServer(layers, 2, 200, 16)
    drafts.serve(a, [s[:n] for s, n in zip(streams, lens)], new)
    drafts.serve(b, streams, new[:, :0])

    def cached(server, cache, s, n):
        return cache[server.table[s].clamp(min=0).long()].flatten(0, 1)[:n]

    for s, n in enumerate(lens):
        for x, y in ((a.k[0], b.k[0]), (a.v[0], b.v[0])):
            p, q = cached(a, x, s, n + steps).float(), cached(b, y, s, n + steps).float()
            assert float((p - q).abs().max()) <= 4 * 2.0 ** -8 * float(q.abs().max())
    assert B.get_last_device_error() == B.MHC_OK
