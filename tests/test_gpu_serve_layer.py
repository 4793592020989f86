"""The layer with its attention sublayer, served in chunks and single tokens,
against whole prompts given at once (GPU).

Both paths round to bf16 at the same places, but a row's keys come in other
pieces, so its sums differ before the rounding: the attention output by up to
one unit in the last place, 2^-8 of its size, and what follows (a projection, the
residual update) keeps that relative to the sublayer's share of the state; four
units in the last place of the state's largest values bound it.
"""

import importlib.util
import os

import pytest
import torch

from mhc_pre_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serving():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_layer.py")
    spec = importlib.util.spec_from_file_location("serve_layer", path)
    mod = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["serve_layer"] = mod
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("Hq,Hk,Dh,window,page", [(20, 4, 128, 0, 64), (8, 8, 64, 100, 16), (6, 1, 96, 0, 48)])
def test_chunks_and_single_tokens_match_whole_prompts(serving, Hq, Hk, Dh, window, page):
    layer = serving.ServedLayer(D=1024, Hq=Hq, Hk=Hk, Dh=Dh, window=window, max_pos=1024)
    g = torch.Generator(device="cuda").manual_seed(2)
    lens, steps = (300, 1, 129), 3
    streams = [torch.randn(n + steps, 4, 1024, generator=g, device="cuda").bfloat16() for n in lens]
    new = torch.stack([s[n:] for s, n in zip(streams, lens)])
    served = serving.serve(layer, [s[:n] for s, n in zip(streams, lens)], new, chunk=77, page=page)
    whole = serving.serve(layer, streams, new[:, :0], chunk=10 ** 6, page=page)
    assert B.get_last_device_error() == B.MHC_OK
    for a, b in zip(served, whole):
        assert a.shape == b.shape and bool(a.isfinite().all())
        assert float((a.float() - b.float()).abs().max()) <= 4 * 2.0 ** -8 * float(b.float().abs().max())
