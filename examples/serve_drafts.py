"""Layers of an mHC model served by drafted trees (speculative decoding), with all
tables of a step made on the GPU:

    mhc_paged_step -> each layer: mhc_pre -> packed projection -> normalise, rotate
            and append -> attention of the trees -> output projection -> mhc_post
            -> mhc_cache_keep, which keeps each sequence's accepted path

There is no vocabulary here: a "token" is its residual streams, and a draft is a
tree of tokens among which the true next ones form a path.  Prompts go in as they
are, then every step drafts a tree for each sequence and keeps its true path.  Run
it (GPU) with

    python examples/serve_drafts.py

It prints how far the kept states are from those of the whole streams at once.
"""

from __future__ import annotations

import math
import os
import random
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from examples.serve_layer import ServedLayer  # noqa: E402
from mhc_pre_gb300 import binding as B  # noqa: E402


class DraftServer:
    """The caches of some layers, and which pages each sequence has: on the GPU."""

    def __init__(self, layers, sequences: int, max_len: int, page: int = 64, pages: int = None):
        first, dev = layers[0], layers[0].w_q.device
        self.layers, self.page = layers, page
        width = -(-max_len // page)
        n = pages or sequences * width
        shape = (n, page, first.Hk, first.Dh)
        # what no step has written is NaN here: it must not reach anything
        self.k, self.v = ([torch.full(shape, float("nan"), dtype=torch.bfloat16, device=dev) for _ in layers]
                          for _ in range(2))
        i32 = dict(dtype=torch.int32, device=dev)
        self.table = torch.full((sequences, width), -1, **i32)
        self.held, self.lens = torch.zeros(sequences, **i32), torch.zeros(sequences, **i32)
        self.free, self.count = torch.randperm(n, device=dev).to(torch.int32), torch.tensor([n], **i32)
        self.max_kv = width * page

    def step(self, x, counts, parents=None, paths=None):
        """x [T, 4, D]: the streams of counts[b] new tokens of each sequence, nodes
        of the trees `parents` if given.  All of them are kept, or `paths[b]` of each.
        Returns the states after the last layer."""
        if parents is not None:
            deepest = max(depths(parents, counts), default=0)
            for layer in self.layers:    # the masks have all ancestors, also those that a window hides
                if 0 < layer.window < deepest:
                    raise ValueError(f"a path of {deepest} drafted tokens is longer than a layer's window of {layer.window}")
        dev, T, n = x.device, x.shape[0], max(counts)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)       # noqa: E731
        s = B.mhc_paged_step(i32(counts), self.lens, self.table, self.held, self.free, self.count, self.page, T,
                             parents=None if parents is None else i32(parents), width=-(-n // 32))
        plans, lay = {}, self.layers[0]
        if parents is None:      # one for all layers with the same window
            for window in {layer.window for layer in self.layers}:
                plans[window] = B.mhc_paged_attn_plan(s.cu_q, s.kv_lens, torch.bfloat16, T, lay.Hq, lay.Hk, lay.Dh,
                                                      self.page, n, self.max_kv, window)
        for layer, k, v in zip(self.layers, self.k, self.v):
            x = self.layer(layer, x, k, v, s, n, plans.get(layer.window))
        if paths is None:
            self.lens = s.kv_lens
        else:
            keep = [len(p) for p in paths]
            path = i32([p + [0] * (max(keep) - len(p)) for p in paths])
            B.mhc_cache_keep(self.k, self.v, self.table, s.cu_q, s.kv_lens, path, i32(keep), lens=self.lens)
        return x

    def layer(self, layer, x, k_cache, v_cache, s, most, plan):
        T, h, k = x.shape[0], layer.Hq * layer.Dh, layer.Hk * layer.Dh
        f = B.mhc_pre(x, layer.phi, layer.b, layer.alpha)
        q, kk, v = (t.view(T, -1, layer.Dh) for t in (f.x_in @ layer.w_qkv).split([h, k, k], 1))
        q = B.mhc_qk_norm_rope_append(q, kk, v, layer.w_q, layer.w_k, k_cache, v_cache, s.slots,
                                      positions=s.positions, cos_sin=layer.cos_sin)
        if plan is not None:
            o = B.mhc_paged_attn(q, k_cache, v_cache, self.table, plan=plan).o
        else:
            o = B.mhc_tree_attn(q, k_cache, v_cache, self.table, s.tree, s.cu_q, s.kv_lens, max_q=most,
                                max_kv=self.max_kv, window=layer.window).o
        return B.mhc_post(x, o.view(T, h) @ layer.w_out, f.H_post, f.H_res)


def depths(parents, counts):
    """How many nodes the path of each node has, of trees laid end to end."""
    out = []
    for n in counts:
        first = len(out)
        for p in parents[first:first + n]:
            out.append(1 if p < 0 else out[first + p] + 1)
    return out


def draft(rng, left: int, most: int):
    """A tree of up to `most` nodes in which a path of up to `left` true tokens
    lies: (parents, numbers of the path's nodes)."""
    n = rng.randrange(1, most + 1)
    path = sorted(rng.sample(range(1, n), min(left, rng.randrange(1, 6), n) - 1)) if n > 1 else []
    path = [0] + path                     # the first node is the last token sampled: it is true
    parents = []
    for i in range(n):
        if i in path:
            at = path.index(i)
            parents.append(path[at - 1] if at else -1)
        else:
            parents.append(rng.randrange(-1, i))
    return parents, path


def serve(server: DraftServer, prompts, new, most=24, seed=0):
    """Runs prompts [len, 4, D] whole, then the streams of new [sequences, steps, 4, D]
    as paths of drafted trees.  Returns each sequence's kept states."""
    rng, S = random.Random(seed), len(prompts)
    counts = [len(p) for p in prompts]
    out = [[part] for part in server.step(torch.cat(list(prompts)), counts).split(counts)]
    done = [0] * S
    while min(done) < new.shape[1]:
        xs, parents, paths, counts = [], [], [], []
        for b in range(S):
            left = new.shape[1] - done[b]
            tree, path = draft(rng, left, most) if left else ([], [])
            x = torch.randn(len(tree), *new.shape[2:], device=new.device).to(new.dtype)
            x[path] = new[b, done[b]:done[b] + len(path)]
            done[b] += len(path)
            xs.append(x)
            parents += tree
            paths.append(path)
            counts.append(len(tree))
        y = server.step(torch.cat(xs), counts, parents, paths)
        for b, part in enumerate(y.split(counts)):
            out[b].append(part[paths[b]])
    return [torch.cat(o) for o in out]


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    layers = [ServedLayer(seed=i) for i in range(2)]
    lens, steps = (300, 1, 129), 40
    streams = [torch.randn(n + steps, 4, layers[0].D, generator=g, device="cuda").bfloat16() for n in lens]
    new = torch.stack([s[n:] for s, n in zip(streams, lens)])
    kept = serve(DraftServer(layers, 3, 448), [s[:n] for s, n in zip(streams, lens)], new)
    whole = serve(DraftServer(layers, 3, 448), streams, new[:, :0])
    assert B.get_last_device_error() == B.MHC_OK
    worst = max(float((a - b).abs().max()) for a, b in zip(kept, whole))
    size = math.sqrt(sum(float(a.float().square().mean()) for a in whole) / len(whole))
    print(f"kept paths of drafted trees against whole streams: largest difference {worst:.3g} of states of size "
          f"{size:.3g}")


if __name__ == "__main__":
    main()
