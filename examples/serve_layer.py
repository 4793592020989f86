"""One mHC layer with an attention sublayer, served over a paged cache:

    mhc_pre -> packed projection -> normalise, rotate and append -> attention
            over the pages -> output projection -> mhc_post

A prompt goes in by chunks, then tokens one at a time; several sequences of
different lengths share the batch and the cache.  Run it (GPU) with

    python examples/serve_layer.py

It prints how far the served states are from those of the whole prompts given
at once.
"""

from __future__ import annotations

import math
import os
import sys
from dataclasses import dataclass, field

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mhc_pre_gb300 import binding as B  # noqa: E402


def rope_table(max_pos: int, rot: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """[max_pos, rot] float32: rot/2 cosines, then rot/2 sines."""
    freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


@dataclass
class Pages:
    """The cache of one layer and which pages each sequence has."""
    k: torch.Tensor                 # [pages, page_size, Hk, Dh]
    v: torch.Tensor
    table: torch.Tensor             # [sequences, most pages] int32, on the host
    lens: list = field(default_factory=list)
    free: list = field(default_factory=list)

    @classmethod
    def make(cls, sequences: int, max_len: int, page: int, Hk: int, Dh: int, device="cuda"):
        each = -(-max_len // page)
        n = sequences * each
        k, v = (torch.empty(n, page, Hk, Dh, dtype=torch.bfloat16, device=device) for _ in range(2))
        return cls(k, v, torch.full((sequences, each), -1, dtype=torch.int32), [0] * sequences,
                   torch.randperm(n).tolist())

    def step(self, counts):
        """Room for counts[b] new tokens of each sequence: the step's device
        tensors (positions, slots, cu_q, kv_lens, page table) and their bounds."""
        page = self.k.shape[1]
        pos, slots = [], []
        for b, n in enumerate(counts):
            for i in range(self.lens[b], self.lens[b] + n):
                if i % page == 0:
                    self.table[b, i // page] = self.free.pop()
                pos.append(i)
                slots.append(int(self.table[b, i // page]) * page + i % page)
            self.lens[b] += n
        d = self.k.device
        cu = [0]
        for n in counts:
            cu.append(cu[-1] + n)
        i32 = dict(dtype=torch.int32, device=d)
        return dict(positions=torch.tensor(pos, **i32), slots=torch.tensor(slots, dtype=torch.int64, device=d),
                    cu_q=torch.tensor(cu, **i32), kv_lens=torch.tensor(self.lens, **i32), table=self.table.to(d),
                    max_q=max(counts), max_kv=max(self.lens))


class ServedLayer:
    """Random weights of an mHC layer (n = 4 streams of D) with an attention
    sublayer of Hq query and Hk key heads of Dh."""

    def __init__(self, D=2560, Hq=20, Hk=4, Dh=128, window=0, max_pos=8192, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        n = lambda *s, std: torch.randn(*s, generator=g, device=device) * std     # noqa: E731
        self.D, self.Hq, self.Hk, self.Dh, self.window = D, Hq, Hk, Dh, window
        self.phi, self.b = n(4 * D, 24, std=0.02), n(24, std=0.1)
        self.alpha = torch.full((3,), 0.01, device=device)
        self.w_qkv = n(D, (Hq + 2 * Hk) * Dh, std=D ** -0.5).bfloat16()
        self.w_out = n(Hq * Dh, D, std=(Hq * Dh) ** -0.5).bfloat16()
        self.w_q, self.w_k = 1 + n(Dh, std=0.1), 1 + n(Dh, std=0.1)
        self.cos_sin = rope_table(max_pos, Dh, device=device)

    def plan(self, T, step, page):
        """The step's split over the GPU: one plan serves all layers."""
        return B.mhc_paged_attn_plan(step["cu_q"], step["kv_lens"], torch.bfloat16, T, self.Hq, self.Hk, self.Dh,
                                     page, step["max_q"], step["max_kv"], self.window)

    def __call__(self, x, pages, step, plan):
        """x [T, 4, D]: the residual streams of the step's tokens, sequence after
        sequence.  Returns them after the layer."""
        T, h, k = x.shape[0], self.Hq * self.Dh, self.Hk * self.Dh
        f = B.mhc_pre(x, self.phi, self.b, self.alpha)
        q, kk, v = (t.view(T, -1, self.Dh) for t in (f.x_in @ self.w_qkv).split([h, k, k], 1))
        q = B.mhc_qk_norm_rope_append(q, kk, v, self.w_q, self.w_k, pages.k, pages.v, step["slots"],
                                      positions=step["positions"], cos_sin=self.cos_sin)
        o = B.mhc_paged_attn(q, pages.k, pages.v, step["table"], plan=plan).o
        return B.mhc_post(x, o.view(T, h) @ self.w_out, f.H_post, f.H_res)


def serve(layer: ServedLayer, prompts, new, chunk, page=64):
    """Runs prompts [len, 4, D] in chunks of at most `chunk` tokens, then the
    tokens of `new` [sequences, steps, 4, D] one at a time.  Returns each
    sequence's states after the layer."""
    S, steps = len(prompts), new.shape[1]
    pages = Pages.make(S, max(len(p) for p in prompts) + steps, page, layer.Hk, layer.Dh)
    done, out = [0] * S, [[] for _ in range(S)]

    def run(parts):
        counts = [len(p) for p in parts]
        step = pages.step(counts)
        x = torch.cat(parts)
        y = layer(x, pages, step, layer.plan(len(x), step, page))
        for b, part in enumerate(y.split(counts)):
            out[b].append(part)

    while any(done[b] < len(prompts[b]) for b in range(S)):
        # a sequence whose prompt is through waits: it has no rows in this step
        parts = [p[done[b]:done[b] + chunk] for b, p in enumerate(prompts)]
        done = [d + len(p) for d, p in zip(done, parts)]
        run(parts)
    for i in range(steps):
        run([new[b, i:i + 1] for b in range(S)])
    return [torch.cat(o) for o in out]


def main():
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = ServedLayer()
    lens, steps = (300, 1, 129), 5
    streams = [torch.randn(n + steps, 4, layer.D, generator=g, device="cuda").bfloat16() for n in lens]
    new = torch.stack([s[n:] for s, n in zip(streams, lens)])
    served = serve(layer, [s[:n] for s, n in zip(streams, lens)], new, chunk=100)
    whole = serve(layer, streams, new[:, :0], chunk=10 ** 6)
    assert B.get_last_device_error() == B.MHC_OK
    worst = max(float((a - b).abs().max()) for a, b in zip(served, whole))
    size = math.sqrt(sum(float(a.float().square().mean()) for a in whole) / len(whole))
    print(f"served in chunks of 100 and single tokens against whole prompts: largest difference {worst:.3g} "
          f"of states of size {size:.3g}")


if __name__ == "__main__":
    main()
