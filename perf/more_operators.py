"""Cases of the operators around a step of speculative serving on the paged
cache, and of the rotation that both training and serving use:

  table    cosines and sines of scaled positions, for long contexts
  rope     the rotation alone (forward, backward, and into the paged cache)
  step     page tables, slots, positions and tree masks of a step's new tokens,
           from the lengths of its sequences
  tree     attention of a tree of drafted tokens over the cache
  keep     the accepted path's keys and values move behind the context

The widths are those of the layer's workloads: D = 5120 is 40 heads of 128,
D = 2560 is 20 heads of 128 or 40 of 64; T = 32768 and 1024 are its batches.
``run`` computes each operator in plain torch where ``own`` is false, and calls
the package where it is true.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a table for contexts 16 times as long as the model was trained on, scaled by parts
        dict(name="table 131072x128 by parts", op="table", rows=131072, rot=128, factor=16.0, original=8192,
             low=1.0, high=32.0, amplitude=1.25),
        # training forward of the large batch (T = 32768, D = 5120), packed documents of 4096 tokens
        dict(name="rope fwd bf16 T32768 h40", op="rope", dtype="bf16", t=32768, hq=40, hk=8, dh=128, rot=128,
             pairs="halves", doc=4096),
        # backward of a short ragged float32 batch, neighbouring pairs, half of each head
        dict(name="rope bwd f32 T1023 h20", op="rope_bwd", dtype="f32", t=1023, hq=20, hk=4, dh=128, rot=64,
             pairs="adjacent", doc=1023),
        # one new token for each of 64 sequences goes into the cache
        dict(name="rope append bf16 T64", op="append", dtype="bf16", t=64, hq=40, hk=8, dh=128, rot=128,
             pairs="halves", doc=1, page=64),
        # a decoding step of 64 sequences, one token each
        dict(name="step B64 decode", op="step", b=64, new="one", n=1, kv=8192, page=64, tree=0, mix=11),
        # a server's step: trees of 64 drafted tokens for most of 512 sequences, others decode or end
        dict(name="step B512 trees", op="step", b=512, new="mixed", n=64, kv=32768, page=16, tree=1, mix=12),
        # the smallest tree call: one sequence, 13 drafted tokens, a short context
        dict(name="tree B1 n13 kv777", op="tree", dtype="bf16", hq=40, hk=8, dh=128, page=64, b=1, n=13, kv=777,
             lens="equal", window=0, softcap=0.0, mix=1),
        # a batch of sequences of very different lengths, trees of up to 32
        dict(name="tree B32 n32 kv8192", op="tree", dtype="bf16", hq=40, hk=8, dh=128, page=64, b=32, n=32, kv=8192,
             lens="ragged", window=0, softcap=0.0, mix=2),
        # long contexts, wide trees
        dict(name="tree B4 n64 kv65536", op="tree", dtype="bf16", hq=40, hk=8, dh=128, page=128, b=4, n=64, kv=65536,
             lens="equal", window=0, softcap=0.0, mix=3),
        # float32, a window and capped scores, small pages
        dict(name="tree f32 B5 n21 w512 cap", op="tree", dtype="f32", hq=20, hk=4, dh=128, page=16, b=5, n=21,
             kv=3000, lens="ragged", window=512, softcap=30.0, mix=4),
        # one layer's caches after a step of one sequence
        dict(name="keep B1 L1", op="keep", dtype="bf16", hk=8, dh=128, page=64, b=1, n=13, kv=777, layers=1, path=4,
             mix=21),
        # all layers' caches after a step of a batch
        dict(name="keep B48 L16", op="keep", dtype="bf16", hk=8, dh=128, page=64, b=48, n=32, kv=400, layers=16,
             path=8, mix=22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """What a pass of the plain form moves, roughly, in float32 values."""
    op = case["op"]
    if op == "tree":
        return 6 * case["b"] * case["hq"] * case["n"] * case["kv"] + 4 * case["b"] * case["kv"] * case["hk"] * case["dh"]
    if op == "table":
        return 24 * case["rows"] * case["rot"]
    if op == "step":
        return 2000 * case["b"] * case["n"]
    if op == "keep":
        return case["layers"] * (4 * case["b"] * (case["kv"] + case["page"]) * case["hk"] * case["dh"] + 100000)
    return 12 * case["t"] * (case["hq"] + case["hk"]) * case["dh"]


def draw(rng):
    most = {c["op"]: 0 for c in listed()}
    for c in listed():
        most[c["op"]] = max(most[c["op"]], _cost(c))
    most["rope"] = most["rope_bwd"] = most["append"] = max(most["rope"], most["rope_bwd"], most["append"])
    while True:
        hq, hk, dh = rng.choice([(40, 8, 128), (20, 4, 128), (40, 8, 64), (16, 16, 64), (8, 1, 128), (12, 4, 96)])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        op = rng.choice(["table", "rope", "rope_bwd", "append", "step", "step", "tree", "tree", "tree", "tree", "keep",
                         "keep"])
        if op == "table":
            factor = rng.choice([1.0, 4.0, 8.0, 16.0, 2.5])
            case = dict(op=op, rows=_log(rng, 64, 131072), rot=rng.choice([32, 64, 96, 128]), factor=factor,
                        original=rng.choice([0, 4096, 8192]), low=1.0, high=rng.choice([4.0, 32.0]),
                        amplitude=rng.choice([1.0, 1.0, 1.25]))
        elif op == "step":
            case = dict(op=op, b=_log(rng, 1, 1024), new=rng.choice(["one", "mixed", "chunks"]), n=1,
                        kv=_log(rng, 64, 65536), page=rng.choice([16, 32, 64, 128, 48]), tree=0,
                        mix=rng.randrange(1 << 20))
            if case["new"] == "mixed":
                case.update(n=_log(rng, 2, 64), tree=1)
            elif case["new"] == "chunks":
                case.update(b=min(case["b"], 64), n=_log(rng, 16, 2048))
        elif op == "tree":
            case = dict(op=op, dtype=dtype, hq=hq, hk=hk, dh=dh, page=rng.choice([16, 32, 64, 128]), b=_log(rng, 1, 64),
                        n=_log(rng, 1, 128), kv=_log(rng, 160, 65536), lens=rng.choice(["ragged", "ragged", "equal"]),
                        window=rng.choice([0, 0, 0, _log(rng, 64, 4096)]), softcap=rng.choice([0.0, 0.0, 0.0, 30.0]),
                        mix=rng.randrange(1 << 20))
        elif op == "keep":
            n = _log(rng, 2, 64)
            case = dict(op=op, dtype=dtype, hk=hk, dh=dh, page=rng.choice([16, 32, 64, 128]), b=_log(rng, 1, 64), n=n,
                        kv=n + _log(rng, 1, 1024), layers=_log(rng, 1, 48), path=rng.randrange(1, n // 2 + 1),
                        mix=rng.randrange(1 << 20))
        else:
            case = dict(op=op, dtype=dtype, t=_log(rng, 1, 32768), hq=hq, hk=hk, dh=dh,
                        rot=rng.choice([dh, dh, dh // 2]), pairs=rng.choice(["halves", "halves", "adjacent"]),
                        doc=_log(rng, 16, 8192))
            if op == "append":
                case["page"] = rng.choice([16, 32, 64, 128])
        if _cost(case) <= most[op] and (dtype == "bf16" or op != "tree" or work(case)["flops"] <= 4e11):
            return case


# ------------------------------------------------- lengths and trees of a case

def _parents(r, n):
    """A tree of n drafted tokens in the order of their drafting: the first
    follows the context, each other one an earlier token."""
    return [-1 if i == 0 else r.randrange(max(0, i - 8), i) for i in range(n)]


def _lens(case):
    """(drafted tokens, cached tokens including them) of each sequence."""
    r = random.Random(case["mix"])
    out = []
    for i in range(case["b"]):
        if case["lens"] == "equal" or i == 0:
            n, m = case["n"], case["kv"]
        else:
            n = r.randrange(max(1, case["n"] // 2), case["n"] + 1)
            m = max(n, _log(r, max(1, case["kv"] // 32), case["kv"]))
        out.append((n, max(n, m)))
    return out


def _trees(case):
    r = random.Random(case["mix"] + 1)
    return [_parents(r, n) for n, _ in _lens(case)]


def _ancestry(parents):
    """For each node the nodes it sees (itself and its ancestors) as one integer's bits."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits


def _words(bits, width):
    """Bits as `width` signed 32-bit words."""
    out = []
    for w in range(width):
        x = bits >> 32 * w & 0xFFFFFFFF
        out.append(x - (1 << 32) if x >> 31 else x)
    return out


def _new_lens(case):
    """New tokens of each sequence of a step, -1 for one that ends."""
    r = random.Random(case["mix"])
    out = []
    for i in range(case["b"]):
        if case["new"] == "one":
            out.append(1)
        elif case["new"] == "chunks":
            out.append(1 if i % 2 else _log(r, max(1, case["n"] // 8), case["n"]))
        else:
            kind = r.randrange(10) if i else 5
            out.append(-1 if kind == 0 else 0 if kind == 1 else 1 if kind < 4 else
                       r.randrange(max(1, case["n"] // 2), case["n"] + 1))
    return out


def work(case):
    op = case["op"]
    if op == "table":
        return {"bytes": 4 * case["rows"] * case["rot"], "flops": 8.0 * case["rows"] * case["rot"]}
    if op == "step":
        t, b = sum(max(0, n) for n in _new_lens(case)), case["b"]
        tree = t * (4 + 4 * -(-case["n"] // 32)) if case["tree"] else 0
        return {"bytes": 12 * t + 24 * b + tree, "flops": 4.0 * t}
    e = 2 if case["dtype"] == "bf16" else 4
    hk, dh = case["hk"], case["dh"]
    if op == "keep":
        moved = case["b"] * (case["path"] - 1)          # the first of a path stays where it is
        return {"bytes": case["layers"] * 4 * moved * hk * dh * e + 4 * case["b"] * (case["path"] + 3), "flops": 0.0}
    hq = case["hq"]
    if op == "tree":
        t = pairs = keys = 0
        for (n, m), tree in zip(_lens(case), _trees(case)):
            seen = [bin(b).count("1") for b in _ancestry(tree)]
            if case["window"]:
                pairs += sum(s + min(m - n, max(0, case["window"] - s)) for s in seen)
                keys += min(m, n + case["window"])
            else:
                pairs += sum(seen) + n * (m - n)
                keys += m
            t += n
        return {"bytes": e * dh * (2 * t * hq + 2 * keys * hk) + 4 * t * hq, "flops": 4.0 * dh * hq * pairs}
    t = case["t"]
    rows = t * (hq + hk) * dh
    table = 4 * min(t, case["doc"]) * case["rot"]
    if op == "append":
        return {"bytes": 2 * (rows + t * hk * dh) * e + table, "flops": 3.0 * rows}
    return {"bytes": 2 * rows * e + table, "flops": 3.0 * rows}


# -------------------------------------------------------------------- inputs

def _randn(gen, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
    return x.to(dtype)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _paged(gen, need, pages):
    """A page table of `need[b]` pages each, in random order, and what is left over."""
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(need), max(need + [1])), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, order[at:]


def _prepare_step(case, seed, gen, s):
    r = random.Random(seed)
    page, new = case["page"], _new_lens(case)
    lens = [r.randrange(max(1, case["kv"] // 32), case["kv"] + 1) for _ in new]
    width = -(-(case["kv"] + max(case["n"], 1)) // page)
    held = [-(-m // page) for m in lens]
    # a server keeps a few pages free; some of a step's sequences may find none
    wanted = sum(max(0, -(-(m + n) // page) - h) for m, n, h in zip(lens, new, held) if n > 0)
    spare = wanted + 5 if r.random() < 0.8 else wanted // 2
    table, rest = _paged(gen, held, sum(held) + spare)
    s["page_table"] = torch.full((case["b"], width), -1, dtype=torch.int32, device="cuda")
    s["page_table"][:, :table.shape[1]] = table
    s["free_pages"] = torch.zeros(sum(held) + spare, dtype=torch.int32, device="cuda")
    s["free_pages"][:spare] = rest
    s["free_count"] = _ints([spare])
    s["lens"], s["held"], s["new_lens"] = _ints(lens), _ints(held), _ints(new)
    s["t"] = sum(max(0, n) for n in new)
    s["width"] = -(-case["n"] // 32)
    if case["tree"]:
        s["parents"] = _ints([p for n in new for p in _parents(r, max(0, n))])
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "table":
        s["base"] = 10000.0 * (1.0 + (seed % 97) / 97.0)      # a model's own
        return s
    if op == "step":
        return _prepare_step(case, seed, gen, s)
    dt = DTYPES[case["dtype"]]
    hk, dh = case["hk"], case["dh"]
    if op == "tree":
        hq, page, lens = case["hq"], case["page"], _lens(case)
        t, need = sum(n for n, _ in lens), [-(-m // page) for _, m in lens]
        pages = sum(need) + 7                          # a cache a little larger than what is in use
        s["q"] = _randn(gen, (t, hq, dh), dt, 1.5)
        s["k_cache"] = _randn(gen, (pages, page, hk, dh), dt, 1.5)
        s["v_cache"] = _randn(gen, (pages, page, hk, dh), dt, 0.5)
        s["page_table"], _ = _paged(gen, need, pages)
        cu = [0]
        for n, _ in lens:
            cu.append(cu[-1] + n)
        s["cu_q"], s["kv_lens"] = _ints(cu), _ints([m for _, m in lens])
        s["max_q"], s["max_kv"] = max(n for n, _ in lens), max(m for _, m in lens)
        width = -(-s["max_q"] // 32)
        s["tree"] = _ints([_words(b, width) for p in _trees(case) for b in _ancestry(p)])
        return s
    if op == "keep":
        r, page, b, n, m = random.Random(seed), case["page"], case["b"], case["n"], case["kv"]
        need = [-(-m // page)] * b
        pages = sum(need) + 3
        shape = (pages, page, hk, dh)
        s["k_caches"] = [_randn(gen, shape, dt) for _ in range(case["layers"])]
        s["v_caches"] = [_randn(gen, shape, dt) for _ in range(case["layers"])]
        s["page_table"], _ = _paged(gen, need, pages)
        s["cu_q"], s["kv_lens"] = _ints([i * n for i in range(b + 1)]), _ints([m] * b)
        # a tree's first token is accepted by itself; the others of the path lie behind its place
        c = case["path"]
        s["path"] = _ints([[0] + sorted(r.sample(range(c, n), c - 1)) for _ in range(b)])
        s["keep"] = _ints([c] * b)
        s["lens"] = _ints([m - n] * b)
        return s
    t, rot, hq = case["t"], case["rot"], case["hq"]
    first = 0 if t > 1 else seed % 8192
    s["positions"] = (torch.arange(t, device="cuda") % case["doc"] + first).to(torch.int32)
    if op == "append" and case["doc"] == 1:            # decoding: every sequence at its own position
        s["positions"] = torch.randint(0, 8192, (t,), generator=gen, device="cuda").to(torch.int32)
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(max(8192, case["doc"]) + 1, dtype=torch.float64, device="cuda")[:, None] * freq
    s["cos_sin"] = torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()     # [n, rot]: cosines, then sines
    if op == "rope_bwd":
        s["g_q"], s["g_k"] = _randn(gen, (t, hq, dh), dt), _randn(gen, (t, hk, dh), dt)
        return s
    s["qkv"] = _randn(gen, (t, (hq + 2 * hk) * dh), dt)     # what the packed projection leaves
    if op == "append":
        page = case["page"]
        pages = -(-t // page) + 3
        s["k_cache"] = _randn(gen, (pages, page, hk, dh), dt)
        s["v_cache"] = _randn(gen, (pages, page, hk, dh), dt)
        order = torch.randperm(pages, generator=gen, device="cuda")
        i = torch.arange(t, device="cuda")
        s["slots"] = (order[i // page] * page + i % page).to(torch.int64)
    return s


def _split(s):
    c = s["case"]
    t, hq, hk, dh = c["t"], c["hq"], c["hk"], c["dh"]
    q, k, v = s["qkv"].split([hq * dh, hk * dh, hk * dh], dim=1)
    return q.view(t, hq, dh), k.view(t, hk, dh), v.view(t, hk, dh)


# ---------------------------------------------------------------- plain forms

def _plain_table(s):
    c = s["case"]
    f = s["base"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
    turns = c["original"] * f / (2.0 * math.pi)                 # of a pair over the trained length
    keep = ((turns - c["low"]) / (c["high"] - c["low"])).clamp(0.0, 1.0)
    f = f * (keep + (1.0 - keep) / c["factor"])
    a = torch.arange(c["rows"], dtype=torch.float64, device="cuda")[:, None] * f
    return (c["amplitude"] * torch.cat([a.cos(), a.sin()], dim=1)).float()


def _rotate(x, s, back=False):
    """Rotates the first `rot` values of each head by the position's angles."""
    c, x = s["case"], x.float()
    rot = c["rot"]
    cos, sin = s["cos_sin"][s["positions"].long()][:, None].split(rot // 2, dim=-1)
    if back:
        sin = -sin
    r, rest = x[..., :rot], x[..., rot:]
    if c["pairs"] == "adjacent":
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r.split(rot // 2, dim=-1)
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, rest], dim=-1)


def _plain_step(s):
    c, page = s["case"], s["case"]["page"]
    table, held, free, count = s["page_table"], s["held"], s["free_pages"], s["free_count"]
    lens, new = s["lens"].long(), s["new_lens"].long()
    over, n = new < 0, new.clamp(min=0)
    b, width = table.shape
    have = held.long()
    # the pages of sequences that end go back on top of the free ones
    col = torch.arange(width, device="cuda")
    back = over[:, None] & (col < have[:, None])
    at = count.long() + (back.flatten().cumsum(0) - 1)
    top = free.numel()
    stack = torch.cat([free, free.new_zeros(1)])
    stack[torch.where(back.flatten(), at, top)] = table.flatten()
    have = torch.where(over, 0, have)
    avail = count.long() + back.sum()
    # each sequence's missing pages, from the top; it gets all of them or none
    need = torch.where(over, 0, (-(-(lens + n) // page) - have).clamp(min=0))
    upto = need.cumsum(0)
    served = ~over & ((need == 0) | (upto <= avail))
    take = torch.where(served, need, 0)
    want = served[:, None] & (col >= have[:, None]) & (col < (have + take)[:, None])
    src = avail - 1 - (upto - need)[:, None] - (col - have[:, None])
    table.copy_(torch.where(want, stack[src.clamp(0, top)], table))
    left = avail - take.sum()
    idx = torch.arange(top, device="cuda")
    free.copy_(torch.where((idx >= count) & (idx < left), stack[:top], free))
    held.copy_((have + take).to(torch.int32))
    count.copy_(left.to(torch.int32))
    kv = torch.where(over, 0, torch.where(served, lens + n, lens))
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    tok = torch.arange(s["t"], device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[seq]
    place = lens[seq] + i
    slots = table[seq, (place // page).clamp(max=width - 1)].long() * page + place % page
    out = {"cu_q": cu.to(torch.int32), "kv_lens": kv.to(torch.int32), "slots": torch.where(served[seq], slots, -1)}
    if c["tree"]:
        # parents all the way up, one level of the trees at a time
        par = s["parents"].long()
        bits = torch.zeros((s["t"], 32 * s["width"]), dtype=torch.bool, device="cuda")
        depth, node = torch.zeros_like(tok), i.clone()
        for _ in range(c["n"]):
            live = node >= 0
            bits[tok, node.clamp(min=0)] |= live
            depth += live
            node = torch.where(live, par[cu[seq] + node.clamp(min=0)], -1)
        w = bits.view(s["t"], s["width"], 32).long() << torch.arange(32, device="cuda")
        w = w.sum(-1)
        out["tree"] = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
        place = lens[seq] + depth - 1
    out["positions"] = place.to(torch.int32)
    out.update(page_table=table, held=held, free_count=count)
    return out


def _plain_tree(s):
    c = s["case"]
    q, kv_lens, cu = s["q"], s["kv_lens"].long(), s["cu_q"].long()
    t, hq, dh = q.shape
    hk, b, mq, mk = c["hk"], c["b"], s["max_q"], s["max_kv"]
    g = hq // hk
    row = torch.arange(mq, device="cuda")
    key = torch.arange(mk, device="cuda")
    q_lens = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + row).clamp(max=t - 1)
    qp = q[at].float().view(b, mq, hk, g, dh).permute(0, 2, 3, 1, 4).reshape(b, hk, g * mq, dh)

    def cached(cache):
        x = cache[s["page_table"].long()].flatten(1, 2)[:, :mk].float()
        return x.masked_fill((key >= kv_lens[:, None])[..., None, None], 0.0)

    sc = qp @ cached(s["k_cache"]).permute(0, 2, 3, 1)
    sc = sc * (1.0 / math.sqrt(dh))
    if c["softcap"] > 0:
        sc = c["softcap"] * torch.tanh(sc / c["softcap"])
    node = torch.arange(mq, device="cuda")
    bits = (s["tree"][:, node // 32] >> (node % 32) & 1).bool()[at]           # [b, mq, mq]
    ctx = kv_lens - q_lens
    seen = (key < ctx[:, None])[:, None].expand(b, mq, mk)
    if c["window"]:
        seen = seen & (key >= (ctx[:, None] + bits.sum(-1) - c["window"])[..., None])
    j = key - ctx[:, None]                                                    # drafted token of a key
    drafted = bits.gather(2, j.clamp(0, mq - 1)[:, None].expand(b, mq, mk))
    seen = torch.where(((j >= 0) & (j < q_lens[:, None]))[:, None], drafted, seen) & (row < q_lens[:, None])[..., None]
    sc = sc.view(b, hk, g, mq, mk).masked_fill(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.masked_fill(m == -math.inf, 0.0))
    del sc
    l = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, g * mq, mk) @ cached(s["v_cache"]).permute(0, 2, 1, 3)).view(b, hk, g, mq, dh)
    o = o / l.masked_fill(l == 0, 1.0)
    lse = (m + torch.log(l)).squeeze(-1)
    tok = torch.arange(t, device="cuda")
    seq = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[seq]
    o = o.permute(0, 3, 1, 2, 4).reshape(b, mq, hq, dh)[seq, i]
    lse = lse.permute(0, 3, 1, 2).reshape(b, mq, hq)[seq, i]
    return {"o": o.to(q.dtype), "lse": lse}


def _plain_keep(s):
    page = s["case"]["page"]
    path, keep = s["path"].long(), s["keep"].long()
    cu = s["cu_q"].long()
    ctx = (s["kv_lens"].long() - (cu[1:] - cu[:-1]))[:, None]
    d = torch.arange(path.shape[1], device="cuda")
    on = d < keep[:, None]

    def slot(j):
        return (s["page_table"].long().gather(1, j // page) * page + j % page)[on]

    src, dst = slot(ctx + torch.where(on, path, 0)), slot(ctx + torch.where(on, d, 0))
    for cache in (*s["k_caches"], *s["v_caches"]):
        flat = cache.view(-1, *cache.shape[2:])
        flat[dst] = flat[src]
    s["lens"].copy_((ctx[:, 0] + keep).to(torch.int32))
    return {"k": s["k_caches"], "v": s["v_caches"], "lens": s["lens"]}


def _plain(s):
    op = s["case"]["op"]
    if op == "table":
        return {"cos_sin": _plain_table(s)}
    if op == "step":
        return _plain_step(s)
    if op == "tree":
        return _plain_tree(s)
    if op == "keep":
        return _plain_keep(s)
    dt = DTYPES[s["case"]["dtype"]]
    if op == "rope_bwd":
        return {"dq": _rotate(s["g_q"], s, back=True).to(dt), "dk": _rotate(s["g_k"], s, back=True).to(dt)}
    q, k, v = _split(s)
    qr, kr = _rotate(q, s).to(dt), _rotate(k, s).to(dt)
    if op == "rope":
        return {"q": qr, "k": kr}
    s["k_cache"].flatten(0, 1)[s["slots"]] = kr
    s["v_cache"].flatten(0, 1)[s["slots"]] = v
    return {"q": qr, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# -------------------------------------------------------------- the package

def _package(s):
    from mhc_pre_gb300 import binding as B
    c = s["case"]
    op = c["op"]
    if op == "table":
        return {"cos_sin": B.mhc_rope_table(c["rows"], c["rot"], base=s["base"], factor=c["factor"],
                                            original=c["original"], low=c["low"], high=c["high"],
                                            amplitude=c["amplitude"])}
    if op == "step":
        r = B.mhc_paged_step(s["new_lens"], s["lens"], s["page_table"], s["held"], s["free_pages"], s["free_count"],
                             page_size=c["page"], T=s["t"], parents=s.get("parents"), width=s["width"])
        out = {"cu_q": r.cu_q, "kv_lens": r.kv_lens, "slots": r.slots}
        if c["tree"]:
            out["tree"] = r.tree
        out["positions"] = r.positions
        out.update(page_table=s["page_table"], held=s["held"], free_count=s["free_count"])
        return out
    if op == "tree":
        r = B.mhc_tree_attn(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["tree"], s["cu_q"], s["kv_lens"],
                            max_q=s["max_q"], max_kv=s["max_kv"], window=c["window"], softcap=c["softcap"])
        return {"o": r.o, "lse": r.lse}
    if op == "keep":
        B.mhc_cache_keep(s["k_caches"], s["v_caches"], s["page_table"], s["cu_q"], s["kv_lens"], s["path"], s["keep"],
                         lens=s["lens"])
        return {"k": s["k_caches"], "v": s["v_caches"], "lens": s["lens"]}
    rope = dict(positions=s["positions"], cos_sin=s["cos_sin"], interleaved=c["pairs"] == "adjacent")
    if op == "rope_bwd":
        r = B.mhc_rope_bwd(s["g_q"], s["g_k"], **rope)
        return {"dq": r.q, "dk": r.k}
    q, k, v = _split(s)
    if op == "rope":
        r = B.mhc_rope(q, k, **rope)
        return {"q": r.q, "k": r.k}
    qr = B.mhc_rope_append(q, k, v, s["k_cache"], s["v_cache"], s["slots"], **rope)
    return {"q": qr, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    return _package(state) if own else _plain(state)


# ------------------------------------------------------------- 64-bit values

def _exact_table(case, s):
    cols = []
    for part in (torch.cos, torch.sin):
        for j in range(case["rot"] // 2):
            f = s["base"] ** (-2.0 * j / case["rot"])
            turns = case["original"] * f / (2.0 * math.pi)
            g = min(1.0, max(0.0, (turns - case["low"]) / (case["high"] - case["low"])))
            f = (1.0 - g) * f / case["factor"] + g * f
            cols.append(case["amplitude"] * part(torch.arange(case["rows"], dtype=torch.float64, device="cuda") * f))
    return {"cos_sin": torch.stack(cols, dim=1)}


def _exact_turn(x, s, back=False):
    """Heads [T, H, dh] turned as complex numbers."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    y = x.double().clone()
    tab = s["cos_sin"].double()[s["positions"].long()]
    by = torch.complex(tab[:, :half], -tab[:, half:] if back else tab[:, half:])[:, None]
    if c["pairs"] == "adjacent":
        z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * by
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :half], y[..., half:rot]) * by
        y[..., :half], y[..., half:rot] = z.real, z.imag
    return y


def _exact_step(case, s):
    """One sequence after the other, on the host."""
    page = case["page"]
    new, lens, held = s["new_lens"].tolist(), s["lens"].tolist(), s["held"].tolist()
    table, free = s["page_table"].tolist(), s["free_pages"].tolist()[:int(s["free_count"])]
    for b, n in enumerate(new):
        if n < 0:
            free += table[b][:held[b]]
            held[b] = 0
    cu, kv, slots, positions, tree = [0], [], [], [], []
    parents = s["parents"].tolist() if case["tree"] else None
    full = False                     # a sequence found too few pages: none are left for later ones
    for b, n in enumerate(new):
        n_new, m = max(0, n), lens[b]
        need = 0 if n < 0 else max(0, -(-(m + n_new) // page) - held[b])
        served = n >= 0 and (need == 0 or (not full and need <= len(free)))
        full = full or (need > 0 and not served)
        if served:
            for _ in range(need):
                table[b][held[b]] = free.pop()
                held[b] += 1
        kv.append(0 if n < 0 else m + n_new if served else m)
        mine = _ancestry(parents[cu[-1]:cu[-1] + n_new]) if parents is not None else None
        for i in range(n_new):
            slots.append(table[b][(m + i) // page] * page + (m + i) % page if served else -1)
            if mine is None:
                positions.append(m + i)
            else:
                positions.append(m + bin(mine[i]).count("1") - 1)
                tree.append(_words(mine[i], s["width"]))
        cu.append(cu[-1] + n_new)
    out = {"cu_q": _ints(cu), "kv_lens": _ints(kv), "slots": _ints(slots, torch.int64)}
    if case["tree"]:
        out["tree"] = _ints(tree)
    out["positions"] = _ints(positions)
    out.update(page_table=_ints(table), held=_ints(held), free_count=_ints([len(free)]))
    return out


def _exact_tree(case, s):
    hq, hk, dh, page = case["hq"], case["hk"], case["dh"], case["page"]
    g = hq // hk
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, ((n, m), parents) in enumerate(zip(_lens(case), _trees(case))):
        pages = s["page_table"][b, : -(-m // page)].long()
        ancestors = _ancestry(parents)
        hidden = torch.zeros((n, m), dtype=torch.bool)
        for i, bits in enumerate(ancestors):
            if case["window"]:
                hidden[i, :max(0, min(m - n, m - n + bin(bits).count("1") - case["window"]))] = True
            hidden[i, m - n:] = torch.tensor([not bits >> j & 1 for j in range(n)])
        hidden = hidden.cuda()
        for h in range(hk):
            kk = s["k_cache"][pages, :, h].reshape(-1, dh)[:m].double()
            vv = s["v_cache"][pages, :, h].reshape(-1, dh)[:m].double()
            for r in range(g):
                z = s["q"][at:at + n, h * g + r].double() @ kk.T / math.sqrt(dh)
                if case["softcap"] > 0:
                    z = case["softcap"] * torch.tanh(z / case["softcap"])
                z[hidden] = -math.inf
                e = torch.logsumexp(z, dim=1)
                lse[at:at + n, h * g + r] = e
                o[at:at + n, h * g + r] = torch.exp(z - e[:, None]) @ vv
        at += n
    return {"o": o, "lse": lse}


def _exact_keep(case, s):
    page, n = case["page"], case["n"]
    table, path, keep = s["page_table"].tolist(), s["path"].tolist(), s["keep"].tolist()
    lens = []
    for b, m in enumerate(s["kv_lens"].tolist()):
        for d in range(keep[b]):
            (pa, ia), (pb, ib) = divmod(m - n + path[b][d], page), divmod(m - n + d, page)
            for cache in (*s["k_caches"], *s["v_caches"]):
                cache[table[b][pb], ib] = cache[table[b][pa], ia]
        lens.append(m - n + keep[b])
    return {"k": s["k_caches"], "v": s["v_caches"], "lens": _ints(lens)}


def exact(case, seed):
    op = case["op"]
    # a whole square of scores is formed for each sequence: above this it takes too long in 64 bits
    if op == "tree" and sum(n * m for n, m in _lens(case)) * case["hq"] * (4 * case["dh"] + 60) > 4e12:
        return None
    # one copy at a time
    if op == "keep" and 2 * case["layers"] * case["b"] * case["path"] > 60000:
        return None
    s = prepare(case, seed)
    if op == "table":
        return _exact_table(case, s)
    if op == "step":
        return _exact_step(case, s)
    if op == "tree":
        return _exact_tree(case, s)
    if op == "keep":
        return _exact_keep(case, s)
    if op == "rope_bwd":
        return {"dq": _exact_turn(s["g_q"], s, True), "dk": _exact_turn(s["g_k"], s, True)}
    q, k, v = _split(s)
    qr, kr = _exact_turn(q, s), _exact_turn(k, s)
    if op == "rope":
        return {"q": qr, "k": kr}
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    page = case["page"]
    where, slot = s["slots"] // page, s["slots"] % page
    kc[where, slot], vc[where, slot] = kr, v.double()
    return {"q": qr, "k_cache": kc, "v_cache": vc}
