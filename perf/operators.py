"""Cases of the attention-sublayer operators: per-head query/key normalisation
with the position rotation (forward, backward, and the serving form that
writes a paged cache), and attention of a chunk of new tokens over that cache.

The widths are those of the layer's workloads: D = 5120 is 40 heads of 128,
D = 2560 is 20 heads of 128 or 40 of 64; T = 32768, 4096, 2048 and 1024 are its
batches.  ``run`` computes each operator in plain float32 torch where ``own``
is false, and calls the package where it is true.
"""

from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6
ROPE_BASE = 10000.0
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # training forward of the large batch (T = 32768, D = 5120), packed documents of 4096 tokens
        dict(name="qk fwd bf16 T32768 h40", op="qk", dtype="bf16", t=32768, hq=40, hk=8, dh=128, rot=128,
             pairs="halves", doc=4096),
        # a short ragged float32 batch, adjacent-pair rotation of half of each head
        dict(name="qk fwd f32 T1023 h20", op="qk", dtype="f32", t=1023, hq=20, hk=4, dh=128, rot=64,
             pairs="adjacent", doc=1023),
        # training backward of the large batch
        dict(name="qk bwd bf16 T32768 h40", op="qk_bwd", dtype="bf16", t=32768, hq=40, hk=8, dh=128, rot=128,
             pairs="halves", doc=4096),
        # backward of a small fine-tuning batch, as many key heads as query heads, heads of 64
        dict(name="qk bwd bf16 T1000 h16", op="qk_bwd", dtype="bf16", t=1000, hq=16, hk=16, dh=64, rot=64,
             pairs="halves", doc=250),
        # one new token of one sequence: pure latency
        dict(name="append bf16 T1", op="append", dtype="bf16", t=1, hq=40, hk=8, dh=128, rot=128,
             pairs="halves", doc=1, page=64),
        # a prompt chunk going into the cache
        dict(name="append bf16 T4096", op="append", dtype="bf16", t=4096, hq=40, hk=8, dh=128, rot=128,
             pairs="halves", doc=4096, page=64),
        # one token over a short context: the smallest attention call
        dict(name="attn decode B1 kv777", op="attn", dtype="bf16", hq=40, hk=8, dh=128, page=64, b=1, q=1,
             kv=777, lens="equal", window=0, softcap=0.0, mix=1),
        # a decode batch of 64 sequences of very different lengths
        dict(name="attn decode B64 kv8192", op="attn", dtype="bf16", hq=40, hk=8, dh=128, page=64, b=64, q=1,
             kv=8192, lens="decode", window=0, softcap=0.0, mix=2),
        # long contexts, two tokens each (one drafted)
        dict(name="attn decode B4 kv131072", op="attn", dtype="bf16", hq=40, hk=8, dh=128, page=128, b=4, q=2,
             kv=131072, lens="equal", window=0, softcap=0.0, mix=3),
        # a chunk of a long prompt over what is cached already
        dict(name="attn chunk 2048 kv32768", op="attn", dtype="bf16", hq=40, hk=8, dh=128, page=64, b=1, q=2048,
             kv=32768, lens="equal", window=0, softcap=0.0, mix=4),
        # whole prompts of odd lengths with a 512-token window and capped scores, heads of 64, small pages
        dict(name="attn prompts B5 w512 cap", op="attn", dtype="bf16", hq=40, hk=8, dh=64, page=16, b=5, q=4096,
             kv=4096, lens="prompt", window=512, softcap=30.0, mix=5),
        # prompt chunks and single tokens in one float32 batch
        dict(name="attn mixed f32 B6", op="attn", dtype="f32", hq=20, hk=4, dh=128, page=32, b=6, q=300,
             kv=2000, lens="mixed", window=0, softcap=0.0, mix=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    """What a pass of the plain form moves, roughly, in float32 values."""
    if case["op"] == "attn":
        return 6 * case["b"] * case["hq"] * case["q"] * case["kv"] + 4 * case["b"] * case["kv"] * case["hk"] * case["dh"]
    return 12 * case["t"] * (case["hq"] + case["hk"]) * case["dh"]


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        hq, hk, dh = rng.choice([(40, 8, 128), (20, 4, 128), (40, 8, 64), (16, 16, 64), (8, 1, 128), (12, 4, 96)])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        op = rng.choice(["qk", "qk_bwd", "append", "attn", "attn", "attn"])
        if op == "attn":
            lens = rng.choice(["decode", "mixed", "prompt", "equal"])
            case = dict(op=op, dtype=dtype, hq=hq, hk=hk, dh=dh, page=rng.choice([16, 32, 64, 128]), lens=lens,
                        window=rng.choice([0, 0, 0, _log(rng, 64, 4096)]), softcap=rng.choice([0.0, 0.0, 0.0, 30.0]),
                        mix=rng.randrange(1 << 20))
            if lens == "decode":
                case.update(b=_log(rng, 1, 128), q=rng.choice([1, 1, 2, 4]), kv=_log(rng, 64, 65536))
            elif lens == "mixed":
                case.update(b=_log(rng, 2, 24), q=_log(rng, 16, 1024), kv=_log(rng, 1024, 16384))
            elif lens == "prompt":
                n = _log(rng, 16, 8192)
                case.update(b=_log(rng, 1, 8), q=n, kv=n)
            else:
                n = _log(rng, 16, 4096)
                case.update(b=_log(rng, 1, 4), q=n, kv=n + _log(rng, 1, 32768))
        else:
            case = dict(op=op, dtype=dtype, t=_log(rng, 1, 32768), hq=hq, hk=hk, dh=dh,
                        rot=rng.choice([dh, dh, dh // 2]), pairs=rng.choice(["halves", "halves", "adjacent"]),
                        doc=_log(rng, 16, 8192))
            if op == "append":
                case["page"] = rng.choice([16, 32, 64, 128])
        if _cost(case) <= most and (dtype == "bf16" or op != "attn" or work(case)["flops"] <= 4e11):
            return case


def _lens(case):
    """(new tokens, cached tokens including them) of each sequence."""
    r = random.Random(case["mix"])
    b, q, kv, kind = case["b"], case["q"], case["kv"], case["lens"]
    out = []
    for i in range(b):
        if kind == "equal" or i == 0:
            n, m = q, kv
        elif kind == "decode":
            n, m = q, max(q, _log(r, max(1, kv // 32), kv))
        elif kind == "prompt":
            n = m = _log(r, max(1, q // 16), q)
        else:  # a step of a server: half the sequences decode, the others bring a chunk
            n = 1 if i % 2 else _log(r, max(1, q // 8), q)
            m = max(n, _log(r, max(1, kv // 16), kv))
        out.append((n, m))
    return out


def _pairs_seen(case):
    """(query, key) pairs that the mask leaves."""
    total, w = 0, case["window"]
    for n, m in _lens(case):
        first = m - n + 1                       # keys that the first query sees without a window
        if w == 0 or m <= w:
            total += n * first + n * (n - 1) // 2
        else:
            below = min(n, max(0, w - first))   # queries that see fewer than w keys
            total += below * first + below * (below - 1) // 2 + (n - below) * w
    return total


def _keys_read(case):
    w = case["window"]
    return sum(m if w == 0 else min(m, w + n - 1) for n, m in _lens(case))


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hk, dh = case["hq"], case["hk"], case["dh"]
    if case["op"] == "attn":
        t = sum(n for n, _ in _lens(case))
        return {"bytes": e * dh * (2 * t * hq + 2 * _keys_read(case) * hk) + 4 * t * hq,
                "flops": 4.0 * dh * hq * _pairs_seen(case)}
    t = case["t"]
    rows = t * (hq + hk) * dh
    table = 4 * min(t, case["doc"]) * case["rot"]
    if case["op"] == "qk":
        return {"bytes": 2 * rows * e + table, "flops": 8.0 * rows}
    if case["op"] == "qk_bwd":
        return {"bytes": 3 * rows * e + table, "flops": 16.0 * rows}
    return {"bytes": 2 * (rows + t * hk * dh) * e + table, "flops": 8.0 * rows}


# -------------------------------------------------------------------- inputs

def _randn(gen, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
    return x.to(dtype)


def _rope_table(n, rot):
    freq = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], dim=1).float().contiguous()      # [n, rot]: cosines, then sines


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    hq, hk, dh = case["hq"], case["hk"], case["dh"]
    s = dict(case=case)
    if case["op"] == "attn":
        lens, page = _lens(case), case["page"]
        t, need = sum(n for n, _ in lens), [-(-m // page) for _, m in lens]
        pages = sum(need) + 7                      # a cache a little larger than what is in use
        s["q"] = _randn(gen, (t, hq, dh), dt, 1.5)
        s["k_cache"] = _randn(gen, (pages, page, hk, dh), dt, 1.5)
        s["v_cache"] = _randn(gen, (pages, page, hk, dh), dt, 0.5)
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros((case["b"], max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        s["page_table"] = table
        cu = [0]
        for n, _ in lens:
            cu.append(cu[-1] + n)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["kv_lens"] = torch.tensor([m for _, m in lens], dtype=torch.int32, device="cuda")
        s["max_q"], s["max_kv"] = max(n for n, _ in lens), max(m for _, m in lens)
        return s
    t, rot = case["t"], case["rot"]
    s["qkv"] = _randn(gen, (t, (hq + 2 * hk) * dh), dt)     # what the packed projection leaves
    s["w_q"] = 1.0 + _randn(gen, (dh,), torch.float32, 0.2)
    s["w_k"] = 1.0 + _randn(gen, (dh,), torch.float32, 0.2)
    first = 0 if t > 1 else seed % 8192
    s["positions"] = (torch.arange(t, device="cuda") % case["doc"] + first).to(torch.int32)
    s["cos_sin"] = _rope_table(max(8192, case["doc"]) + 1, rot)
    if case["op"] == "qk_bwd":
        s["g_q"], s["g_k"] = _randn(gen, (t, hq, dh), dt), _randn(gen, (t, hk, dh), dt)
    if case["op"] == "append":
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


# ---------------------------------------------------------------- plain form

def _rotate(x, cos_sin, positions, rot, adjacent, back=False):
    """Rotates the first `rot` values of each head by the position's angles."""
    cos, sin = cos_sin[positions.long()][:, None].split(rot // 2, dim=-1)
    if back:
        sin = -sin
    r, rest = x[..., :rot], x[..., rot:]
    if adjacent:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r.split(rot // 2, dim=-1)
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, rest], dim=-1)


def _norm_rotate(x, w, s):
    c = s["case"]
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
    return _rotate(y, s["cos_sin"], s["positions"], c["rot"], c["pairs"] == "adjacent")


def _norm_rotate_bwd(g, x, w, s):
    c = s["case"]
    g = _rotate(g.float(), s["cos_sin"], s["positions"], c["rot"], c["pairs"] == "adjacent", back=True)
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh = x * r
    gw = g * w
    return r * (gw - xh * (gw * xh).mean(-1, keepdim=True)), (g * xh).sum((0, 1))


def _plain_attn(s):
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
    pos = (kv_lens - q_lens)[:, None] + row                                   # [b, mq]
    seen = (key <= pos[..., None]) & (row < q_lens[:, None])[..., None]
    if c["window"]:
        seen = seen & (key > pos[..., None] - c["window"])
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


def _plain(s):
    op = s["case"]["op"]
    if op == "attn":
        return _plain_attn(s)
    q, k, v = _split(s)
    if op == "qk_bwd":
        dq, dw_q = _norm_rotate_bwd(s["g_q"], q, s["w_q"], s)
        dk, dw_k = _norm_rotate_bwd(s["g_k"], k, s["w_k"], s)
        return {"dq": dq.to(q.dtype), "dk": dk.to(q.dtype), "dw_q": dw_q, "dw_k": dw_k}
    qn = _norm_rotate(q, s["w_q"], s).to(q.dtype)
    kn = _norm_rotate(k, s["w_k"], s).to(q.dtype)
    if op == "qk":
        return {"q": qn, "k": kn}
    s["k_cache"].flatten(0, 1)[s["slots"]] = kn
    s["v_cache"].flatten(0, 1)[s["slots"]] = v
    return {"q": qn, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# -------------------------------------------------------------- the package

def _package(s):
    from mhc_pre_gb300 import binding as B
    c = s["case"]
    if c["op"] == "attn":
        r = B.mhc_paged_attn(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["cu_q"], s["kv_lens"],
                             max_q=s["max_q"], max_kv=s["max_kv"], window=c["window"], softcap=c["softcap"])
        return {"o": r.o, "lse": r.lse}
    q, k, v = _split(s)
    rope = dict(positions=s["positions"], cos_sin=s["cos_sin"], eps=EPS, interleaved=c["pairs"] == "adjacent")
    if c["op"] == "qk":
        r = B.mhc_qk_norm_rope(q, k, s["w_q"], s["w_k"], **rope)
        return {"q": r.q, "k": r.k}
    if c["op"] == "qk_bwd":
        r = B.mhc_qk_norm_rope_bwd(s["g_q"], s["g_k"], q, k, s["w_q"], s["w_k"], **rope)
        return {"dq": r.dq, "dk": r.dk, "dw_q": r.dw_q, "dw_k": r.dw_k}
    qn = B.mhc_qk_norm_rope_append(q, k, v, s["w_q"], s["w_k"], s["k_cache"], s["v_cache"], s["slots"], **rope)
    return {"q": qn, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    return _package(state) if own else _plain(state)


# ------------------------------------------------------------- 64-bit values

def _exact_head(x, w, s, g=None):
    """One operand's heads [T, H, dh] through the normalisation and rotation as
    complex numbers; with `g`, the gradients of <g, output>."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    x, w = x.double(), w.double()
    tab = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(tab[:, :half], tab[:, half:])[:, None]

    def turned(y, by):
        y = y.clone()
        if c["pairs"] == "adjacent":
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * by
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(y[..., :half], y[..., half:rot]) * by
            y[..., :half], y[..., half:rot] = z.real, z.imag
        return y

    n = x.shape[-1]
    rms = ((x ** 2).sum(-1, keepdim=True) / n + EPS) ** 0.5
    if g is None:
        return turned(x / rms * w, turn)
    h = turned(g.double(), turn.conj())
    dw = (h * x / rms).sum((0, 1))
    u = h * w
    return u / rms - x * (u * x).sum(-1, keepdim=True) / (n * rms ** 3), dw


def _exact_attn(case, s):
    hq, hk, dh, page = case["hq"], case["hk"], case["dh"], case["page"]
    g = hq // hk
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(_lens(case)):
        pages = s["page_table"][b, : -(-m // page)].long()
        i = torch.arange(n, device="cuda")[:, None] + (m - n)
        j = torch.arange(m, device="cuda")[None, :]
        hidden = (j > i) | ((j <= i - case["window"]) if case["window"] else (j < 0))
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


def exact(case, seed):
    # a whole square of scores is formed for each sequence: above this it takes too long in 64 bits
    if case["op"] == "attn" and sum(n * m for n, m in _lens(case)) * case["hq"] * (4 * case["dh"] + 60) > 4e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(case, s)
    q, k, v = _split(s)
    if case["op"] == "qk_bwd":
        dq, dw_q = _exact_head(q, s["w_q"], s, s["g_q"])
        dk, dw_k = _exact_head(k, s["w_k"], s, s["g_k"])
        return {"dq": dq, "dk": dk, "dw_q": dw_q, "dw_k": dw_k}
    qn, kn = _exact_head(q, s["w_q"], s), _exact_head(k, s["w_k"], s)
    if case["op"] == "qk":
        return {"q": qn, "k": kn}
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    page = case["page"]
    where, slot = s["slots"] // page, s["slots"] % page
    kc[where, slot], vc[where, slot] = kn, v.double()
    return {"q": qn, "k_cache": kc, "v_cache": vc}
