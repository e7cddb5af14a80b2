"""Measured cases of the chunk operators: the rotary cache write, attention of a chunk of new tokens over the
paged cache, the accumulated attention mass of its keys, and eviction by that mass.

`run` computes each operator in elementary torch operations, or, where `own` is true, by the library's calls.
Lengths are plain functions of the case (ragged batches take them from the case's "ragged" number), values come
from the seed.
"""
import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"


# ---- cases --------------------------------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a batch of 64 sequences: the smallest write, launch latency counts
        dict(name="write-decode-64", op="write", batch=64, hq=32, hk=8, dim=128, page=64, q=1, kv=1024, ragged=1,
             axes=1, rot=128, interleaved=False, adjacent=False, fused=True),
        # a video prompt: three axes (time, height, width) interleaved over the pairs, G = 7
        dict(name="write-video-8k", op="write", batch=1, hq=28, hk=4, dim=128, page=64, q=8191, kv=9000, ragged=0,
             axes=3, rot=128, interleaved=True, adjacent=False, fused=False),
        # several prompts' chunks at once from a fused projection, half of each head rotated in adjacent pairs
        dict(name="write-prompts-32k", op="write", batch=5, hq=64, hk=8, dim=128, page=128, q=8192, kv=16384, ragged=3,
             axes=2, rot=64, interleaved=False, adjacent=True, fused=True),
        # one new token of one conversation: latency
        dict(name="decode-1-2k", op="attend", batch=1, hq=32, hk=8, dim=128, page=64, q=1, kv=2049, ragged=0,
             cap=0.0, window=0, alibi=False, docs=0, prefix=False),
        # a decode step of a serving batch with ragged contexts, G = 7
        dict(name="decode-32-ragged", op="attend", batch=32, hq=28, hk=4, dim=128, page=64, q=1, kv=32768, ragged=5,
             cap=0.0, window=0, alibi=False, docs=0, prefix=False),
        # a prompt piece over a long context: the ordinary chunked prefill, and the largest case
        dict(name="chunk-2k-on-32k", op="attend", batch=1, hq=32, hk=8, dim=128, page=64, q=2048, kv=34816, ragged=0,
             cap=0.0, window=0, alibi=False, docs=0, prefix=False),
        # packed documents with capped scores and a sliding window, odd lengths, padding tokens that see nothing
        dict(name="chunk-docs-cap", op="attend", batch=3, hq=64, hk=8, dim=128, page=128, q=1531, kv=8192, ragged=7,
             cap=30.0, window=2048, alibi=False, docs=1500, prefix=False),
        # a bidirectional prefix with a distance bias, narrow heads without sharing, small pages
        dict(name="chunk-prefix-bias", op="attend", batch=2, hq=16, hk=16, dim=64, page=16, q=777, kv=4095, ragged=9,
             cap=0.0, window=0, alibi=True, docs=0, prefix=True),
        # mass added by one decode step of a batch
        dict(name="mass-decode-8", op="mass", batch=8, hq=32, hk=8, dim=128, page=64, q=1, kv=16384, ragged=11,
             cap=0.0, window=0, alibi=False, docs=0, prefix=False, last=0),
        # mass given by the last 64 tokens of a prompt's last chunk to a 64K context
        dict(name="mass-last64-64k", op="mass", batch=1, hq=32, hk=8, dim=128, page=64, q=200, kv=65536, ragged=0,
             cap=0.0, window=0, alibi=False, docs=0, prefix=False, last=64),
        # a 32K cache cut to 4K keys a head
        dict(name="evict-32k-4k", op="evict", batch=1, hq=32, hk=8, dim=128, page=64, kv=32768, ragged=0, budget=4096,
             sink=4, recent=512),
        # a ragged batch cut to an odd budget, some sequences shorter than it
        dict(name="evict-ragged-6", op="evict", batch=6, hq=28, hk=4, dim=128, page=64, kv=16383, ragged=13, budget=2001,
             sink=64, recent=129),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: sizes log-uniform, odd ones likely."""
    op = rng.choice(["write", "attend", "attend", "mass", "evict"])
    hq, hk = rng.choice([(32, 8), (28, 4), (64, 8), (16, 16), (8, 1), (12, 2)])
    c = dict(op=op, hq=hq, hk=hk, dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 64, 128]),
             ragged=rng.randrange(1, 1 << 20))
    if op == "write":
        c.update(batch=_log(rng, 1, 64), axes=rng.choice([1, 2, 3, 4]), interleaved=rng.random() < 0.5,
                 adjacent=rng.random() < 0.5, fused=rng.random() < 0.5)
        c["rot"] = c["dim"] if rng.random() < 0.6 else c["dim"] // 2
        c["q"] = _log(rng, 1, max(2, 16384 // c["batch"]))
        c["kv"] = c["q"] + _log(rng, 1, 2048)
        return c
    if op == "evict":
        c.update(batch=_log(rng, 1, 8), kv=_log(rng, 300, 32768))
        c["budget"] = max(40, int(c["kv"] * rng.uniform(0.05, 0.6)))
        c["sink"] = rng.choice([0, 4, 16])
        c["recent"] = rng.choice([0, 1, c["budget"] // 4])
        return c
    c.update(batch=_log(rng, 1, 32), cap=rng.choice([0.0, 0.0, 20.0, 50.0]), window=rng.choice([0, 0, 0, 1000]),
             alibi=rng.random() < 0.3, docs=rng.choice([0, 0, 700]), prefix=rng.random() < 0.3)
    if op == "mass":
        c["last"] = rng.choice([0, 0, 16, 33])
    if rng.random() < 0.4:
        c["q"] = rng.choice([1, 1, 2, 5])
        c["kv"] = _log(rng, 64, 32768)
    else:
        c["q"] = _log(rng, 2, 2048)
        c["kv"] = c["q"] + _log(rng, 1, 16384)
    # no larger than the largest listed chunk, in pairs of tokens and keys over all sequences and heads
    while c["batch"] * c["q"] * c["kv"] * hq > 0.7 * 2048 * 34816 * 32 or c["batch"] * c["kv"] * hk > 4000000:
        c["batch"], c["kv"] = max(1, c["batch"] // 2), max(c["q"], int(c["kv"] * 0.8))
        c["q"] = max(1, int(c["q"] * 0.9))
    return c


def _lens(c):
    """(new tokens, keys after them) of each sequence: the case's own sizes, or ragged ones up to them."""
    q, kv, n = c.get("q", 1), c["kv"], c["batch"]
    if not c["ragged"]:
        return [(q, kv)] * n
    r = random.Random(c["ragged"])
    out = [(q, kv)]
    for _ in range(n - 1):
        ql = q if q <= 2 else r.randint(max(1, q // 3), q)
        out.append((ql, r.randint(max(ql, kv // 8), kv)))
    r.shuffle(out)
    return out


def _mask_vectors(c):
    """Per token: its sequence, position, and first and last visible key (last < first: it sees none)."""
    seq, pos, lo, hi, docs = [], [], [], [], []
    for b, (q, kv) in enumerate(_lens(c)):
        t = np.arange(kv - q, kv)
        first = np.zeros(q, np.int64)
        if c["docs"]:
            first = t // (c["docs"] + b) * (c["docs"] + b)  # documents of about that length, packed
            first[max(1, q - 3):] = kv                      # padding tokens: they see nothing
        a = np.maximum(first, t - c["window"] + 1 if c["window"] else 0)
        z = np.maximum(t, _prefix(q, kv) - 1) if c["prefix"] else t
        seq.append(np.full(q, b)), pos.append(t), lo.append(a), hi.append(np.minimum(z, kv - 1)), docs.append(first)
    return tuple(np.concatenate(v) for v in (seq, pos, lo, hi, docs))


def _prefix(q, kv):
    return kv - q + (q + 2) // 3  # the prefix ends inside the chunk


def work(case):
    c = case
    d, hq, hk, lens = c["dim"], c["hq"], c["hk"], _lens(c)
    tok = sum(q for q, _ in lens)
    if c["op"] == "write":
        return {"bytes": 4.0 * tok * (hq + 2 * hk) * d + 4.0 * tok * c["axes"], "flops": 3.0 * tok * (hq + hk) * c["rot"]}
    if c["op"] == "evict":
        kept = sum(min(kv, c["budget"]) for _, kv in lens)
        return {"bytes": hk * (4.0 * sum(kv for _, kv in lens) + kept * (8.0 * d + 8.0)), "flops": 0.0}
    seq, _, lo, hi, _ = _mask_vectors(c)
    if c["op"] == "mass" and c["last"]:
        use = np.concatenate([np.arange(q) >= q - c["last"] for q, _ in lens])
        seq, lo, hi = seq[use], lo[use], hi[use]
    pairs = float(np.maximum(hi - lo + 1, 0).sum())
    keys = 0
    for b in range(c["batch"]):
        m = (seq == b) & (hi >= lo)
        keys += int(hi[m].max() - lo[m].min() + 1) if m.any() else 0
    if c["op"] == "attend":
        return {"bytes": 4.0 * tok * hq * d + 4.0 * tok * hq + 4.0 * keys * hk * d, "flops": 4.0 * pairs * hq * d}
    total = sum(kv for _, kv in lens)
    return {"bytes": 2.0 * len(seq) * hq * d + 4.0 * len(seq) * hq + 2.0 * keys * hk * d + 8.0 * total * hk,
            "flops": 2.0 * pairs * hq * d}


# ---- inputs ---------------------------------------------------------------------------------------------------
def _sections(c):
    """Pairs of each axis: the first axis takes what the others leave."""
    n, a = c["rot"] // 2, c["axes"]
    rest = n // (a + 1)
    return [n - rest * (a - 1)] + [rest] * (a - 1)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    b, hq, hk, d, p, lens = c["batch"], c["hq"], c["hk"], c["dim"], c["page"], _lens(c)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)

    pps = -(-max(kv for _, kv in lens) // p)
    more = -(-c["budget"] // p) if c["op"] == "evict" else 0
    phys = b * (pps + more) + 3
    # pages in a shuffled order, as a cache in use hands them out
    perm = torch.randperm(phys, generator=g, device=DEV).to(torch.int32)
    s = dict(c=c, lens=lens, seed=int(seed), pps=pps, table=perm[:b * pps].view(b, pps).contiguous(),
             k_pool=rand(phys, hk, p, d), v_pool=rand(phys, hk, p, d),
             kv_len=_ints([kv for _, kv in lens]), cu_q=_ints([0] + list(np.cumsum([q for q, _ in lens]))))
    tok = sum(q for q, _ in lens)
    if c["op"] == "write":
        q_tok, k_tok, v_tok = rand(tok, hq, d), rand(tok, hk, d), rand(tok, hk, d)
        if c["fused"]:  # views of one projection's output
            both = torch.cat([q_tok, k_tok, v_tok], 1).contiguous()
            q_tok, k_tok, v_tok = both[:, :hq], both[:, hq:hq + hk], both[:, hq + hk:]
        t = torch.cat([torch.arange(kv - q, kv, device=DEV) for q, kv in lens])
        grid = [t // 96, t // 12 % 64, t % 12 * 5] if c["axes"] > 1 else [t]
        s.update(q_tok=q_tok, k_tok=k_tok, v_tok=v_tok, q=torch.empty(tok, hq, d, dtype=torch.bfloat16, device=DEV),
                 positions=torch.stack([grid[a % len(grid)] + (100000 if a == 0 else 0)
                                        for a in range(c["axes"])]).to(torch.int32).contiguous(),
                 inv_freq=(500000.0 ** (-torch.arange(c["rot"] // 2, dtype=torch.float64, device=DEV) * 2 / c["rot"])).float())
    elif c["op"] == "evict":
        # masses as they come: a few heavy keys, many light ones, and exact zeros
        m = torch.exp(1.5 * torch.randn(b, hk, pps * p, generator=g, device=DEV)) * 0.01
        m *= (torch.rand(m.shape, generator=g, device=DEV) > 0.3)
        s.update(mass=m, dst=perm[b * pps:b * (pps + more)].view(b, more).contiguous(),
                 kept=torch.empty(b, hk, c["budget"], dtype=torch.int32, device=DEV),
                 new_len=torch.empty(b, dtype=torch.int32, device=DEV),
                 mass_out=torch.zeros(b, hk, more * p, device=DEV))
    else:
        # a common direction of queries and first keys: the attention sink
        u = torch.nn.functional.normalize(torch.randn(hk, d, generator=g, device=DEV), dim=-1)
        first = s["table"][:, 0].long()
        s["k_pool"][first, :, :4] += (3.0 * u)[None, :, None].to(torch.bfloat16)
        q = (rand(tok, hq, d).view(tok, hk, hq // hk, d) + u[None, :, None].to(torch.bfloat16)).reshape(tok, hq, d)
        s.update(q=q.contiguous(), scale=1.0 / math.sqrt(d),
                 slopes=2.0 ** (-8.0 * torch.arange(1, hq + 1, device=DEV, dtype=torch.float32) / hq) if c["alibi"] else None,
                 first_key=_ints(_mask_vectors(c)[4].tolist()) if c["docs"] else None,
                 prefix_len=_ints([_prefix(q, kv) for q, kv in lens]) if c["prefix"] else None)
        if c["op"] == "attend":
            s.update(out=torch.empty(tok, hq, d, dtype=torch.bfloat16, device=DEV), lse=torch.empty(tok, hq, device=DEV))
        else:
            s["lse"] = _attend(s)[1]  # what the attention of the same tokens left
            s["mass"] = torch.rand(b, hk, pps * p, generator=g, device=DEV)
    if own:
        s["plan"] = _plan(s)
    return s


# ---- the plain form ---------------------------------------------------------------------------------------------
def _cache(pool, table, n, dtype=torch.float32):
    """The first n keys of every sequence: [B][H_kv][n][D]."""
    p = pool.shape[2]
    x = pool[table[:, :-(-n // p)].long()].to(dtype)
    return x.permute(0, 2, 1, 3, 4).reshape(x.shape[0], pool.shape[1], -1, pool.shape[3])[:, :, :n]


def _padded(s):
    """Tokens of the sequences in rows of equal length: their index, and which rows are tokens."""
    ql = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    i = torch.arange(max(q for q, _ in s["lens"]), device=DEV)
    real = i[None] < ql[:, None]
    return torch.where(real, s["cu_q"][:-1, None].long() + i[None], 0), real, ql


def _scores(s):
    """Scores [B][H_kv][G][L][keys] with the masked ones at -inf, and the rows' index."""
    c = s["c"]
    n, kvl = max(kv for _, kv in s["lens"]), s["kv_len"].long()
    at, real, ql = _padded(s)
    b, length = at.shape
    hk, gr, d = c["hk"], c["hq"] // c["hk"], c["dim"]
    q = s["q"].float()[at].view(b, length, hk, gr, d).permute(0, 2, 3, 1, 4).reshape(b, hk, gr * length, d)
    x = torch.matmul(q, _cache(s["k_pool"], s["table"], n).transpose(-1, -2)).view(b, hk, gr, length, n)
    x *= s["scale"]
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    pos = (kvl - ql)[:, None] + torch.arange(length, device=DEV)[None]
    key = torch.arange(n, device=DEV)
    if c["alibi"]:
        far = (pos[:, :, None] - key).abs().float()
        x -= s["slopes"].view(1, hk, gr, 1, 1) * far[:, None, None]
    lo = torch.zeros_like(pos) if s["first_key"] is None else s["first_key"].long()[at]
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    hi = pos if s["prefix_len"] is None else torch.maximum(pos, s["prefix_len"].long()[:, None] - 1)
    hi = torch.minimum(hi, kvl[:, None] - 1)
    seen = (key >= lo[:, :, None]) & (key <= hi[:, :, None]) & real[:, :, None]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    return x, at, real


def _rows(x, real):
    """[B][H_kv][G][L][...] back to token-major rows."""
    return x.flatten(1, 2).movedim(1, 2)[real]


def _attend(s):
    x, at, real = _scores(s)
    c = s["c"]
    m = x.amax(-1, keepdim=True)
    base = torch.where(m.isinf(), 0.0, m)
    x.sub_(base).exp_()
    l = x.sum(-1, keepdim=True)
    b, hk, gr, length, n = x.shape
    v = torch.matmul(x.view(b, hk, gr * length, n), _cache(s["v_pool"], s["table"], n)).view(b, hk, gr, length, -1)
    o = torch.where(l > 0, v / l, 0.0)
    lse = torch.where(l > 0, base + torch.log(l), -math.inf)[..., 0]
    return _rows(o, real).to(torch.bfloat16), _rows(lse, real)


def _mass(s):
    x, at, real = _scores(s)
    c = s["c"]
    b, hk, gr, length, n = x.shape
    lse = s["lse"][at].view(b, length, hk, gr).permute(0, 2, 3, 1)[..., None]
    x.sub_(torch.where(lse.isinf(), 0.0, lse)).exp_()
    _, _, ql = _padded(s)
    if c["last"]:
        x *= (torch.arange(length, device=DEV)[None] >= (ql - c["last"])[:, None]).view(b, 1, 1, length, 1)
    add = x.sum((2, 3))
    key, kvl = torch.arange(n, device=DEV), s["kv_len"].long()
    old = s["mass"][:, :, :n]
    new = add + torch.where((key < (kvl - ql)[:, None])[:, None], old, 0.0)
    s["mass"][:, :, :n] = torch.where((key < kvl[:, None])[:, None], new, old)
    return s["mass"]


def _axis_of(c):
    """The axis that turns each pair."""
    sec = _sections(c)
    j = torch.arange(c["rot"] // 2, device=DEV)
    if c["interleaved"]:
        a = j % c["axes"]
        return torch.where(j < c["axes"] * torch.tensor(sec, device=DEV)[a], a, 0)
    return torch.bucketize(j, torch.cumsum(torch.tensor(sec, device=DEV), 0), right=True)


def _turn(x, cos, sin, c):
    r = c["rot"]
    y = x.float()
    if c["adjacent"]:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        new = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        new = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([new, y[..., r:]], -1).to(torch.bfloat16)


def _slots(s):
    """Page and slot of every new token."""
    at, real, ql = _padded(s)
    pos = ((s["kv_len"].long() - ql)[:, None] + torch.arange(at.shape[1], device=DEV)[None])
    p = s["c"]["page"]
    page = torch.gather(s["table"].long(), 1, torch.where(real, pos // p, 0))
    return page[real], (pos % p)[real]


def _write(s):
    c = s["c"]
    angle = s["positions"].double()[_axis_of(c)].T * s["inv_freq"].double()  # far positions: 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s["q"].copy_(_turn(s["q_tok"], cos, sin, c))
    page, slot = _slots(s)
    s["k_pool"][page, :, slot] = _turn(s["k_tok"], cos, sin, c)
    s["v_pool"][page, :, slot] = s["v_tok"]
    return s["q"], s["k_pool"], s["v_pool"]


def _evict(s):
    c = s["c"]
    b, hk, n = s["mass"].shape
    key, kvl = torch.arange(n, device=DEV), s["kv_len"].long()[:, None]
    forced = (key < c["sink"]) | (key >= kvl - c["recent"])
    rank = torch.where(forced[:, None], math.inf, s["mass"])
    rank = torch.where((key < kvl)[:, None], rank, -math.inf)
    pick = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :c["budget"]]
    new = torch.clamp(kvl[:, 0], max=c["budget"])
    short = c["budget"] - pick.shape[-1]  # a budget past the longest sequence
    pick = torch.cat([pick, torch.full((b, hk, short), n, device=DEV)], -1) if short > 0 else pick
    j = torch.arange(c["budget"], device=DEV)
    have = (j[None] < new[:, None])[:, None].expand(b, hk, -1)
    pick = torch.sort(torch.where(have, pick, n), dim=-1).values
    s["kept"].copy_(torch.where(have, pick, -1))
    s["new_len"].copy_(new)
    p = c["page"]
    bi, hi, ji = torch.nonzero(have, as_tuple=True)
    src = pick[bi, hi, ji]
    from_page, to_page = s["table"].long()[bi, src // p], s["dst"].long()[bi, ji // p]
    s["k_pool"][to_page, hi, ji % p] = s["k_pool"][from_page, hi, src % p]
    s["v_pool"][to_page, hi, ji % p] = s["v_pool"][from_page, hi, src % p]
    s["mass_out"][bi, hi, ji] = s["mass"][bi, hi, src]
    return s["kept"], s["new_len"], s["k_pool"], s["v_pool"], s["mass_out"]


# ---- the library's calls -----------------------------------------------------------------------------------------
def _plan(s):
    """What a server keeps beside the cache: the shape, the parameters and the attention's workspace."""
    import block_sparse_long_kap_b200 as C
    c, lens = s["c"], s["lens"]
    shape = C.ChunkShape(c["batch"], c["hq"], c["hk"], c["dim"], c["page"], total_q=sum(q for q, _ in lens),
                         max_q=max(q for q, _ in lens), max_kv=max(kv for _, kv in lens), pages_per_seq=s["pps"],
                         num_phys_pages=s["k_pool"].shape[0])
    if c["op"] == "write":
        return C, shape, C.RopeParams(sections=tuple(_sections(c)), interleaved=c["interleaved"], adjacent=c["adjacent"])
    if c["op"] == "evict":
        return C, shape, C.EvictParams(budget=c["budget"], sink=c["sink"], recent=c["recent"])
    score = C.ScoreParams(softcap=c["cap"], window=c["window"], slopes=s["slopes"], first_key=s["first_key"],
                          prefix_len=s["prefix_len"])
    if c["op"] == "attend":
        s["ws"] = torch.empty(C.cosa_chunk_attention_workspace_size(shape), dtype=torch.uint8, device=DEV)
    return C, shape, score


def _own(s):
    C, shape, par = s["plan"]
    op = s["c"]["op"]
    if op == "write":
        C.cosa_chunk_write(shape, par, s["q_tok"], s["k_tok"], s["v_tok"], s["positions"], s["inv_freq"], s["cu_q"],
                           s["kv_len"], s["table"], s["q"], s["k_pool"], s["v_pool"])
        return s["q"], s["k_pool"], s["v_pool"]
    if op == "attend":
        C.cosa_chunk_attention(shape, s["q"], s["k_pool"], s["v_pool"], s["table"], s["cu_q"], s["kv_len"], s["out"],
                               s["ws"], score=par, lse=s["lse"])
        return s["out"], s["lse"]
    if op == "mass":
        C.cosa_attention_mass(shape, s["q"], s["k_pool"], s["table"], s["cu_q"], s["kv_len"], s["lse"], s["mass"],
                              score=par, last_q=s["c"]["last"], decay=1.0)
        return s["mass"]
    C.cosa_cache_evict(shape, par, s["k_pool"], s["v_pool"], s["table"], s["kv_len"], s["mass"], s["dst"], s["kept"],
                       s["new_len"], mass_out=s["mass_out"])
    return s["kept"], s["new_len"], s["k_pool"], s["v_pool"], s["mass_out"]


def run(state):
    if own:
        return _own(state)
    return {"write": _write, "attend": _attend, "mass": _mass, "evict": _evict}[state["c"]["op"]](state)


# ---- the definition, in 64 bits -----------------------------------------------------------------------------------
def exact(case, seed):
    """Each operator from its formula, one sequence and head at a time."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"write": _exact_write, "attend": _exact_attend, "mass": _exact_attend, "evict": _exact_evict}[case["op"]](s)


def _exact_write(s):
    c = s["c"]
    sec, half = _sections(c), c["rot"] // 2
    axis = []
    for j in range(half):
        if c["interleaved"]:
            a = j % c["axes"]
            axis.append(a if a and j < c["axes"] * sec[a] else 0)
        else:
            axis.append(next(a for a in range(c["axes"]) if j < sum(sec[:a + 1])))
    outs = {}
    for name in ("q", "k"):
        x = s[name + "_tok"].double()
        y = x.clone()
        for j in range(half):
            i0, i1 = (2 * j, 2 * j + 1) if c["adjacent"] else (j, j + half)
            w = (s["positions"][axis[j]].double() * s["inv_freq"][j].double())[:, None]
            y[..., i0] = x[..., i0] * torch.cos(w) - x[..., i1] * torch.sin(w)
            y[..., i1] = x[..., i0] * torch.sin(w) + x[..., i1] * torch.cos(w)
        outs[name] = y
    kp, vp, at, p = s["k_pool"].double(), s["v_pool"].double(), 0, c["page"]
    for b, (q, kv) in enumerate(s["lens"]):
        t = torch.arange(kv - q, kv, device=DEV)
        pages = s["table"][b].long()[t // p]
        kp[pages, :, t % p] = outs["k"][at:at + q]
        vp[pages, :, t % p] = s["v_tok"][at:at + q].double()
        at += q
    return outs["q"], kp, vp


def _exact_attend(s):
    c = s["c"]
    hq, hk, d, p = c["hq"], c["hk"], c["dim"], c["page"]
    mass_of = c["op"] == "mass"
    if mass_of:
        new = s["mass"].double()
    else:
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    seq, pos, lo, hi, _ = (torch.from_numpy(v).to(DEV) for v in _mask_vectors(c))
    at = 0
    for b, (q, kv) in enumerate(s["lens"]):
        pages = s["table"][b].long()[torch.arange(kv, device=DEV) // p]
        slots = torch.arange(kv, device=DEV) % p
        key = torch.arange(kv, device=DEV)
        rows = slice(at, at + q)
        at += q
        seen = (key >= lo[rows, None]) & (key <= hi[rows, None])
        for h in range(hq):
            g = h // (hq // hk)
            k = s["k_pool"][pages, g, slots].double()
            x = s["q"][rows, h].double() @ k.T / math.sqrt(d)
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if c["alibi"]:
                x = x - s["slopes"][h].double() * (pos[rows, None] - key).abs()
            if mass_of:
                if h % (hq // hk) == 0:
                    total = torch.zeros(kv, dtype=torch.float64, device=DEV)
                w = torch.where(seen, torch.exp(x - s["lse"][rows, h].double()[:, None]), 0.0)
                total += (w[max(0, q - c["last"]):] if c["last"] else w).sum(0)
                if h % (hq // hk) == hq // hk - 1:
                    total[:kv - q] += new[b, g, :kv - q]
                    new[b, g, :kv] = total
                continue
            x = torch.where(seen, x, -math.inf)
            lse[rows, h] = torch.logsumexp(x, -1)
            w = torch.where(seen, torch.exp(x - lse[rows, h][:, None]), 0.0)
            out[rows, h] = w @ s["v_pool"][pages, g, slots].double()
    return new if mass_of else (out, lse)


def _exact_evict(s):
    c = s["c"]
    kp, vp, mo, p = s["k_pool"].double(), s["v_pool"].double(), s["mass_out"].double(), c["page"]
    kept = np.full((c["batch"], c["hk"], c["budget"]), -1, np.int32)
    mass = s["mass"].double().cpu().numpy()
    new_len = []
    for b, (_, kv) in enumerate(s["lens"]):
        n = min(kv, c["budget"])
        new_len.append(n)
        must = [k for k in range(kv) if k < c["sink"] or k >= kv - c["recent"]][:n]
        for h in range(c["hk"]):
            rest = np.setdiff1d(np.arange(kv), must)
            by = np.lexsort((rest, -mass[b, h, rest]))  # heaviest first, then the lower position
            keep = np.sort(np.concatenate([np.array(must, np.int64), rest[by][:n - len(must)]])).astype(np.int64)
            kept[b, h, :n] = keep
            src, j = torch.from_numpy(keep).to(DEV), torch.arange(n, device=DEV)
            f, t = s["table"][b].long()[src // p], s["dst"][b].long()[j // p]
            kp[t, h, j % p] = s["k_pool"][f, h, src % p].double()
            vp[t, h, j % p] = s["v_pool"][f, h, src % p].double()
            mo[b, h, :n] = s["mass"][b, h, src].double()
    return kept, np.array(new_len, np.int32), kp, vp, mo
