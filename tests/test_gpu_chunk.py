"""GPU parity of the chunk operators (rotary write, attention, mass, eviction) against the
float64 oracle, at the sizes and masks where they can go wrong.

Tolerances, from the formats.  A rounding to bf16 is off by at most 2^-8 of the value.
  write      one rounding, after fp32 products: 2^-8 |ref| + 2^-20 (|x| + |y|).
  scores     fp32 accumulation of D products: ds = D 2^-24 scale max|q| . |k|, and c 2^-21 more
             under a cap c (an exponential and a reciprocal good to 2^-22, or a polynomial).
  attention  weights rounded to bf16 and the result once more, a score error of ds moves a
             weight by that share and the sum by as much: (2^-8 + 2 ds) sum w|v| + 2^-8 |ref|.
  lse        ds + the fp32 sum of n terms, n 2^-24, + 2^-22 |lse|.
  mass       per weight ds + 2^-22 (|lse| + 2), the sum over rows as many times 2^-24.
  eviction   exact.
"""
import math

import numpy as np
import pytest
import torch

import block_sparse_long_kap_b200 as C
from oracle import chunk_oracle as K

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


class Case:
    """A ragged batch: lens = [(new tokens, keys)], a shuffled page table, and NaN in every slot of
    the pools that holds no key."""

    def __init__(self, lens, hq, hk, D=128, P=64, seed=0, extra_q=3, extra_pages=1, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hk, self.D, self.P = lens, hq, hk, D, P
        B = len(lens)
        self.cu = np.concatenate([[0], np.cumsum([q for q, _ in lens])]).astype(np.int32)
        self.kv = np.array([kv for _, kv in lens], np.int32)
        self.T = int(self.cu[-1]) + extra_q
        self.pps = max(1, -(-int(self.kv.max()) // P)) + extra_pages
        self.phys = B * self.pps + 2
        perm = torch.randperm(self.phys, generator=g)
        self.table = perm[:B * self.pps].view(B, self.pps).to(torch.int32)
        self.k_pool = torch.full((self.phys, hk, P, D), float("nan"))
        self.v_pool = torch.full((self.phys, hk, P, D), float("nan"))
        for b, (_, kv) in enumerate(lens):
            for p in range(-(-kv // P)):
                n = min(P, kv - p * P)
                self.k_pool[self.table[b, p], :, :n] = torch.randn(hk, n, D, generator=g) * spread
                self.v_pool[self.table[b, p], :, :n] = torch.randn(hk, n, D, generator=g)
            # entries past the sequence's pages name nothing
            self.table[b, -(-kv // P):] = -1
        self.q = torch.randn(self.T, hq, D, generator=g)
        self.q[int(self.cu[-1]):] = float("nan")
        self.g = g
        bf = torch.bfloat16
        self.k_pool, self.v_pool, self.q = self.k_pool.to(bf), self.v_pool.to(bf), self.q.to(bf)
        self.shape = C.ChunkShape(B, hq, hk, D, P, total_q=self.T, max_q=max(max(q for q, _ in lens), 1),
                                  max_kv=max(int(self.kv.max()), 1), pages_per_seq=self.pps,
                                  num_phys_pages=self.phys)
        self.scale = 1.0 / math.sqrt(D)
        self.d = {n: getattr(self, n).cuda() for n in ("k_pool", "v_pool", "q", "table")}
        self.d["cu"], self.d["kv"] = torch.from_numpy(self.cu).cuda(), torch.from_numpy(self.kv).cuda()

    def score(self, opt):
        """(ScoreParams, oracle keywords) of a named option."""
        kw, dev = {}, {}
        for o in opt.split("+"):
            if o == "cap":
                kw["softcap"] = 5.0
            if o == "bigcap":
                kw["softcap"] = 50.0
            if o == "window":
                kw["window"] = 70
            if o == "bias":
                kw["slopes"] = np.float32(2.0) ** -np.linspace(0.5, 6, self.hq).astype(np.float32)
            if o == "docs":  # packed documents of 50 keys; every fifth token sees nothing
                t = np.concatenate([np.arange(kv - q, kv) for q, kv in self.lens] + [[0] * (self.T - self.cu[-1])])
                f = (t // 50 * 50).astype(np.int32)
                f[4::5] = t[4::5] + 1 + (np.arange(len(t))[4::5] % 2) * 100000
                kw["first_key"] = f
            if o == "prefix":
                kw["prefix_len"] = np.array([max(0, kv - q + q // 2) for q, kv in self.lens], np.int32)
        for n in ("slopes", "first_key", "prefix_len"):
            dev[n] = torch.from_numpy(kw[n]).cuda() if n in kw else None
        return C.ScoreParams(softcap=kw.get("softcap", 0.0), window=kw.get("window", 0), **dev), kw

    def ds(self, kw):
        """Bound of a score's error."""
        kmax = float(torch.nan_to_num(self.k_pool.float()).norm(dim=-1).max())
        qmax = float(torch.nan_to_num(self.q.float()).norm(dim=-1).max())
        return self.D * 2.0**-24 * self.scale * kmax * qmax + kw.get("softcap", 0.0) * 2.0**-21

    def attend(self, score=None, q=None, stream=None, ws=None, d=None):
        d = d or self.d
        out = torch.full((self.T, self.hq, self.D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((self.T, self.hq), 7.0, device="cuda")
        if ws is None:
            ws = torch.full((C.cosa_chunk_attention_workspace_size(self.shape),), 255, dtype=torch.uint8, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())  # the buffers were filled there
        C.cosa_chunk_attention(self.shape, d["q"] if q is None else q, d["k_pool"], d["v_pool"], d["table"], d["cu"],
                               d["kv"], out, ws, score=score, lse=lse, stream=stream)
        if stream is not None:  # and are not handed out again before this stream is done with them
            for t in (out, lse, ws):
                t.record_stream(stream)
        return out, lse

    def oracle(self, kw):
        return K.chunk_attention(_np(self.q), _np(self.k_pool), _np(self.v_pool), self.table.numpy(), self.cu, self.kv,
                                 self.scale, **kw)

    def check(self, out, lse, kw, ref=None):
        o, l, spread = ref or self.oracle(kw)
        n, ds = int(self.cu[-1]), self.ds(kw)
        got, gl = _np(out), _np(lse)
        tol = (2.0**-8 + 2 * ds) * spread + 2.0**-8 * np.abs(o)
        bad = np.abs(got - o)[:n] > tol[:n]
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - o)[:n].max())
        assert np.array_equal(np.isinf(gl[:n]), np.isinf(l[:n]))
        fin = np.isfinite(l[:n])
        tl = ds + int(self.kv.max()) * 2.0**-24 + 2.0**-22 * np.abs(l[:n][fin])
        assert (np.abs(gl[:n][fin] - l[:n][fin]) <= tl).all()
        assert (got[:n][~np.isfinite(l[:n])] == 0).all()
        assert (got[n:] == 7).all() and (gl[n:] == 7).all()  # rows behind the last sequence
        assert C.cosa_get_status() == 0


# ---- attention ------------------------------------------------------------------------------------
ATTEND = [
    # lens, hq, hk, D, P
    ([(1, 1)], 1, 1, 128, 64),
    ([(1, 127), (1, 128), (1, 129), (1, 1)], 8, 2, 128, 64),
    ([(1, 300), (0, 77), (3, 3), (2, 515)], 7, 1, 128, 16),
    ([(5, 5), (130, 261), (31, 31)], 8, 2, 128, 128),
    ([(64, 64), (65, 200), (1, 1)], 4, 4, 128, 32),
    ([(129, 140), (127, 390)], 2, 2, 64, 16),
    ([(40, 321), (300, 300)], 14, 2, 128, 64),
    ([(2, 33), (9, 100)], 128, 1, 64, 64),
    ([(20, 1000), (1, 2), (33, 700)], 16, 1, 128, 64),
    ([(3, 4000)], 4, 1, 64, 32),
]


@pytest.mark.parametrize("i", range(len(ATTEND)))
@pytest.mark.parametrize("opt", ["plain", "window", "docs", "cap", "bias+prefix"])
def test_attention_parity(i, opt):
    lens, hq, hk, D, P = ATTEND[i]
    c = Case(lens, hq, hk, D, P, seed=i)
    score, kw = c.score(opt)
    c.check(*c.attend(None if opt == "plain" else score), kw)


@pytest.mark.parametrize("opt", ["cap+bias", "bigcap+docs+window", "bias+docs+prefix", "cap+window+prefix",
                                 "bigcap+bias+docs+window+prefix", "docs+window+prefix"])
@pytest.mark.parametrize("i", [2, 3, 5])
def test_attention_parity_of_combined_options(i, opt):
    lens, hq, hk, D, P = ATTEND[i]
    c = Case(lens, hq, hk, D, P, seed=20 + i)
    score, kw = c.score(opt)
    c.check(*c.attend(score), kw)


@pytest.mark.parametrize("opt", ["plain", "cap", "bigcap"])
@pytest.mark.parametrize("q", [2, 70])
def test_logits_far_apart_move_the_exponent_base(opt, q):
    """Keys thirty times as long: logits of hundreds, row maxima that jump block after block."""
    c = Case([(q, 900)], 4, 1, 128, 64, seed=5, spread=30.0)
    score, kw = c.score(opt)
    c.check(*c.attend(score), kw)


@pytest.mark.parametrize("kv", [120, 900])  # one block: a whole tile; eight: cut between CTAs
@pytest.mark.parametrize("q,D", [(2, 128), (30, 128), (70, 64), (110, 128)])
def test_a_nan_key_reaches_the_rows_that_see_it_and_no_others(kv, q, D):
    c = Case([(q, kv)], 4, 2, D, 64, seed=84)
    first = np.zeros(c.T, np.int32)
    first[1::2] = 8  # odd tokens see only later keys
    c.k_pool[c.table[0, 0], 0, 5, D // 2] = float("nan")  # key 5 of KV head 0
    c.d["k_pool"].copy_(c.k_pool)
    out, lse = c.attend(C.ScoreParams(first_key=torch.from_numpy(first).cuda()))
    o, l, spread = c.oracle(dict(first_key=first))
    hit = np.isnan(l)[:q]
    assert hit.sum() == 2 * len(range(0, q, 2))
    got, gl = _np(out)[:q], _np(lse)[:q]
    assert np.isnan(gl[hit]).all() and np.isnan(got[hit]).all()
    tol = (2.0**-8 + 2 * c.ds({})) * spread + 2.0**-8 * np.abs(o)
    assert (np.abs(got - o[:q])[~hit] <= tol[:q][~hit]).all()
    assert (np.abs(gl - l[:q])[~hit] <= c.ds({}) + kv * 2.0**-24 + 2.0**-22 * np.abs(l[:q][~hit])).all()
    assert C.cosa_get_status() == 0


@pytest.mark.parametrize("q,D", [(3, 128), (20, 128), (3, 64), (100, 64)])
def test_distances_at_positions_past_what_fp32_counts(q, D):
    """2^24 + 1001 keys (the pages named over and over): a float no longer holds every position, and
    a bias by distance needs it to one key.  Steep slopes leave the last 2,000 keys to compare."""
    n, P = 2**24 + 1001, 128
    c = Case([(q, 1024)], 2, 1, D, P, seed=85)
    g = torch.Generator().manual_seed(86)
    table = c.table[0, torch.randint(0, 8, (1, -(-n // P)), generator=g)]
    c.kv, c.table, c.pps = np.array([n], np.int32), table, table.shape[1]
    c.shape.max_kv, c.shape.pages_per_seq = n, c.pps
    c.d["table"], c.d["kv"] = table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda")
    slopes = np.array([0.5, 0.25], np.float32)
    score = C.ScoreParams(slopes=torch.from_numpy(slopes).cuda())
    out, lse = c.attend(score)
    off = (n - 2048) // P * P
    args = _np(c.q), _np(c.k_pool)
    o, l, spread = K.chunk_attention(*args, _np(c.v_pool), table[:, off // P:].numpy(), c.cu, c.kv - off, c.scale,
                                     slopes=slopes)
    tol = (2.0**-8 + 2 * c.ds({})) * spread + 2.0**-8 * np.abs(o)
    assert (np.abs(_np(out) - o)[:q] <= tol[:q]).all()
    assert (np.abs(_np(lse) - l)[:q] <= c.ds({}) + 2048 * 2.0**-24 + 2.0**-22 * (np.abs(l[:q]) + 2)).all()
    mass = torch.zeros(1, 1, c.pps * P, device="cuda")
    C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass, score=score)
    want = K.attention_mass(*args, table[:, off // P:].numpy(), c.cu, c.kv - off, _np(lse),
                            np.zeros((1, 1, c.pps * P - off)), c.scale, slopes=slopes)
    got = _np(mass)
    rel = c.ds({}) + 2.0**-22 * (np.abs(l[:q]).max() + 2) + 2 * q * 2.0**-24
    # a weight's share of the distance's own rounding: slope x distance x 2^-23 in its exponent
    far = slopes.max() * (n - off) * 2.0**-23
    assert (np.abs(got[..., off:] - want) <= (rel + far) * want + 1e-30).all()
    assert (got[..., :off] < 1e-30).all()
    assert C.cosa_get_status() == 0


@pytest.mark.parametrize("q,D", [(2, 128), (40, 64)])
def test_extreme_mask_values(q, D):
    """Lengths of a prefix and first keys at the ends of int32, windows at its top."""
    c = Case([(q, 300), (q, 300), (q, 300)], 4, 2, D, 64, seed=87)
    first = np.zeros(c.T, np.int64)
    first[0::3], first[1::3] = -2**31, 2**31 - 1
    kw = dict(first_key=first.astype(np.int32), prefix_len=np.array([-2**31, 2**31 - 1, 0], np.int32), window=2**31 - 1)
    score = C.ScoreParams(window=2**31 - 1, first_key=torch.from_numpy(kw["first_key"]).cuda(),
                          prefix_len=torch.from_numpy(kw["prefix_len"]).cuda())
    ref = c.oracle(dict(kw, first_key=np.maximum(first, 0)))
    out, lse = c.attend(score)
    c.check(out, lse, {}, ref)
    mass = torch.zeros(3, 2, c.pps * 64, device="cuda")
    C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass, score=score)
    want = K.attention_mass(_np(c.q), _np(c.k_pool), c.table.numpy(), c.cu, c.kv, _np(lse), np.zeros(mass.shape), c.scale,
                            **dict(kw, first_key=np.maximum(first, 0)))
    rel = c.ds({}) + 2.0**-22 * (np.abs(ref[1][np.isfinite(ref[1])]).max() + 2) + 2 * q * 2.0**-24
    assert (np.abs(_np(mass) - want) <= rel * want + 1e-30).all()
    assert C.cosa_get_status() == 0


def test_strided_queries_and_null_lse():
    c = Case([(3, 50), (17, 200)], 8, 2, seed=1)
    fused = torch.full((c.T, 8 + 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = c.d["q"]
    out, lse = c.attend(q=fused[:, 2:10])
    c.check(out, lse, {})
    ws = torch.empty(C.cosa_chunk_attention_workspace_size(c.shape), dtype=torch.uint8, device="cuda")
    out2 = torch.full_like(out, 7.0)
    C.cosa_chunk_attention(c.shape, c.d["q"], c.d["k_pool"], c.d["v_pool"], c.d["table"], c.d["cu"], c.d["kv"], out2, ws)
    assert torch.equal(out, out2)


def test_whole_prompt_equals_the_dense_kernel():
    N, hq, hk, D, P = 1024, 8, 2, 128, 64
    c = Case([(N, N)], hq, hk, D, P, seed=3, extra_q=0, extra_pages=0)
    out, lse = c.attend()
    sh = C.Shape(1, hq, hk, N, D, P, 128, num_phys_pages=c.phys)
    q = c.d["q"].permute(1, 0, 2).contiguous()[None]
    o2, l2 = torch.empty_like(q), torch.empty(1, hq, N, device="cuda")
    C.cosa_dense_attention(sh, q, c.d["k_pool"], c.d["v_pool"], c.d["table"], o2, lse=l2)
    # both within two bf16 roundings of the exact result, whose size is at most that of V
    assert (out.permute(1, 0, 2)[None].float() - o2.float()).abs().max() <= 2 * 2.0**-8 * 2 * 5
    assert (lse.T[None] - l2).abs().max() <= 2 * c.ds({}) + 2.0**-13


def test_many_sequences_and_one_long_one_share_the_work():
    """Tiles cut between CTAs: a 20K cache of one head beside 200 short ones; rows against a
    float64 softmax on the GPU."""
    lens = [(1, 20011)] + [(1, 1 + 7 * i % 300) for i in range(200)]
    c = Case(lens, 4, 1, seed=9)
    out, lse = c.attend()
    for b in (0, 1, 57, 200):
        kv = lens[b][1]
        k = torch.arange(kv)
        pages = c.table[b, k // c.P].long()
        Kb, Vb = (x[pages, 0, k % c.P].cuda().double() for x in (c.k_pool, c.v_pool))
        s = c.d["q"][c.cu[b]].double() @ Kb.T * c.scale
        w = torch.softmax(s, -1)
        o, spread = w @ Vb, w @ Vb.abs()
        assert ((out[c.cu[b]].double() - o).abs() <= (2.0**-8 + 2 * c.ds({})) * spread + 2.0**-8 * o.abs()).all()
        assert (lse[c.cu[b]].double() - torch.logsumexp(s, -1)).abs().max() <= c.ds({}) + kv * 2.0**-24 + 2.0**-18
    assert C.cosa_get_status() == 0


def test_same_bits_on_every_run_and_with_a_loose_bound():
    c = Case([(1, 3000), (2, 100), (1, 2000)], 8, 1, seed=4)
    a = c.attend()
    for _ in range(3):
        b = c.attend()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # a bound on the lengths looser than they are sizes nothing that the result depends on
    c.shape.max_kv = c.pps * c.P
    b = c.attend()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_at_once_and_a_side_stream():
    a, b = Case([(300, 700)], 8, 2, seed=6), Case([(1, 5000), (1, 20)], 8, 2, seed=7)
    ra, rb = a.oracle({}), b.oracle({})
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        x, y = a.attend(stream=s1), b.attend(stream=s2)
    torch.cuda.synchronize()
    a.check(*x, {}, ra)
    b.check(*y, {}, rb)


def test_captured_graph_follows_lengths_and_two_graphs_share_a_workspace():
    c = Case([(1, 400), (1, 77)], 8, 2, seed=8)
    ws = torch.empty(C.cosa_chunk_attention_workspace_size(c.shape), dtype=torch.uint8, device="cuda")
    out = torch.empty(c.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(c.T, 8, device="cuda")
    mass = torch.zeros(2, 2, c.pps * c.P, device="cuda")

    def run(with_mass):
        C.cosa_chunk_attention(c.shape, c.d["q"], c.d["k_pool"], c.d["v_pool"], c.d["table"], c.d["cu"], c.d["kv"], out, ws, lse=lse)
        if with_mass:
            C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass, decay=0.0)

    run(True)
    torch.cuda.synchronize()
    graphs = []
    for m in (False, True):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(m)
        graphs.append(g)
    for kv in ([400, 77], [129, 1], [64, 65]):
        c.d["kv"].copy_(torch.tensor(kv, dtype=torch.int32))
        for g in graphs:
            out.fill_(7.0)
            lse.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        ref = K.chunk_attention(_np(c.q), _np(c.k_pool), _np(c.v_pool), c.table.numpy(), c.cu, np.array(kv), c.scale)
        c.check(out, lse, {}, ref)
        for b in range(2):
            assert (mass[b, :, :kv[b]].sum(-1) - 4).abs().max() < 1e-4


# ---- mass -----------------------------------------------------------------------------------------
MASS = [
    ([(1, 1), (1, 130), (1, 257)], 8, 2, 128, 64),
    ([(1, 300), (0, 77), (3, 3), (2, 515)], 7, 1, 128, 16),
    ([(40, 321), (130, 300)], 14, 2, 128, 64),   # several tiles
    ([(70, 90), (9, 600)], 4, 4, 64, 32),        # two tiles (held)
    ([(100, 640), (20, 41)], 16, 1, 128, 128),
    ([(2, 33)], 128, 1, 64, 64),
]


@pytest.mark.parametrize("i", range(len(MASS)))
@pytest.mark.parametrize("opt,last,decay", [("plain", 0, 1.0), ("docs", 0, 0.0), ("window", 3, 0.5),
                                            ("cap", 0, 1.0), ("bias+prefix", 7, 0.9),
                                            ("bigcap+bias+docs+window+prefix", 0, 2.0)])
def test_mass_parity(i, opt, last, decay):
    lens, hq, hk, D, P = MASS[i]
    c = Case(lens, hq, hk, D, P, seed=40 + i)
    score, kw = c.score(opt)
    _, lse = c.attend(score)
    lse[int(c.cu[-1]):] = float("nan")
    old = torch.rand(len(lens), hk, c.pps * P, generator=c.g)
    if decay == 0.0:
        old[:] = float("nan")
    mass = old.cuda()
    C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass, score=score,
                          last_q=last, decay=decay)
    want = K.attention_mass(_np(c.q), _np(c.k_pool), c.table.numpy(), c.cu, c.kv, _np(lse), _np(old), c.scale,
                            last_q=last, decay=decay, **kw)
    got = _np(mass)
    fin = np.isfinite(_np(lse))
    rel = c.ds(kw) + 2.0**-22 * (np.abs(_np(lse)[fin]).max() + 2) + (c.shape.max_q * hq // hk) * 2.0**-24
    for b, (n, kv) in enumerate(lens):
        keys = kv if n else 0
        assert (np.abs(got[b, :, :keys] - want[b, :, :keys]) <= rel * np.abs(want[b, :, :keys]) + 1e-30).all()
        assert np.array_equal(got[b, :, keys:], _np(old)[b, :, keys:], equal_nan=True)
    assert C.cosa_get_status() == 0


def test_mass_same_bits_on_every_run():
    c = Case([(200, 900), (1, 40)], 8, 2, seed=50)
    _, lse = c.attend()
    res = []
    for _ in range(3):
        m = torch.zeros(2, 2, c.pps * c.P, device="cuda")
        C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, m)
        res.append(m)
    assert torch.equal(res[0], res[1]) and torch.equal(res[0], res[2])


# ---- write ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("D,P,sections,interleaved,adjacent", [
    (128, 64, (64,), False, False), (128, 16, (24, 20, 20), False, False), (128, 128, (24, 20, 20), True, False),
    (64, 32, (8, 4, 4), True, True), (128, 64, (16, 0, 8, 8), False, True), (64, 64, (8,), False, False), (128, 64, (), False, False)])
@pytest.mark.parametrize("fused,inplace", [(False, False), (True, False), (True, True)])
def test_write_parity(D, P, sections, interleaved, adjacent, fused, inplace):
    lens = [(3, 70), (0, 5), (1, 1), (40, 129)]
    c = Case(lens, 6, 2, D, P, seed=60)
    g = c.g
    both = torch.randn(c.T, 10, D, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (max(1, len(sections)), c.T), generator=g, dtype=torch.int32)
    pos[0, 0], pos[0, 1] = 2**31 - 1, -5
    half = sum(sections)
    freq = (500000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()
    dev = both.cuda()
    qt, kt, vt = (x if fused else x.contiguous() for x in (dev[:, :6], dev[:, 6:8], dev[:, 8:]))
    q = qt if inplace else torch.full((c.T, 6, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kp, vp = c.d["k_pool"].clone(), c.d["v_pool"].clone()
    rope = C.RopeParams(sections, interleaved, adjacent) if sections else None
    C.cosa_chunk_write(c.shape, rope, qt, kt, vt, pos.cuda(), freq.cuda(), c.d["cu"], c.d["kv"], c.d["table"], q, kp, vp)
    torch.cuda.synchronize()
    assert C.cosa_get_status() == 0
    x = both.float().numpy().astype(np.float64)
    q0 = x[:, :6] if inplace else np.full((c.T, 6, D), 7.0)
    wq, wk, wv = K.chunk_write(x[:, :6], x[:, 6:8], x[:, 8:], pos.numpy(), freq.numpy(), sections, interleaved, adjacent,
                               c.cu, c.kv, c.table.numpy(), q0, _np(c.k_pool), _np(c.v_pool))
    # |x| + |y| of a pair is at most twice the largest value
    for got, want in ((q, wq), (kp, wk)):
        got, big = _np(got), 2 * np.abs(x).max()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        ok = np.abs(got - want) <= 2.0**-8 * np.abs(want) + 2.0**-20 * big
        assert (ok | np.isnan(want)).all()
    assert np.array_equal(_np(vp), wv, equal_nan=True)
    assert np.array_equal(_np(q)[int(c.cu[-1]):], q0[int(c.cu[-1]):])


# ---- eviction -------------------------------------------------------------------------------------
@pytest.mark.parametrize("kvs,hk,D,P,budget,sink,recent", [
    ([1, 9, 10, 11, 300], 2, 128, 64, 10, 2, 3), ([5000, 4097, 64], 3, 64, 16, 700, 0, 0),
    ([1000], 1, 128, 128, 999, 4, 100), ([777, 2000], 2, 64, 32, 64, 64, 0), ([777, 2000], 2, 64, 32, 64, 30, 34),
    ([40, 50], 1, 128, 64, 100, 5, 5), ([3000], 1, 128, 64, 1, 0, 0), ([0, 200], 1, 64, 64, 7, 0, 1)])
@pytest.mark.parametrize("kind", ["random", "ties", "special"])
def test_evict_parity(kvs, hk, D, P, budget, sink, recent, kind):
    c = Case([(min(1, kv), kv) for kv in kvs], 2 * hk, hk, D, P, seed=70, extra_pages=0)
    B, g = len(kvs), c.g
    mass = torch.rand(B, hk, c.pps * P, generator=g)
    if kind == "ties":
        mass = torch.randint(0, 3, mass.shape, generator=g).float()
    if kind == "special":
        pick = torch.randint(0, 8, mass.shape, generator=g)
        for i, v in enumerate((float("nan"), float("inf"), -0.0, 0.0, -1.5, float("-inf"))):
            mass[pick == i] = v
    mass[:, :, max(kvs):] = float("nan")
    need = -(-budget // P)
    dst = torch.arange(B * need, dtype=torch.int32).view(B, need) + c.phys
    kp = torch.cat([c.k_pool, torch.full((B * need, hk, P, D), 7.0, dtype=torch.bfloat16)]).cuda()
    vp = torch.cat([c.v_pool, torch.full((B * need, hk, P, D), 7.0, dtype=torch.bfloat16)]).cuda()
    c.shape.num_phys_pages = c.phys + B * need
    before = kp.clone(), vp.clone()
    kept = torch.full((B, hk, budget), -9, dtype=torch.int32, device="cuda")
    mo = torch.full((B, hk, need * P), 7.0, device="cuda")
    kv = c.d["kv"].clone()
    C.cosa_cache_evict(c.shape, C.EvictParams(budget, sink, recent), kp, vp, c.d["table"], kv, mass.cuda(), dst.cuda(), kept,
                       kv, mass_out=mo)  # new_len over kv_len
    torch.cuda.synchronize()
    assert C.cosa_get_status() == 0
    wk, wn, k2, v2, wm = K.cache_evict(_np(before[0]), _np(before[1]), c.table.numpy(), c.kv, mass.numpy(), dst.numpy(), budget,
                                       sink, recent)
    assert np.array_equal(_np(kept), wk) and np.array_equal(_np(kv), wn)
    assert np.array_equal(_np(kp), k2, equal_nan=True) and np.array_equal(_np(vp), v2, equal_nan=True)
    for (b, h), m in wm.items():
        assert np.array_equal(_np(mo)[b, h, :len(m)], m.astype(np.float64), equal_nan=True)
        assert (_np(mo)[b, h, len(m):] == 7).all()
    # without the optional output, new lengths apart
    kept2, n2 = torch.empty_like(kept), torch.empty_like(kv)
    C.cosa_cache_evict(c.shape, C.EvictParams(budget, sink, recent), kp, vp, c.d["table"], c.d["kv"], mass.cuda(), dst.cuda(), kept2, n2)
    assert torch.equal(kept, kept2) and torch.equal(kv, n2)


def test_evict_of_a_cache_past_what_shared_memory_holds():
    kv, P, D, budget = 400001, 128, 64, 1234
    pps = -(-kv // P)
    need = -(-budget // P)
    pool = torch.zeros(pps + need, 1, P, D, dtype=torch.bfloat16, device="cuda")
    pool[:pps].view(-1, D)[:, 0] = (torch.arange(pps * P, device="cuda") % 251).to(torch.bfloat16)
    table = torch.arange(pps, dtype=torch.int32, device="cuda")[None]
    dst = torch.arange(pps, pps + need, dtype=torch.int32, device="cuda")[None]
    g = torch.Generator().manual_seed(1)
    mass = torch.randint(0, 5000, (1, 1, pps * P), generator=g).float()
    s = C.ChunkShape(1, 1, 1, D, P, 1, 1, kv, pps, pps + need)
    kept = torch.empty(1, 1, budget, dtype=torch.int32, device="cuda")
    n = torch.empty(1, dtype=torch.int32, device="cuda")
    C.cosa_cache_evict(s, C.EvictParams(budget, 10, 20), pool, pool, table, torch.tensor([kv], dtype=torch.int32, device="cuda"),
                       mass.cuda(), dst, kept, n)
    m = mass[0, 0].numpy()
    rest = np.arange(10, kv - 20)
    order = rest[np.lexsort((rest, -m[rest]))][:budget - 30]
    want = np.sort(np.concatenate([np.arange(10), order, np.arange(kv - 20, kv)]))
    assert np.array_equal(_np(kept)[0, 0], want) and int(n) == budget
    assert np.array_equal(_np(pool[pps:].view(-1, D)[:budget, 0]), want % 251)


# ---- what is wrong on the device --------------------------------------------------------------------
def test_bad_lengths_leave_their_sequence_out():
    for cu, kv in (([0, 3, 9, 12], [50, 4, 60]),       # more new tokens than keys
                   ([0, 3, 2, 5], [50, 40, 60]),       # cu_q goes back
                   ([0, 3, 6, 4000], [50, 40, 60]),    # past the rows
                   ([0, 3, 6, 9], [50, 10**9, 60]),    # past the bound
                   ([-1, 3, 6, 9], [50, 40, 60])):
        c = Case([(3, 50), (6, 40), (3, 60)], 4, 2, seed=80)
        good = [b for b in range(3) if 0 <= cu[b] <= cu[b + 1] <= c.T and cu[b + 1] - cu[b] <= min(kv[b], c.shape.max_q) and kv[b] <= 60]
        c.d["cu"], c.d["kv"] = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, kv))
        out, lse = c.attend()
        torch.cuda.synchronize()
        assert C.cosa_get_status() == 1
        mass = torch.full((3, 2, c.pps * c.P), 5.0, device="cuda")
        C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass)
        assert C.cosa_get_status() == 1
        kp, vp, q = c.d["k_pool"].clone(), c.d["v_pool"].clone(), torch.full((c.T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        kv_tok = torch.ones(c.T, 2, 128, dtype=torch.bfloat16, device="cuda")
        C.cosa_chunk_write(c.shape, None, c.d["q"], kv_tok, kv_tok, None, None, c.d["cu"], c.d["kv"], c.d["table"], q, kp, vp)
        assert C.cosa_get_status() == 1
        rows = np.zeros(c.T, bool)
        for b in good:
            rows[cu[b]:cu[b + 1]] = True
        for b in range(3):
            assert (b in good) == bool((mass[b] != 5.0).any())
        assert (_np(out)[~rows] == 7).all() and (_np(lse)[~rows] == 7).all() and (_np(q)[~rows] == 7).all()
        assert (_np(lse)[rows] != 7).all()
        assert C.cosa_get_status() == 0


def test_more_tiles_than_rows_give_runs_nothing():
    """Overlapping sequences (cu_q going back and forth) add up to more tiles than the workspace
    has room for: refused on the device as a whole."""
    c = Case([(200, 900)] * 4, 4, 2, seed=81, extra_q=0)
    cu = [0, 800, 0, 800, 0]
    c.d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    c.shape.max_q = 800
    out, lse = c.attend()
    torch.cuda.synchronize()
    assert C.cosa_get_status() == 1
    assert (out == 7).all() and (lse == 7).all()


def test_pages_outside_the_pool_are_reported_and_never_touched():
    for bad in (-1, 2**31 - 1, None):
        c = Case([(3, 200), (2, 100)], 4, 2, seed=82)
        c.d["table"][0, 1] = c.phys if bad is None else bad
        out, lse = c.attend()
        torch.cuda.synchronize()
        assert C.cosa_get_status() == 1
        # its keys read as zeros: scores 0, values 0; the other sequence is untouched by it
        k2, v2 = c.k_pool.clone(), c.v_pool.clone()
        k2[c.table[0, 1]], v2[c.table[0, 1]] = 0, 0
        o, l, spread = K.chunk_attention(_np(c.q), _np(k2), _np(v2), c.table.numpy(), c.cu, c.kv, c.scale)
        n = int(c.cu[-1])
        assert (np.abs(_np(out) - o)[:n] <= ((2.0**-8 + 2 * c.ds({})) * spread + 2.0**-8 * np.abs(o))[:n]).all()
        mass = torch.zeros(2, 2, c.pps * c.P, device="cuda")
        C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass)
        assert C.cosa_get_status() == 1
        assert (mass[0, :, :200].sum(-1) - 6).abs().max() < 1e-3
        # a write behind 64 keys lands on the bad page: only the good sequence's pages change
        c.d["kv"].copy_(torch.tensor([70, 100], dtype=torch.int32))
        kp, vp = c.d["k_pool"].clone(), c.d["v_pool"].clone()
        tok = torch.ones(c.T, 2, 128, dtype=torch.bfloat16, device="cuda")
        C.cosa_chunk_write(c.shape, None, c.d["q"], tok, tok, None, None, c.d["cu"], c.d["kv"], c.d["table"], torch.empty_like(c.d["q"]), kp, vp)
        assert C.cosa_get_status() == 1
        changed = [p for p in range(c.phys) if not torch.equal(torch.nan_to_num(kp[p].float()), torch.nan_to_num(c.d["k_pool"][p].float()))]
        assert set(changed) <= {int(c.table[1, 1])}
        dst = torch.tensor([[0], [c.phys]], dtype=torch.int32, device="cuda")
        kept, n2 = torch.empty(2, 2, 20, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
        before = kp.clone()
        C.cosa_cache_evict(c.shape, C.EvictParams(20), kp, vp, c.d["table"], c.d["kv"], mass, dst, kept, n2)
        assert C.cosa_get_status() == 1
        same = [p for p in range(1, c.phys) if torch.equal(torch.nan_to_num(kp[p].float()), torch.nan_to_num(before[p].float()))]
        assert len(same) == c.phys - 1


@pytest.mark.parametrize("q,D", [(1, 128), (30, 128), (70, 64)])
def test_after_a_timeout_that_nobody_read_nothing_is_written(q, D):
    """A launch that finds COSA_ERR_TIMEOUT pending runs nothing, whatever its workspace held: here
    ones, which as a join list would name row 1 (and lie in range)."""
    from helpers import shape_of, to_dev
    from test_gpu_fault import _case
    wl, x, _, sel = _case()
    xd, shape = to_dev(x), shape_of(wl, x)
    order, count = (torch.from_numpy(sel[n]).cuda() for n in ("order", "count"))
    osk = torch.zeros(wl.batch, wl.num_q_heads, wl.seq_len, 128, dtype=torch.bfloat16, device="cuda")
    c = Case([(q, 900), (q, 500)], 4, 2, D, 64, seed=83)
    want = c.attend()
    ws = torch.ones(C.cosa_chunk_attention_workspace_size(c.shape) // 4, dtype=torch.int32, device="cuda")
    C.cosa_debug_osk_wait_fault(0, 20_000_000)  # the bounded wait of another call runs out
    C.cosa_osk_attention(shape, C.OskParams(1e-4), xd["q"], xd["k_pool"], xd["v_pool"], xd["page_table"], order, count, osk)
    out, lse = c.attend(ws=ws)
    torch.cuda.synchronize()
    assert C.cosa_get_status() == 4
    assert (out == 7).all() and (lse == 7).all()
    got = c.attend(ws=ws)
    assert torch.equal(got[0][:2 * q], want[0][:2 * q]) and torch.equal(got[1][:2 * q], want[1][:2 * q])
    assert C.cosa_get_status() == 0


# ---- a run of them together ---------------------------------------------------------------------------
def test_a_prompt_in_chunks_decoded_and_evicted():
    """A prompt enters in three chunks with rotary positions of three axes, two tokens are decoded, the
    cache is cut by accumulated mass, two more are decoded: every output against the oracle run on
    the cache as the calls left it."""
    hq, hk, D, P, pps = 8, 2, 128, 16, 24
    g = torch.Generator().manual_seed(90)
    phys = 60
    kp, vp = (torch.full((phys, hk, P, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    perm = torch.randperm(phys, generator=g).to(torch.int32)
    table = perm[:2 * pps].view(2, pps).cuda()
    rope, freq = C.RopeParams((24, 20, 20), interleaved=True), (10000.0 ** (-torch.arange(64) / 64)).cuda()
    mass = torch.zeros(2, hk, pps * P, device="cuda")
    kv = np.zeros(2, np.int64)
    seen = np.zeros(2, np.int64)  # true positions, which the eviction does not change

    def step(lens, table, mass, last_q=0):
        nonlocal kv, seen
        T = sum(lens)
        kv, pps_ = kv + np.array(lens), table.shape[1]
        s = C.ChunkShape(2, hq, hk, D, P, T, max(lens), int(kv.max()), pps_, phys)
        cu = torch.tensor([0, lens[0], T], dtype=torch.int32, device="cuda")
        kvd = torch.tensor(kv, dtype=torch.int32, device="cuda")
        qkv = torch.randn(T, hq + 2 * hk, D, generator=g).to(torch.bfloat16).cuda()
        t = torch.cat([torch.arange(seen[b], seen[b] + lens[b]) for b in range(2)])
        pos = torch.stack([t, t // 7, t % 7]).to(torch.int32).cuda()
        seen = seen + np.array(lens)
        q = qkv[:, :hq]
        C.cosa_chunk_write(s, rope, q, qkv[:, hq:hq + hk], qkv[:, hq + hk:], pos, freq, cu, kvd, table, q, kp, vp)
        out = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(T, hq, device="cuda")
        ws = torch.empty(C.cosa_chunk_attention_workspace_size(s), dtype=torch.uint8, device="cuda")
        C.cosa_chunk_attention(s, q, kp, vp, table, cu, kvd, out, ws, lse=lse)
        C.cosa_attention_mass(s, q, kp, table, cu, kvd, lse, mass, last_q=last_q, decay=0.9)
        o, l, spread = K.chunk_attention(_np(q), _np(kp), _np(vp), _np(table), _np(cu), kv, D**-0.5)
        ds = D * 2.0**-24 * D**-0.5 * 40 * 40
        assert (np.abs(_np(out) - o) <= (2.0**-8 + 2 * ds) * spread + 2.0**-8 * np.abs(o)).all()
        assert np.abs(_np(lse) - l).max() <= ds + 2.0**-12
        return s, kvd

    for lens in ([100, 33], [57, 120], [90, 40], [1, 1], [1, 1]):
        s, kvd = step(lens, table, mass)
    dst = perm[2 * pps:2 * pps + 12].view(2, 6).cuda()
    kept = torch.empty(2, hk, 90, dtype=torch.int32, device="cuda")
    small = torch.zeros(2, hk, 6 * P, device="cuda")
    C.cosa_cache_evict(s, C.EvictParams(90, sink=4, recent=16), kp, vp, table, kvd, mass, dst, kept, kvd, mass_out=small)
    assert kvd.tolist() == [90, 90] and (kept[:, :, :4] == torch.arange(4, device="cuda")).all()
    assert torch.equal(small[:, :, :90], torch.gather(mass, 2, kept.long()))
    kv = np.array([90, 90])
    step([1, 1], dst, small)
    step([2, 3], dst, small)
    assert C.cosa_get_status() == 0
