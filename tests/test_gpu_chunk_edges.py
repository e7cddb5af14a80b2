"""GPU parity of the chunk operators at the edges of what a call may say.

Tolerances as in test_gpu_chunk.py, but for a capped score, whose error is taken relative to the
score: the polynomial is off by 2^-22.1 of it at most, the exponential's form (used from
|y| = 0.625 on, where tanh y > 0.55) by 2^-21.5, with six fp32 roundings of 2^-24 each at most beside
them: together under 2^-20 |s|.
"""
import numpy as np
import pytest
import torch

import block_sparse_long_kap_b200 as C
from oracle import chunk_oracle as K
from test_gpu_chunk import Case, _np

pytestmark = pytest.mark.gpu


def _check_rows(c, out, lse, kw, ds):
    o, l, spread = c.oracle(kw)
    n = int(c.cu[-1])
    tol = (2.0**-8 + 2 * ds) * spread + 2.0**-8 * np.abs(o)
    assert (np.abs(_np(out) - o)[:n] <= tol[:n]).all()
    assert (np.abs(_np(lse) - l)[:n] <= ds + int(c.kv.max()) * 2.0**-24 + 2.0**-22 * np.abs(l[:n])).all()


def _check_mass(c, score, kw, lse, ds):
    mass = torch.zeros(len(c.lens), c.hk, c.pps * c.P, device="cuda")
    C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass, score=score)
    want = K.attention_mass(_np(c.q), _np(c.k_pool), c.table.numpy(), c.cu, c.kv, _np(lse), np.zeros(mass.shape), c.scale, **kw)
    n = int(c.cu[-1])
    rel = ds + 2.0**-22 * (np.abs(_np(lse)[:n]).max() + 2) + (c.shape.max_q * c.hq // c.hk) * 2.0**-24
    assert (np.abs(_np(mass) - want) <= rel * want + 1e-30).all()


# ---- a cap far above the scores -----------------------------------------------------------------------
FORMS = [(2, 128), (8, 128), (30, 128), (110, 128), (3, 64), (70, 64)]  # transposed, one tile, a pair of tiles


@pytest.mark.parametrize("q,D", FORMS)
@pytest.mark.parametrize("cap", [1e4, 1e6, 1e8, 1e30, 8.5e37])
def test_a_cap_far_above_the_scores_leaves_them(q, D, cap):
    c = Case([(q, 700), (q, 130)], 4, 2, D, 64, seed=100)
    kw = dict(softcap=cap)
    score = C.ScoreParams(softcap=cap)
    raw = c.ds({}) / (D * 2.0**-24)  # scale max|q| . max|k|: no score is larger
    ds = c.ds({}) + 2.0**-20 * raw
    out, lse = c.attend(score)
    _check_rows(c, out, lse, kw, ds)
    _check_mass(c, score, kw, lse, ds)
    assert C.cosa_get_status() == 0


@pytest.mark.parametrize("q,D", FORMS)
@pytest.mark.parametrize("cap", [1e-44, 1e-38])
def test_a_cap_of_nothing_makes_every_score_zero(q, D, cap):
    c = Case([(q, 700), (q, 130)], 4, 2, D, 64, seed=105)
    kw, score = dict(softcap=cap), C.ScoreParams(softcap=cap)
    out, lse = c.attend(score)
    _check_rows(c, out, lse, kw, 2.0**-20)
    _check_mass(c, score, kw, lse, 2.0**-20)


@pytest.mark.parametrize("opt", ["plain", "bias"])
@pytest.mark.parametrize("q,D", FORMS)
def test_one_score_at_the_cap_leaves_the_small_ones_beside_it(q, D, opt):
    """Key 5 of every sequence lies 10^5 below the others and at the cap: it weighs nothing, and
    what is worked out for it must not cost the others their precision."""
    c = Case([(q, 700), (q, 130)], 4, 2, D, 64, seed=101)
    c.q[:, :, 0] = 1.0
    raw = c.ds({}) / (D * 2.0**-24)
    ds = c.ds({}) + 2.0**-20 * raw
    for b in range(2):
        c.k_pool[c.table[b, 0], :, 5] = 0
        c.k_pool[c.table[b, 0], :, 5, 0] = -(2.0**20)
    c.d["q"].copy_(c.q)
    c.d["k_pool"].copy_(c.k_pool)
    kw = dict(softcap=1e5)
    if opt == "bias":
        kw["slopes"] = np.float32(2.0) ** -np.linspace(5, 9, 4).astype(np.float32)
        ds += 700 * 2.0**-5 * 2.0**-22  # the bias, rounded twice
    score = C.ScoreParams(softcap=1e5, slopes=torch.from_numpy(kw["slopes"]).cuda() if "slopes" in kw else None)
    out, lse = c.attend(score)
    _check_rows(c, out, lse, kw, ds)
    _check_mass(c, score, kw, lse, ds)
    assert C.cosa_get_status() == 0


@pytest.mark.parametrize("cap", [20.0, 1e5])
def test_mass_of_many_tiles_under_a_cap(cap):
    """A chunk past two tiles: the streamed form."""
    c = Case([(200, 400)], 8, 2, 128, 64, seed=102)
    kw, score = dict(softcap=cap), C.ScoreParams(softcap=cap)
    ds = c.ds({}) + 2.0**-20 * c.ds({}) / (128 * 2.0**-24)
    out, lse = c.attend(score)
    _check_rows(c, out, lse, kw, ds)
    _check_mass(c, score, kw, lse, ds)


# ---- eviction from a page outside the pool ----------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [-1, 2**31 - 1, None])
def test_kept_keys_of_a_bad_page_arrive_as_zeros(D, bad):
    """A page-table entry outside the pool reads as zeros: before an eviction and after it."""
    P, budget = 64, 150
    c = Case([(1, 200), (1, 170)], 4, 2, D, P, seed=103, extra_pages=0)
    need = -(-budget // P)
    fresh = torch.full((2 * need, 2, P, D), float("nan"), dtype=torch.bfloat16)
    kp, vp = (torch.cat([x, fresh]).cuda() for x in (c.k_pool, c.v_pool))
    c.shape.num_phys_pages = c.phys + 2 * need
    table = c.table.clone()
    table[0, 1] = c.shape.num_phys_pages if bad is None else bad
    dst = torch.arange(2 * need, dtype=torch.int32).view(2, need) + c.phys
    mass = torch.rand(2, 2, c.pps * P, generator=c.g)
    kept = torch.empty(2, 2, budget, dtype=torch.int32, device="cuda")
    n = torch.empty(2, dtype=torch.int32, device="cuda")
    mo = torch.full((2, 2, need * P), 7.0, device="cuda")
    before = kp.clone(), vp.clone()
    C.cosa_cache_evict(c.shape, C.EvictParams(budget, 4, 16), kp, vp, table.cuda(), c.d["kv"], mass.cuda(), dst.cuda(), kept, n,
                       mass_out=mo)
    torch.cuda.synchronize()
    assert C.cosa_get_status() == 1
    # the same with that page there, and zero
    k2, v2 = (np.nan_to_num(_np(x)) for x in before)
    k2[c.table[0, 1]] = v2[c.table[0, 1]] = 0
    wk, wn, k2, v2, wm = K.cache_evict(k2, v2, c.table.numpy(), c.kv, mass.numpy(), dst.numpy(), budget, 4, 16)
    assert np.array_equal(_np(kept), wk) and np.array_equal(_np(n), wn)
    for b in range(2):
        j = np.arange(budget)
        page, slot = dst[b].numpy()[j // P], j % P
        for got, want in ((kp, k2), (vp, v2)):
            assert np.array_equal(_np(got)[page, :, slot], want[page, :, slot])
        for h in range(2):
            assert np.array_equal(_np(mo)[b, h, :budget], wm[b, h].astype(np.float64))
    for got, was in ((kp, before[0]), (vp, before[1])):  # the old pages are as they were
        assert np.array_equal(_np(got)[:c.phys], _np(was)[:c.phys], equal_nan=True)


# ---- lengths that go back ---------------------------------------------------------------------------------
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("cu,lens", [
    ([0, 3, 2, 5], [(3, 50), (6, 40), (3, 60)]),            # rows of two sequences at once
    ([0, 100, 1, 101], [(100, 130), (3, 40), (100, 120)]),  # ninety-nine of them
    ([0, 5, 0, 4, 9], [(5, 60), (2, 30), (4, 44), (5, 70)]),
    ([4, 9, 2, 2, 6], [(5, 60), (2, 30), (1, 44), (4, 70)])])
def test_a_sequence_of_decreasing_ends_leaves_its_neighbours_whole(cu, lens, inplace):
    """Only the sequence whose own ends go back is left out: the others' queries and slots are all
    written, also of rows that two of them own, each row turned once."""
    c = Case(lens, 4, 2, 128, 64, seed=104)
    good = [b for b in range(len(lens)) if cu[b + 1] >= cu[b]]
    c.d["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    g = c.g
    both = torch.randn(c.T, 8, 128, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 16, (1, c.T), generator=g, dtype=torch.int32)
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()
    dev = both.cuda()
    qt, kt, vt = dev[:, :4], dev[:, 4:6], dev[:, 6:]
    q = qt if inplace else torch.full((c.T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    kp, vp = c.d["k_pool"].clone(), c.d["v_pool"].clone()
    C.cosa_chunk_write(c.shape, C.RopeParams((64,)), qt, kt, vt, pos.cuda(), freq.cuda(), c.d["cu"], c.d["kv"], c.d["table"], q, kp, vp)
    torch.cuda.synchronize()
    assert C.cosa_get_status() == 1
    x = both.float().numpy().astype(np.float64)
    wq, wk, wv = x[:, :4] if inplace else np.full((c.T, 4, 128), 7.0), _np(c.k_pool), _np(c.v_pool)
    # (the turned rows do not depend on the sequence: each good one's are taken from one call)
    for b in good:
        wq, wk, wv = K.chunk_write(x[:, :4], x[:, 4:6], x[:, 6:], pos.numpy(), freq.numpy(), (64,), False, False,
                                   np.array([cu[b], cu[b + 1]]), c.kv[b:b + 1], c.table.numpy()[b:b + 1], wq, wk, wv)
    tol = lambda w: 2.0**-8 * np.abs(w) + 2.0**-20 * 2 * np.abs(x).max()
    for got, want in ((q, wq), (kp, wk)):
        got = _np(got)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert ((np.abs(got - want) <= tol(want)) | np.isnan(want)).all()
    assert np.array_equal(_np(vp), wv, equal_nan=True)


# ---- weights of few rows ----------------------------------------------------------------------------------
@pytest.mark.parametrize("lens,hq,hk", [([(1, 2049)], 32, 8), ([(1, 700), (2, 1300), (0, 9)], 28, 4), ([(4, 515)], 16, 4)])
@pytest.mark.parametrize("opt", ["plain", "cap", "bias+prefix"])
def test_few_rows_keep_their_weights_whole(lens, hq, hk, opt):
    """Up to 16 rows at D = 128 the weights meet V as two bf16 halves, 2^-16 of them at most left over:
    beside the scores only the result's own rounding is seen."""
    c = Case(lens, hq, hk, 128, 64, seed=106)
    score, kw = c.score(opt)
    out, lse = c.attend(score)
    o, l, spread = c.oracle(kw)
    n, ds = int(c.cu[-1]), c.ds(kw)
    # fp32 sums over the keys: n 2^-24 of the spread at most, in the products and in the divisor
    tol = (2.0**-16 + 2 * ds + 2 * int(c.kv.max()) * 2.0**-24) * spread + 2.0**-8 * np.abs(o)
    assert (np.abs(_np(out) - o)[:n] <= tol[:n]).all()
    assert C.cosa_get_status() == 0


# ---- large prompts ------------------------------------------------------------------------------------------
def _exact_rows(q, k_pool, v_pool, table, kv, scale, pos0):
    """Causal attention of consecutive tokens of one sequence in 64 bits on the GPU, [tokens][H_q][D]:
    out, lse, sum of w |v|, sum of w^2 v^2."""
    n, hq, hk, P = q.shape[0], q.shape[1], k_pool.shape[1], k_pool.shape[2]
    key = torch.arange(kv, device="cuda")
    pages = table.long()[key // P]
    res = []
    for h in range(hq):
        K_, V_ = (x[pages, h // (hq // hk), key % P].double() for x in (k_pool, v_pool))
        x = q[:, h].double() @ K_.T * scale
        x.masked_fill_(key[None] > pos0 + torch.arange(n, device="cuda")[:, None], -float("inf"))
        w = torch.softmax(x, -1)
        res.append((w @ V_, torch.logsumexp(x, -1), w @ V_.abs(), (w * w) @ (V_ * V_)))
    return [torch.stack(r, 1) for r in zip(*res)]


LARGE = [
    ([(1024, 1024)], 8, 2, 128, 64),               # the whole prompt
    ([(1100, 3001)], 8, 2, 128, 64),               # a piece of one: pairs of tiles cut between CTAs
    ([(1531, 7000)], 4, 4, 64, 16),
    ([(700, 4100), (1, 2000), (1300, 1300)], 7, 1, 128, 128),
]


def _check_large(out, lse, ref, ds, kv):
    o, l, spread, w2v2 = ref
    err = (out.double() - o).abs()
    # for any signs of the roundings
    assert (err <= (2.0**-8 + 2 * ds) * spread + 2.0**-8 * o.abs()).all()
    assert ((lse.double() - l).abs() <= ds + kv * 2.0**-24 + 2.0**-22 * l.abs()).all()
    # The weights' roundings are independent from key to key, each of mean square (2^-8 w)^2 / 3 at most
    # (uniform over half a step of up to 2^-8), so an element's error has a mean square of
    # (2^-8)^2 / 3 (sum w^2 v^2 + o^2); summed over the elements of a row, three times that, and the
    # scores' share for any signs.  A half block of values lost or doubled is ten times as much.
    rms = (2.0**-8) * (w2v2 + o * o).sum(-1).sqrt()
    assert (err.norm(dim=-1) <= rms + 2 * ds * spread.norm(dim=-1)).all()


@pytest.mark.parametrize("lens,hq,hk,D,P", LARGE)
def test_every_element_of_a_large_prompt(lens, hq, hk, D, P):
    """Over a thousand keys random values average to a twentieth of their size: the bounds are those of an
    element's own size and spread, not of V's."""
    c = Case(lens, hq, hk, D, P, seed=107)
    out, lse = c.attend()
    for b, (n, kv) in enumerate(lens):
        rows = slice(int(c.cu[b]), int(c.cu[b]) + n)
        ref = _exact_rows(c.d["q"][rows], c.d["k_pool"], c.d["v_pool"], c.d["table"][b], kv, c.scale, kv - n)
        _check_large(out[rows], lse[rows], ref, c.ds({}), kv)
    assert C.cosa_get_status() == 0


# ---- the prompt's path and the chunks' on one cache ------------------------------------------------------------
@pytest.mark.parametrize("D,P", [(128, 64), (64, 64), (128, 128)])
def test_a_sparse_prefill_decoded_by_chunks(D, P):
    """cosa_prefill_write and the ordered-skipping attention take the prompt (head-major q and lse), the
    chunk calls what comes after it (token-major), on the same pools and page table; the cache is cut and
    decoded on."""
    N, hq, hk, B, budget = 1024, 8, 2, 2, 400
    g = torch.Generator().manual_seed(108)
    pps, need = N // P + 2, -(-budget // P) + 1
    phys = B * (pps + need) + 3
    perm = torch.randperm(phys, generator=g).to(torch.int32)
    table, dst = perm[:B * pps].view(B, pps).cuda(), perm[B * pps:B * (pps + need)].view(B, need).cuda()
    kp, vp = (torch.full((phys, hk, P, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tok = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    q_tok, k_tok, v_tok = tok(B, N, hq, D), tok(B, N, hk, D), tok(B, N, hk, D)
    sh = C.Shape(B, hq, hk, N, D, P, 128, pages_per_seq=pps, num_phys_pages=phys)
    kap = C.KapParams(budget=1.0, q_sub=32, k_sub=16, sink_pages=1)
    q = torch.empty(B, hq, N, D, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(C.cosa_kap_workspace_size(sh, kap), dtype=torch.uint8, device="cuda")
    C.cosa_prefill_write(sh, kap, q_tok, k_tok, v_tok, table, q, kp, vp, workspace=ws)
    order = torch.empty(B, hq, N // 128, C.cosa_kap_kcap(sh, kap), dtype=torch.int32, device="cuda")
    count = torch.empty(B, hq, N // 128, dtype=torch.int32, device="cuda")
    C.cosa_kap_rank(sh, kap, order, count, ws)
    out, lse = torch.empty_like(q), torch.empty(B, hq, N, device="cuda")
    C.cosa_osk_attention(sh, C.OskParams(eps=0.0), q, kp, vp, table, order, count, out, lse=lse)
    ds = D * 2.0**-24 * D**-0.5 * float(q_tok.float().norm(dim=-1).max() * k_tok.float().norm(dim=-1).max())
    # all pages, none skipped: the chunk attention of the whole prompt over the same cache agrees
    s = C.ChunkShape(B, hq, hk, D, P, B * N, N, N, pps, phys)
    cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, N, 2 * N], [N, N]))
    wsc = torch.empty(C.cosa_chunk_attention_workspace_size(s), dtype=torch.uint8, device="cuda")
    o2, l2 = torch.empty(B * N, hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(B * N, hq, device="cuda")
    C.cosa_chunk_attention(s, q_tok.view(B * N, hq, D), kp, vp, table, cu, kv, o2, wsc, lse=l2)
    mass = torch.zeros(B, hk, pps * P, device="cuda")
    C.cosa_attention_mass(s, q_tok.view(B * N, hq, D), kp, table, cu, kv, l2, mass, last_q=16)
    for b in range(B):
        ref = _exact_rows(q_tok[b], kp, vp, table[b], N, D**-0.5, 0)
        _check_large(out[b].transpose(0, 1), lse[b].T, ref, ds, N)
        _check_large(o2[b * N:b * N + N], l2[b * N:b * N + N], ref, ds, N)

    def step(lens, kv, table):
        T, width = sum(lens), table.shape[1]
        s = C.ChunkShape(B, hq, hk, D, P, T, max(lens), int(max(kv)), width, phys)
        x = tok(T, hq + 2 * hk, D)
        cu, kvd = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, lens[0], T], list(kv)))
        qt, o, l = x[:, :hq], torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, hq, device="cuda")
        w = torch.empty(C.cosa_chunk_attention_workspace_size(s), dtype=torch.uint8, device="cuda")
        C.cosa_chunk_write(s, None, qt, x[:, hq:hq + hk], x[:, hq + hk:], None, None, cu, kvd, table, qt, kp, vp)
        C.cosa_chunk_attention(s, qt, kp, vp, table, cu, kvd, o, w, lse=l)
        wo, wl, spread = K.chunk_attention(_np(qt), _np(kp), _np(vp), _np(table), _np(cu), np.array(kv), D**-0.5)
        assert (np.abs(_np(o) - wo) <= (2.0**-8 + 4 * ds) * spread + 2.0**-8 * np.abs(wo)).all()
        assert (np.abs(_np(l) - wl) <= 2 * ds + N * 2.0**-23 + 2.0**-22 * np.abs(wl)).all()
        return s, kvd

    step([1, 1], [N + 1, N + 1], table)
    s, kvd = step([40, 1], [N + 41, N + 2], table)
    kept = torch.empty(B, hk, budget, dtype=torch.int32, device="cuda")
    n = torch.empty(B, dtype=torch.int32, device="cuda")
    C.cosa_cache_evict(s, C.EvictParams(budget, sink=4, recent=64), kp, vp, table, kvd, mass, dst[:, :-(-budget // P)].contiguous(),
                       kept, n)
    assert n.tolist() == [budget, budget]
    step([1, 1], [budget + 1, budget + 1], dst)  # the page after the kept keys' is the next one to fill
    step([3, 20], [budget + 4, budget + 21], dst)
    assert C.cosa_get_status() == 0


# ---- pages that a window has left behind ------------------------------------------------------------------------
@pytest.mark.parametrize("entry", ["none", "another's"])
@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("q,D", FORMS)
def test_pages_before_the_window_may_be_given_up(q, D, P, entry):
    """Their entries name nothing, or a page that holds something else by now (NaN), wherever in a block of
    keys they end: no error, and every key that a token sees is there.  A page with one such key is still
    missed."""
    window = 70
    c = Case([(q, 700), (q, 333)], 4, 2, D, P, seed=109)
    kw, score = dict(window=window), C.ScoreParams(window=window)
    keep = [(kv - q - window + 1) // P for q, kv in c.lens]  # the first page that the first token sees
    free = sorted(set(range(c.phys)) - set(c.table.flatten().tolist()))[0]
    assert torch.isnan(c.v_pool[free].float()).all()
    for b, n in enumerate(keep):
        c.d["table"][b, :max(n, 0)] = -1 if entry == "none" else free
    out, lse = c.attend(score)
    _check_rows(c, out, lse, kw, c.ds({}))
    old = torch.rand(2, 2, c.pps * P, generator=c.g)
    for last in (0, 1):
        mass = old.cuda()
        C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass, score=score, last_q=last)
        want = K.attention_mass(_np(c.q), _np(c.k_pool), c.table.numpy(), c.cu, c.kv, _np(lse), _np(old), c.scale, last_q=last, **kw)
        rel = c.ds({}) + 2.0**-22 * (np.abs(_np(lse)[:2 * q]).max() + 2) + q * 2 * 2.0**-24
        for b, (_, kv) in enumerate(c.lens):
            assert (np.abs(_np(mass) - want)[b, :, :kv] <= rel * want[b, :, :kv] + 1e-30).all()
    assert C.cosa_get_status() == 0
    c.d["table"][1, keep[1]] = -1
    c.attend(score)
    assert C.cosa_get_status() == 1
    C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass, score=score)
    assert C.cosa_get_status() == 1


# ---- more sequences than threads --------------------------------------------------------------------------------
@pytest.mark.parametrize("D,qs", [(128, (1, 0, 2)), (64, (1, 3, 0)), (128, (1, 40, 0))])
def test_batches_past_a_block_of_threads(D, qs):
    """1,300 sequences: past the 256, 384 and 1,024 threads that list them in one go."""
    g = torch.Generator().manual_seed(110)
    B, P = 1300, 16
    kvs = torch.randint(41, 60, (B,), generator=g).tolist()
    c = Case([(qs[b % 3], kvs[b]) for b in range(B)], 4, 2, D, P, seed=111)
    out, lse = c.attend()
    _check_rows(c, out, lse, {}, c.ds({}))
    _check_mass_of_full(c, lse)
    both = torch.randn(c.T, 8, D, generator=g).to(torch.bfloat16).cuda()
    kp, vp = c.d["k_pool"].clone(), c.d["v_pool"].clone()
    q = torch.full((c.T, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    C.cosa_chunk_write(c.shape, None, both[:, :4], both[:, 4:6], both[:, 6:], None, None, c.d["cu"], c.d["kv"], c.d["table"], q, kp, vp)
    assert C.cosa_get_status() == 0
    n = int(c.cu[-1])
    seq = np.repeat(np.arange(B), np.diff(c.cu))
    pos = c.kv[seq] - c.cu[seq + 1] + np.arange(n)
    page, slot = c.table.long()[seq, pos // P], torch.from_numpy(pos % P)
    assert torch.equal(q[:n], both[:n, :4]) and (q[n:] == 7).all()
    wk, wv = c.d["k_pool"].clone(), c.d["v_pool"].clone()
    wk[page, :, slot], wv[page, :, slot] = both[:n, 4:6], both[:n, 6:]
    assert torch.equal(torch.nan_to_num(kp.float(), 99.0), torch.nan_to_num(wk.float(), 99.0))
    assert torch.equal(torch.nan_to_num(vp.float(), 99.0), torch.nan_to_num(wv.float(), 99.0))


def _check_mass_of_full(c, lse):
    """A key's mass, and with it each sequence's: a token gives its group's heads one each."""
    mass = torch.full((len(c.lens), c.hk, c.pps * c.P), 5.0, device="cuda")
    C.cosa_attention_mass(c.shape, c.d["q"], c.d["k_pool"], c.d["table"], c.d["cu"], c.d["kv"], lse, mass, decay=0.0)
    assert C.cosa_get_status() == 0
    ds = c.ds({}) + 2.0**-22 * 12 + 60 * 2.0**-24
    got = _np(mass)
    for b, (n, kv) in enumerate(c.lens):
        if n == 0:
            assert (got[b] == 5).all()
            continue
        assert (np.abs(got[b, :, :kv].sum(-1) - n * c.hq // c.hk) <= ds * (n * c.hq // c.hk)).all()
        assert (got[b, :, kv:] == 5).all()



# ---- calls that nothing above makes ------------------------------------------------------------------------------
@pytest.mark.parametrize("scale", [1e-3, 0.7])
@pytest.mark.parametrize("q,D", FORMS)
def test_a_scale_of_the_callers(q, D, scale):
    c = Case([(q, 400), (q, 130)], 4, 2, D, 64, seed=112)
    c.shape.softmax_scale = scale
    c.scale = np.float32(scale).item()
    kw, score = dict(softcap=50.0), C.ScoreParams(softcap=50.0)
    for kw, score in (({}, None), (kw, score)):
        out, lse = c.attend(score)
        _check_rows(c, out, lse, kw, c.ds(kw))
        _check_mass(c, score, kw, lse, c.ds(kw))


@pytest.mark.parametrize("q", [1, 3])
def test_no_lse_asked_of_the_few_row_form(q):
    c = Case([(q, 3000), (q, 100)], 8, 2, 128, 64, seed=113)
    out, _ = c.attend()
    ws = torch.empty(C.cosa_chunk_attention_workspace_size(c.shape), dtype=torch.uint8, device="cuda")
    out2 = torch.full_like(out, 7.0)
    C.cosa_chunk_attention(c.shape, c.d["q"], c.d["k_pool"], c.d["v_pool"], c.d["table"], c.d["cu"], c.d["kv"], out2, ws)
    assert torch.equal(out, out2)


class _Server:
    """One decode step and the cut behind it: write, attention, mass, eviction, on its own buffers."""

    def __init__(self, seed, D=128, P=32, B=3, pps=40, budget=300):
        g = torch.Generator().manual_seed(seed)
        hq, hk, need = 8, 2, -(-budget // P)
        phys = B * (pps + need)
        perm = torch.randperm(phys, generator=g).to(torch.int32)
        r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
        self.kp, self.vp = r(phys, hk, P, D), r(phys, hk, P, D)
        self.table, self.dst = perm[:B * pps].view(B, pps).cuda(), perm[B * pps:].view(B, need).cuda()
        self.x = r(B, hq + 2 * hk, D)
        self.kv = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros(1, B, dtype=torch.int32, device="cuda")
        self.freq = (10000.0 ** (-torch.arange(D // 2) / (D // 2))).float().cuda()
        self.shape = C.ChunkShape(B, hq, hk, D, P, B, 1, pps * P, pps, phys)
        self.q = torch.empty(B, hq, D, dtype=torch.bfloat16, device="cuda")
        self.out, self.lse = torch.empty_like(self.q), torch.empty(B, hq, device="cuda")
        self.ws = torch.empty(C.cosa_chunk_attention_workspace_size(self.shape), dtype=torch.uint8, device="cuda")
        self.mass = torch.rand(B, hk, pps * P, generator=g).cuda()
        self.kept = torch.empty(B, hk, budget, dtype=torch.int32, device="cuda")
        self.n = torch.empty(B, dtype=torch.int32, device="cuda")
        self.small = torch.empty(B, hk, need * P, device="cuda")
        self.evict, self.hq, self.hk = C.EvictParams(budget, 4, 50), hq, hk
        self.state = {k: v.clone() for k, v in vars(self).items() if torch.is_tensor(v)}

    def set(self, kv):
        for k, v in self.state.items():
            getattr(self, k).copy_(v)
        self.kv.copy_(torch.tensor(kv, dtype=torch.int32))
        self.pos.copy_(self.kv[None] - 1)

    def run(self, stream=None):
        h, k = self.hq, self.hk
        C.cosa_chunk_write(self.shape, C.RopeParams((self.freq.numel(),)), self.x[:, :h], self.x[:, h:h + k], self.x[:, h + k:],
                           self.pos, self.freq, self.cu, self.kv, self.table, self.q, self.kp, self.vp, stream=stream)
        C.cosa_chunk_attention(self.shape, self.q, self.kp, self.vp, self.table, self.cu, self.kv, self.out, self.ws, lse=self.lse,
                               stream=stream)
        C.cosa_attention_mass(self.shape, self.q, self.kp, self.table, self.cu, self.kv, self.lse, self.mass, stream=stream)
        C.cosa_cache_evict(self.shape, self.evict, self.kp, self.vp, self.table, self.kv, self.mass, self.dst, self.kept, self.n,
                           mass_out=self.small, stream=stream)

    def result(self):
        torch.cuda.synchronize()
        res = [x.clone() for x in (self.kp, self.vp, self.q, self.out, self.lse, self.mass, self.kept, self.n)]
        for b, n in enumerate(self.n.tolist()):
            res.append(self.small[b, :, :n].clone())
        return res


LENGTHS = [[1, 1280, 299], [301, 300, 700], [1024, 33, 1279]]


@pytest.mark.parametrize("D", [64, 128])
def test_a_whole_step_captured_and_replayed_with_other_lengths(D):
    s = _Server(114, D)
    want = []
    for kv in LENGTHS:
        s.set(kv)
        s.run()
        want.append(s.result())
    s.set(LENGTHS[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for kv, w in zip(LENGTHS, want):
        s.set(kv)
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(s.result(), w))
    assert C.cosa_get_status() == 0


def test_two_whole_steps_at_once_on_two_streams():
    a, b = _Server(115), _Server(116, 64, 16, pps=80)
    want = []
    for s in (a, b):
        s.set(LENGTHS[2])
        s.run()
        want.append(s.result())
        s.set(LENGTHS[2])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s, st in zip((a, b), streams):
        s.run(stream=st)
    for s, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(s.result(), w))
    assert C.cosa_get_status() == 0


def test_pools_and_rows_past_what_32_bits_count():
    """Pages and query rows whose elements lie past 2^31, and tokens at the end of a long row list."""
    P, hk, hq, D, n = 64, 2, 4, 128, 5
    phys = 2**31 // (hk * P * D) + 40
    kp, vp = (torch.empty(phys, hk, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    T, width = 270000, 8000  # 2.16e9 elements of a fused projection
    fused = torch.empty(T, width, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(117)
    kv, pps = 1000, 16
    table = torch.arange(phys - 20, phys - 20 + pps, dtype=torch.int32)[None]
    small = [torch.randn(pps, hk, P, D, generator=g).to(torch.bfloat16) for _ in range(2)]
    for pool, x in zip((kp, vp), small):
        pool[phys - 20:phys - 20 + pps] = x.cuda()
    tok = torch.randn(n, (hq + 2 * hk) * D, generator=g).to(torch.bfloat16)
    fused[T - n:, :tok.shape[1]] = tok.cuda()
    rows = fused[:, :tok.shape[1]].view(T, hq + 2 * hk, D)
    sh = C.ChunkShape(1, hq, hk, D, P, T, n, kv, pps, phys)
    cu, kvd = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([T - n, T], [kv]))
    td = table.cuda()
    qr = rows[:, :hq]
    C.cosa_chunk_write(sh, None, qr, rows[:, hq:hq + hk], rows[:, hq + hk:], None, None, cu, kvd, td, qr, kp, vp)
    out = torch.zeros(T, hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(T, hq, device="cuda")
    ws = torch.empty(C.cosa_chunk_attention_workspace_size(sh), dtype=torch.uint8, device="cuda")
    mass = torch.zeros(1, hk, pps * P, device="cuda")
    xs = tok.view(n, hq + 2 * hk, D).float().numpy().astype(np.float64)
    q, (sk, sv) = xs[:, :hq], (_np(x) for x in small)
    near = np.arange(pps)[None]
    _, sk, sv = K.chunk_write(q, xs[:, hq:hq + hk], xs[:, hq + hk:], None, None, (), False, False, np.array([0, n]),
                              np.array([kv]), near, q, sk, sv)
    o, l, spread = K.chunk_attention(q, sk, sv, near, np.array([0, n]), np.array([kv]), D**-0.5)
    ds = D * 2.0**-24 * D**-0.5 * np.linalg.norm(q, axis=-1).max() * np.linalg.norm(sk, axis=-1).max()
    C.cosa_chunk_attention(sh, qr, kp, vp, td, cu, kvd, out, ws, lse=lse)
    assert (np.abs(_np(out[T - n:]) - o) <= (2.0**-8 + 2 * ds) * spread + 2.0**-8 * np.abs(o)).all()
    assert (np.abs(_np(lse[T - n:]) - l) <= ds + kv * 2.0**-24 + 2.0**-22 * np.abs(l)).all()
    sh.max_q = kv  # a looser bound: the tiled form
    ws = torch.empty(C.cosa_chunk_attention_workspace_size(sh), dtype=torch.uint8, device="cuda")
    out.zero_()
    C.cosa_chunk_attention(sh, qr, kp, vp, td, cu, kvd, out, ws, lse=lse)
    assert (np.abs(_np(out[T - n:]) - o) <= (2.0**-8 + 2 * ds) * spread + 2.0**-8 * np.abs(o)).all()
    assert not out[:T - n].any()
    C.cosa_attention_mass(sh, qr, kp, td, cu, kvd, lse, mass)
    want = K.attention_mass(q, sk, near, np.array([0, n]), np.array([kv]), _np(lse[T - n:]), np.zeros((1, hk, pps * P)), D**-0.5)
    rel = ds + 2.0**-22 * (np.abs(l).max() + 2) + n * 2 * 2.0**-24
    assert (np.abs(_np(mass) - want) <= rel * want + 1e-30).all()
    dst = torch.arange(phys - 4, phys, dtype=torch.int32, device="cuda")[None]
    kept, left = torch.empty(1, hk, 200, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
    C.cosa_cache_evict(sh, C.EvictParams(200, 4, 20), kp, vp, td, kvd, mass, dst, kept, left)
    assert C.cosa_get_status() == 0 and int(left) == 200
    for h in range(hk):
        src = _np(kept)[0, h]
        assert (np.diff(src) > 0).all()
        for pool, x in ((kp, sk), (vp, sv)):
            got = _np(pool[phys - 4:])[:, h].reshape(-1, D)[:200]
            assert np.array_equal(got, x[src // P, h, src % P])


@pytest.mark.parametrize("opt", ["plain", "cap", "prefix", "window"])
@pytest.mark.parametrize("q,D", FORMS)
def test_slopes_of_either_sign(q, D, opt):
    """A falling, a rising and no slope at all side by side: far keys ahead of near ones in some heads."""
    c = Case([(q, 1900), (q, 130)], 8, 2, D, 64, seed=118)
    score, kw = c.score(opt)
    kw["slopes"] = np.array([0.5, -0.5, 0.0, -0.01, 2.0, -2.0, 0.001, -30.0], np.float32)
    score.slopes = torch.from_numpy(kw["slopes"]).cuda()
    out, lse = c.attend(score)
    # the bias is rounded as a product with log2 e and as a sum: 2^-22 of it, where it weighs at all (within
    # 60 of the row's largest, which is at a distance of 1900 at most)
    ds = c.ds(kw) + 1900 * 30.0 * 2.0**-22
    _check_rows(c, out, lse, kw, ds)
    _check_mass(c, score, kw, lse, ds)
    assert C.cosa_get_status() == 0


@pytest.mark.parametrize("cap", [5.0, 50.0])
@pytest.mark.parametrize("q,D", [(1, 64), (20, 64), (300, 64), (2, 128), (200, 128)])
def test_mass_under_a_cap_is_as_exact_as_without(q, D, cap):
    """Small scores: the cap's own error, 2^-20 of a score, is next to nothing beside the fp32 product's."""
    c = Case([(q, 700), (min(q, 90), 90)], 4, 2, D, 64, seed=119, spread=0.01)
    kw, score = dict(softcap=cap), C.ScoreParams(softcap=cap)
    ds = c.ds({}) + 2.0**-20 * c.ds({}) / (D * 2.0**-24)
    out, lse = c.attend(score)
    _check_mass(c, score, kw, lse, ds)


def test_a_decreasing_end_among_thousands_of_sequences_is_looked_over_in_passing():
    """4,096 sequences of eight tokens, one of whose ends goes back by sixteen: two others' rows are owned
    twice, all are written, and the call stays a call of milliseconds."""
    B, n, P, D = 4096, 8, 16, 64
    ends = np.arange(B + 1, dtype=np.int32) * n
    ends[2000] -= 16
    sh = C.ChunkShape(B, 1, 1, D, P, B * n, 24, 32, 2, 2 * B)
    g = torch.Generator().manual_seed(120)
    x = torch.randn(B * n, 3, D, generator=g).to(torch.bfloat16).cuda()
    table = torch.arange(2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    cu, kv = torch.from_numpy(ends).cuda(), torch.full((B,), 24, dtype=torch.int32, device="cuda")
    kp, vp = (torch.full((2 * B, 1, P, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.full((B * n, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    times = []
    for _ in range(3):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        C.cosa_chunk_write(sh, None, x[:, :1], x[:, 1:2], x[:, 2:], None, None, cu, kv, table, q, kp, vp)
        e[1].record()
        torch.cuda.synchronize()
        times.append(e[0].elapsed_time(e[1]))
        assert C.cosa_get_status() == 1
    assert min(times) < 500
    want = torch.full((B, 2 * P, D), 7.0, dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        m = int(ends[b + 1] - ends[b])
        if m > 0:
            want[b, 24 - m:24] = x[int(ends[b]):int(ends[b + 1]), 1]
    assert torch.equal(kp.view(B, 2 * P, D), want)
    assert torch.equal(q, x[:, :1])

