"""Pins of the chunk operators' CPU oracle: closed forms, torch's own attention in float64 and
brute force, none of them sharing code with it."""
import math

import numpy as np
import pytest
import torch

from oracle import chunk_oracle as K


def _cache(rng, B, H, P, D, pps):
    phys = B * pps + 2
    table = rng.permutation(phys)[:B * pps].reshape(B, pps).astype(np.int32)
    return rng.standard_normal((phys, H, P, D)), rng.standard_normal((phys, H, P, D)), table


def _logical(pool, table, b, n):
    return np.concatenate([pool[p] for p in table[b]], axis=1)[:, :n]


@pytest.mark.parametrize("interleaved,sections,want", [
    (False, (3, 2, 1), [0, 0, 0, 1, 1, 2]),
    (True, (4, 2, 2), [0, 1, 2, 0, 1, 2, 0, 0]),
    (True, (5,), [0, 0, 0, 0, 0]),
    (True, (6, 1), [0, 1, 0, 0, 0, 0, 0])])
def test_axis_of_pairs(interleaved, sections, want):
    assert K.rope_axis_of(sections, interleaved) == want


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_is_a_complex_product_and_keeps_relative_angles(adjacent):
    rng = np.random.default_rng(0)
    T, D, sec = 5, 16, (6,)
    x, pos = rng.standard_normal((T, 1, D)), rng.integers(0, 1000, (1, T))
    f = 10000.0 ** (-np.arange(6) / 6)
    y = K._rotate(x, pos, f, sec, False, adjacent)
    z = x[..., 0:12:2] + 1j * x[..., 1:12:2] if adjacent else x[..., :6] + 1j * x[..., 6:12]
    z = z * np.exp(1j * pos[0][:, None, None] * f)
    got = y[..., 0:12:2] + 1j * y[..., 1:12:2] if adjacent else y[..., :6] + 1j * y[..., 6:12]
    assert np.allclose(got, z, atol=1e-12) and np.array_equal(y[..., 12:], x[..., 12:])
    # products depend on the difference of positions alone
    a = K._rotate(x, pos, f, sec, False, adjacent)[:, 0] @ K._rotate(x, pos, f, sec, False, adjacent)[:, 0].T
    b = K._rotate(x, pos + 77, f, sec, False, adjacent)[:, 0] @ K._rotate(x, pos + 77, f, sec, False, adjacent)[:, 0].T
    assert np.allclose(a, b, atol=1e-9)


def test_write_places_tokens_behind_the_keys():
    rng = np.random.default_rng(1)
    kp, vp, table = _cache(rng, 2, 2, 4, 16, 3)
    cu, kv = np.array([0, 3, 5]), np.array([7, 2])
    q, k, v = (rng.standard_normal((6, h, 16)) for h in (4, 2, 2))
    q2, k2, v2 = K.chunk_write(q, k, v, None, None, (), False, False, cu, kv, table, np.zeros_like(q), kp, vp)
    for b in range(2):
        n = cu[b + 1] - cu[b]
        assert np.array_equal(_logical(k2, table, b, kv[b])[:, kv[b] - n:], k[cu[b]:cu[b + 1]].swapaxes(0, 1))
        assert np.array_equal(_logical(v2, table, b, kv[b])[:, :kv[b] - n], _logical(vp, table, b, kv[b] - n))
    assert np.array_equal(q2[:5], q[:5]) and not q2[5].any()
    assert (k2 != kp).any(-1).sum() == 5 * 2


@pytest.mark.parametrize("opt", ["plain", "window", "docs", "prefix", "bias"])
def test_attention_against_torch_with_an_explicit_mask(opt):
    rng = np.random.default_rng(2)
    B, Hq, H, P, D = 2, 4, 2, 4, 8
    kp, vp, table = _cache(rng, B, H, P, D, 5)
    cu, kv = np.array([0, 5, 9]), np.array([17, 4])
    q = rng.standard_normal((9, Hq, D))
    kw = {}
    if opt == "window":
        kw["window"] = 3
    if opt == "docs":
        kw["first_key"] = np.array([0, 12, 12, 15, 17, 0, 1, 1, 3], np.int32)
    if opt == "prefix":
        kw["prefix_len"] = np.array([15, 2], np.int32)
    if opt == "bias":
        kw["slopes"] = np.array([0.5, 0.25, 0.1, 0.0])
    out, lse, _ = K.chunk_attention(q, kp, vp, table, cu, kv, 0.3, **kw)
    for b in range(B):
        n = cu[b + 1] - cu[b]
        t = kv[b] - n + np.arange(n)
        key = np.arange(kv[b])
        mask = key[None] <= t[:, None]
        if opt == "window":
            mask &= key[None] > t[:, None] - 3
        if opt == "docs":
            mask &= key[None] >= kw["first_key"][cu[b]:cu[b + 1], None]
        if opt == "prefix":
            mask |= (key < kw["prefix_len"][b])[None]
        bias = np.where(mask, 0.0, -np.inf)[None].repeat(Hq, 0)
        if opt == "bias":
            bias = bias - kw["slopes"][:, None, None] * np.abs(t[:, None] - key[None])
        Kb = torch.from_numpy(_logical(kp, table, b, kv[b]).repeat(2, 0))
        Vb = torch.from_numpy(_logical(vp, table, b, kv[b]).repeat(2, 0))
        qb = torch.from_numpy(q[cu[b]:cu[b + 1]].swapaxes(0, 1).copy())
        want = torch.nn.functional.scaled_dot_product_attention(
            qb[None], Kb[None], Vb[None], attn_mask=torch.from_numpy(bias)[None], scale=0.3)[0].numpy()
        s = (qb @ Kb.transpose(-1, -2)).numpy() * 0.3 + bias
        for i in range(n):
            if not mask[i].any():
                assert not out[cu[b] + i].any() and np.isinf(lse[cu[b] + i]).all()
            else:
                assert np.allclose(out[cu[b] + i], want[:, i], atol=1e-12)
                assert np.allclose(lse[cu[b] + i], np.log(np.exp(s[:, i]).sum(-1)), atol=1e-12)


def test_cap_bounds_scores_and_vanishes_when_large():
    rng = np.random.default_rng(3)
    kp, vp, table = _cache(rng, 1, 1, 4, 8, 3)
    q = rng.standard_normal((2, 2, 8))
    cu, kv = np.array([0, 2]), np.array([10])
    a = K.chunk_attention(q, kp, vp, table, cu, kv, 1.0)
    b = K.chunk_attention(q, kp, vp, table, cu, kv, 1.0, softcap=1e6)
    assert np.allclose(a[0], b[0], atol=1e-9) and np.allclose(a[1], b[1], atol=1e-9)
    tiny = K.chunk_attention(q, kp, vp, table, cu, kv, 1.0, softcap=1e-9)
    assert np.allclose(tiny[1][1], math.log(10), atol=1e-6)  # all scores equal


def test_mass_of_all_rows_adds_up_to_their_number():
    rng = np.random.default_rng(4)
    kp, vp, table = _cache(rng, 2, 2, 4, 8, 4)
    cu, kv = np.array([0, 6, 7]), np.array([13, 9])
    q = rng.standard_normal((7, 4, 8))
    _, lse, _ = K.chunk_attention(q, kp, vp, table, cu, kv, 0.4)
    old = rng.random((2, 2, 16))
    m = K.attention_mass(q, kp, table, cu, kv, lse, old, 0.4, decay=0.0)
    assert np.allclose(m[0, :, :13].sum(-1), 12) and np.allclose(m[1, :, :9].sum(-1), 2)
    assert np.array_equal(m[0, :, 13:], old[0, :, 13:])
    m2 = K.attention_mass(q, kp, table, cu, kv, lse, old, 0.4, decay=0.5)
    assert np.allclose(m2[0, :, :7] - m[0, :, :7], 0.5 * old[0, :, :7])
    assert np.allclose(m2[0, :, 7:], m[0, :, 7:])  # new keys start from nothing
    last = K.attention_mass(q, kp, table, cu, kv, lse, old, 0.4, last_q=2, decay=0.0)
    assert np.allclose(last[0, :, :13].sum(-1), 4)


def test_eviction_keeps_the_heaviest_by_enumeration():
    import itertools
    rng = np.random.default_rng(5)
    kp, vp, table = _cache(rng, 1, 2, 4, 8, 4)
    dst = np.array([[0, 1]], np.int32)
    mass = rng.integers(0, 4, (1, 2, 16)).astype(np.float32)  # many ties
    kept, n, k2, v2, _ = K.cache_evict(kp, vp, table, np.array([11]), mass, dst, 6, 1, 2)
    assert n[0] == 6
    for h in range(2):
        assert kept[0, h, 0] == 0 and list(kept[0, h, -2:]) == [9, 10]
        best = max(itertools.combinations(range(1, 9), 3), key=lambda c: (mass[0, h, list(c)].sum(), [-i for i in c]))
        assert mass[0, h, list(best)].sum() == mass[0, h, kept[0, h, 1:4]].sum()
        border = mass[0, h, kept[0, h, 1:4]].min()
        ties = [k for k in range(1, 9) if mass[0, h, k] == border]
        took = [k for k in kept[0, h, 1:4] if mass[0, h, k] == border]
        assert took == ties[:len(took)]
        for j, k in enumerate(kept[0, h]):
            assert np.array_equal(k2[dst[0, j // 4], h, j % 4], kp[table[0, k // 4], h, k % 4])
