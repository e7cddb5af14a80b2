"""CPU oracle of the chunk operators (numpy, float64): the rotary cache write, attention of
new tokens over a paged cache, the accumulated attention mass of its keys, and eviction by
that mass.  One function per operator, written from the formulas in include/cosa.h, one
sequence and head at a time; it shares no code with the CUDA path.

Arguments are numpy arrays with the layouts of include/cosa.h; nothing is modified, results
are returned (pools as new float64 arrays).
"""
from __future__ import annotations

import numpy as np

__all__ = ["chunk_write", "chunk_attention", "attention_mass", "cache_evict", "rope_axis_of",
           "visible"]


def rope_axis_of(sections, interleaved):
    """The axis that turns each rotary pair."""
    axes, out = len(sections), []
    for j in range(sum(sections)):
        if interleaved:
            a = j % axes
            out.append(a if a > 0 and j < axes * sections[a] else 0)
        else:
            a = 0
            while j >= sum(sections[:a + 1]):
                a += 1
            out.append(a)
    return out


def _rotate(x, positions, inv_freq, sections, interleaved, adjacent):
    """x [T][H][D]."""
    y = np.array(x, dtype=np.float64)
    half = sum(sections)
    for j, axis in enumerate(rope_axis_of(sections, interleaved)):
        i0, i1 = (2 * j, 2 * j + 1) if adjacent else (j, j + half)
        w = positions[axis].astype(np.float64) * np.float64(inv_freq[j])
        c, s = np.cos(w)[:, None], np.sin(w)[:, None]
        y[..., i0] = x[..., i0] * c - x[..., i1] * s
        y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def chunk_write(q_tok, k_tok, v_tok, positions, inv_freq, sections, interleaved, adjacent, cu_q,
                kv_len, page_table, q, k_pool, v_pool):
    """(q, k_pool, v_pool) after the call; rows and slots that it does not write keep theirs."""
    q, k_pool, v_pool = (np.array(a, dtype=np.float64) for a in (q, k_pool, v_pool))
    P = k_pool.shape[2]
    if sections:
        qr = _rotate(q_tok, positions, inv_freq, sections, interleaved, adjacent)
        kr = _rotate(k_tok, positions, inv_freq, sections, interleaved, adjacent)
    else:
        qr, kr = q_tok.astype(np.float64), k_tok.astype(np.float64)
    for b in range(len(kv_len)):
        n = cu_q[b + 1] - cu_q[b]
        for i in range(n):
            t, tok = kv_len[b] - n + i, cu_q[b] + i
            page = page_table[b, t // P]
            q[tok] = qr[tok]
            k_pool[page, :, t % P] = kr[tok]
            v_pool[page, :, t % P] = v_tok[tok]
    return q, k_pool, v_pool


def visible(t, kv, window=0, first_key=0, prefix=0):
    """Which of kv keys a token at position t sees (bool [kv])."""
    k = np.arange(kv)
    lo = max(first_key, t - window + 1) if window > 0 else first_key
    return (k >= lo) & ((k <= t) | (k < prefix))


def _scores(qv, keys, scale, softcap, slope, t):
    s = keys @ qv * scale
    if softcap > 0:
        s = softcap * np.tanh(s / softcap)
    if slope is not None:
        s = s - slope * np.abs(t - np.arange(len(keys)))
    return s


def _keys(pool, table, b, h, kv):
    P = pool.shape[2]
    k = np.arange(kv)
    return np.asarray(pool[table[b][k // P], h, k % P], dtype=np.float64)


def chunk_attention(q, k_pool, v_pool, page_table, cu_q, kv_len, scale, softcap=0.0, window=0,
                    slopes=None, first_key=None, prefix_len=None):
    """(out, lse, spread): spread is sum of weight * |v| per output element, the scale of its
    rounding errors.  Rows past the last sequence are zero."""
    T, Hq, D = q.shape
    G = Hq // k_pool.shape[1]
    out, spread = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    for b in range(len(kv_len)):
        n, kv = int(cu_q[b + 1] - cu_q[b]), int(kv_len[b])
        if n == 0:
            continue
        for h in range(Hq):
            K = _keys(k_pool, page_table, b, h // G, kv)
            V = _keys(v_pool, page_table, b, h // G, kv)
            for i in range(n):
                t, tok = kv - n + i, int(cu_q[b]) + i
                m = visible(t, kv, window, 0 if first_key is None else int(first_key[tok]),
                            0 if prefix_len is None else int(prefix_len[b]))
                if not m.any():
                    continue
                s = _scores(q[tok, h].astype(np.float64), K, scale, softcap,
                            None if slopes is None else float(slopes[h]), t)[m]
                top = s.max()
                w = np.exp(s - top)
                lse[tok, h] = top + np.log(w.sum())
                w /= w.sum()
                out[tok, h] = w @ V[m]
                spread[tok, h] = w @ np.abs(V[m])
    return out, lse, spread


def attention_mass(q, k_pool, page_table, cu_q, kv_len, lse, mass, scale, last_q=0, decay=1.0,
                   softcap=0.0, window=0, slopes=None, first_key=None, prefix_len=None):
    """mass after the call."""
    mass = np.array(mass, dtype=np.float64)
    Hq = q.shape[1]
    G = Hq // k_pool.shape[1]
    for b in range(len(kv_len)):
        n, kv = int(cu_q[b + 1] - cu_q[b]), int(kv_len[b])
        if n == 0:
            continue
        for hk in range(k_pool.shape[1]):
            K = _keys(k_pool, page_table, b, hk, kv)
            add = np.zeros(kv)
            for i in range(max(0, n - last_q) if last_q > 0 else 0, n):
                t, tok = kv - n + i, int(cu_q[b]) + i
                m = visible(t, kv, window, 0 if first_key is None else int(first_key[tok]),
                            0 if prefix_len is None else int(prefix_len[b]))
                for h in range(hk * G, hk * G + G):
                    s = _scores(q[tok, h].astype(np.float64), K, scale, softcap,
                                None if slopes is None else float(slopes[h]), t)
                    add[m] += np.exp(s[m] - float(lse[tok, h]))
            old = mass[b, hk, :kv].copy()
            old[kv - n:] = 0.0
            old = decay * old if decay else np.zeros(kv)
            mass[b, hk, :kv] = old + add
    return mass


def cache_evict(k_pool, v_pool, page_table, kv_len, mass, dst_table, budget, sink, recent):
    """(kept, new_len, k_pool, v_pool, {(b, h): kept masses})."""
    k_pool, v_pool = np.array(k_pool), np.array(v_pool)
    src_k, src_v = k_pool.copy(), v_pool.copy()
    B, H, P = len(kv_len), k_pool.shape[1], k_pool.shape[2]
    kept = np.full((B, H, budget), -1, np.int32)
    new_len, masses = np.minimum(kv_len, budget).astype(np.int32), {}
    for b in range(B):
        kv, n = int(kv_len[b]), int(new_len[b])
        for h in range(H):
            if kv <= budget:
                keep = list(range(kv))
            else:
                keep = list(range(sink)) + list(range(kv - recent, kv))
                rest = list(range(sink, kv - recent))
                v = mass[b, h].astype(np.float64)
                # the largest first; NaN below everything; equal ones by position
                rest.sort(key=lambda k: (np.isnan(v[k]), 0.0 if np.isnan(v[k]) else -v[k], k))
                keep = sorted(keep + rest[:budget - sink - recent])
            kept[b, h, :n] = keep
            masses[b, h] = mass[b, h, keep]
            for j, k in enumerate(keep):
                f, d = page_table[b, k // P], dst_table[b, j // P]
                k_pool[d, h, j % P] = src_k[f, h, k % P]
                v_pool[d, h, j % P] = src_v[f, h, k % P]
    return kept, new_len, k_pool, v_pool, masses
