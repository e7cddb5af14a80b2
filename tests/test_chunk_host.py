"""Argument checks of the chunk entry points (no GPU): every bad call is refused on the host
before any CUDA call, by the C interface and by the binding."""
import ctypes

import pytest
import torch

import block_sparse_long_kap_b200 as C

GOOD = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, page_size=64, total_q=10, max_q=6,
            max_kv=200, pages_per_seq=4, num_phys_pages=8)


def _size(**kw):
    s = C.ChunkShape(**{**GOOD, **kw}).c()
    out = ctypes.c_size_t(0)
    return C.lib().cosa_chunk_attention_workspace_size(ctypes.byref(s), ctypes.byref(out)), out.value


@pytest.mark.parametrize("bad,code", [
    (dict(batch=0), 1), (dict(num_kv_heads=3), 1), (dict(total_q=0), 1), (dict(max_q=11), 1),
    (dict(max_q=0), 1), (dict(max_kv=257), 1), (dict(max_kv=5), 1), (dict(pages_per_seq=-1), 1),
    (dict(num_phys_pages=-3), 1), (dict(softmax_scale=-1.0), 1), (dict(softmax_scale=float("nan")), 1),
    (dict(head_dim=96), 2), (dict(page_size=8, pages_per_seq=40), 2), (dict(page_size=48, pages_per_seq=5), 2),
    (dict(page_size=256), 2), (dict(num_q_heads=258, num_kv_heads=2), 2), (dict(batch=4097), 2),
    (dict(num_phys_pages=(1 << 30) + 1), 2)])
def test_shapes_outside_the_supported_set(bad, code):
    assert _size(**bad)[0] == code


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
def test_supported_pages_and_dims(page, dim):
    st, n = _size(page_size=page, head_dim=dim, pages_per_seq=200 // page + 1)
    assert st == 0 and n > 0


def test_workspace_does_not_depend_on_the_cache_length():
    a = _size(max_kv=200)[1]
    b = _size(max_kv=1 << 20, pages_per_seq=1 << 14, num_phys_pages=1 << 15)[1]
    assert a == b
    # partial rows of at most two tiles a CTA and the plan: a decode step needs little, a
    # prompt some tens of megabytes whatever its length
    small = _size(batch=64, total_q=64, max_q=1)[1]
    big = _size(batch=1, total_q=100000, max_q=100000, max_kv=200000, pages_per_seq=4000)[1]
    assert small < 4 << 20 and 36 << 20 < big < 40 << 20


def test_null_and_misaligned_pointers_strides_and_workspace():
    L = C.lib()
    s = C.ChunkShape(**GOOD).c()
    ref, sc = ctypes.byref(s), None
    ws = _size()[1]
    ok = [ref, sc, 16, 8 * 128, 16, 16, 16, 16, 16, 16, None, 256, ws, None]
    for i in (2, 4, 5, 6, 7, 8, 9):
        bad = list(ok)
        bad[i] = None
        assert L.cosa_chunk_attention(*bad) == 1, i
    for i in (2, 4, 5, 9):
        bad = list(ok)
        bad[i] = 8
        assert L.cosa_chunk_attention(*bad) == 1, i
    for stride in (8 * 128 - 8, 8 * 128 + 4, -1024):
        bad = list(ok)
        bad[3] = stride
        assert L.cosa_chunk_attention(*bad) == 1
    for w, n in ((None, ws), (256, ws - 1), (128, ws)):
        bad = list(ok)
        bad[11], bad[12] = w, n
        assert L.cosa_chunk_attention(*bad) == 5
    for cap, window in ((-1.0, 0), (float("inf"), 0), (float("nan"), 0), (0.0, -1)):
        p = C._Score(cap, window, None, None, None)
        bad = list(ok)
        bad[1] = ctypes.byref(p)
        assert L.cosa_chunk_attention(*bad) == 1
    assert L.cosa_chunk_attention(None, *ok[1:]) == 1
    assert L.cosa_chunk_attention_workspace_size(ref, None) == 1


def test_write_checks():
    L = C.lib()
    s = C.ChunkShape(**GOOD).c()
    good = C.RopeParams(sections=(32, 16, 16)).c()

    def call(rope=good, at=None, value=None, **kw):
        a = [ctypes.byref(s), None if rope is None else ctypes.byref(rope), 16, 1024, 16, 256, 16, 256,
             16, 16, 16, 16, 16, 32, 1024, 16, 16, None]
        if at is not None:
            a[at] = value
        return L.cosa_chunk_write(*a)

    for at in (2, 4, 6, 8, 9, 10, 11, 12, 13, 15, 16):
        assert call(at=at, value=None) == 1, at
    for at in (2, 4, 6, 13, 15, 16):
        assert call(at=at, value=24) == 1, at
    for at, value in ((3, 1016), (5, 248), (7, 260), (14, 1000)):
        assert call(at=at, value=value) == 1
    for sec, code in (((3,), 2), ((65,), 1), ((-8, 16), 1), ((0,), 1), ((20,), 2)):
        assert call(C.RopeParams(sections=sec).c()) == code, sec
    for field, value in (("axes", 5), ("axes", -1), ("interleaved", 2), ("adjacent", -1)):
        r = C.RopeParams(sections=(32, 16, 16)).c()
        setattr(r, field, value)
        assert call(r) == 1
    # in place, but with another stride
    a = [ctypes.byref(s), None, 16, 1024, 32, 256, 48, 256, None, None, 64, 64, 64, 16, 2048, 64, 64, None]
    assert L.cosa_chunk_write(*a) == 1


def test_mass_and_evict_checks():
    L = C.lib()
    s = C.ChunkShape(**GOOD).c()
    ref = ctypes.byref(s)
    ok = [ref, None, 16, 1024, 16, 16, 16, 16, 16, 0, 1.0, 16, None]
    for i in (2, 4, 5, 6, 7, 8, 11):
        bad = list(ok)
        bad[i] = None
        assert L.cosa_attention_mass(*bad) == 1, i
    for i, v in ((9, -1), (10, -0.5), (10, float("nan")), (10, float("inf")), (3, 1000)):
        bad = list(ok)
        bad[i] = v
        assert L.cosa_attention_mass(*bad) == 1, (i, v)
    e = C.EvictParams(50, 4, 10).c()
    ok = [ref, ctypes.byref(e), 16, 16, 16, 16, 16, 16, 16, 16, None, None]
    for i in (1, 2, 3, 4, 5, 6, 7, 8, 9):
        bad = list(ok)
        bad[i] = None
        assert L.cosa_cache_evict(*bad) == 1, i
    bad = list(ok)
    bad[6] = bad[10] = 64  # masses written over the ones being read
    assert L.cosa_cache_evict(*bad) == 1
    for budget, sink, recent in ((0, 0, 0), (10, -1, 0), (10, 0, -1), (10, 6, 5),
                                 (10, 2**31 - 1, 2**31 - 1)):
        bad = list(ok)
        x = C.EvictParams(budget, sink, recent).c()
        bad[1] = ctypes.byref(x)
        assert L.cosa_cache_evict(*bad) == 1


def test_binding_refuses_host_tensors_shapes_and_types(monkeypatch):
    monkeypatch.setattr(C, "_current_device", lambda: 0)
    s = C.ChunkShape(**GOOD)
    q = torch.zeros(10, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(8, 2, 64, 128, dtype=torch.bfloat16)
    pt, cu, kv = (torch.zeros(n, dtype=torch.int32) for n in ((2, 4), (3,), (2,)))
    ws = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="current device"):
        C.cosa_chunk_attention(s, q, pool, pool, pt, cu, kv, q, ws)
    with pytest.raises(ValueError, match="shape"):
        C.cosa_chunk_attention(s, q[:9], pool, pool, pt, cu, kv, q, ws)
    with pytest.raises(TypeError, match="dtype"):
        C.cosa_chunk_attention(s, q.float(), pool, pool, pt, cu, kv, q, ws)
    with pytest.raises(ValueError, match="contiguous"):
        C.cosa_chunk_attention(s, q.transpose(1, 2).contiguous().transpose(1, 2), pool, pool, pt, cu, kv, q, ws)
    with pytest.raises(ValueError, match="required"):
        C.cosa_attention_mass(s, None, pool, pt, cu, kv, ws, ws)
    with pytest.raises(ValueError, match="4 rotary axes"):
        C.RopeParams(sections=(8, 8, 8, 8, 8)).c()


@pytest.mark.parametrize("cap", [8.6e37, 3.4e38])
def test_caps_past_what_fp32_can_double_are_refused(cap):
    L, s, ws = C.lib(), C.ChunkShape(**GOOD).c(), _size()[1]
    p = C._Score(cap, 0, None, None, None)
    ref, sc = ctypes.byref(s), ctypes.byref(p)
    assert L.cosa_chunk_attention(ref, sc, 16, 1024, 16, 16, 16, 16, 16, 16, None, 256, ws, None) == 1
    assert L.cosa_attention_mass(ref, sc, 16, 1024, 16, 16, 16, 16, 16, 0, 1.0, 16, None) == 1


@pytest.mark.parametrize("page_size", [0, -16])
def test_binding_of_the_eviction_names_what_is_wrong_with_the_shape(monkeypatch, page_size):
    """(a page size of zero divided the budget)"""
    monkeypatch.setattr(C, "_current_device", lambda: -1)  # where host tensors say they are
    s = C.ChunkShape(**{**GOOD, "page_size": page_size})
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32)
    stream = type("Stream", (), {"cuda_stream": 0})
    with pytest.raises((C.CosaError, ValueError), match="cosa_cache_evict: |shape"):
        pool = torch.zeros(8, 2, max(page_size, 0), 128, dtype=torch.bfloat16)
        C.cosa_cache_evict(s, C.EvictParams(10), pool, pool, i32(2, 4), i32(2), torch.zeros(2, 2, 0), i32(2, 10), i32(2, 2, 10), i32(2),
                           stream=stream)
