"""Refusals of the event-history calls, checked on the host before anything touches a device."""
import ctypes

import pytest
import torch

import dlrm_embedding_interaction_amd as dl
from dlrm_embedding_interaction_amd import history as hi

P = 4096    # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    return dl.load()


def att(dtype=0, heads=4, kv=2, dim=64, window=10, sinks=0, scale=0.125):
    return hi._Attention(dtype, heads, kv, dim, window, sinks, scale, 0)


def cache(n_pages=10, page=16, kv=2, dim=64, slots=4, max_pages=8, ptr=P):
    return hi._Cache(n_pages, page, kv, dim, slots, max_pages, *([ptr] * 9))


def encode(lib, a, batch=2, n=10, off=P, ib=8, q=P, ldq=256, k=P, ldk=128, v=P, ldv=128, out=P, ldo=256):
    return lib.dlrm_history_attention(ctypes.byref(a) if a is not None else None, batch, n, off, ib, q, ldq, k, ldk,
                                      v, ldv, None, out, ldo, None)


def test_encode_refusals(lib):
    assert encode(lib, None) == dl.DLRM_E_NULL
    for name in ("off", "q", "k", "v", "out"):
        assert encode(lib, att(), **{name: None}) == dl.DLRM_E_NULL
    bad = [att(dtype=3), att(dtype=-1), att(heads=3), att(heads=0), att(kv=0), att(dim=0), att(window=0),
           att(window=-5), att(sinks=-1), att(scale=float("nan")), att(scale=float("inf"))]
    for a in bad:
        assert encode(lib, a) == dl.DLRM_E_SHAPE
    for a in (att(dim=48), att(dim=256), att(heads=8192)):
        assert encode(lib, a) == dl.DLRM_E_UNSUPPORTED
    for kw in (dict(batch=0), dict(n=-1), dict(ib=2), dict(ldq=255), dict(ldk=127), dict(ldv=127), dict(ldo=255)):
        assert encode(lib, att(), **kw) == dl.DLRM_E_SHAPE
    assert encode(lib, att(), n=1 << 31) == dl.DLRM_E_UNSUPPORTED
    assert encode(lib, att(), batch=1 << 31) == dl.DLRM_E_UNSUPPORTED
    assert encode(lib, att(), n=0, q=None, k=None, v=None, out=None) == dl.DLRM_OK    # nothing to do, no launch


def test_cache_refusals(lib):
    ref = ctypes.byref
    ws, big = 4096, 1 << 40
    calls = {
        "init": lambda c: lib.dlrm_history_init(c, None),
        "append": lambda c: lib.dlrm_history_append(c, 2, None, 0, 4, P, 8, P, 128, P, 128, ws, big, None),
        "lookup": lambda c: lib.dlrm_history_lookup(c, ref(att()), 2, None, 1, P, 256, P, 256, ws, big, None),
        "fork": lambda c: lib.dlrm_history_fork(c, 1, P, P, ws, big, None),
        "truncate": lambda c: lib.dlrm_history_truncate(c, 1, P, P, ws, big, None),
        "trim": lambda c: lib.dlrm_history_trim(c, 1, P, 10, 0, ws, big, None),
        "compact": lambda c: lib.dlrm_history_compact(c, ws, big, None),
    }
    for name, call in calls.items():
        assert call(None) == dl.DLRM_E_NULL, name
        assert call(ref(cache(ptr=None))) == dl.DLRM_E_NULL, name
        for kw in (dict(n_pages=0), dict(page=0), dict(kv=0), dict(dim=0), dict(slots=0), dict(max_pages=0)):
            assert call(ref(cache(**kw))) == dl.DLRM_E_SHAPE, (name, kw)
        for kw in (dict(page=128), dict(page=8), dict(dim=96), dict(kv=5000), dict(max_pages=1 << 28),
                   dict(n_pages=(1 << 30) + 1)):
            assert call(ref(cache(**kw))) == dl.DLRM_E_UNSUPPORTED, (name, kw)
        c = cache()
        c.k = P + 8
        assert call(ref(c)) == dl.DLRM_E_SHAPE, name


def test_append_refusals(lib):
    c = ctypes.byref(cache())
    need = lib.dlrm_history_workspace_bytes(c, 2, 0, 0)
    assert need > 0

    def f(batch=2, slots=None, dtype=0, n=4, off=P, ib=8, k=P, ldk=128, v=P, ldv=128, ws=P, size=need):
        return lib.dlrm_history_append(c, batch, slots, dtype, n, off, ib, k, ldk, v, ldv, ws, size, None)
    for kw in (dict(off=None), dict(k=None), dict(v=None)):
        assert f(**kw) == dl.DLRM_E_NULL
    for kw in (dict(batch=0), dict(n=-1), dict(dtype=5), dict(ib=3), dict(ldk=127), dict(ldv=1), dict(batch=5)):
        assert f(**kw) == dl.DLRM_E_SHAPE
    assert f(n=1 << 31) == dl.DLRM_E_UNSUPPORTED
    assert f(slots=P, batch=1 << 30) == dl.DLRM_E_UNSUPPORTED
    for kw in (dict(ws=None), dict(size=16), dict(ws=P + 16)):
        assert f(**kw) == dl.DLRM_E_WORKSPACE


def test_lookup_refusals(lib):
    c = ctypes.byref(cache())
    need = lib.dlrm_history_workspace_bytes(c, 2, 3, 4)
    assert need > 0

    def f(a=att(), batch=2, slots=None, queries=3, q=P, ldq=256, out=P, ldo=256, ws=P, size=need):
        return lib.dlrm_history_lookup(c, ctypes.byref(a) if a is not None else None, batch, slots, queries, q, ldq,
                                       out, ldo, ws, size, None)
    for kw in (dict(a=None), dict(q=None), dict(out=None)):
        assert f(**kw) == dl.DLRM_E_NULL
    for kw in (dict(a=att(kv=4)), dict(a=att(dim=32)), dict(a=att(window=0)), dict(batch=0), dict(queries=0),
               dict(batch=5), dict(ldq=255), dict(ldo=255)):
        assert f(**kw) == dl.DLRM_E_SHAPE
    assert f(slots=P, batch=1 << 29, queries=16) == dl.DLRM_E_UNSUPPORTED
    for kw in (dict(ws=None), dict(size=0), dict(ws=P + 64)):
        assert f(**kw) == dl.DLRM_E_WORKSPACE


def test_page_call_refusals(lib):
    c = ctypes.byref(cache())
    need = lib.dlrm_history_workspace_bytes(c, 1, 0, 0)
    big = 1 << 31
    assert lib.dlrm_history_fork(c, 0, P, P, P, need, None) == dl.DLRM_E_SHAPE
    assert lib.dlrm_history_fork(c, big, P, P, P, need, None) == dl.DLRM_E_UNSUPPORTED
    assert lib.dlrm_history_fork(c, 1, None, P, P, need, None) == dl.DLRM_E_NULL
    assert lib.dlrm_history_fork(c, 1, P, None, P, need, None) == dl.DLRM_E_NULL
    assert lib.dlrm_history_truncate(c, 1, None, P, P, need, None) == dl.DLRM_E_NULL
    assert lib.dlrm_history_truncate(c, -1, P, P, P, need, None) == dl.DLRM_E_SHAPE
    assert lib.dlrm_history_trim(c, 1, P, 0, 0, P, need, None) == dl.DLRM_E_SHAPE
    assert lib.dlrm_history_trim(c, 1, P, 1, -1, P, need, None) == dl.DLRM_E_SHAPE
    for f in (lambda ws, n: lib.dlrm_history_fork(c, 1, P, P, ws, n, None),
              lambda ws, n: lib.dlrm_history_truncate(c, 1, P, None, ws, n, None),
              lambda ws, n: lib.dlrm_history_trim(c, 1, P, 1, 0, ws, n, None),
              lambda ws, n: lib.dlrm_history_compact(c, ws, n, None)):
        assert f(None, need) == dl.DLRM_E_WORKSPACE
        assert f(P, 100) == dl.DLRM_E_WORKSPACE
        assert f(P + 4, need) == dl.DLRM_E_WORKSPACE


def test_workspace_bytes(lib):
    f = lib.dlrm_history_workspace_bytes
    c = ctypes.byref(cache())
    assert f(None, 1, 0, 0) == 0
    for args in ((0, 0, 0), (-1, 0, 0), (1, -1, 4), (1, 1, 0), (1, 1, 3), (1, 1, 5000), (1 << 29, 16, 4)):
        assert f(c, *args) == 0, args
    assert f(c, 1, 0, 0) % 256 == 0
    assert f(c, 100000, 0, 0) >= 1600000          # 16 bytes for each history of an append


def test_binding_refuses_what_is_not_on_the_gpu():
    q = torch.zeros((4, 2, 64))
    with pytest.raises(TypeError):
        dl.history_attention(q, q, q, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError):
        dl.history_attention(q.double(), q, q, torch.zeros(1, dtype=torch.int64))
    with pytest.raises(TypeError):
        dl.HistoryCache.wrap(*([torch.zeros(1)] * 9))
