"""Refusals of the calls that continue event histories with beams, checked on the host before anything touches a device;
run once more with the host code under the address and undefined-behaviour sanitizers."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import dlrm_embedding_interaction_amd as dl
from dlrm_embedding_interaction_amd import history as hi
from test_history_abi import att, cache

P = 4096    # never dereferenced: validation fails first
MUCH = 1 << 40
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib():
    return dl.load()


def sel(dtype=1, beams=4, keep=4, items=1000, end=-1):
    return hi._Select(dtype, beams, keep, end, items)


def test_select_refusals(lib):
    need = lib.dlrm_history_select_workspace_bytes(ctypes.byref(sel()), 2)
    assert need > 0

    def f(d=sel(), batch=2, x=P, ld=1000, scores=P, may=None, ldm=0, ended=None, s=P, p=P, i=P, ws=P, size=need):
        return lib.dlrm_history_select(ctypes.byref(d) if d is not None else None, batch, x, ld, scores, may, ldm,
                                       ended, s, p, i, ws, size, None)
    for kw in (dict(d=None), dict(x=None), dict(s=None), dict(p=None), dict(i=None)):
        assert f(**kw) == dl.DLRM_E_NULL
    for d in (sel(dtype=3), sel(dtype=-1), sel(beams=0), sel(keep=0), sel(items=0), sel(keep=-1)):
        assert f(d=d) == dl.DLRM_E_SHAPE
    for kw in (dict(batch=0), dict(batch=-4), dict(ld=999), dict(may=P, ldm=999), dict(may=P, ldm=-1)):
        assert f(**kw) == dl.DLRM_E_SHAPE
    for d in (sel(beams=129), sel(keep=129), sel(items=(1 << 25) + 1)):
        assert f(d=d) == dl.DLRM_E_UNSUPPORTED
    assert f(batch=1 << 40, size=MUCH) == dl.DLRM_E_UNSUPPORTED
    for kw in (dict(ws=None), dict(size=need - 1), dict(ws=P + 16)):
        assert f(**kw) == dl.DLRM_E_WORKSPACE
    one = sel(beams=1, keep=1, items=1)
    assert f(d=one, batch=1 << 23) == dl.DLRM_E_WORKSPACE


def test_select_workspace_bytes(lib):
    f = lib.dlrm_history_select_workspace_bytes
    assert f(None, 2) == 0
    for d, batch in ((sel(), 0), (sel(beams=0), 2), (sel(keep=200), 2), (sel(items=0), 2), (sel(dtype=9), 2)):
        assert f(ctypes.byref(d), batch) == 0
    assert f(ctypes.byref(sel()), 3) % 256 == 0
    assert f(ctypes.byref(sel(items=1 << 25, beams=128, keep=128)), 64) > 64 * 128 * 128 * 8


def test_reorder_refusals(lib):
    c = ctypes.byref(cache())
    need = lib.dlrm_history_workspace_bytes(c, 1, 0, 0)

    def f(c=c, n=1, group=4, slots=P, parents=P, ws=P, size=need):
        return lib.dlrm_history_reorder(c, n, group, slots, parents, ws, size, None)
    assert f(c=None) == dl.DLRM_E_NULL
    assert f(c=ctypes.byref(cache(ptr=None))) == dl.DLRM_E_NULL
    assert f(parents=None) == dl.DLRM_E_NULL
    for kw in (dict(n=0), dict(group=0), dict(group=-1), dict(slots=None, n=2), dict(slots=None, group=5)):
        assert f(**kw) == dl.DLRM_E_SHAPE
    for kw in (dict(group=129), dict(n=1 << 31), dict(n=1 << 25)):
        assert f(**kw) == dl.DLRM_E_UNSUPPORTED
    for kw in (dict(ws=None), dict(size=16), dict(ws=P + 8)):
        assert f(**kw) == dl.DLRM_E_WORKSPACE


def test_lookup_shared_refusals(lib):
    c = ctypes.byref(cache())
    need = lib.dlrm_history_shared_workspace_bytes(c, 4, 2, 3, 4)
    assert need > 0

    def f(c=c, a=att(), batch=4, slots=P, n=2, groups=None, ib=8, queries=3, q=P, ldq=256, out=P, ldo=256, ws=P,
          size=need):
        return lib.dlrm_history_lookup_shared(c, ctypes.byref(a) if a is not None else None, batch, slots, n, groups, ib,
                                              queries, q, ldq, out, ldo, ws, size, None)
    for kw in (dict(c=None), dict(a=None), dict(q=None), dict(out=None), dict(c=ctypes.byref(cache(ptr=None)))):
        assert f(**kw) == dl.DLRM_E_NULL
    for kw in (dict(a=att(kv=4)), dict(a=att(dim=32)), dict(a=att(window=0)), dict(batch=0), dict(queries=0), dict(n=0),
               dict(n=3), dict(slots=None, batch=6), dict(ldq=255), dict(ldo=255), dict(groups=P, ib=2), dict(n=-2)):
        assert f(**kw) == dl.DLRM_E_SHAPE, kw
    for kw in (dict(a=att(dim=48)), dict(batch=1 << 29, queries=16), dict(groups=P, n=1 << 31),
               dict(batch=1 << 26, queries=1, size=1 << 60), dict(groups=P, n=1 << 24, size=1 << 60)):
        assert f(**kw) == dl.DLRM_E_UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(size=need - 1), dict(ws=P + 64), dict(groups=P, n=5)):
        assert f(**kw) == dl.DLRM_E_WORKSPACE


def test_shared_workspace_bytes(lib):
    f = lib.dlrm_history_shared_workspace_bytes
    c = ctypes.byref(cache())
    assert f(None, 1, 1, 1, 4) == 0
    for args in ((0, 1, 1, 4), (1, 0, 1, 4), (1, 1, 0, 4), (1, 1, 1, 0), (1, 1, 1, 3), (1, 1, 1, 5000),
                 (1 << 29, 1, 16, 4)):
        assert f(c, *args) == 0, args
    assert f(c, 8, 2, 1, 4) % 256 == 0


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros((2, 3, 50))
    with pytest.raises(TypeError):
        dl.history_select(x)
    with pytest.raises(TypeError):
        dl.history_select(x.double())


def test_beams_abi_under_address_and_undefined_behaviour_sanitizers():
    if os.environ.get("LD_PRELOAD"):
        pytest.skip("this is the sanitized run")
    import test_history_sanitizers as hs
    import test_sanitizers as ts
    from dlrm_embedding_interaction_amd import _build
    try:
        cc = _build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    rt = ts._clang_asan_runtime(cc)
    if not rt:
        pytest.skip("clang AddressSanitizer runtime not found next to hipcc")
    code = hs.CHILD.format(root=hs.ROOT, here=HERE, lib=ts._sanitized_library(), tests=[os.path.abspath(__file__)])
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, LD_PRELOAD=rt, **ts.SAN_ENV),
                       capture_output=True, text=True, timeout=600)
    if r.returncode != 0:
        pytest.fail(f"sanitized run exited {r.returncode}\n{r.stdout[-3000:]}\n{r.stderr[-6000:]}")
    assert "passed" in r.stdout
