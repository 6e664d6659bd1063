"""The embedding calls on a machine without a GPU: workspace sizes and the
argument checks, all of which come before any CUDA call."""
import ctypes

import pytest
import torch

import error_feedback_b200 as ef
from error_feedback_b200 import build as efbuild

F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def lib():
    efbuild.build()
    return ef.lib()


def test_workspace_sizes(lib):
    assert ef.embedding_lookup_workspace_bytes() >= 320
    a = ef.embedding_grad_workspace_bytes(1000, 5000, 64)
    b = ef.embedding_grad_workspace_bytes(2000, 5000, 64)
    assert 0 < a < b
    assert ef.embedding_grad_workspace_bytes(0, 0, 0) > 0
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (2**31, 1, 1), (1, 2**31, 1), (1, 1, 2**24 + 1)):
        assert ef.embedding_grad_workspace_bytes(*bad) == 0


WS = 1 << 20      # an aligned address that no rejected call touches

LOOKUP = dict(w=4096, wt=F32, ldw=8, ids=8192, idb=4, T=3, V=5, D=8, scale=1.0, out=16384, ot=F32,
              ldo=8, ws=WS, wsb=1 << 16)
GRAD = dict(dy=4096, dt=F32, ldd=8, ids=8192, idb=4, T=3, V=5, D=8, scale=1.0, pad=-1, out=16384,
            ot=F32, ldo=8, acc=0, ws=WS, wsb=1 << 24)
ROWS = dict(dy=4096, dt=F32, ldd=8, ids=8192, idb=4, T=3, V=5, D=8, scale=1.0, pad=-1, rows=4096,
            out=16384, ot=F32, ldo=8, count=8192, ws=WS, wsb=1 << 24)


def _call(fn, args, **change):
    a = {**args, **change}
    a["scale"] = ctypes.c_float(a["scale"])
    return fn(*a.values(), None)


COMMON = [dict(T=-1), dict(V=-1), dict(D=-1), dict(T=2**31), dict(D=2**24 + 1), dict(idb=2),
          dict(ids=None), dict(ids=8193), dict(out=None), dict(out=16386), dict(ot=3), dict(ot=-1),
          dict(ldo=7), dict(ws=None), dict(ws=WS + 8)]


@pytest.mark.parametrize("change", COMMON + [dict(out=4096), dict(w=None), dict(w=4098), dict(wt=7), dict(ldw=7)])
def test_lookup_rejects(lib, change):
    assert _call(lib.embedding_lookup, LOOKUP, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", COMMON + [dict(out=4096), dict(dy=None), dict(dy=4098), dict(dt=9), dict(ldd=7),
                                             dict(ids=8196, idb=8)])
def test_grad_rejects(lib, change):
    assert _call(lib.embedding_grad, GRAD, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", COMMON + [dict(out=4096), dict(rows=None), dict(rows=4097), dict(count=None),
                                             dict(count=8194)])
def test_rows_rejects(lib, change):
    assert _call(lib.embedding_grad_rows, ROWS, **change) == ef.ERR_INVALID_ARG


def test_small_workspace(lib):
    assert _call(lib.embedding_lookup, LOOKUP, wsb=64) == ef.ERR_WORKSPACE
    assert _call(lib.embedding_grad, GRAD, wsb=1024) == ef.ERR_WORKSPACE
    assert _call(lib.embedding_grad_rows, ROWS, wsb=1024) == ef.ERR_WORKSPACE


def test_binding_rejects_cpu_tensors(lib):
    w, ids = torch.zeros(4, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        ef.embedding_lookup(w, ids)
    with pytest.raises(ValueError):
        ef.embedding_grad(torch.zeros(3, 8), ids, 4)
    with pytest.raises(ValueError):
        ef.embedding_grad_rows(torch.zeros(3, 8), ids, 4)


def test_binding_rejects_workspaces_that_are_not_contiguous():
    """An expanded tensor reports more bytes than it holds."""
    from types import SimpleNamespace
    ws = torch.empty(1, dtype=torch.uint8).expand(1 << 20)
    with pytest.raises(ValueError, match="contiguous"):
        ef._workspace(1024, ws.device, ws)
    with pytest.raises(ValueError, match="contiguous"):
        ef._on_device(ws, SimpleNamespace(index=ws.get_device()))
