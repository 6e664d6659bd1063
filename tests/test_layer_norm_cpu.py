"""The layer norm calls on a machine without a GPU: workspace sizes and the
argument checks, all of which come before any CUDA call."""
import ctypes

import pytest
import torch

import error_feedback_b200 as ef
from error_feedback_b200 import build as efbuild

F32, BF16 = 0, 1
WS = 1 << 20      # an aligned address that no rejected call touches


@pytest.fixture(scope="module")
def lib():
    efbuild.build()
    return ef.lib()


def test_workspace_sizes(lib):
    a = ef.layer_norm_grad_workspace_bytes(1000, 64)
    assert 0 < a < ef.layer_norm_grad_workspace_bytes(1000, 65)
    assert ef.layer_norm_grad_workspace_bytes(0, 1) > 0
    assert ef.layer_norm_grad_workspace_bytes(2**31 - 1, 2**24) > 0
    for bad in ((-1, 1), (1, 0), (1, -1), (2**31, 1), (1, 2**24 + 1)):
        assert ef.layer_norm_grad_workspace_bytes(*bad) == 0


NORM = dict(x=4096, xt=F32, ldx=8, w=8192, wt=F32, b=8448, bt=F32, T=3, D=8, eps=1e-5, out=16384, ot=F32, ldo=8,
            mean=32768, rstd=33024)
GRAD = dict(dy=4096, dt=F32, ldd=8, x=8192, xt=F32, ldx=8, mean=32768, rstd=33024, w=40960, wt=F32, T=3, D=8,
            gx=16384, ldg=8, gw=49152, gwt=F32, gb=53248, gbt=F32, acc=0, ws=WS, wsb=1 << 24)


def _call(fn, args, **change):
    a = {**args, **change}
    assert a.keys() == args.keys()
    if "eps" in a:
        a["eps"] = ctypes.c_float(a["eps"])
    return fn(*a.values(), None)


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(T=2**31), dict(D=0), dict(D=-1), dict(D=2**24 + 1), dict(ldx=7), dict(ldo=7), dict(xt=3),
    dict(ot=-1), dict(x=None), dict(x=4098), dict(out=None), dict(out=16386), dict(wt=4), dict(w=8194), dict(bt=-2),
    dict(b=8449), dict(mean=32770), dict(rstd=33025), dict(eps=-1.0), dict(eps=float("nan")),
    dict(out=4096, ot=BF16), dict(out=4096, ldo=9)])
def test_norm_rejects(lib, change):
    assert _call(lib.layer_norm, NORM, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(T=2**31), dict(D=0), dict(D=2**24 + 1), dict(ldd=7), dict(ldx=7), dict(ldg=7), dict(dt=3),
    dict(xt=-1), dict(dy=None), dict(dy=4097), dict(x=None), dict(x=8194), dict(mean=None), dict(rstd=None),
    dict(mean=32769), dict(w=40962), dict(wt=9), dict(gx=None), dict(gx=16386), dict(gw=49153), dict(gwt=5),
    dict(gb=53250), dict(gbt=-1), dict(gb=49152), dict(ws=None), dict(ws=WS + 8), dict(gx=8192, ldg=9),
    dict(gx=4096, dt=BF16), dict(gx=4096, ldg=9)])
def test_grad_rejects(lib, change):
    assert _call(lib.layer_norm_grad, GRAD, **change) == ef.ERR_INVALID_ARG


def test_small_workspace_and_no_rows(lib):
    assert _call(lib.layer_norm_grad, GRAD, wsb=0) == ef.ERR_WORKSPACE
    assert _call(lib.layer_norm, NORM, T=0, x=None, out=None) == ef.OK
    assert _call(lib.layer_norm_grad, GRAD, T=0, gw=None, gb=None, ws=None, wsb=0) == ef.OK


def test_binding_rejects_cpu_tensors(lib):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        ef.layer_norm(x)
    with pytest.raises(ValueError):
        ef.layer_norm_grad(x, x, torch.zeros(4), torch.ones(4))
