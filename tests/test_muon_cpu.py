"""muon_update on a machine without a GPU: workspace sizes and the argument
checks, all of which come before any CUDA call."""
import ctypes

import pytest
import torch

import error_feedback_b200 as ef
from error_feedback_b200 import build as efbuild


@pytest.fixture(scope="module")
def lib():
    efbuild.build()
    return ef.lib()


COEF = (3.4445, -4.7750, 2.0315)
WS = 1 << 20      # an aligned address that no rejected call touches
ARGS = dict(grad=4096, gt=0, ldg=8, sg=48, mom=8192, B=2, rows=6, cols=8, mu=0.9, nesterov=1,
            eps=1e-7, coef=COEF, steps=1, scale=1.0, out=16384, ot=0, ldo=8, so=48, ws=WS,
            wsb=1 << 28)


def _call(lib, **change):
    a = {**ARGS, **change}
    for k in ("mu", "eps", "scale"):
        a[k] = ctypes.c_float(a[k])
    if a["coef"] is not None:
        a["coef"] = (ctypes.c_float * len(a["coef"]))(*a["coef"])
    return lib.muon_update(*a.values(), None)


def test_workspace_sizes(lib):
    f, b = torch.float32, torch.bfloat16
    assert 0 < ef.muon_workspace_bytes(1, 64, 27, b) <= ef.muon_workspace_bytes(1, 64, 27, f)
    assert ef.muon_workspace_bytes(1, 64, 27) < ef.muon_workspace_bytes(4, 64, 27)
    assert ef.muon_workspace_bytes(0, 0, 0) > 0
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, -1), (65536, 1, 1), (1, 2**20 + 1, 1), (1, 1, 2**20 + 1)):
        assert ef.muon_workspace_bytes(*bad) == 0
    assert lib.muon_workspace_bytes(1, 1, 1, 3) == 0


@pytest.mark.parametrize("change", [
    dict(gt=3), dict(ot=-1), dict(B=-1), dict(rows=-1), dict(cols=2**20 + 1), dict(ldg=7),
    dict(ldo=7), dict(sg=47), dict(so=47), dict(grad=None), dict(out=None), dict(grad=4098),
    dict(out=16386), dict(mom=8194), dict(ws=None), dict(ws=WS + 8), dict(coef=None),
    dict(steps=0), dict(steps=65), dict(eps=-1.0), dict(eps=float("nan")),
    dict(coef=(float("nan"), 0, 0)), dict(coef=(5.0, 0, 0)), dict(coef=(4.0, -17.0, 0.0)),
    dict(coef=(1.0, 2.0, 2.0)), dict(coef=(0.0, 0.0, 16.5)), dict(mom=4096), dict(mom=16384),
    dict(out=4096, so=56), dict(out=4096, ot=1), dict(rows=2**20, cols=2**20, B=4, ldg=2**20,
    ldo=2**20, sg=2**40, so=2**40, wsb=2**62)])
def test_rejects(lib, change):
    assert _call(lib, **change) == ef.ERR_INVALID_ARG


def test_rejects_polynomials_that_grow_over_the_steps(lib):
    # |p| <= 1.6 on [0, 1], but p(1.6) = 2.56, p(2.56) = 4.096 (the third step)
    steps3 = (1.6, 0.0, 0.0) * 3
    assert _call(lib, coef=steps3, steps=3) == ef.ERR_INVALID_ARG


def test_small_workspace(lib):
    assert _call(lib, wsb=1024) == ef.ERR_WORKSPACE


def test_binding_rejects(lib):
    with pytest.raises(ValueError):
        ef.muon_update(torch.zeros(4, 8))
    for bad in ((1.0, 2.0), [(1.0, 2.0, 3.0)] * 4, [], 5 * [(1.0, 2.0)]):
        with pytest.raises(ValueError):
            ef._coefficients(bad, 5)
    c, steps = ef._coefficients([(1.0, 2.0, 3.0), (4.0, 5.0, 6.0)], 2)
    assert list(c) == [1.0, 2.0, 3.0, 4.0, 5.0, 6.0] and steps == 2
