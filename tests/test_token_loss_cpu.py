"""The calls over a vocabulary on a machine without a GPU: workspace sizes and the
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
    assert 320 <= ef.token_logprobs_workspace_bytes() <= ef._STATUS_WS
    assert 320 <= ef.distill_loss_workspace_bytes() <= ef._STATUS_WS


LOGP = dict(z=4096, zt=F32, ldz=8, ids=8192, idb=4, T=3, V=8, scale=1.0, pad=-1, top=2, lp=12288, en=12544, ls=12800,
            ti=13056, tp=13312, ws=WS, wsb=512)
GRAD = dict(z=4096, zt=F32, ldz=8, ids=8192, idb=4, T=3, V=8, scale=1.0, pad=-1, ls=12800, en=12544, g=12288, h=13056,
            dz=16384, ot=F32, ldo=8, ws=WS, wsb=512)
DISTILL = dict(z=4096, zt=F32, ldz=8, ids=8192, idb=4, t=12288, tt=F32, T=3, V=8, K=2, scale=1.0, w=12544, loss=12800,
               dz=16384, ot=F32, ldo=8, ws=WS, wsb=512)


def _call(fn, args, **change):
    a = {**args, **change}
    assert a.keys() == args.keys()
    a["scale"] = ctypes.c_float(a["scale"])
    return fn(*a.values(), None)


COMMON = [dict(T=-1), dict(T=2**31), dict(V=0), dict(V=2**24 + 1), dict(zt=3), dict(ldz=7), dict(z=None), dict(z=4098),
          dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(ws=None),
          dict(ws=WS + 8)]


@pytest.mark.parametrize("change", COMMON + [
    dict(idb=2), dict(ids=8196, idb=8), dict(ids=None), dict(top=-1), dict(top=129), dict(lp=12289), dict(en=12546),
    dict(ls=12801), dict(ti=13058), dict(tp=13313), dict(V=2**19, ldz=2**19), dict(V=2**20, ldz=2**20, zt=BF16)])
def test_logprobs_rejects(lib, change):
    assert _call(lib.token_logprobs, LOGP, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", COMMON + [
    dict(idb=2), dict(ids=8193), dict(ids=None), dict(ls=None), dict(ls=12801), dict(en=None), dict(en=12545),
    dict(g=12290), dict(h=13057), dict(dz=None), dict(dz=16386), dict(ot=5), dict(ldo=7), dict(dz=4096, ldo=9),
    dict(dz=4096, ot=BF16)])
def test_logprobs_grad_rejects(lib, change):
    assert _call(lib.token_logprobs_grad, GRAD, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", COMMON + [
    dict(idb=1), dict(ids=None), dict(ids=8194), dict(t=None), dict(t=12290), dict(tt=-1), dict(K=-1), dict(K=257),
    dict(w=12545), dict(loss=12802), dict(dz=16385), dict(ot=7), dict(ldo=7), dict(dz=4096, ldo=9),
    dict(dz=4096, ot=BF16)])
def test_distill_rejects(lib, change):
    assert _call(lib.distill_loss, DISTILL, **change) == ef.ERR_INVALID_ARG


def test_small_workspace(lib):
    for fn, args in ((lib.token_logprobs, LOGP), (lib.token_logprobs_grad, GRAD), (lib.distill_loss, DISTILL)):
        assert _call(fn, args, wsb=64) == ef.ERR_WORKSPACE


def test_binding_rejects_cpu_tensors(lib):
    z, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        ef.token_logprobs(z, ids)
    with pytest.raises(ValueError):
        ef.token_logprobs_grad(z, ids, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError):
        ef.distill_loss(z, ids.view(4, 1), torch.zeros(4, 1))
