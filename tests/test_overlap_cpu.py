"""Arguments of the layer norm calls and the losses that share memory are refused before any CUDA
call, unless the header allows them; columns of one buffer share none.  (An argument that is not
refused is shown by the next check, of a workspace that is too small.)"""
import pytest

import error_feedback_b200 as ef
from error_feedback_b200 import build as efbuild
from test_layer_norm_cpu import BF16, F32, GRAD as NORM_GRAD, NORM, WS, _call as norm_call
from test_token_loss_cpu import DISTILL, GRAD, LOGP, _call


@pytest.fixture(scope="module")
def lib():
    efbuild.build()
    return ef.lib()


# (T = 3 rows of D = V = 8: 32 bytes each, 96 in all)

@pytest.mark.parametrize("change", [
    dict(out=4096 + 32), dict(out=4096 + 4), dict(out=4096 + 92), dict(out=4096 - 4), dict(out=4096 - 92),
    dict(out=4096 + 32, ldo=16), dict(out=4096 + 60, ldx=16, ldo=16), dict(out=4096 + 36, ldx=16, ldo=16),
    dict(out=4096 + 28, ldx=16, ldo=16), dict(out=4096 + 2, ot=BF16), dict(out=8192 + 16), dict(out=8448 - 64),
    dict(mean=4096 + 4), dict(rstd=4096 + 92), dict(mean=16384 + 8), dict(rstd=32768), dict(rstd=32768 + 8),
    dict(mean=8192), dict(rstd=8448 + 28), dict(mean=4096, ldx=16), dict(out=4096, mean=4096)])
def test_norm(lib, change):
    assert norm_call(lib.layer_norm, NORM, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(gx=8192 + 32), dict(gx=8192 - 4), dict(gx=4096 + 4), dict(gx=4096 - 92), dict(gx=4096, x=4096 + 32),
    dict(gx=32768 - 92), dict(gx=33024 + 8), dict(gx=40960 + 28), dict(gw=53248 + 16), dict(gb=49152 + 28),
    dict(gw=16384 + 92), dict(gb=16384), dict(gw=WS + 256), dict(gx=WS + 512), dict(x=WS + 256), dict(dy=WS - 4),
    dict(mean=WS)])
def test_norm_grad(lib, change):
    assert norm_call(lib.layer_norm_grad, NORM_GRAD, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(gx=8192), dict(gx=4096), dict(dy=8192), dict(dy=8192, gx=8192), dict(gx=8192 + 96), dict(gx=8192 - 96),
    dict(x=8192, gx=8192 + 32, dy=8192 + 64, ldx=24, ldg=24, ldd=24), dict(gx=8192 + 32, ldx=40, ldg=40),
    dict(gw=40960), dict(gb=53248 - 32), dict(T=0, gx=8192 + 4)])
def test_norm_grad_allows(lib, change):
    assert norm_call(lib.layer_norm_grad, NORM_GRAD, **{**change, "wsb": 0}) == ef.ERR_WORKSPACE


@pytest.mark.parametrize("change", [
    dict(lp=4096 + 92), dict(en=4096), dict(ls=8192), dict(en=12288 + 8), dict(ls=12544), dict(ti=13312 + 20),
    dict(tp=13056), dict(ti=4096 + 64), dict(tp=8192 + 8), dict(lp=WS + 64), dict(z=WS + 256), dict(ids=WS)])
def test_logprobs(lib, change):
    assert _call(lib.token_logprobs, LOGP, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(dz=4096 + 32), dict(dz=4096 - 4), dict(dz=4096 + 36, ldz=16, ldo=16), dict(dz=8192 - 92), dict(dz=12800),
    dict(dz=12544 + 8), dict(dz=12288 - 92), dict(dz=13056 + 8), dict(dz=WS + 64), dict(ls=WS), dict(z=WS - 92)])
def test_logprobs_grad(lib, change):
    assert _call(lib.token_logprobs_grad, GRAD, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(dz=4096 + 32), dict(dz=4096 - 4), dict(dz=8192 + 20), dict(dz=12288 + 20), dict(dz=12544), dict(dz=12800 - 92),
    dict(loss=12544 + 4), dict(loss=4096 + 92), dict(loss=8192), dict(loss=12288 - 8), dict(loss=WS), dict(w=WS + 8)])
def test_distill(lib, change):
    assert _call(lib.distill_loss, DISTILL, **change) == ef.ERR_INVALID_ARG


@pytest.mark.parametrize("name,args,change", [
    ("token_logprobs", LOGP, dict(lp=4096 + 96)), ("token_logprobs", LOGP, dict(lp=4096 + 32, ldz=16, T=1)),
    ("token_logprobs", LOGP, dict(top=0, ti=4096, tp=4096)), ("token_logprobs_grad", GRAD, dict(dz=4096)),
    ("token_logprobs_grad", GRAD, dict(g=12544, h=12544)), ("token_logprobs_grad", GRAD, dict(dz=4096 + 32, ldz=16, ldo=16)),
    ("token_logprobs_grad", GRAD, dict(dz=4096 - 32, ldz=24, ldo=24)), ("distill_loss", DISTILL, dict(dz=4096)),
    ("distill_loss", DISTILL, dict(loss=12544)), ("distill_loss", DISTILL, dict(dz=4096 + 96)),
    ("distill_loss", DISTILL, dict(K=0, ids=4096, t=4096))])
def test_losses_allow(lib, name, args, change):
    assert _call(getattr(lib, name), args, **{**change, "wsb": 0}) == ef.ERR_WORKSPACE


def test_rows_of_other_strides(lib):
    """Every second row's gap of a buffer, row by row against a list of bytes."""
    def bytes_of(at, ld, size):
        return {at + r * ld * size + i for r in range(3) for i in range(8 * size)}

    seen = set()
    for at in range(4096 - 160, 4096 + 400, 20):
        for ldz, ldo, ot in ((8, 16, F32), (20, 10, F32), (12, 24, BF16), (40, 9, F32), (30, 15, F32)):
            want = bool(bytes_of(4096, ldz, 4) & bytes_of(at, ldo, 2 if ot == BF16 else 4))
            if at == 4096:
                continue
            got = _call(lib.token_logprobs_grad, GRAD, ldz=ldz, dz=at, ldo=ldo, ot=ot, wsb=0)
            assert got == (ef.ERR_INVALID_ARG if want else ef.ERR_WORKSPACE), (at, ldz, ldo, ot)
            seen.add(want)
    assert seen == {False, True}
