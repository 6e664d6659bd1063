"""The workspace of layer_norm_grad: as large as the column sums that a call keeps, no larger."""
import pytest
import torch

import error_feedback_b200 as ef
from error_feedback_b200 import build as efbuild


@pytest.mark.parametrize("T,D,parts", [(0, 64, 1), (5, 64, 2), (1000, 64, 250), (131072, 64, 296), (131072, 4096, 296),
                                       (131072, 4097, 148), (10**6, 8192, 148), (10**6, 8193, 64), (16384, 16384, 64),
                                       (10000, 2**20, 64), (40, 2**20, 10)])
def test_bytes(T, D, parts):
    """Rows of two sums of D in fp32, a row for each block that keeps them."""
    efbuild.build()
    need = parts * 2 * D * 4
    assert need < ef.layer_norm_grad_workspace_bytes(T, D) <= need + 1024


@pytest.mark.gpu
@pytest.mark.parametrize("D", [8, 128, 200, 256, 500, 1001, 1024, 2048, 4095, 4096, 4104, 8192, 8200, 16384, 16400, 20001])
@pytest.mark.parametrize("T", [3, 50, 2500])
@pytest.mark.parametrize("xt,dt", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
                                   (torch.bfloat16, torch.float32)])
def test_nothing_behind_it_is_written(T, D, xt, dt):
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    x = torch.randn(T, D, generator=gen, device="cuda").to(xt)
    dy = torch.randn(T, D, generator=gen, device="cuda").to(dt)
    _, mean, rstd = ef.layer_norm(x)
    n = ef.layer_norm_grad_workspace_bytes(T, D)
    buf = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    _, dw, db = ef.layer_norm_grad(dy, x, mean, rstd, ws=buf[:n])
    assert (buf[n:] == 0xA5).all()
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    u = 2.0**-24
    for got, term in ((dw, dy.double() * xh), (db, dy.double())):
        # (two roundings of xh, its product, and a chain of adds no longer than all rows)
        assert ((got.double() - term.sum(0)).abs() <= (T + 30) * u * term.abs().sum(0) + 1e-30).all()
