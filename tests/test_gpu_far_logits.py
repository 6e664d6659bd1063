"""token_logprobs_grad on the GPU against a 64-bit softmax of the logits, not of the call's own
log of the sum: rows far from 0, rows that a mask of finite value leaves with nothing else, and
ordinary ones.

u = 2^-24, ex2 is off by at most 2^-22 of its value, c = scale log2 e by u of itself.
An ordinary row (|lse| <= 128) has p = exp(scale z - lse), so p is off by the error of lse, one
rounding of the difference, of its product with log2 e and of that constant.  The others are
summed again: p_i = 2^t_i / s with t_i = c (z_i - max) up to a whole number, d_i = |t_i| + 1, so
p is off by u (2 d_i + the mean of 2 d) ln 2, by the sum's own error and by ex2's twice."""
import math

import pytest
import torch

import error_feedback_b200 as ef
import test_gpu_token_loss as calls

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U, EX2, INF = 2.0**-24, 2.0**-22, math.inf


def _rows(V, dtype, ld=None, offset=0):
    """Rows of every kind, repeated; a row's first kind is ordinary."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(14, V, generator=g, device="cuda") * 3
    big = 6e4 if dtype == torch.float16 else 1e9
    every = torch.arange(V, device="cuda")
    z[1] = -big
    z[2] = torch.finfo(dtype).min
    z[3] += 5e3
    z[4] -= 2e4
    z[5] += 5e4 if dtype == torch.float16 else 1e6
    z[6] = torch.where(every % 3 == 0, -big, -big + 64)
    z[7] = torch.where(every % 2 == 1, -big, z[7])
    z[8] = -INF
    z[9] = torch.finfo(dtype).max
    z[10] = torch.where(every % 5 == 4, -INF, z[10] + 4e2)
    z[11] *= 50
    z[12] = torch.where(every == V // 2, 1e3, -big)
    z = z.to(dtype)
    if ld is None:
        return z
    buf = torch.zeros(14 * ld + offset + 8, dtype=dtype, device="cuda")
    rows = buf[offset:offset + 14 * ld].view(14, ld)[:, :V]
    return rows.copy_(z)


def _exact(z, ids, scale, g, h):
    """The gradient in 64 bits, and how far a call may be from it before its last rounding."""
    T, V = z.shape
    x = z.double() * scale
    empty = (x == -INF).all(1, keepdim=True)
    logp = torch.log_softmax(x, 1)
    p = torch.where(x == -INF, 0.0, logp.exp())
    lp = torch.where(p > 0, logp, 0.0)
    H = -(p * lp).sum(1, keepdim=True)
    lse = torch.logsumexp(x, 1, keepdim=True)
    G = torch.where(ids >= 0, g.double(), 0.0)[:, None]
    h = h.double()[:, None] if h is not None else torch.zeros_like(G)
    hot = torch.zeros_like(x)
    hot[torch.arange(T, device="cuda"), ids.clamp(min=0)] = 1.0
    want = torch.where(empty, 0.0, scale * (G * (hot - p) - h * p * (lp + H)))
    top = x.max(1, keepdim=True).values
    d = torch.where(p > 0, (x - top).abs() * 1.4427 + 1, 0.0)
    mean = (p * d).sum(1, keepdim=True)
    e_s = EX2 + U * (V / 2048 + 40 + 4 * mean)
    rel = e_s + EX2 + U * (4 * d + 8)
    # the log of the sum: its own error, the scale's (c), two roundings; log p the same again
    near = e_s + U * (4 * lse.abs() + 4 * math.log(V) + 40) + EX2 + 8 * U * (lp.abs() + 1)
    rel = torch.where(lse.abs() <= 128, rel + near, rel)
    e_h = (e_s + U * 40) * (2 + 2 * mean) + 8 * U * (H + math.log(V) + 9)
    size = G.abs() + h.abs() * (lp.abs() + H)
    e_log = h.abs() * (e_h + rel + U * (8 * lp.abs() + 8 * math.log(V) + 40))
    err = scale * (p * (size * (rel + 8 * U) + e_log) + 4 * U * G.abs() * hot + size * 2.0**-125)
    return want, torch.where(empty, 0.0, torch.nan_to_num(err))


def _check(z, scale, entropy, out=None, out_dtype=None):
    T, V = z.shape
    gen = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
    ids[12] = V // 2
    g = torch.randn(T, generator=gen, device="cuda")
    h = torch.randn(T, generator=gen, device="cuda") if entropy else None
    want, err = _exact(z, ids, scale, g, h)
    _, en, ls, _, _ = ef.token_logprobs(z, ids, scale=scale)
    got = ef.token_logprobs_grad(z, ids, ls, grad_logprob=g, entropy=en, grad_entropy=h, scale=scale, out=out,
                                 out_dtype=out_dtype)
    y = got.double()
    eps = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * (eps if got.dtype != torch.float32 else 2.0)
    bad = ~((y - want).abs() <= err * (1 + eps) + want.abs() * eps + tiny)
    assert not bad.any(), f"{int(bad.sum())} off, rows {bad.any(1).nonzero()[:, 0].tolist()}, first " \
        f"{float(y[bad][0])} for {float(want[bad][0])} (bound {float(err[bad][0])})"
    if not entropy and got.dtype == torch.float32:
        # a row of it adds up to 0
        assert (y.sum(1).abs() <= err.sum(1) + want.abs().sum(1) * eps + V * tiny).all()
    return got


@pytest.mark.parametrize("V", [1, 2, 33, 1000, 5003, 40001, 131072])
@pytest.mark.parametrize("zt,ot", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("entropy", [False, True])
def test_far_rows(V, zt, ot, entropy):
    z = _rows(V, TYPES[zt])
    _check(z, 1.0, entropy, out_dtype=TYPES[ot])
    got = _check(z, 0.25, entropy, out_dtype=TYPES[ot])
    if zt == ot:
        here = z.clone()
        gen = torch.Generator(device="cuda").manual_seed(3)
        ids = torch.randint(0, V, (14,), generator=gen, device="cuda")
        ids[12] = V // 2
        g = torch.randn(14, generator=gen, device="cuda")
        h = torch.randn(14, generator=gen, device="cuda") if entropy else None
        _, en, ls, _, _ = ef.token_logprobs(z, ids, scale=0.25)
        ef.token_logprobs_grad(here, ids, ls, grad_logprob=g, entropy=en, grad_entropy=h, scale=0.25, out=here)
        assert torch.equal(here, got)


def test_scale_past_the_type():
    """scale z passes fp32's range, z does not."""
    z = _rows(700, torch.float32)
    z[5], z[6] = -3e38, 3e38
    _check(z, 2.0, False)
    _check(z, 2.0, True)


@pytest.mark.parametrize("ld,ldo,off", [(1001, 1001, 0), (1008, 1016, 8), (1030, 1001, 3), (1024, 1024, 1)])
@pytest.mark.parametrize("zt,ot", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_far_rows_that_start_anywhere(ld, ldo, off, zt, ot):
    z = _rows(1001, TYPES[zt], ld, off)
    buf = torch.full((14 * ldo + off + 8,), 7.0, dtype=TYPES[ot], device="cuda")
    rows = buf[off:off + 14 * ldo].view(14, ldo)
    _check(z, 1.0, True, out=rows[:, :1001])
    assert (rows[:, 1001:] == 7.0).all() and (buf[:off] == 7.0).all() and (buf[off + 14 * ldo:] == 7.0).all()


def test_many_far_rows_padding_and_capture():
    z = _rows(3001, torch.bfloat16).repeat(150, 1)
    T = z.shape[0]
    ids = torch.arange(T, device="cuda") * 7 % 3001
    ids[5::28] = -1
    g = torch.linspace(-1, 1, T, device="cuda")
    g[6::28] = 0.0
    _, en, ls, _, _ = ef.token_logprobs(z, ids)
    ws = torch.empty(ef.token_logprobs_workspace_bytes(), dtype=torch.uint8, device="cuda")
    got = ef.token_logprobs_grad(z, ids, ls, grad_logprob=g, ws=ws)
    assert (got[5::28] == 0).all() and (got[6::28] == 0).all()
    want, err = _exact(z, ids, 1.0, torch.where(ids < 0, 0.0, g), None)
    assert ((got.double() - want).abs() <= err + want.abs() * 2.0**-8 + 2.0**-133).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = ef.token_logprobs_grad(z, ids, ls, grad_logprob=g, ws=ws)
    again.fill_(3)
    graph.replay()
    assert torch.equal(again, got)


@pytest.mark.parametrize("T,V", [(501, V) for V in (33, 500, 2000, 4097, 8192, 16385, 40001)] +
                         [(900, 33), (900, 500), (900, 2000), (1800, 4000), (1800, 8000)])
@pytest.mark.parametrize("zt", ["f32", "bf16"])
def test_far_and_masked_rows_of_every_team(T, V, zt):
    """Rows of one warp, four and eight: all three calls, with a row masked by -1e9 throughout."""
    z = calls._logits(T, V, TYPES[zt])
    z[3] = -INF
    z[5] = -1e9
    z[7, ::2] = -INF
    ids = calls._ids(T, V)
    calls._check_forward(z, ids, 1.0, 17)
    _check(z, 1.0, True)
    tids, tl = calls._teacher(T, V, 9)
    w = torch.rand(T, device="cuda")
    w[::5] = 0
    keep = [r for r in range(T) if r not in (3, 7)]       # (a teacher's token at -inf: loss +inf)
    zk = z[keep].contiguous()
    tk = [t[keep].contiguous() for t in (tids, tl, w)]
    calls._check_distill(zk, *tk[:2], tk[2], 0.7)
    calls._check_distill(zk, *tk[:2], None, 0.7, grad=False)


@pytest.mark.parametrize("T,V", [(3, 50), (3, 40001), (600, 3000), (2000, 900)])
def test_minus_inf_beside_inf(T, V):
    """A row with +inf or NaN is NaN at its tokens of -inf too, as a log softmax is; no other row."""
    z = calls._logits(T, V, torch.float32)
    ids = calls._ids(T, V)
    ids[1] = 4
    want = ef.token_logprobs(z, ids, top=V if V < 100 else 3)
    for value in (INF, math.nan):
        y = z.clone()
        y[1] = -INF
        y[1, 7] = value
        lp, en, ls, ti, tp = got = ef.token_logprobs(y, ids, top=V if V < 100 else 3)
        assert lp[1].isnan() and en[1].isnan() and ls[1].isnan() and tp[1].isnan().all()
        assert ti[1, :3].tolist() == [7, 0, 1]
        assert ef.token_logprobs_grad(y, ids, ls, grad_logprob=torch.ones(T, device="cuda"))[1].isnan().all()
        others = [r for r in range(T) if r != 1]
        assert all(torch.equal(a[others], b[others]) for a, b in zip(want, got))
