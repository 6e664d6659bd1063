"""token_logprobs, token_logprobs_grad and distill_loss on the GPU against 64-bit
formulas.

u = 2^-24 is half a step of fp32; ex2 is off by at most 2^-22 of its value.  The
calls hold p_i as 2^t_i / s with t_i = c z_i - m, where c = scale log2 e is off by u
of itself, m lies at most 9 above and below c max z, and t_i is rounded once.  The
sum s has positive terms: it is off by their errors' mean and u for each add of
the longest chain, whose roundings (V / 64 of a row's one warp, V / 256 of four, V / 512 of
eight, of either sign) add up to less than V / 2048 + 40 of them: 128 at V = 8,192 have a
deviation of 7, 586 at 150,000 of 14.  All the tolerances below follow from that."""
import math

import pytest
import torch

import error_feedback_b200 as ef

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U, EX2 = 2.0**-24, 2.0**-22
INF = math.inf


def _logits(T, V, dtype, ld=0, offset=0, seed=0, spread=3.0, peak=True):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * T + V)
    ld = ld or V
    buf = torch.randn(T * ld + offset + 8, generator=g, device="cuda").mul_(spread)
    z = buf[offset:offset + T * ld].view(T, ld)
    if peak and T:
        at = torch.randint(0, V, (T,), generator=g, device="cuda")
        z[torch.arange(T, device="cuda"), at] += 8.0
    return buf.to(dtype)[offset:offset + T * ld].view(T, ld)[:, :V]


def _ids(T, V, seed=0, dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed + T)
    return torch.randint(0, V, (T,), generator=g, device="cuda").to(dtype)


class Exact:
    """64-bit softmax of rows and how far the calls may be from it."""

    def __init__(self, z, scale):
        self.V = z.shape[1]
        self.x = z.double() * scale
        self.logp = torch.log_softmax(self.x, 1)
        self.logp = torch.where(self.x == -INF, -INF, self.logp)
        self.p = self.logp.exp()
        self.lse = torch.logsumexp(self.x, 1)
        self.entropy = -torch.xlogy(self.p, self.p).sum(1)
        x = torch.where(self.x == -INF, 0.0, self.x) * 1.4427
        top = self.x.max(1, keepdim=True).values * 1.4427
        # |t| + |c z|, roundings in u.  (A row past 2^16 is summed with differences: no |c z|.)
        far = top.abs() > 65000
        self.round = (x - torch.where(top == -INF, 0.0, top)).abs() + 9 + torch.where(far, 0.0, x.abs())
        self.n = self.V / 2048 + 40
        self.e_s = EX2 + U * (self.n + (self.p * self.round).sum(1))

    def err_logp(self):
        return self.e_s[:, None] + U * (2 * self.round + 4 * self.logp.clamp(min=-1e30).abs() + 8 * math.log(self.V) + 40)

    def err_lse(self):
        return self.e_s + U * (3 * self.lse.abs() + 4 * math.log(self.V) + 40)

    def err_entropy(self):
        t = (self.p * self.round).sum(1)
        e_u = (self.p * self.round * (EX2 + U * (self.n + self.round))).sum(1) + U * t
        return self.e_s * (1 + t) + e_u + 8 * U * (self.entropy + math.log(self.V) + 9 + t)


def _near(got, want, err, dtype=torch.float32):
    got = got.double()
    same = (got == want) | (got.isnan() & want.isnan())
    eps = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * (eps if dtype != torch.float32 else 2.0)   # (ex2 flushes)
    bad = ~(same | ((got - want).abs() <= err * (1 + eps) + want.abs() * eps + tiny))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
        f"{got[bad][0]} for {want[bad][0]} (bound {(err + 0 * want)[bad][0]})"


def _best(z, K):
    """Ids of the K largest, the lower first among equal ones."""
    return torch.sort(z.float(), dim=1, descending=True, stable=True).indices[:, :K]


def _check_forward(z, ids, scale, top, padding_idx=-1, ws=None, status=0):
    T, V = z.shape
    ws = ws if ws is not None else torch.full((ef.token_logprobs_workspace_bytes(),), 0xA5, dtype=torch.uint8,
                                              device="cuda")
    lp, en, ls, ti, tp = ef.token_logprobs(z, ids, scale=scale, top=top, padding_idx=padding_idx, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == status
    e = Exact(z, scale)
    skip = torch.zeros(T, dtype=torch.bool, device="cuda") if ids is None else ids.reshape(-1) == padding_idx
    keep = ~skip
    if ids is None:
        assert lp is None
    else:
        i = ids.reshape(-1).long()
        ok = keep & (i >= 0) & (i < V)
        assert (lp[~ok] == 0).all()
        rows = torch.arange(T, device="cuda")[ok]
        _near(lp[ok], e.logp[rows, i[ok]], e.err_logp()[rows, i[ok]])
    _near(en[keep], e.entropy[keep], e.err_entropy()[keep])
    _near(ls[keep], e.lse[keep], e.err_lse()[keep])
    assert (en[skip] == 0).all() and (ls[skip] == 0).all()
    if top == 0:
        assert ti is None and tp is None
        return
    k = min(top, V)
    want = _best(z, k)
    assert torch.equal(ti[keep][:, :k].long(), want[keep])
    _near(tp[keep][:, :k], e.logp.gather(1, want)[keep], e.err_logp().gather(1, want)[keep])
    assert (ti[skip] == -1).all() and (tp[skip] == -INF).all()
    assert (ti[:, k:] == -1).all() and (tp[:, k:] == -INF).all()


SHAPES = [(1, 1), (3, 2), (1, 7), (4, 31), (2, 64), (9, 100), (5, 257), (3, 1000), (40, 1031), (2, 4096), (1, 32768),
          (600, 5000), (3, 50021), (1, 131072), (17, 131071), (2, 262144)]


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("zt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale,top", [(1.0, 0), (0.5, 20), (2.0, 128)])
def test_forward(T, V, zt, scale, top):
    z = _logits(T, V, TYPES[zt])
    _check_forward(z, _ids(T, V, 1, torch.int32 if T % 2 else torch.int64), scale, top)


@pytest.mark.parametrize("top", [1, 2, 63, 64, 65, 127, 128])
@pytest.mark.parametrize("V", [100, 3000, 40000])
def test_tops(V, top):
    _check_forward(_logits(7, V, torch.bfloat16), None, 1.0, top)


@pytest.mark.parametrize("ld,off", [(1001, 0), (1008, 8), (1030, 3), (1001, 1)])
@pytest.mark.parametrize("zt", ["f32", "bf16"])
def test_forward_strides(ld, off, zt):
    _check_forward(_logits(50, 1001, TYPES[zt], ld, off), _ids(50, 1001), 1.0, 9)


@pytest.mark.parametrize("zt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "two", "runs", "signs", "zeros"])
def test_ties_and_orders(zt, kind):
    V = 20_011
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    z = {"equal": torch.full_like(i, -2.5), "ascending": i * 1e-3, "descending": -i * 1e-3, "two": (i % 2) * 3,
         "runs": (i // 97) % 5, "signs": torch.where(i % 3 == 0, -1.0, 1.0) * ((i * 7919) % 13),
         "zeros": torch.where(i % 2 == 0, 0.0, -0.0)}[kind].to(TYPES[zt]).repeat(3, 1)
    for top in (1, 50, 128):
        _check_forward(z, _ids(3, V), 1.0, top)


@pytest.mark.parametrize("zt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [2, 600])
def test_masks(T, zt):
    """Forbidden tokens at -inf, at the type's lowest value or at -1e4; rows with one, two or no
    token left, and rows of nothing but masks of finite value."""
    V = 3001
    for mask in (-INF, torch.finfo(TYPES[zt]).min, -1e4):
        z = _logits(T, V, TYPES[zt])
        g = torch.Generator(device="cuda").manual_seed(1)
        z[torch.rand(T, V, generator=g, device="cuda") < 0.9] = mask
        z[0] = mask
        z[1] = mask
        z[1, 2990] = 1.5
        _check_forward(z, _ids(T, V), 1.0, 30)
        _check_forward(z, _ids(T, V), 0.25, 0)


def test_far_values():
    """Rows far from 0, whose c z would lose all bits: by a common offset, and masks of
    several sizes with nothing else."""
    z = _logits(8, 2500, torch.float32)
    z[0] += 1e6
    z[1] -= 1e6
    z[2] = -1e9
    z[3] = torch.where(torch.arange(2500, device="cuda") % 3 == 0, -1e9, -1e9 + 64)
    z[4] = torch.where(torch.arange(2500, device="cuda") % 3 == 0, -3e38, -2e38)
    z[5] *= 1e30
    z[6] += 5e4
    z[7] = 3e38
    _check_forward(z, _ids(8, 2500), 1.0, 12)
    big = z.repeat(80, 1)
    assert torch.equal(ef.token_logprobs(big)[1][:8], ef.token_logprobs(big)[1][-8:])


@pytest.mark.parametrize("T", [6, 700])
def test_special_values_stay_in_their_row(T):
    z = _logits(T, 4000, torch.float32)
    ids = _ids(T, 4000)
    want = ef.token_logprobs(z, ids, top=5)
    y = z.clone()
    y[1, 77], y[2, 3999], y[4, 0] = math.nan, INF, -INF
    got = ef.token_logprobs(y, ids, top=5)
    for r in (1, 2):
        assert got[0][r].isnan() and got[1][r].isnan() and got[2][r].isnan() and got[4][r].isnan().all()
    assert int(got[3][1, 0]) == 77 and int(got[3][2, 0]) == 3999
    others = [r for r in range(T) if r not in (1, 2, 4)]
    assert all(torch.equal(a[others], b[others]) for a, b in zip(want, got))


@pytest.mark.parametrize("T", [40, 9000])
def test_padding_and_bad_ids(T):
    V = 300
    z = _logits(T, V, torch.bfloat16)
    z[3] = math.nan
    ids = _ids(T, V)
    ids[3] = ids[T - 1] = -100
    _check_forward(z, ids, 1.0, 4, padding_idx=-100)
    ids[5], ids[7] = V, -1
    z[3] = 0
    _check_forward(z, ids, 1.0, 4, padding_idx=-100, status=ef.ERR_BAD_INPUT)
    ids[5], ids[7] = 0, 1
    _check_forward(z, ids, 1.0, 4, padding_idx=-100)


def test_shapes_and_given_outputs():
    z = _logits(12, 50, torch.float32).view(3, 4, 50)
    ids = _ids(12, 50).view(3, 4)
    want = ef.token_logprobs(z, ids, top=3)
    assert want[0].shape == (12,) and want[3].shape == (12, 3) and want[3].dtype == torch.int32
    outs = dict(logprob=torch.empty(12, device="cuda"), entropy=torch.empty(12, device="cuda"),
                lse=torch.empty(12, device="cuda"), top_ids=torch.empty(12, 3, dtype=torch.int32, device="cuda"),
                top_logprobs=torch.empty(12, 3, device="cuda"))
    got = ef.token_logprobs(z, ids, top=3, **outs)
    assert all(a is b for a, b in zip(got, outs.values())) and all(torch.equal(a, b) for a, b in zip(got, want))
    e = ef.token_logprobs(z[:0], ids[:0], top=3)
    assert e[0].shape == (0,) and e[4].shape == (0, 3)
    assert ef.token_logprobs(z[0, 0])[2].shape == (1,)


def test_rows_past_2_31_elements():
    T, V = 20_000, 131_072
    z = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    for r in range(0, T, 2000):
        z[r:r + 2000].normal_(0, 3)
    at = torch.tensor([0, 16_383, 16_384, 19_999], device="cuda")
    ids = _ids(T, V)
    got = ef.token_logprobs(z, ids, top=7)
    _check_forward(z[at], ids[at], 1.0, 7)
    # (four rows alone are shared by clusters: the sums' order differs)
    assert torch.equal(got[3][at], _best(z[at], 7).int())
    e = Exact(z[at], 1.0)
    _near(got[2][at], e.lse, e.err_lse())
    g = -torch.ones(T, device="cuda")
    ef.token_logprobs_grad(z, ids, got[2], grad_logprob=g, out=z)
    want = e.p.clone()
    want[torch.arange(4, device="cuda"), ids[at]] -= 1.0
    _near(z[at], want, e.p * (EX2 + 40 * U * e.round) + 8 * U * want.abs() + U, torch.bfloat16)


# ----------------------------------------------------------------- gradient

def _check_gradient(z, ids, scale, g, h, out=None, out_dtype=None, padding_idx=-1):
    T, V = z.shape
    lp, en, ls, _, _ = ef.token_logprobs(z, ids, scale=scale, padding_idx=padding_idx)
    z0 = z.clone()
    got = ef.token_logprobs_grad(z, ids, ls, grad_logprob=g, entropy=en if h is not None else None, grad_entropy=h,
                                 scale=scale, padding_idx=padding_idx, out=out, out_dtype=out_dtype)
    x = z0.double() * scale
    t = torch.where(x == -INF, -INF, x - ls.double()[:, None])
    p = t.exp()
    i = ids.reshape(-1).long() if ids is not None else torch.full((T,), -1, device="cuda")
    skip = i == padding_idx if ids is not None else torch.zeros(T, dtype=torch.bool, device="cuda")
    ok = (i >= 0) & (i < V)
    G = torch.where(ok, g.double(), 0.0) if g is not None else torch.zeros(T, dtype=torch.float64, device="cuda")
    H = h.double() if h is not None else torch.zeros_like(G)
    skip = skip | ((G == 0) & (H == 0)) | (ls == -INF)
    hot = torch.zeros_like(x)
    hot[torch.arange(T, device="cuda")[ok], i[ok]] = 1.0
    tc = t.clamp(min=-1e4)
    k = G[:, None] + H[:, None] * (tc + en.double()[:, None])
    want = scale * (G[:, None] * hot - p * k)
    size = G.abs()[:, None] + H.abs()[:, None] * (tc.abs() + en.double().abs()[:, None])
    # p: t is rounded once and its product with log2 e (a constant off by u) twice
    rel = EX2 + 6 * U * (tc.abs() + x.clamp(min=-1e30).abs() * 0 + 1)
    err = scale * (p * size * (rel + 6 * U) + 4 * U * (G.abs()[:, None] * hot))
    # (p below 2^-126 is 0)
    err = err + scale * size * 2.0**-126
    want[skip] = 0.0
    err[skip] = 0.0
    assert got.shape == z.shape
    assert (got[skip] == 0).all()
    _near(got, want, err, got.dtype)
    return got


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("zt,ot", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "bf16"), ("f32", "f16")])
def test_gradient(T, V, zt, ot):
    z = _logits(T, V, TYPES[zt])
    ids = _ids(T, V, 3)
    g = torch.randn(T, device="cuda")
    h = torch.randn(T, device="cuda")
    _check_gradient(z, ids, 0.5, g, h, out_dtype=TYPES[ot])
    _check_gradient(z, ids, 1.0, g, None, out_dtype=TYPES[ot])
    _check_gradient(z, None, 1.0, None, h, out_dtype=TYPES[ot])


@pytest.mark.parametrize("ld,ldo,off", [(1001, 1001, 0), (1008, 1016, 8), (1030, 1001, 3), (1024, 1024, 1)])
@pytest.mark.parametrize("zt,ot", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_gradient_strides(ld, ldo, off, zt, ot):
    T, V = 30, 1001
    z = _logits(T, V, TYPES[zt], ld, off)
    buf = torch.full((T * ldo + off + 8,), 7.0, dtype=TYPES[ot], device="cuda")
    rows = buf[off:off + T * ldo].view(T, ldo)
    _check_gradient(z, _ids(T, V), 1.0, torch.randn(T, device="cuda"), None, out=rows[:, :V])
    assert (rows[:, V:] == 7.0).all() and (buf[:off] == 7.0).all() and (buf[off + T * ldo:] == 7.0).all()


def test_gradient_in_place_padding_masks():
    T, V = 60, 2003
    z = _logits(T, V, torch.bfloat16)
    z[:, ::3] = -INF
    z[5] = -INF
    z[7] = math.nan
    z[8, 10] = math.nan
    ids = _ids(T, V) // 3 * 3 + 1
    ids[7] = -1
    g, h = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    g[11] = h[11] = 0.0
    keep = [r for r in range(T) if r != 8]
    zk, idk = z[keep].contiguous(), ids[keep].contiguous()
    want = _check_gradient(zk, idk, 1.0, g[keep], h[keep])
    got = _check_gradient(zk, idk, 1.0, g[keep], h[keep], out=zk)
    assert got.data_ptr() == zk.data_ptr() and torch.equal(got, want)
    lp, en, ls, _, _ = ef.token_logprobs(z, ids)
    assert ef.token_logprobs_grad(z, ids, ls, grad_logprob=g)[8].isnan().all()


@pytest.mark.parametrize("T", [40, 9000])
def test_gradient_bad_ids(T):
    z = _logits(T, 300, torch.float32)
    ids = _ids(T, 300)
    ids[4] = 300
    ls = ef.token_logprobs(z, ids)[2]
    ws = torch.full((ef.token_logprobs_workspace_bytes(),), 0xA5, dtype=torch.uint8, device="cuda")
    g = torch.ones(T, device="cuda")
    d = ef.token_logprobs_grad(z, ids, ls, grad_logprob=g, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == ef.ERR_BAD_INPUT
    assert (d[4] == 0).all() and (d[5] != 0).any()
    ids[4] = -1
    ef.token_logprobs_grad(z, ids, ls, grad_logprob=g, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0


def test_gradient_against_autograd_and_differences():
    T, V = 6, 500
    z = _logits(T, V, torch.float32)
    ids = _ids(T, V)
    gen = torch.Generator(device="cuda").manual_seed(2)
    g, h = (torch.randn(T, generator=gen, device="cuda") for _ in range(2))
    lp, en, ls, _, _ = ef.token_logprobs(z, ids, scale=0.7)
    got = ef.token_logprobs_grad(z, ids, ls, g, en, h, scale=0.7).double()
    s = float(torch.tensor(0.7))

    def loss(z):
        logp = torch.log_softmax(z * s, 1)
        return (logp.gather(1, ids[:, None])[:, 0] * g.double() - (logp.exp() * logp).sum(1) * h.double()).sum()

    z64 = z.double().requires_grad_()
    loss(z64).backward()
    # (lse and p in fp32: some tens of 2^-24)
    assert float((got - z64.grad).norm() / z64.grad.norm()) < 1e-5
    d = torch.randn(T, V, generator=gen, device="cuda").double()
    diff = (loss(z.double() + 1e-5 * d) - loss(z.double() - 1e-5 * d)) / 2e-5
    assert float(abs(diff - (got * d).sum())) < 1e-5 * float(got.norm() * d.norm())


# ------------------------------------------------------------- distillation

def _teacher(T, V, K, seed=0, dtype=torch.float32, distinct=True):
    g = torch.Generator(device="cuda").manual_seed(seed + T + K)
    if distinct and K <= V:
        ids = torch.rand(T, V, generator=g, device="cuda").argsort(1)[:, :K] if V <= 5000 else \
            (torch.randint(0, V, (T, 1), generator=g, device="cuda") + torch.arange(K, device="cuda") * (V // K)) % V
    else:
        ids = torch.randint(0, V, (T, K), generator=g, device="cuda")
    return ids.to(torch.int32 if K % 2 else torch.int64).contiguous(), \
        (torch.randn(T, K, generator=g, device="cuda") * 3).to(dtype)


def _check_distill(z, ids, tl, weight, scale, grad=True, out=None, out_dtype=None, status=0):
    T, V = z.shape
    K = ids.shape[1]
    z0 = z.clone()
    ws = torch.full((ef.distill_loss_workspace_bytes(),), 0xA5, dtype=torch.uint8, device="cuda")
    loss, dz = ef.distill_loss(z, ids, tl, weight=weight, scale=scale, grad=grad, grad_logits=out, out_dtype=out_dtype,
                               ws=ws)
    assert ef.topk_ef_last_device_status(ws) == status
    w = torch.ones(T, dtype=torch.float64, device="cuda") if weight is None else weight.double()
    i = ids.long()
    ok = (i >= 0) & (i < V)
    t = torch.where(ok, tl.double(), -INF) * scale
    none = (t == -INF).all(1) | (w == 0)
    q = torch.nan_to_num(torch.softmax(t, 1), nan=0.0) if K else t
    logq = torch.log_softmax(t, 1) if K else t
    e = Exact(z0, scale)
    ic = i.clamp(0, V - 1)
    logp, elogp = e.logp.gather(1, ic), e.err_logp().gather(1, ic)
    term = torch.where(q > 0, q * (logq - logp), 0.0)
    tt = torch.where(q > 0, (t - (t.max(1, keepdim=True).values if K else 0)).abs(), 0.0)
    # q: ex2 and its argument's roundings, the sum of 256 the same way (20 adds), a division
    e_q = 2 * EX2 + U * (8 * tt + 30)
    want = w * term.sum(1)
    err = w.abs() * (torch.where(q > 0, q * (elogp + EX2 + U * (6 * tt + 30 + 4 * logq.abs())), 0.0) +
                     term.abs() * (e_q + 30 * U)).sum(1)
    want[none] = 0.0
    err[none] = 0.0
    assert (loss[none] == 0).all()
    _near(loss, want, err)
    if not grad and out is None:
        assert dz is None
        return loss, dz
    qv = torch.zeros_like(e.p).scatter_add_(1, ic, torch.where(ok, q, 0.0))
    eqv = torch.zeros_like(e.p).scatter_add_(1, ic, torch.where(ok, q * (e_q + 16 * U), 0.0))
    f = (w * scale)[:, None]
    want = f * (e.p - qv)
    err = f.abs() * (e.p * (e.e_s[:, None] + EX2 + U * (2 * e.round + 8)) + eqv + 4 * U * (e.p + qv))
    # (2^t below 2^-126 is 0, s at least 1/2: p may lose 2^-125, times f)
    err = err + f.abs() * 2.0**-125
    want[none] = 0.0
    err[none] = 0.0
    assert (dz[none] == 0).all()
    _near(dz, want, err, dz.dtype)
    return loss, dz


@pytest.mark.parametrize("T,V", SHAPES)
@pytest.mark.parametrize("zt,ot,K", [("f32", "f32", 20), ("bf16", "bf16", 64), ("f16", "f16", 1), ("bf16", "f32", 33),
                                     ("f32", "bf16", 256)])
def test_distill(T, V, zt, ot, K):
    z = _logits(T, V, TYPES[zt])
    ids, tl = _teacher(T, V, K, distinct=K <= V, dtype=TYPES[ot])
    w = torch.rand(T, device="cuda") + 0.1
    w[T // 2] = 0.0 if T > 1 else 1.0
    loss, dz = _check_distill(z, ids, tl, w, 0.5, out_dtype=TYPES[ot])
    # (the loss alone is summed in another order, within the same bound)
    _check_distill(z, ids, tl, w, 0.5, grad=False)
    again = ef.distill_loss(z, ids, tl, weight=w, scale=0.5, grad=True, out_dtype=TYPES[ot])
    assert torch.equal(again[0], loss) and torch.equal(again[1], dz)
    if zt == ot:
        here = z.clone()
        got = ef.distill_loss(here, ids, tl, weight=w, scale=0.5, grad_logits=here)
        assert torch.equal(got[1], dz) and got[1].data_ptr() == here.data_ptr() and torch.equal(got[0], loss)


@pytest.mark.parametrize("ld,ldo,off", [(1001, 1001, 0), (1008, 1016, 8), (1030, 1001, 3), (1024, 1024, 1)])
@pytest.mark.parametrize("zt,ot", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
def test_distill_strides(ld, ldo, off, zt, ot):
    T, V = 30, 1001
    z = _logits(T, V, TYPES[zt], ld, off)
    ids, tl = _teacher(T, V, 12)
    buf = torch.full((T * ldo + off + 8,), 7.0, dtype=TYPES[ot], device="cuda")
    rows = buf[off:off + T * ldo].view(T, ldo)
    _check_distill(z, ids, tl, None, 1.0, out=rows[:, :V])
    assert (rows[:, V:] == 7.0).all() and (buf[:off] == 7.0).all() and (buf[off + T * ldo:] == 7.0).all()


@pytest.mark.parametrize("T", [5, 800])
def test_distill_repeated_empty_and_bad_entries(T):
    V, K = 700, 40
    z = _logits(T, V, torch.float32)
    ids, tl = _teacher(T, V, K, distinct=False)
    ids[:, 3] = ids[:, 7] = ids[:, 39]
    ids[0] = 11
    ids[1] = -1
    ids[2, 5:] = -7
    tl[3, :] = -INF
    tl[4, ::2] = -INF
    ids[4, 1] = ids[4, 0]
    _check_distill(z, ids, tl, None, 1.0)
    ids[4, 0], ids[3, 2] = V, V + 5
    _check_distill(z, ids, tl, None, 1.0, status=ef.ERR_BAD_INPUT)
    ids[4, 0], ids[3, 2] = 1, 1
    _check_distill(z, ids, tl, None, 1.0)
    _check_distill(z, ids[:, :0].contiguous(), tl[:, :0].contiguous(), None, 1.0)


def test_distill_masks_and_special_values():
    T, V, K = 9, 3000, 10
    z = _logits(T, V, torch.float32)
    ids, tl = _teacher(T, V, K)
    z[:, ::2] = -INF
    ids = (ids | 1)
    z[3] = -1e9
    z[4] = torch.finfo(torch.float32).min
    _check_distill(z, ids, tl, None, 1.0)
    w = torch.ones(T, device="cuda")
    want = ef.distill_loss(z, ids, tl, weight=w, grad=True)
    z[1, 5], z[2, 7] = math.nan, INF
    tl[5, 0] = math.nan
    z[6, int(ids[6, 0])] = -INF
    z[7] = -INF
    z[8] = math.nan
    w[8] = 0.0
    loss, dz = ef.distill_loss(z, ids, tl, weight=w, grad=True)
    assert loss[1].isnan() and loss[2].isnan() and loss[5].isnan() and loss[6] == INF and loss[7] == INF
    assert dz[1].isnan().all() and dz[5, ids[5].long()].isnan().all()
    assert dz[6].isfinite().all() and dz[7].isfinite().all() and (dz[8] == 0).all() and loss[8] == 0
    assert torch.equal(dz[[0, 3, 4]], want[1][[0, 3, 4]]) and torch.equal(loss[[0, 3, 4]], want[0][[0, 3, 4]])


def test_distill_against_autograd_and_differences():
    T, V, K = 5, 400, 16
    z = _logits(T, V, torch.float32)
    ids, tl = _teacher(T, V, K, distinct=False)
    gen = torch.Generator(device="cuda").manual_seed(2)
    w = torch.rand(T, generator=gen, device="cuda")
    got_loss, got = ef.distill_loss(z, ids, tl, weight=w, scale=0.5, grad=True)

    def loss(z):
        q = torch.softmax(tl.double() * 0.5, 1)
        logp = torch.log_softmax(z * 0.5, 1).gather(1, ids.long())
        return (w.double() * (q * (q.log() - logp)).sum(1)).sum()

    z64 = z.double().requires_grad_()
    want = loss(z64)
    want.backward()
    want = want.detach()
    assert float(abs(got_loss.double().sum() - want)) < 1e-5 * float(want)
    assert float((got.double() - z64.grad).norm() / z64.grad.norm()) < 1e-5
    d = torch.randn(T, V, generator=gen, device="cuda").double()
    diff = (loss(z.double() + 1e-5 * d) - loss(z.double() - 1e-5 * d)) / 2e-5
    assert float(abs(diff - (got.double() * d).sum())) < 1e-5 * float(got.double().norm() * d.norm())


# --------------------------------------------------------------- the set together

@pytest.mark.parametrize("T", [3, 500])
def test_teacher_to_student(T):
    """A teacher's alternatives are a student's targets: where both are the same model, the
    loss is 0 up to the mass that the teacher's set leaves out."""
    V, K = 3000, 32
    z = _logits(T, V, torch.bfloat16)
    _, _, _, ids, lp = ef.token_logprobs(z, top=K)
    loss, dz = _check_distill(z, ids, lp, None, 1.0)
    kept = lp.double().exp().sum(1)
    e = Exact(z, 1.0)
    _near(loss, -kept.log(), 4 * e.e_s + 400 * U)
    pad = torch.full((T,), -1, device="cuda")
    _, _, _, ids, lp = ef.token_logprobs(z, pad, top=K)
    loss, dz = ef.distill_loss(z, ids, lp, grad=True)
    assert (loss == 0).all() and (dz == 0).all()


@pytest.mark.parametrize("T,V", [(3, 40000), (400, 3000), (9000, 60)])
def test_capture_and_streams(T, V):
    z = _logits(T, V, torch.bfloat16)
    ids = _ids(T, V)
    tids, tl = _teacher(T, V, 8, distinct=False)
    g = torch.randn(T, device="cuda")
    ws = [torch.empty(512, dtype=torch.uint8, device="cuda") for _ in range(3)]

    def run(ws, **kw):
        a = ef.token_logprobs(z, ids, top=5, ws=ws[0], **kw)
        b = ef.token_logprobs_grad(z, ids, a[2], grad_logprob=g, entropy=a[1], grad_entropy=g, ws=ws[1], **kw)
        c = ef.distill_loss(z, tids, tl, grad=True, ws=ws[2], **kw)
        return [*a, b, *c]

    want = run(ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(ws)
    for _ in range(2):
        for t in got:
            t.fill_(5)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(ef.topk_ef_last_device_status(w) == 0 for w in ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run([None] * 3, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refuses():
    z = torch.randn(4, 30, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    for kw in (dict(ids=ids[:3]), dict(ids=ids.float()), dict(ids=ids.cpu()), dict(logprob=f), dict(entropy=f[:3]),
               dict(lse=f.half()), dict(top=2, top_ids=torch.zeros(4, 2, device="cuda")),
               dict(top=2, top_logprobs=torch.zeros(4, 3, device="cuda")), dict(top_logprobs=torch.zeros(4, 3, device="cuda")),
               dict(ws=torch.empty(512, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            ef.token_logprobs(z, **kw)
    for kw in (dict(top=129), dict(top=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=INF),
               dict(ws=torch.empty(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ef.TopkEfError):
            ef.token_logprobs(z, **kw)
    with pytest.raises(ef.TopkEfError):
        ef.token_logprobs(z[:, :0])
    with pytest.raises(ef.TopkEfError):
        ef.token_logprobs(torch.empty(1, 2**19 + 1, device="cuda"), top=1)
    with pytest.raises(ValueError):
        ef.token_logprobs(z.t())
    for kw in (dict(lse=None), dict(lse=f, grad_entropy=f), dict(lse=f, ids=None, grad_logprob=f),
               dict(lse=f, out=torch.empty(4, 29, device="cuda")), dict(lse=f, out=z, out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            ef.token_logprobs_grad(z, **{"ids": ids, **kw})
    with pytest.raises(ef.TopkEfError):
        ef.token_logprobs_grad(z, ids, f, scale=0.0)
    t = torch.zeros(4, 2, device="cuda")
    i2 = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for args, kw in (((i2[:3].contiguous(), t), {}), ((i2, t[:, :1]), {}), ((i2, None), {}), ((i2, t), dict(weight=f[:2])),
                     ((i2, t), dict(loss=f.half())), ((i2, t), dict(grad_logits=z[:3])), ((i2, t.double()), {})):
        with pytest.raises(ValueError):
            ef.distill_loss(z, *args, **kw)
    with pytest.raises(ef.TopkEfError):
        ef.distill_loss(z, torch.zeros(4, 257, dtype=torch.int32, device="cuda"), torch.zeros(4, 257, device="cuda"))
    with pytest.raises(ef.TopkEfError):
        ef.distill_loss(z, i2, t, scale=-2.0)


@pytest.mark.parametrize("T,V", [(501, V) for V in (1, 33, 500, 2000, 4097, 8192, 16385, 40001)] +
                         [(900, 1), (900, 33), (900, 500), (900, 2000), (1800, 4000), (1800, 8000)])
@pytest.mark.parametrize("zt", ["f32", "bf16"])
def test_more_rows_than_run_at_once(T, V, zt):
    """Rows of one warp, four and eight."""
    z = _logits(T, V, TYPES[zt])
    z[3] = -INF
    z[5] = -1e9
    z[7, ::2] = -INF
    ids = _ids(T, V)
    ids[11] = -1
    _check_forward(z, ids, 1.0, 17)
    _check_gradient(z, ids, 1.0, torch.randn(T, device="cuda"), torch.randn(T, device="cuda"))
    tids, tl = _teacher(T, V, 9, distinct=9 <= V)
    w = torch.rand(T, device="cuda")
    w[::5] = 0
    keep = [r for r in range(T) if r not in (3, 7)]       # (a teacher's token at -inf: loss +inf)
    zk = z[keep].contiguous()
    tk = [t[keep].contiguous() for t in (tids, tl, w)]
    _check_distill(zk, *tk[:2], tk[2], 0.7)
    _check_distill(zk, *tk[:2], None, 0.7, grad=False)


@pytest.mark.parametrize("T,V,ld,off,zt,top", [
    (1000, 1000, 1000, 0, "bf16", 31), (1000, 1003, 1007, 5, "bf16", 32), (900, 130, 131, 1, "bf16", 128),
    (1000, 512, 512, 0, "f32", 128), (1000, 2011, 2011, 3, "f32", 100), (900, 17, 17, 9, "f32", 3),
    (1900, 8000, 8000, 0, "bf16", 100), (1900, 7001, 7003, 1, "bf16", 20), (1900, 4000, 4001, 7, "f32", 128),
    (1900, 8192, 8192, 0, "f16", 64), (900, 20000, 20000, 0, "bf16", 64), (900, 20001, 20005, 3, "f32", 17),
    (1600, 60001, 60001, 0, "bf16", 128), (1600, 45001, 45001, 0, "f32", 40)])
def test_many_rows(T, V, ld, off, zt, top):
    """Rows of one warp and of four, their tops from short groups and long ones."""
    z = _logits(T, V, TYPES[zt], ld=ld, offset=off)
    z[0] = -INF
    z[1] = -INF
    z[1, V // 2:V // 2 + 3] = 1.0
    z[2] = 0.5
    z[3] = -1e9 if zt != "f16" else -6e4
    z[4, ::2] = -INF
    z[5] = torch.arange(V, device="cuda").remainder(7).to(z.dtype)
    z[6, :-1] = -INF
    z[7] = -torch.arange(V, device="cuda").float().to(z.dtype)
    z[8, 1:] = -INF
    z[9] = 0.0
    z[9, 1::2] = -0.0
    _check_forward(z, _ids(T, V), 1.0, top)
    _check_forward(z, _ids(T, V), 1.0, 0)


@pytest.mark.parametrize("V,zt,top", [(2**19 - 64, "f32", 128), (2**20 - 64, "bf16", 100), (700_001, "f32", 0),
                                      (3_000_000, "bf16", 0)])
def test_long_rows(V, zt, top):
    z = _logits(2, V, TYPES[zt])
    _check_forward(z, _ids(2, V), 1.0, top)
    _check_gradient(z, _ids(2, V), 1.0, torch.randn(2, device="cuda"), torch.randn(2, device="cuda"))
    tids, tl = _teacher(2, V, 20)
    _check_distill(z, tids, tl, None, 1.0)


def test_all_entries_the_same_token():
    z = _logits(6, 900, torch.float32)
    ids = torch.full((6, 256), 417, dtype=torch.int64, device="cuda")
    _check_distill(z, ids, torch.randn(6, 256, device="cuda"), None, 1.0)


@pytest.mark.parametrize("scale", [1e-3, 1e-6, 50.0, 1e4])
@pytest.mark.parametrize("zt", ["f32", "bf16", "f16"])
def test_scales(scale, zt):
    """Near uniform and near one-hot rows, forbidden tokens among them."""
    z = _logits(5, 2100, TYPES[zt], peak=False)
    z[:, ::7] = -INF
    scale = float(torch.tensor(scale, dtype=torch.float32))
    _check_forward(z, _ids(5, 2100), scale, 10)
    tids, tl = _teacher(5, 2100, 8)
    tids = tids // 7 * 7 + 1
    _check_distill(z, tids, tl * 0.1, None, scale)


def test_two_calls_at_once():
    zs = [_logits(700, 9000, torch.bfloat16, seed=s) for s in (1, 2)]
    ids = [_ids(700, 9000, s) for s in (1, 2)]
    teach = [_teacher(700, 9000, 16, s) for s in (1, 2)]

    def run(i, s):
        a = ef.token_logprobs(zs[i], ids[i], top=9, stream=s)
        b = ef.token_logprobs_grad(zs[i], ids[i], a[2], grad_logprob=a[0], entropy=a[1], grad_entropy=a[1], stream=s)
        return [*a, b, *ef.distill_loss(zs[i], *teach[i], grad=True, stream=s)]

    want = [run(i, None) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [run(i, s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g, v in zip(got, want) for p, q in zip(g, v))
