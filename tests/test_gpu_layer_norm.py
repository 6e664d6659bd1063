"""layer_norm and layer_norm_grad on the GPU against 64-bit formulas.

u = 2^-24 is half a step of fp32.  A sum of n terms added in any order is off by
at most depth u times the sum of magnitudes (to first order), where depth is the
longest chain of adds: at most 16 in a thread, 5 in a warp and 32 over warps
in the register kernels, D / 512 + 40 in the kernels for long rows, and for the
column sums at most T / blocks of a block's rows and the blocks in eighths."""
import itertools

import pytest
import torch

import error_feedback_b200 as ef

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = 2.0**-24


def _strided(rows, cols, dtype, ld, offset, seed, scale=1.0, shift=0.0):
    """A [rows, cols] view with row stride ld that starts `offset` elements into its buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(rows * ld + offset + 8, generator=g, device="cuda").mul_(scale).add_(shift).to(dtype)
    return buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def _near(got, want, err, dtype):
    """got within err of want before its rounding to dtype."""
    got = got.double()
    eps = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * eps
    bound = err * (1 + eps) + want.abs() * eps + tiny
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: " \
        f"{got[bad][0]} for {want[bad][0]} (bound {bound[bad][0]})"


def _depth(D):
    return 64 + D // 512


def _forward64(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = (d.square().mean(1) + eps).rsqrt()
    xh = d * rstd[:, None]
    y = xh * (1.0 if w is None else w.double()) + (0.0 if b is None else b.double())
    return y, mean, rstd, xh


def _check_forward(out, mean, rstd, x, w, b, eps):
    y, m, r, xh = _forward64(x, w, b, eps)
    n = _depth(x.shape[1])
    d = x.double() - x.double()[:, :1]
    # the mean: n adds of the elements, their sum with a factor that is rounded; past 16 deviations
    # from 0 a rounded mean and n adds of the distances from it instead
    dist = x.double() - m[:, None]
    plain = (n + 3) * U * x.double().abs().mean(1)
    err_m = torch.where(m.square() > 256 * dist.square().mean(1), (n + 2) * U * dist.abs().mean(1) + 4 * U * m.abs(), plain)
    assert ((mean.double() - m).abs() <= err_m + 1e-45).all()
    # squares: two roundings each and n adds; the means that they are taken from,
    # off by err_m (less the sum with c), enter twice; the root 2 steps and eps's own
    rel = 0.5 * ((n + 4) * U + 4 * (n + 2) * U * d.abs().mean(1) * r) + 6 * U + U
    rel = rel + 0.5 * ((n + 2) * U * d.abs().mean(1) * r) ** 2
    # (rest^2 is taken off the squares of distances that a rounded mean of n roundings leaves)
    rel = rel + (n + 4) * U * ((n + 2) * U * x.double().abs().mean(1) * r) ** 2
    assert ((rstd.double() - r).abs() <= rel * r).all()
    wm = torch.ones(x.shape[1], dtype=torch.float64, device="cuda") if w is None else w.double().abs()
    bm = 0.0 if b is None else b.double().abs()
    # x - mean = (x - m_w) - rest: m_w is off by n roundings of the mean's size at most, rest is
    # the mean of what that leaves and off by n roundings of it (all there is where the elements
    # are equal)
    second = ((n + 2) * U) ** 2 * x.double().abs().mean(1)[:, None]
    err = wm * r[:, None] * ((n + 3) * U * d.abs().mean(1)[:, None] + 2 * U * d.abs() + second)
    err = err + (xh.abs() * wm) * (rel[:, None] + 2 * U) + U * (xh.abs() * wm + bm)
    _near(out, y, err, out.dtype)


SHAPES = [(1, 1), (3, 2), (1, 8), (5, 31), (9, 64), (2, 255), (700, 256), (33, 257), (17, 512), (40, 520),
          (1, 1000), (513, 1001), (3, 1024), (6, 1030), (2, 2048), (150, 2056), (1, 4096), (310, 4096),
          (3, 4097), (4, 8192), (2, 8200), (3, 16384), (2, 16385), (3, 20000), (1, 70001)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("xt,ot", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "f32")])
def test_forward(T, D, xt, ot):
    x = _strided(T, D, TYPES[xt], D, 0, T + D, 2.0, 0.5)
    w = _strided(1, D, TYPES[xt], D, 0, 1, 0.3, 1.0)[0].contiguous()
    b = _strided(1, D, TYPES[ot], D, 0, 2)[0].contiguous()
    out, mean, rstd = ef.layer_norm(x, w, b, out_dtype=TYPES[ot])
    assert out.dtype == TYPES[ot] and out.shape == x.shape
    _check_forward(out, mean, rstd, x, w, b, 1e-5)
    again = ef.layer_norm(x, w, b, out_dtype=TYPES[ot])
    assert all(torch.equal(p, q) for p, q in zip((out, mean, rstd), again))


@pytest.mark.parametrize("types", list(itertools.product(TYPES, TYPES)))
def test_every_pair_of_types(types):
    xt, ot = types
    for D in (40, 300, 1100, 3000, 9001, 17000):
        x = _strided(3, D, TYPES[xt], D, 0, D)
        out, mean, rstd = ef.layer_norm(x, out_dtype=TYPES[ot])
        _check_forward(out, mean, rstd, x, None, None, 1e-5)
        dy = _strided(3, D, TYPES[ot], D, 0, D + 1, 1e-1)
        _check_gradient(dy, x, mean, rstd, None, ef.layer_norm_grad(dy, x, mean, rstd))


@pytest.mark.parametrize("ldx,ldo,off", [(72, 72, 0), (64, 80, 8), (61, 61, 0), (67, 64, 3), (64, 61, 1)])
@pytest.mark.parametrize("xt,ot", [("f32", "bf16"), ("bf16", "bf16")])
def test_strides(ldx, ldo, off, xt, ot):
    x = _strided(50, 61, TYPES[xt], ldx, off, 3)
    buf = torch.full((50 * ldo + off + 8,), 7.0, dtype=TYPES[ot], device="cuda")
    rows = buf[off:off + 50 * ldo].view(50, ldo)
    out, mean, rstd = ef.layer_norm(x, eps=1e-3, out=rows[:, :61])
    _check_forward(out, mean, rstd, x, None, None, 1e-3)
    assert (rows[:, 61:] == 7.0).all() and (buf[:off] == 7.0).all() and (buf[off + 50 * ldo:] == 7.0).all()
    dy = _strided(50, 61, TYPES[xt], ldo, off, 4)
    buf = torch.full((50 * ldx + off + 8,), 7.0, dtype=TYPES[xt], device="cuda")
    rows = buf[off:off + 50 * ldx].view(50, ldx)
    got = ef.layer_norm_grad(dy, x, mean, rstd, grad_x=rows[:, :61])
    _check_gradient(dy, x, mean, rstd, None, got)
    assert (rows[:, 61:] == 7.0).all() and (buf[:off] == 7.0).all() and (buf[off + 50 * ldx:] == 7.0).all()


@pytest.mark.parametrize("D", [1, 7, 100, 1000, 4096, 20000])
@pytest.mark.parametrize("shift", [0.0, 300.0, -1e5])
def test_offsets_and_outliers(D, shift):
    """A common offset, a first element far from the others, equal elements."""
    x = _strided(6, D, torch.float32, D, 0, D, 1.0, shift)
    x[1, 0] += 1000.0
    x[2, D // 2] -= 3e4
    x[3] = shift
    out, mean, rstd = ef.layer_norm(x)
    _check_forward(out, mean, rstd, x, None, None, 1e-5)


@pytest.mark.parametrize("D", [64, 900, 4096, 17000])
def test_special_values_stay_in_their_row(D):
    x = _strided(6, D, torch.float32, D, 0, 5)
    ref = ef.layer_norm(x)
    y = x.clone()
    y[1, D - 1], y[3, 0], y[4, D // 3] = float("nan"), float("inf"), float("-inf")
    out, mean, rstd = ef.layer_norm(y)
    for r in (1, 3, 4):
        assert out[r].isnan().all() and rstd[r].isnan()
    for r in (0, 2, 5):
        assert all(torch.equal(a[r], b[r]) for a, b in zip((out, mean, rstd), ref))


def test_shapes_defaults_and_in_place():
    x = torch.randn(3, 5, 48, device="cuda", dtype=torch.bfloat16)
    out, mean, rstd = ef.layer_norm(x)
    assert out.shape == x.shape and out.dtype == x.dtype and mean.shape == rstd.shape == (15,)
    o2, m2, r2 = ef.layer_norm(x, stats=False)
    assert m2 is None and r2 is None and torch.equal(o2, out)
    o3, m3, r3 = ef.layer_norm(x, stats=False, mean=mean.clone())
    assert torch.equal(m3, mean) and r3 is None
    y = x.clone()
    ef.layer_norm(y, out=y)
    assert torch.equal(y, out)
    one = torch.randn(48, device="cuda")
    assert ef.layer_norm(one)[0].shape == (48,)
    e, m, r = ef.layer_norm(x[:0])
    assert e.shape == (0, 5, 48) and m.numel() == 0
    z = torch.randn(4, 20000, device="cuda")
    want = ef.layer_norm(z)[0]
    ef.layer_norm(z, out=z)
    assert torch.equal(z, want)


# ----------------------------------------------------------------- gradient

def _check_gradient(dy, x, mean, rstd, w, got, old=None):
    T, D = x.shape
    n = _depth(D)
    X, Y, r = x.double(), dy.double(), rstd.double()[:, None]
    d = X - mean.double()[:, None]
    xh = d * r
    W = torch.ones(D, dtype=torch.float64, device="cuda") if w is None else w.double()
    g = Y * W
    s1, s2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - s1 - xh * s2)
    # xh and g carry 2 and 1 roundings, the sums n adds and their products, the
    # result three more
    m1, m2 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
    err = r * ((n + 3) * U * m1 + (n + 8) * U * m2 * xh.abs() + 5 * U * (g.abs() + s1.abs() + (xh * s2).abs()))
    _near(got[0], dx, err, got[0].dtype)
    if got[1] is None:
        return
    # a block's rows one after another, the blocks in eighths, the eighths: of T rows no
    # chain is longer than T / 148 + 2368 / 8 + 24 nor than T + 24
    k = min(T, T // 148 + 296) + 24
    for out, term, o in ((got[1], Y * xh, 0), (got[2], Y, 1)):
        want, mag = term.sum(0), term.abs().sum(0)
        if old is not None:
            want, mag = want + old[o].double(), mag + old[o].double().abs()
        _near(out, want, (k + 5) * U * mag, out.dtype)


def _run_gradient(T, D, xt, dt, wt, gt, acc=False):
    x = _strided(T, D, TYPES[xt], D, 0, T + D, 2.0, 0.5)
    dy = _strided(T, D, TYPES[dt], D, 0, T + D + 1, 1e-2)
    w = None if wt is None else _strided(1, D, TYPES[wt], D, 0, 1, 0.3, 1.0)[0].contiguous()
    _, mean, rstd = ef.layer_norm(x, w)
    gw = torch.randn(D, device="cuda").to(TYPES[gt])
    gb = torch.randn(D, device="cuda").to(TYPES[gt])
    old = (gw.clone(), gb.clone()) if acc else None
    ws = torch.full((ef.layer_norm_grad_workspace_bytes(T, D),), 0xFF, dtype=torch.uint8, device="cuda")
    got = ef.layer_norm_grad(dy, x, mean, rstd, w, accumulate=acc, grad_weight=gw, grad_bias=gb, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0
    _check_gradient(dy, x, mean, rstd, w, got, old)
    if not acc:
        again = ef.layer_norm_grad(dy, x, mean, rstd, w, out_dtype=TYPES[gt])
        assert all(torch.equal(p, q) for p, q in zip(got, again))
        # in place of either input
        for which in (x, dy):
            if which.dtype == x.dtype:
                a, b = x.clone(), dy.clone()
                to = a if which is x else b
                assert torch.equal(ef.layer_norm_grad(b, a, mean, rstd, w, affine=False, grad_x=to)[0], got[0])


@pytest.mark.parametrize("T,D", SHAPES + [(3000, 64), (5001, 1001), (2500, 4096), (20000, 16)])
@pytest.mark.parametrize("xt,dt,wt", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f32", "bf16", None),
                                      ("f16", "f16", "f32")])
def test_gradient(T, D, xt, dt, wt):
    _run_gradient(T, D, xt, dt, wt, "f32")


@pytest.mark.parametrize("T,D", [(1, 40), (600, 100), (70, 3001), (9, 9000)])
@pytest.mark.parametrize("gt", ["f32", "bf16", "f16"])
def test_gradient_accumulates(T, D, gt):
    _run_gradient(T, D, "bf16", "bf16", "f32", gt, acc=True)


def test_gradient_parts_and_empty():
    x = torch.randn(7, 40, device="cuda")
    dy = torch.randn(7, 40, device="cuda")
    _, mean, rstd = ef.layer_norm(x)
    gx, gw, gb = ef.layer_norm_grad(dy, x, mean, rstd)
    a, none_w, none_b = ef.layer_norm_grad(dy, x, mean, rstd, affine=False)
    assert torch.equal(a, gx) and none_w is None and none_b is None
    e = ef.layer_norm_grad(dy[:0], x[:0], mean[:0], rstd[:0])
    assert e[0].shape == (0, 40) and (e[1] == 0).all() and (e[2] == 0).all()
    w0, b0 = gw.clone(), gb.clone()
    ef.layer_norm_grad(dy[:0], x[:0], mean[:0], rstd[:0], accumulate=True, grad_weight=gw, grad_bias=gb)
    assert torch.equal(gw, w0) and torch.equal(gb, b0)


@pytest.mark.parametrize("D", [48, 1001])
def test_gradient_against_autograd_and_differences(D):
    g = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn(9, D, generator=g, device="cuda")
    w = torch.randn(D, generator=g, device="cuda")
    b = torch.randn(D, generator=g, device="cuda")
    dy = torch.randn(9, D, generator=g, device="cuda")
    _, mean, rstd = ef.layer_norm(x, w, b)
    got = ef.layer_norm_grad(dy, x, mean, rstd, w)
    leaves = [t.double().requires_grad_() for t in (x, w, b)]

    def loss(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return ((d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b) * dy.double()).sum()

    loss(*leaves).backward()
    for have, leaf in zip(got, leaves):
        # (sums of up to D terms in fp32, a few hundred roundings of 2^-24)
        assert float((have.double() - leaf.grad).norm() / leaf.grad.norm()) < 2e-5
        step = torch.randn(leaf.shape, generator=g, device="cuda").double()
        h = 1e-5
        args = [t.detach() for t in leaves]
        i = next(k for k, t in enumerate(leaves) if t is leaf)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * step, args[i] - h * step
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # (h^2 times a third derivative, and cancellation of 2^-53 |loss| / h)
        assert float((diff - (have.double() * step).sum()).abs()) < 2e-5 * float(leaf.grad.norm() * step.norm())


def test_capture_and_streams():
    x = torch.randn(300, 1000, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(300, 1000, device="cuda", dtype=torch.bfloat16)
    want = ef.layer_norm(x)
    wantg = ef.layer_norm_grad(dy, x, want[1], want[2])
    out, mean, rstd = (torch.empty_like(t) for t in want)
    gx, gw, gb = (torch.empty_like(t) for t in wantg)
    ws = torch.empty(ef.layer_norm_grad_workspace_bytes(300, 1000), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ef.layer_norm(x, out=out, mean=mean, rstd=rstd)
        ef.layer_norm_grad(dy, x, mean, rstd, grad_x=gx, grad_weight=gw, grad_bias=gb, ws=ws)
    for _ in range(3):
        for t in (out, mean, rstd, gx, gw, gb):
            t.fill_(3.0)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip((out, mean, rstd, gx, gw, gb), want + wantg))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = ef.layer_norm(x, stream=s)
    gg = ef.layer_norm_grad(dy, x, got[1], got[2], stream=s)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got + gg, want + wantg))


def test_rows_past_2_31_elements():
    T, D = 70_000, 32_768
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    for r in range(0, T, 10_000):
        x[r:r + 10_000].normal_()
    at = torch.tensor([0, 65_535, 65_536, 69_999], device="cuda")
    out, mean, rstd = ef.layer_norm(x)
    part = ef.layer_norm(x[at])
    assert all(torch.equal(a[at], b) for a, b in zip((out, mean, rstd), part))
    g, gw, gb = ef.layer_norm_grad(out, x, mean, rstd, grad_x=out)
    part = ef.layer_norm_grad(part[0], x[at], part[1], part[2], affine=False)
    assert torch.equal(g[at], part[0])


def test_binding_refuses():
    x = torch.randn(4, 16, device="cuda")
    _, mean, rstd = ef.layer_norm(x)
    bad = [dict(weight=torch.ones(15, device="cuda")), dict(weight=torch.ones(32, device="cuda")[::2]),
           dict(bias=torch.ones(16)), dict(weight=torch.ones(16, device="cuda", dtype=torch.float64)),
           dict(out=torch.empty(4, 15, device="cuda")), dict(out=torch.empty(5, 16, device="cuda")),
           dict(mean=torch.empty(3, device="cuda")), dict(rstd=torch.empty(4, device="cuda", dtype=torch.float16)),
           dict(out=x, out_dtype=torch.float16)]
    for kw in bad:
        with pytest.raises(ValueError):
            ef.layer_norm(x, **kw)
    with pytest.raises(ef.TopkEfError):
        ef.layer_norm(x, eps=-1.0)
    with pytest.raises(ef.TopkEfError):
        ef.layer_norm(x[:, :0])
    with pytest.raises(ValueError):
        ef.layer_norm(x.t())
    bad = [dict(grad_x=torch.empty(4, 16, device="cuda", dtype=torch.float16)), dict(accumulate=True),
           dict(grad_weight=torch.empty(15, device="cuda")), dict(affine=False, grad_bias=torch.empty(16, device="cuda")),
           dict(ws=torch.empty(1 << 20, dtype=torch.uint8))]
    for kw in bad:
        with pytest.raises(ValueError):
            ef.layer_norm_grad(x, x, mean, rstd, **kw)
    with pytest.raises(ValueError):
        ef.layer_norm_grad(x[:3], x, mean, rstd)
    with pytest.raises(ValueError):
        ef.layer_norm_grad(x, x, None, rstd)
    with pytest.raises(ef.TopkEfError):
        ef.layer_norm_grad(x, x, mean, rstd, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("D", [100, 128, 129, 200, 500, 512, 513, 1000, 1500, 2048, 3001, 4096, 6000, 8191, 8200, 12000, 16383])
@pytest.mark.parametrize("xt,dt", [("bf16", "bf16"), ("f32", "f32"), ("f16", "f32"), ("f32", "bf16")])
def test_more_rows_than_run_at_once(D, xt, dt):
    """Every length class with blocks that walk over several rows, to the last row alone."""
    T = 148 * 3 * max(1, 4096 // D) + 321 if D < 8192 else 500
    x = _strided(T, D, TYPES[xt], D, 0, D, 2.0, 0.5)
    dy = _strided(T, D, TYPES[dt], D, 0, D + 1, 1e-2)
    w = _strided(1, D, torch.float32, D, 0, 1, 0.3, 1.0)[0].contiguous()
    b = _strided(1, D, torch.float32, D, 0, 2)[0].contiguous()
    out, mean, rstd = ef.layer_norm(x, w, b)
    _check_forward(out, mean, rstd, x, w, b, 1e-5)
    _check_gradient(dy, x, mean, rstd, w, ef.layer_norm_grad(dy, x, mean, rstd, w))
    y = x.clone()
    ef.layer_norm(y, w, b, out=y)
    assert torch.equal(y, out)


@pytest.mark.parametrize("off", [1, 2, 4])
@pytest.mark.parametrize("wt", ["f32", "bf16"])
def test_weights_that_start_anywhere(off, wt):
    x = _strided(9, 1024, torch.bfloat16, 1024, 0, 1)
    buf = torch.randn(1024 + 8, device="cuda").to(TYPES[wt])
    w = buf[off:off + 1024]
    out, mean, rstd = ef.layer_norm(x, w, w)
    _check_forward(out, mean, rstd, x, w, w, 1e-5)
    dy = _strided(9, 1024, torch.bfloat16, 1024, 0, 2)
    gw = torch.full((1024 + 8,), 3.0, device="cuda")
    got = ef.layer_norm_grad(dy, x, mean, rstd, w, grad_weight=gw[off:off + 1024])
    _check_gradient(dy, x, mean, rstd, w, got)
    assert (gw[:off] == 3.0).all() and (gw[off + 1024:] == 3.0).all()


def test_one_weight_gradient_alone():
    """The C call writes either sum without the other."""
    x, dy = torch.randn(50, 64, device="cuda"), torch.randn(50, 64, device="cuda")
    _, mean, rstd = ef.layer_norm(x)
    gx, gw, gb = ef.layer_norm_grad(dy, x, mean, rstd)
    ws = torch.empty(ef.layer_norm_grad_workspace_bytes(50, 64), dtype=torch.uint8, device="cuda")
    to, one = torch.empty_like(gx), torch.empty_like(gw)
    st = torch.cuda.current_stream().cuda_stream
    for which, want in ((0, gw), (1, gb)):
        ptrs = [one.data_ptr() if k == which else None for k in range(2)]
        rc = ef.lib().layer_norm_grad(dy.data_ptr(), 0, 64, x.data_ptr(), 0, 64, mean.data_ptr(), rstd.data_ptr(), None, 0,
                                      50, 64, to.data_ptr(), 64, ptrs[0], 0, ptrs[1], 0, 0, ws.data_ptr(), ws.numel(), st)
        assert rc == 0 and torch.equal(one, want) and torch.equal(to, gx)


def test_two_calls_at_once():
    xs = [torch.randn(3000, 1024, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    dys = [torch.randn(3000, 1024, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    want = []
    for x, dy in zip(xs, dys):
        y = ef.layer_norm(x)
        want.append((*y, *ef.layer_norm_grad(dy, x, y[1], y[2])))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, x, dy in zip(streams, xs, dys):
            y = ef.layer_norm(x, stream=s)
            got.append((*y, *ef.layer_norm_grad(dy, x, y[1], y[2], stream=s)))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g, v in zip(got, want) for p, q in zip(g, v))
