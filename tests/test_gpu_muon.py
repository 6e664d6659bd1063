"""muon_update on the GPU against the same iteration in 64 bits.

Tolerances (2-norm of the difference over the 2-norm of the result):
 * fp32 output: "as exact as plain fp32 products": four times the error that
   the iteration with fp32 matrix products has on the same input, plus the
   2^-22 to which a pair of fp16 values holds an operand.
 * 16-bit output: a 64-bit model of the documented roundings (X, A and B to
   fp16 where a product reads them, a X from hi + lo) gives the error that they
   make on the same input; roundings at other values fall differently, so
   twice that, plus half a step of the output's rounding."""
import math

import pytest
import torch

import error_feedback_b200 as ef

pytestmark = pytest.mark.gpu

COEF = (3.4445, -4.7750, 2.0315)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _iterate(u, coefs, eps, dtype, quant=None):
    """The iteration of one matrix in `dtype`; quant(t, scale): the rounding
    of what a product reads."""
    quant = quant or (lambda t, s: t)
    u = u.to(dtype)
    x = u / (torch.sqrt((u.double() ** 2).sum()).to(dtype) + eps)
    s = 2.0 ** min(13, math.ceil(0.5 * math.log2(u.numel())))
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for a, b, c in coefs:
        xq = quant(x, s)
        g = quant(xq @ xq.T, 2048.0)
        x = a * x + quant(b * g + c * (g @ g), 2048.0) @ xq
    return x.T if tall else x


def _fp16(t, s):
    return (t * s).to(torch.float16).to(t.dtype) / s


def _rel(x, y):
    n = torch.linalg.norm(y.double())
    d = torch.linalg.norm(x.double() - y.double())
    return float(d / n) if n > 0 else float(d)


def _tolerance(u, coefs, eps, out):
    want = _iterate(u, coefs, eps, torch.float64)
    if out == torch.float32:
        return want, 4 * _rel(_iterate(u, coefs, eps, torch.float32), want) + 2.0**-22
    model = _rel(_iterate(u, coefs, eps, torch.float64, _fp16), want)
    return want, 2 * model + torch.finfo(out).eps / 2


def _make(shape, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, m, n = shape
    x = torch.randn(B, m, n, generator=g, device="cuda")
    if kind == "strong":
        x += 3 * torch.randn(B, m, 1, generator=g, device="cuda") @ torch.randn(B, 1, n, generator=g, device="cuda")
    elif kind == "rank1":
        x = torch.randn(B, m, 1, generator=g, device="cuda") @ torch.randn(B, 1, n, generator=g, device="cuda")
    elif kind == "ones":
        x = torch.ones(B, m, n, device="cuda")
    return x * 1e-3


SHAPES = [(1, 1, 1), (1, 1, 1000), (1, 1000, 1), (1, 64, 27), (1, 27, 64), (1, 128, 256),
          (2, 129, 257), (3, 257, 129), (5, 16, 16), (1, 512, 700), (2, 700, 512), (1, 65, 2049),
          (1, 300, 300), (40, 130, 70), (1, 1030, 1100), (3, 256, 128), (1, 129, 128), (1, 128, 257),
          (200, 40, 33), (2, 65, 255), (1, 100, 2000), (2, 1999, 100), (2, 17, 1025), (1, 128, 2048),
          (3, 2048, 128), (1, 90, 513), (60, 50, 700), (1, 128, 2049), (2, 20, 4096),
          (1, 3000, 128), (9, 40, 2100), (1, 100, 4097)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("gt,ot", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "f16"),
                                   ("bf16", "f32")])
def test_shapes(shape, gt, ot):
    x = _make(shape, "strong", sum(shape)).to(TYPES[gt])
    ws = torch.full((ef.muon_workspace_bytes(*shape, TYPES[ot]),), 0x7F, dtype=torch.uint8, device="cuda")
    out = ef.muon_update(x, out_dtype=TYPES[ot], scale=0.3, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0
    for b in range(shape[0]):
        want, tol = _tolerance(x[b], [COEF] * 5, 1e-7, TYPES[ot])
        r = _rel(out[b], 0.3 * want)
        assert r <= tol, f"matrix {b}: {r} > {tol}"
    assert torch.equal(out, ef.muon_update(x, out_dtype=TYPES[ot], scale=0.3))


@pytest.mark.parametrize("kind", ["plain", "rank1", "ones"])
@pytest.mark.parametrize("ot", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 300, 400), (1, 513, 257)])
def test_spectra(kind, ot, shape):
    x = _make(shape, kind, 5)
    want, tol = _tolerance(x[0], [COEF] * 5, 1e-7, TYPES[ot])
    assert _rel(ef.muon_update(x, out_dtype=TYPES[ot])[0], want) <= tol


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("gt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 40, 100), (2, 77, 33), (2, 30, 1500), (1, 900, 77), (1, 200, 300)])
def test_momentum(nesterov, gt, shape):
    mom = _make(shape, "strong", 1)
    mu = 0.9
    for step in range(2):
        g = _make(shape, "strong", 2 + step).to(TYPES[gt])
        # fp32: one rounding of the product and the sum
        want_m = (mom.double() * float(torch.tensor(mu, dtype=torch.float32)) + g.double())
        out = ef.muon_update(g, momentum=mom, mu=mu, nesterov=nesterov)
        assert torch.equal(mom, want_m.float())
        u = (mom.double() * float(torch.tensor(mu, dtype=torch.float32)) + g.double()).float() \
            if nesterov else mom
        for b in range(shape[0]):
            want, tol = _tolerance(u[b], [COEF] * 5, 1e-7, torch.float32)
            assert _rel(out[b], want) <= tol


@pytest.mark.parametrize("steps", [1, 2, 9])
@pytest.mark.parametrize("ot", ["f32", "bf16"])
def test_steps_and_coefficients(steps, ot):
    x = _make((1, 150, 90), "strong", 8)
    each = [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (15 / 8, -10 / 8, 3 / 8)]
    coefs = [each[i % 3] for i in range(steps)]
    out = ef.muon_update(x, coefficients=coefs, steps=steps, out_dtype=TYPES[ot])
    want, tol = _tolerance(x[0], [tuple(float(torch.tensor(v)) for v in c) for c in coefs], 1e-7, TYPES[ot])
    assert _rel(out[0], want) <= tol


def test_result_is_orthogonal():
    """The cubic iteration converges: all singular values near 1."""
    x = _make((1, 60, 200), "plain", 4)
    out = ef.muon_update(x, coefficients=(1.5, -0.5, 0.0), steps=20)[0].double()
    s = torch.linalg.svdvals(out)
    assert float((s - 1).abs().max()) < 1e-5


@pytest.mark.parametrize("gt,ot", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("B,m,n,ldg,ldo,off", [(1, 50, 70, 72, 80, 8), (2, 70, 50, 51, 53, 1),
                                               (3, 33, 64, 64, 64, 4), (2, 700, 90, 91, 93, 1),
                                               (2, 90, 700, 704, 703, 3), (1, 300, 310, 312, 311, 1), (1, 1500, 1301, 1304, 1303, 1),
                                               (1, 1300, 1500, 1500, 1501, 0), (1, 1100, 1288, 1288, 1296, 8)])
def test_strides(gt, ot, B, m, n, ldg, ldo, off):
    g = torch.Generator(device="cuda").manual_seed(1)
    sg, so = m * ldg + 16, m * ldo + 24
    buf = torch.randn(off + B * sg, generator=g, device="cuda").to(TYPES[gt])
    x = buf[off:].as_strided((B, m, n), (sg, ldg, 1), off)
    obuf = torch.full((off + B * so,), 7.0, dtype=TYPES[ot], device="cuda")
    out = obuf.as_strided((B, m, n), (so, ldo, 1), off)
    ef.muon_update(x, out=out)
    assert torch.equal(out, ef.muon_update(x.contiguous(), out_dtype=TYPES[ot]))
    out.fill_(7.0)
    assert (obuf == 7.0).all()


@pytest.mark.parametrize("shape", [(40, 60), (50, 900), (900, 50), (300, 200)])
def test_out_may_be_grad_in_another_type(shape):
    """One matrix: the same memory, rows at the same place, half the bytes."""
    x = torch.randn(*shape, device="cuda")
    want = ef.muon_update(x.clone(), out_dtype=torch.bfloat16)
    out = x.view(torch.bfloat16)[:, :shape[1]]
    assert torch.equal(ef.muon_update(x, out=out), want)


def test_out_may_be_grad_and_part_of_a_bucket():
    bucket = torch.randn(10_000, device="cuda")
    keep = bucket.clone()
    x = bucket[1000:1000 + 40 * 60].view(40, 60)
    want = ef.muon_update(x.clone())
    assert ef.muon_update(x, out=x) is x
    assert torch.equal(x, want)
    assert torch.equal(bucket[:1000], keep[:1000]) and torch.equal(bucket[3400:], keep[3400:])


@pytest.mark.parametrize("ot", ["f32", "bf16"])
@pytest.mark.parametrize("n", [50, 600, 2500])
def test_zero_tiny_huge_nan(ot, n):
    """Each matrix of the batch on its own: zeros stay zero, a tiny one is held
    by eps, a huge one (whose squares pass fp32's range) is normalised, NaN and
    infinity stay in theirs."""
    x = _make((6, 40, n), "strong", 3)
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e25
    x[3, 5, 7] = float("nan")
    x[4, 5, 7] = float("inf")
    out = ef.muon_update(x, out_dtype=TYPES[ot])
    assert (out[0] == 0).all() and out[3].isnan().all() and out[4].isnan().any()
    for b in (1, 2, 5):
        # (the small one only scaled: 64 bits hold the squares of both)
        want, tol = _tolerance(x[b].double() if b == 2 else x[b], [COEF] * 5, 1e-7, TYPES[ot])
        if b == 2:
            tol = _tolerance(x[5], [COEF] * 5, 1e-7, TYPES[ot])[1]
        if b == 1:
            tol = max(tol, 2.0**-8)
        assert _rel(out[b], want) <= tol


def test_empty():
    for shape in ((0, 5, 5), (2, 0, 5), (2, 5, 0)):
        assert ef.muon_update(torch.zeros(shape, device="cuda")).shape == shape


def test_captured_call_replays_on_new_inputs():
    shape = (2, 90, 130)
    g, mom = _make(shape, "strong", 1), torch.zeros(shape, device="cuda")
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ef.muon_workspace_bytes(*shape, torch.bfloat16), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ef.muon_update(g, momentum=mom, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ef.muon_update(g, momentum=mom, out=out, ws=ws)
    for k in range(3):
        g.copy_(_make(shape, "plain", 10 + k))
        m2 = mom.clone()
        graph.replay()
        want = ef.muon_update(g, momentum=m2, out_dtype=torch.bfloat16)
        assert torch.equal(out, want) and torch.equal(mom, m2)
    assert ef.topk_ef_last_device_status(ws) == 0


def test_two_streams_at_once():
    x = [_make((1, 300, 500), "strong", k) for k in range(2)]
    want = [ef.muon_update(t) for t in x]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [ef.muon_update(t, stream=q) for t, q in zip(x, s)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("bad", [
    lambda x: ef.muon_update(x.double()), lambda x: ef.muon_update(x.t()), lambda x: ef.muon_update(x[0]),
    lambda x: ef.muon_update(x, momentum=x.bfloat16()), lambda x: ef.muon_update(x, momentum=x[:2]),
    lambda x: ef.muon_update(x, out=x[:2]), lambda x: ef.muon_update(x, steps=0),
    lambda x: ef.muon_update(x, coefficients=(9.0, 0.0, 0.0)), lambda x: ef.muon_update(x, eps=-1.0),
    lambda x: ef.muon_update(x[:1].expand(4, 6)),
    lambda x: ef.muon_update(x, ws=torch.empty(300, dtype=torch.uint8, device="cuda"))])
def test_binding_refuses(bad):
    with pytest.raises((ValueError, ef.TopkEfError)):
        bad(torch.zeros(4, 6, device="cuda"))


def _pair(t, s):
    """What a pair of fp16 values (hi, and the rest times 2^11) holds of t."""
    y = t.double() * s
    hi = y.to(torch.float16).double()
    lo = ((y - hi) * 2048).to(torch.float16).double() / 2048
    return ((hi + lo) / s).to(t.dtype)


def _worst(x, y, dim):
    """The largest relative error of a row (dim 1) or column (dim 0)."""
    n = torch.linalg.norm(y.double(), dim=dim)
    return float((torch.linalg.norm(x.double() - y.double(), dim=dim) / n).max())


@pytest.mark.parametrize("kind", ["one large row", "graded rows", "graded columns"])
@pytest.mark.parametrize("m,n", [(64, 64), (100, 1500), (300, 1500), (1500, 300), (1100, 1280),
                                 (2100, 2304), (2304, 2100)])
def test_rows_of_different_size(kind, m, n):
    """fp32 output, row by row and column by column: small rows keep their bits.
    Allowed: four times the error of plain fp32 products, twice that of a 64-bit
    model in which X, A and B are held as pairs, and 2^-22 for the operands of
    the last product."""
    x = _make((1, m, n), "plain", m + n)[0]
    if kind == "one large row":
        x[1:] *= 1e-5
    elif kind == "graded rows":
        x *= torch.logspace(0, -6, m, device="cuda")[:, None]
    else:
        x *= torch.logspace(0, -6, n, device="cuda")
    want = _iterate(x, [COEF] * 5, 1e-7, torch.float64)
    plain = _iterate(x, [COEF] * 5, 1e-7, torch.float32)
    model = _iterate(x, [COEF] * 5, 1e-7, torch.float64, _pair)
    out = ef.muon_update(x)
    for dim in (0, 1):
        tol = 4 * _worst(plain, want, dim) + 2 * _worst(model, want, dim) + 2.0**-22
        assert _worst(out, want, dim) <= tol


@pytest.mark.parametrize("kind", ["plain", "strong", "ones"])
@pytest.mark.parametrize("m,n", [(300, 300), (512, 700), (1500, 200), (1100, 1300)])
def test_fp16_output_is_rounded_once(kind, m, n):
    """Off by half a step of fp16 (and half its smallest subnormal), besides what
    fp32 output may be off by."""
    x = _make((1, m, n), kind, m + n)[0]
    want, tol = _tolerance(x, [COEF] * 5, 1e-7, torch.float32)
    out = ef.muon_update(x, out_dtype=torch.float16)
    small = 2.0**-25 * math.sqrt(m * n) / float(torch.linalg.norm(want))
    assert _rel(out, want) <= tol + torch.finfo(torch.float16).eps / 2 + small


# Shapes by the kernels that take them: pairs' 256 x 256 tiles, whole and halved, in
# one and in several rounds; one tile with a long K; tiles of 64 columns.
LARGE = [(1, 2300, 2600), (1, 2600, 2300), (1, 3000, 3100), (3, 1100, 1200), (2, 1664, 1600)]
LONG = [(1, 128, 24640), (1, 28672, 100), (1, 1, 30000), (1, 300, 30000), (1, 1200, 8000), (1, 8000, 1200),
        (1, 1500, 4000), (2, 60, 60000)]
NARROW = [(1, 64, 5000), (2, 5000, 50), (1, 32, 6001)]


@pytest.mark.parametrize("shape", LARGE + LONG + NARROW)
@pytest.mark.parametrize("gt,ot", [("f32", "f32"), ("bf16", "bf16"), ("f32", "f16")])
def test_shapes_by_kernel(shape, gt, ot):
    x = _make(shape, "strong", sum(shape)).to(TYPES[gt])
    ws = torch.full((ef.muon_workspace_bytes(*shape, TYPES[ot]),), 0x7F, dtype=torch.uint8, device="cuda")
    out = ef.muon_update(x, out_dtype=TYPES[ot], ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0
    for b in range(shape[0]):
        want, tol = _tolerance(x[b], [COEF] * 5, 1e-7, TYPES[ot])
        assert _rel(out[b], want) <= tol
    assert torch.equal(out, ef.muon_update(x, out_dtype=TYPES[ot]))


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("gt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 200, 320), (2, 320, 192), (2, 1100, 1280), (1, 100, 4224)])
def test_momentum_of_whole_rows_of_64(nesterov, gt, shape):
    """Contiguous matrices whose rows are multiples of 64 take a path of their own."""
    mom = _make(shape, "strong", 1)
    mu = float(torch.tensor(0.9, dtype=torch.float32))
    for step in range(2):
        g = _make(shape, "strong", 2 + step).to(TYPES[gt])
        want_m = (mom.double() * mu + g.double()).float()
        out = ef.muon_update(g, momentum=mom, mu=0.9, nesterov=nesterov)
        assert torch.equal(mom, want_m)
        u = (mom.double() * mu + g.double()).float() if nesterov else mom
        for b in range(shape[0]):
            want, tol = _tolerance(u[b], [COEF] * 5, 1e-7, torch.float32)
            assert _rel(out[b], want) <= tol


@pytest.mark.parametrize("steps", [1, 2, 9])
@pytest.mark.parametrize("m,n,ot", [(200, 300, "f32"), (300, 200, "bf16"), (1100, 1280, "bf16"),
                                    (1280, 1100, "bf16"), (1664, 1600, "f32")])
def test_steps_and_coefficients_by_kernel(steps, m, n, ot):
    x = _make((1, m, n), "strong", 8)
    each = [(1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (15 / 8, -10 / 8, 3 / 8)]
    coefs = [each[i % 3] for i in range(steps)]
    out = ef.muon_update(x, coefficients=coefs, steps=steps, out_dtype=TYPES[ot])
    want, tol = _tolerance(x[0], [tuple(float(torch.tensor(v)) for v in c) for c in coefs], 1e-7, TYPES[ot])
    assert _rel(out[0], want) <= tol


@pytest.mark.parametrize("m,n,ot", [(100, 90, "f32"), (200, 300, "f32"), (300, 200, "bf16"), (128, 4200, "f32"),
                                    (320, 192, "f32"), (1100, 1280, "bf16"), (1664, 1600, "f32")])
def test_zero_tiny_huge_nan_by_kernel(m, n, ot):
    """As test_zero_tiny_huge_nan, with a matrix whose norm is near fp32's end.  The
    tiny one's products vanish beside a X: five steps that each round a pair
    (2^-22) and an fp32 product and sum (2^-23), and the scaling at both ends."""
    x = _make((7, m, n), "strong", 3)
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e25
    x[3, 5, 7] = float("nan")
    x[4, 5, 7] = float("inf")
    x[6] = x[6] / x[6].abs().max() * 1e38
    out = ef.muon_update(x, out_dtype=TYPES[ot])
    assert (out[0] == 0).all() and out[3].isnan().all() and out[4].isnan().any()
    tol = _tolerance(x[5], [COEF] * 5, 1e-7, TYPES[ot])[1]
    for b in (2, 5, 6):
        assert _rel(out[b], _iterate(x[b].double(), [COEF] * 5, 1e-7, torch.float64)) <= tol
    tiny = 5 * (2.0**-22 + 2.0**-23) + 2 * 2.0**-22 + (0 if ot == "f32" else torch.finfo(TYPES[ot]).eps / 2)
    assert _rel(out[1], _iterate(x[1].double(), [COEF] * 5, 1e-7, torch.float64)) <= tiny


@pytest.mark.parametrize("m,n", [(60, 70), (200, 300), (320, 192)])
def test_norm_near_the_smallest_values(m, n):
    """eps = 0: the factor that brings X to its scale is no fp32 value."""
    x = _make((1, m, n), "strong", 4)[0] * 1e-34
    want, tol = _tolerance(x.double(), [COEF] * 5, 0.0, torch.float32)
    tol = _tolerance(_make((1, m, n), "strong", 4)[0], [COEF] * 5, 0.0, torch.float32)[1]
    assert _rel(ef.muon_update(x, eps=0.0), want) <= tol


@pytest.mark.parametrize("shape,ot", [((1, 200, 300), "f32"), ((1, 1100, 1280), "bf16"), ((1, 1664, 1600), "f32")])
def test_captured_call_replays_by_kernel(shape, ot):
    g, mom = _make(shape, "strong", 1), torch.zeros(shape, device="cuda")
    out = torch.empty(shape, dtype=TYPES[ot], device="cuda")
    ws = torch.empty(ef.muon_workspace_bytes(*shape, TYPES[ot]), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ef.muon_update(g, momentum=mom, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ef.muon_update(g, momentum=mom, out=out, ws=ws)
    for k in range(3):
        g.copy_(_make(shape, "plain", 10 + k))
        m2 = mom.clone()
        graph.replay()
        want = ef.muon_update(g, momentum=m2, out_dtype=TYPES[ot])
        assert torch.equal(out, want) and torch.equal(mom, m2)
    assert ef.topk_ef_last_device_status(ws) == 0


@pytest.mark.parametrize("shape,ot", [((1, 1100, 1280), "bf16"), ((1, 1664, 1600), "f32"), ((30, 100, 600), "f32")])
def test_two_streams_at_once_by_kernel(shape, ot):
    x = [_make(shape, "strong", k) for k in range(2)]
    want = [ef.muon_update(t, out_dtype=TYPES[ot]) for t in x]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [ef.muon_update(t, out_dtype=TYPES[ot], stream=q) for t, q in zip(x, s)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
