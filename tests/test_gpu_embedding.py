"""embedding_lookup, embedding_grad and embedding_grad_rows on the GPU.

The lookup is one fp32 product and one rounding: bit-exact against torch.
The sums are compared with 64-bit sums element by element.  n fp32 adds in
any order, the product with the scale and (accumulate) the add to the old
value are off by at most (n + 2) 2^-24 of the sum of the magnitudes (to first
order; one more term covers the rest), and the output's rounding by half a
step of the result (and half the smallest subnormal)."""
import numpy as np
import pytest
import torch

import error_feedback_b200 as ef

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _strided(rows, cols, dtype, ld, offset, seed, scale=1.0):
    """A [rows, cols] view with row stride ld that starts `offset` elements into its buffer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.randn(rows * ld + offset + 8, generator=g, device="cuda").mul_(scale).to(dtype)
    return buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]


def _ids(kind, T, V, seed, dtype=torch.int64):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        a = rng.integers(0, V, T)
    elif kind == "same":
        a = np.full(T, V // 2)
    elif kind == "zipf":
        a = np.minimum(np.floor(np.exp(rng.random(T) * np.log(V + 1.0))).astype(np.int64) - 1, V - 1)
    elif kind == "two":
        a = np.where(rng.random(T) < 0.5, 0, V - 1)
    else:                                    # ascending runs of 40
        a = np.minimum(np.arange(T) // 40, V - 1)
    return torch.from_numpy(a.astype(np.int64)).to(dtype).cuda()


# ------------------------------------------------------------------- lookup

@pytest.mark.parametrize("wt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("ot", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,V,D,ldw,ldo,off", [
    (1, 1, 1, 1, 1, 0), (1, 100, 4096, 4096, 4096, 0), (7, 50, 1001, 1001, 1001, 0),
    (33, 9, 1024, 1032, 1040, 8), (5, 20, 1030, 1032, 1032, 0), (300, 31, 24, 24, 27, 3),
    (9000, 100, 72, 72, 72, 0)])
def test_lookup(wt, ot, T, V, D, ldw, ldo, off):
    w = _strided(V, D, TYPES[wt], ldw, off, 1)
    ids = _ids("uniform", T, V, 2, torch.int32 if T % 2 else torch.int64)
    out = torch.full((T, ldo), 7.0, dtype=TYPES[ot], device="cuda")
    ws = torch.empty(ef.embedding_lookup_workspace_bytes(), dtype=torch.uint8, device="cuda")
    scale = 0.37
    ef.embedding_lookup(w, ids, scale=scale, out=out[:, :D], ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0
    want = (w[ids.long()].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")).to(TYPES[ot])
    assert torch.equal(out[:, :D], want)
    assert (out[:, D:] == 7.0).all()


def test_lookup_shapes_and_defaults():
    w = torch.randn(11, 16, device="cuda")
    ids = torch.randint(0, 11, (3, 5), device="cuda")
    out = ef.embedding_lookup(w, ids)
    assert out.shape == (3, 5, 16) and torch.equal(out, w[ids])
    assert ef.embedding_lookup(w, ids, out_dtype=torch.bfloat16).dtype == torch.bfloat16
    assert ef.embedding_lookup(w, ids[:0]).shape == (0, 5, 16)
    assert ef.embedding_lookup(w[:, :0], ids).shape == (3, 5, 0)


@pytest.mark.parametrize("T", [5, 9000])
def test_lookup_bad_ids_are_reported_and_contained(T):
    w = torch.randn(10, 40, device="cuda")
    ids = torch.randint(0, 10, (T,), device="cuda")
    ws = torch.empty(ef.embedding_lookup_workspace_bytes(), dtype=torch.uint8, device="cuda")
    ids[1], ids[3], ids[T - 1] = -1, 10, 2**40
    out = ef.embedding_lookup(w, ids, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == ef.ERR_BAD_INPUT
    ok = (ids >= 0) & (ids < 10)
    assert torch.equal(out[ok], w[ids[ok]]) and (out[~ok] == 0).all() and int((~ok).sum()) == 3
    ef.embedding_lookup(w, ids.clamp(0, 9), ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0


def test_lookup_special_values():
    w = torch.tensor([[float("inf"), float("-inf"), float("nan"), -0.0, 1e-40, 3e38]], device="cuda")
    out = ef.embedding_lookup(w, torch.zeros(2, dtype=torch.int32, device="cuda"), scale=2.0)
    want = (w * 2.0).expand(2, 6)
    assert torch.equal(out.isnan(), want.isnan())
    assert torch.equal(out.nan_to_num(1.0).view(torch.int32), want.nan_to_num(1.0).contiguous().view(torch.int32))


# ----------------------------------------------------------------- gradient

def _want(dy, ids, V, scale, pad, old):
    """64-bit gradient and the bound on the fp32 sums' error."""
    d = dy.double().cpu().numpy()
    i = ids.cpu().numpy().astype(np.int64)
    keep = (i != pad) & (i >= 0) & (i < V)
    g = np.zeros((V, d.shape[1]))
    mag = np.zeros_like(g)
    np.add.at(g, i[keep], d[keep])
    np.add.at(mag, i[keep], np.abs(d[keep]))
    n = np.bincount(i[keep], minlength=V)[:, None]
    s = abs(float(np.float32(scale)))
    g *= float(np.float32(scale))
    mag *= s
    touched = n[:, 0] > 0
    if old is not None:
        o = old.double().cpu().numpy()
        g = np.where(touched[:, None], g + o, o)
        mag += np.abs(o)
    err = (n + 3) * 2.0**-24 * mag
    return g, np.where(touched[:, None], err, 0.0), touched


def _check(got, want, err, dtype):
    got = got.double().cpu().numpy()
    eps = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2
    bound = err * (1 + eps) + np.abs(want) * eps + (tiny if dtype != torch.float32 else 0.0)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{got[bad][0]} for {want[bad][0]} (bound {bound[bad][0]})"


def _run_grad(dt, ot, T, V, D, kind, ldd=0, ldo=0, off=0, pad=-1, acc=False, idt=torch.int64, seed=0):
    dy = _strided(max(T, 1), D, TYPES[dt], ldd or D, off, seed + 1, 1e-2)[:T]
    ids = _ids(kind, T, V, seed + 2, idt)
    out = _strided(V, D, TYPES[ot], ldo or D, off, seed + 3)
    old = out.clone()
    around = out.as_strided((V, ldo or D), (ldo or D, 1))[:, D:].clone()
    ws = torch.full((ef.embedding_grad_workspace_bytes(T, V, D),), 0xA5, dtype=torch.uint8, device="cuda")
    ef.embedding_grad(dy, ids, V, scale=1.7, padding_idx=pad, accumulate=acc, out=out, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0
    want, err, touched = _want(dy, ids, V, 1.7, pad, old if acc else None)
    _check(out, want, err, TYPES[ot])
    assert torch.equal(out.as_strided((V, ldo or D), (ldo or D, 1))[:, D:], around)
    if acc:        # rows of absent ids are left bit for bit
        t = torch.from_numpy(touched).cuda()
        assert torch.equal(out[~t], old[~t])
    # the row-sparse form holds the same bits, and a second call gives the same
    rows = torch.full((min(T, V) + 1,), -7, dtype=torch.int32, device="cuda")
    val = torch.full((min(T, V) + 1, D), 5.0, dtype=TYPES[ot], device="cuda")
    _, _, count = ef.embedding_grad_rows(dy, ids, V, scale=1.7, padding_idx=pad, out_rows=rows,
                                         out_val=val, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0
    c = int(count.item())
    assert np.array_equal(rows[:c].cpu().numpy(), np.nonzero(touched)[0])
    assert (rows[c:] == -7).all() and (val[c:] == 5.0).all()
    dense = ef.embedding_grad(dy, ids, V, scale=1.7, padding_idx=pad, out_dtype=TYPES[ot])
    assert torch.equal(dense[rows[:c].long()], val[:c])
    assert torch.equal(dense, ef.embedding_grad(dy, ids, V, scale=1.7, padding_idx=pad, out_dtype=TYPES[ot]))
    if not acc:
        assert torch.equal(dense, out)


@pytest.mark.parametrize("T,V,D,kind", [
    (512, 100, 520, "zipf"), (513, 100, 520, "zipf"), (512, 40, 72, "same"), (511, 2**18, 260, "uniform"),
    (1, 1, 1, "same"), (1, 40000, 8, "uniform"), (2, 3, 7, "same"), (31, 5, 33, "uniform"),
    (33, 1000, 1024, "uniform"), (500, 513, 100, "zipf"), (500, 3, 1001, "uniform"),
    (4096, 511, 64, "zipf"), (4097, 512, 40, "two"), (5000, 300, 1032, "runs"),
    (10000, 1, 16, "same"), (10000, 2**18 + 5, 9, "uniform"), (30011, 5021, 101, "zipf")])
@pytest.mark.parametrize("dt,ot", [("f32", "f32"), ("bf16", "f32"), ("f16", "bf16"), ("bf16", "bf16")])
def test_grad_shapes(T, V, D, kind, dt, ot):
    _run_grad(dt, ot, T, V, D, kind)


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("dt,ot", [("f32", "f32"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("ldd,ldo,off", [(64, 64, 8), (72, 80, 0), (65, 67, 1), (61, 64, 0)])
def test_grad_strides_and_padding(acc, dt, ot, ldd, ldo, off):
    _run_grad(dt, ot, 700, 90, 61, "zipf", ldd, ldo, off, pad=2, acc=acc, idt=torch.int32)


@pytest.mark.parametrize("kind", ["same", "two", "zipf", "uniform"])
def test_grad_long(kind):
    """More than 32 sort tiles, and runs over thousands of sum tiles."""
    _run_grad("f32", "f32", 300_001, 1500, 12, kind, acc=kind == "two", pad=0 if kind == "zipf" else -1)


def test_grad_only_padding_and_empty():
    dy = torch.randn(6, 10, device="cuda")
    ids = torch.full((6,), 4, dtype=torch.int64, device="cuda")
    g = ef.embedding_grad(dy, ids, 9, padding_idx=4)
    assert g.shape == (9, 10) and (g == 0).all()
    rows, val, count = ef.embedding_grad_rows(dy, ids, 9, padding_idx=4)
    assert int(count) == 0
    old = torch.randn(9, 10, device="cuda")
    keep = old.clone()
    ef.embedding_grad(dy, ids, 9, padding_idx=4, accumulate=True, out=old)
    assert torch.equal(old, keep)
    ef.embedding_grad(dy[:0], ids[:0], 9, accumulate=True, out=old)
    assert torch.equal(old, keep)
    ef.embedding_grad(dy[:0], ids[:0], 9, out=old)
    assert (old == 0).all()
    assert int(ef.embedding_grad_rows(dy[:0], ids[:0], 9)[2]) == 0
    # ids outside the table that are the padding id are no error
    ws = torch.empty(ef.embedding_grad_workspace_bytes(6, 9, 10), dtype=torch.uint8, device="cuda")
    g = ef.embedding_grad(dy, torch.full_like(ids, -100), 9, padding_idx=-100, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == 0 and (g == 0).all()


@pytest.mark.parametrize("T", [3, 700, 9000])
def test_empty_table(T):
    """No rows at all: every id is outside."""
    ids, dy = torch.zeros(T, dtype=torch.int64, device="cuda"), torch.ones(T, 8, device="cuda")
    ws = torch.empty(ef.embedding_grad_workspace_bytes(T, 0, 8), dtype=torch.uint8, device="cuda")
    count = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    rows, val, _ = ef.embedding_grad_rows(dy, ids, 0, out_count=count, ws=ws)
    assert int(count) == 0 and rows.numel() == 0
    assert ef.topk_ef_last_device_status(ws) == ef.ERR_BAD_INPUT
    assert ef.embedding_grad(dy, ids, 0).shape == (0, 8)
    assert (ef.embedding_lookup(dy[:0], ids) == 0).all()


@pytest.mark.parametrize("T", [300, 3000, 9000])
def test_offsets_past_32_bits(T):
    """A table of more than 2^31 elements: the last rows, and the first."""
    V, D = 2_200_000, 1024
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.cat([torch.arange(V - T + 5, V), torch.arange(5)]).cuda()
    w[ids] = torch.randn(T, D, device="cuda").bfloat16()
    out = ef.embedding_lookup(w, ids)
    assert torch.equal(out, w[ids])
    w.fill_(1.0)
    ef.embedding_grad(out, ids, V, out=w)
    assert torch.equal(w[ids], out) and float(w[5:V - T + 5].abs().max()) == 0.0
    ef.embedding_grad(out, ids, V, out=w, accumulate=True, scale=-1.0)
    assert float(w[ids].abs().max()) == 0.0


def test_grad_bad_ids_are_reported_and_contained():
    T, V, D = 50, 20, 33
    dy = torch.randn(T, D, device="cuda")
    ids = torch.randint(0, V, (T,), device="cuda")
    ids[0], ids[7], ids[49] = -5, V, 2**33
    ws = torch.empty(ef.embedding_grad_workspace_bytes(T, V, D), dtype=torch.uint8, device="cuda")
    g = ef.embedding_grad(dy, ids, V, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == ef.ERR_BAD_INPUT
    want, err, _ = _want(dy, ids, V, 1.0, -1, None)
    _check(g, want, err, torch.float32)
    rows, val, count = ef.embedding_grad_rows(dy, ids, V, ws=ws)
    assert ef.topk_ef_last_device_status(ws) == ef.ERR_BAD_INPUT
    assert torch.equal(g[rows[:int(count)].long()], val[:int(count)])


def test_grad_nan_and_inf_stay_in_their_rows():
    dy = torch.ones(8, 4, device="cuda")
    dy[2, 1], dy[5, 3] = float("nan"), float("inf")
    ids = torch.tensor([0, 1, 2, 0, 1, 3, 3, 0], device="cuda")
    g = ef.embedding_grad(dy, ids, 5)
    assert g[2, 1].isnan() and g[3, 3].isinf()
    g[2, 1] = g[3, 3] = 0
    assert g.isfinite().all()


def test_grad_matches_differences_of_the_lookup():
    """<dy, lookup(W + h E) - lookup(W - h E)> / 2h == <grad, E>: the lookup is
    linear, so the two agree up to rounding (all values are small integers
    over a power of two: exactly)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, V, D = 300, 40, 24
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    w, e = (torch.randint(-8, 9, (V, D), generator=g, device="cuda").float() for _ in range(2))
    dy = torch.randint(-8, 9, (T, D), generator=g, device="cuda").float()
    up, down = (ef.embedding_lookup(w + s * e, ids, scale=0.5).double() for s in (1.0, -1.0))
    left = ((up - down) / 2 * dy.double()).sum()
    right = (ef.embedding_grad(dy, ids, V, scale=0.5).double() * e.double()).sum()
    assert left == right


# --------------------------------------------------- streams, graphs, device

def test_captured_calls_replay_on_new_inputs():
    T, V, D = 700, 300, 96
    w = torch.randn(V, D, device="cuda")
    ids = _ids("zipf", T, V, 1)
    dy = torch.randn(T, D, device="cuda")
    ws = torch.empty(ef.embedding_grad_workspace_bytes(T, V, D), dtype=torch.uint8, device="cuda")
    lws = torch.empty(ef.embedding_lookup_workspace_bytes(), dtype=torch.uint8, device="cuda")
    out, gw = torch.empty(T, D, device="cuda"), torch.empty(V, D, device="cuda")
    rows = torch.empty(V, dtype=torch.int32, device="cuda")
    val, count = torch.empty(V, D, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")

    def step():
        ef.embedding_lookup(w, ids, out=out, ws=lws)
        ef.embedding_grad(dy, ids, V, out=gw, ws=ws)
        ef.embedding_grad_rows(dy, ids, V, out_rows=rows, out_val=val, out_count=count, ws=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        ids.copy_(_ids("uniform" if k else "same", T, V, 5 + k))
        dy.normal_()
        graph.replay()
        assert torch.equal(out, w[ids])
        want, err, touched = _want(dy, ids, V, 1.0, -1, None)
        _check(gw, want, err, torch.float32)
        c = int(count)
        assert c == touched.sum() and torch.equal(gw[rows[:c].long()], val[:c])
    ids[0] = V
    graph.replay()
    assert ef.topk_ef_last_device_status(lws) == ef.ERR_BAD_INPUT
    ids[0] = 0
    graph.replay()
    assert ef.topk_ef_last_device_status(lws) == 0 and ef.topk_ef_last_device_status(ws) == 0


def test_stream_argument():
    """Outputs and workspace that the call allocates belong to its stream."""
    s = torch.cuda.Stream()
    w = torch.randn(1000, 512, device="cuda")
    ids = torch.randint(0, 1000, (4000,), device="cuda")
    dy = torch.randn(4000, 512, device="cuda")
    torch.cuda.synchronize()
    want = ef.embedding_grad(dy, ids, 1000)
    torch.cuda.synchronize()
    for _ in range(5):
        out = ef.embedding_lookup(w, ids, stream=s)
        g = ef.embedding_grad(dy, ids, 1000, stream=s)
        torch.empty(4000 * 512, device="cuda").fill_(3.0)
        s.synchronize()
        assert torch.equal(out, w[ids]) and torch.equal(g, want)


@pytest.mark.parametrize("bad", [
    lambda w, i, d: ef.embedding_lookup(w.double(), i), lambda w, i, d: ef.embedding_lookup(w.t(), i),
    lambda w, i, d: ef.embedding_lookup(w, i.short()), lambda w, i, d: ef.embedding_lookup(w, i.cpu()),
    lambda w, i, d: ef.embedding_lookup(w, i, out=torch.empty(5, 7, device="cuda")),
    lambda w, i, d: ef.embedding_lookup(w[:1].expand(10, 8), i),
    lambda w, i, d: ef.embedding_grad(d[:3], i, 10), lambda w, i, d: ef.embedding_grad(d, i, 10, accumulate=True),
    lambda w, i, d: ef.embedding_grad(d, i, 10, out=torch.empty(9, 8, device="cuda")),
    lambda w, i, d: ef.embedding_grad(d, i, 10, ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
    lambda w, i, d: ef.embedding_grad(d, i, -1),
    lambda w, i, d: ef.embedding_grad_rows(d, i, 10, out_rows=torch.empty(4, dtype=torch.int32, device="cuda")),
    lambda w, i, d: ef.embedding_grad_rows(d, i, 10, out_count=torch.empty(1, dtype=torch.int64, device="cuda"))])
def test_binding_refuses(bad):
    w, ids = torch.zeros(10, 8, device="cuda"), torch.zeros(5, dtype=torch.int64, device="cuda")
    with pytest.raises((ValueError, ef.TopkEfError)):
        bad(w, ids, torch.zeros(5, 8, device="cuda"))


@pytest.mark.parametrize("T", [600, 5000, 20000])
@pytest.mark.parametrize("dt,ot,ldo", [("bf16", "f32", 1504), ("f32", "bf16", 1501)])
def test_grad_accumulates_over_several_slabs(T, dt, ot, ldo):
    """Added to what is there, by each way to sort, with rows of more columns than
    one block takes."""
    _run_grad(dt, ot, T, 3000, 1500, "zipf", ldo=ldo, acc=True)
