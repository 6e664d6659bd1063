"""The embedding and Muon operators: cases, inputs, plain forms and 64-bit values.

With ``own`` false ``run`` computes the operators with elementary torch
operations in 32 bits; with ``own`` true it calls ``error_feedback_b200``.
Operators ("op" of a case):

* ``lookup``: out[t] = scale * W[id_t]
* ``grad``:   g[v] = (accumulate ? g[v] : 0) + scale * sum of dy[t] over id_t = v
* ``rows``:   the same sums for the distinct ids only: ascending ids, sums, count
* ``muon``:   momentum, then the quintic Newton-Schulz iteration
"""
import math

import torch

own = False

COEF = (3.4445, -4.7750, 2.0315)      # a, b, c of p(x) = a x + b x^3 + c x^5
STEPS = 5
EPS = 1e-7
MU = 0.95

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
IDS = {"i32": torch.int32, "i64": torch.int64}


def listed():
    return [
        # one token of a decoding step: latency
        {"name": "lookup 1 token", "op": "lookup", "T": 1, "V": 32768, "D": 4096,
         "w": "bf16", "out": "bf16", "ids": "i64"},
        # a training micro-batch (4 sequences of 4,096) of a large vocabulary
        {"name": "lookup batch", "op": "lookup", "T": 16384, "V": 131072, "D": 4096,
         "w": "bf16", "out": "bf16", "ids": "i64"},
        # fp32 master weights read into bf16 activations, odd sizes, rows not 16-byte aligned
        {"name": "lookup odd, f32 to bf16", "op": "lookup", "T": 30011, "V": 50021, "D": 1001,
         "w": "f32", "out": "bf16", "ids": "i32"},
        # one short sequence added to a gradient that is there already (micro-batches)
        {"name": "grad short, accumulate", "op": "grad", "T": 500, "V": 32768, "D": 1024,
         "dy": "bf16", "out": "f32", "ids": "i64", "acc": True, "pad": -1},
        # a training batch into the fp32 bucket, the whole table written
        {"name": "grad batch", "op": "grad", "T": 32768, "V": 131072, "D": 4096,
         "dy": "bf16", "out": "f32", "ids": "i64", "acc": False, "pad": -1},
        # fp32 gradients, odd sizes, a padding token among the frequent ones
        {"name": "grad odd, f32", "op": "grad", "T": 30011, "V": 50021, "D": 1001,
         "dy": "f32", "out": "f32", "ids": "i32", "acc": False, "pad": 1},
        # the row-sparse set of one short batch
        {"name": "rows short", "op": "rows", "T": 2048, "V": 50021, "D": 768,
         "dy": "f32", "out": "f32", "ids": "i32", "pad": 0},
        # a long batch whose frequent tokens hold thousands of positions
        {"name": "rows long", "op": "rows", "T": 131072, "V": 131072, "D": 1024,
         "dy": "bf16", "out": "f32", "ids": "i64", "pad": -1},
        # VGG-16's first convolution as a matrix: launches and waits are all of it
        {"name": "muon 64x27", "op": "muon", "B": 1, "m": 64, "n": 27,
         "g": "f32", "out": "f32", "momentum": True},
        # VGG-16's 512-channel convolutions, updates back into the fp32 bucket
        {"name": "muon 3x512x4608", "op": "muon", "B": 3, "m": 512, "n": 4608,
         "g": "f32", "out": "f32", "momentum": True},
        # a fully connected layer, bf16 update
        {"name": "muon 4096x4096", "op": "muon", "B": 1, "m": 4096, "n": 4096,
         "g": "f32", "out": "bf16", "momentum": True},
        # VGG-16's largest layer (tall), bf16 gradient, no momentum
        {"name": "muon 25088x4096", "op": "muon", "B": 1, "m": 25088, "n": 4096,
         "g": "bf16", "out": "bf16", "momentum": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "grad", "rows", "muon", "muon"])
    if op == "muon":
        g = rng.choice(["f32", "bf16"])
        out = rng.choice(["f32", "bf16"])
        while True:
            c = {"op": op, "B": rng.choice([1, 1, 2, 3, 5]), "m": _log(rng, 16, 8192),
                 "n": _log(rng, 16, 8192), "g": g, "out": out, "momentum": rng.random() < 0.5}
            if work(c)["flops"] < 2e12:
                return c
    ids = rng.choice(["i32", "i64"])
    V, T, D = _log(rng, 1000, 200000), _log(rng, 1, 131072), _log(rng, 32, 8192)
    while T * D > 1 << 27 or V * D > 1 << 29:
        T, D, V = max(1, T * 3 // 4), max(32, D * 7 // 8), max(1000, V * 7 // 8)
    if op == "lookup":
        return {"op": op, "T": T, "V": V, "D": D, "ids": ids,
                "w": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"])}
    c = {"op": op, "T": T, "V": V, "D": D, "ids": ids, "dy": rng.choice(["f32", "bf16"]),
         "out": rng.choice(["f32", "bf16"]), "pad": rng.choice([-1, 0, 3])}
    if op == "grad":
        c["acc"] = rng.random() < 0.5
    return c


def _ids(c, gen):
    """Tokens by Zipf's law (the probability of id i falls as 1 / (i + 1)):
    vocabularies are laid out by frequency."""
    u = torch.rand(c["T"], generator=gen, device="cuda", dtype=torch.float64)
    i = torch.exp(u * math.log(c["V"] + 1.0)).floor().long() - 1
    return i.clamp_(0, c["V"] - 1).to(IDS[c["ids"]])


def _matrix(shape, gen, dtype):
    """A gradient's spectrum: 8 strong directions over noise of full rank."""
    B, m, n = shape
    r = min(8, m, n)
    x = torch.randn(B, m, n, generator=gen, device="cuda")
    u = torch.randn(B, m, r, generator=gen, device="cuda")
    v = torch.randn(B, r, n, generator=gen, device="cuda")
    s = 2.0 * torch.rand(B, 1, r, generator=gen, device="cuda")
    return ((x + (u * s) @ v) * 1e-3).to(dtype)


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape, dtype, scale):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale).to(dtype)

    if c["op"] == "muon":
        shape = (c["B"], c["m"], c["n"])
        s = {"case": c, "g": _matrix(shape, gen, TYPES[c["g"]]),
             "out": torch.empty(shape, dtype=TYPES[c["out"]], device="cuda"),
             "scale": 0.2 * math.sqrt(max(c["m"], c["n"])), "momentum": None}
        if c["momentum"]:
            s["momentum"] = _matrix(shape, gen, torch.float32)
        return s
    T, V, D = c["T"], c["V"], c["D"]
    s = {"case": c, "ids": _ids(c, gen), "scale": math.sqrt(D)}
    if c["op"] == "lookup":
        s["w"] = randn(V, D, dtype=TYPES[c["w"]], scale=0.02)
        s["out"] = torch.empty(T, D, dtype=TYPES[c["out"]], device="cuda")
        return s
    s["dy"] = randn(T, D, dtype=TYPES[c["dy"]], scale=1e-2)
    if c["op"] == "grad":
        # accumulate: what the micro-batches before this one left
        s["out"] = (randn(V, D, dtype=TYPES[c["out"]], scale=0.1) if c["acc"]
                    else torch.empty(V, D, dtype=TYPES[c["out"]], device="cuda"))
        return s
    cap = min(T, V)
    # slots past the count are not written
    s["rows"] = torch.full((cap,), -1, dtype=torch.int32, device="cuda")
    s["val"] = torch.zeros(cap, D, dtype=TYPES[c["out"]], device="cuda")
    s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"]](s, c)


# ------------------------------------------------------------- plain forms

def _plain_lookup(s, c):
    s["out"].copy_(s["w"][s["ids"]].float() * s["scale"])
    return s["out"]


def _contributions(s, c):
    x = s["dy"].float() * s["scale"]
    if c["pad"] >= 0:
        x = x * (s["ids"] != c["pad"]).float()[:, None]
    return x


def _plain_grad(s, c):
    x = _contributions(s, c)
    if not c["acc"]:
        g = torch.zeros(c["V"], c["D"], device="cuda")
        g.index_add_(0, s["ids"], x)
        s["out"].copy_(g)
    elif s["out"].dtype == torch.float32:
        s["out"].index_add_(0, s["ids"], x)
    else:
        g = s["out"].float()
        g.index_add_(0, s["ids"], x)
        s["out"].copy_(g)
    return s["out"]


def _plain_rows(s, c):
    x = _contributions(s, c)
    key, order = torch.sort(s["ids"], stable=True)
    keep = key != c["pad"]
    head = keep.clone()
    head[1:] &= key[1:] != key[:-1]
    slot = torch.cumsum(head, 0) - 1
    count = head.sum()
    cap = s["rows"].numel()
    at = torch.arange(cap, device="cuda") < count
    slot = slot.clamp(min=0)
    rows = torch.zeros(cap, dtype=torch.int32, device="cuda")
    rows.index_add_(0, slot, key.int() * head.int())
    val = torch.zeros(cap, c["D"], device="cuda")
    val.index_add_(0, slot, x[order])
    s["rows"].copy_(torch.where(at, rows, s["rows"]))
    s["val"].copy_(torch.where(at[:, None], val, s["val"].float()))
    s["count"].copy_(count.reshape(1))
    return {"rows": s["rows"], "val": s["val"], "count": s["count"]}


def _plain_muon(s, c):
    u = s["g"].float()
    if c["momentum"]:
        s["momentum"].mul_(MU).add_(u)
        u = u + MU * s["momentum"]
    a, b, d = COEF
    x = u / (torch.sqrt((u * u).sum((1, 2), keepdim=True)) + EPS)
    tall = c["m"] > c["n"]
    if tall:
        x = x.mT
    for _ in range(STEPS):
        g = x @ x.mT
        x = a * x + (b * g + d * (g @ g)) @ x
    if tall:
        x = x.mT
    s["out"].copy_(x * s["scale"])
    return {"out": s["out"], "momentum": s["momentum"]}


_plain = {"lookup": _plain_lookup, "grad": _plain_grad, "rows": _plain_rows, "muon": _plain_muon}


# ------------------------------------------------- the framework's operators

def _workspace(s, nbytes):
    """The workspace that a user's program keeps beside its buffers."""
    ws = s.get("ws")
    if ws is None:
        ws = s["ws"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return ws


def _own_lookup(s, c):
    import error_feedback_b200 as ef
    ws = _workspace(s, lambda: ef.embedding_lookup_workspace_bytes())
    return ef.embedding_lookup(s["w"], s["ids"], scale=s["scale"], out=s["out"], ws=ws)


def _own_grad(s, c):
    import error_feedback_b200 as ef
    ws = _workspace(s, lambda: ef.embedding_grad_workspace_bytes(c["T"], c["V"], c["D"]))
    return ef.embedding_grad(s["dy"], s["ids"], c["V"], scale=s["scale"], padding_idx=c["pad"],
                             accumulate=c["acc"], out=s["out"], ws=ws)


def _own_rows(s, c):
    import error_feedback_b200 as ef
    ws = _workspace(s, lambda: ef.embedding_grad_workspace_bytes(c["T"], c["V"], c["D"]))
    ef.embedding_grad_rows(s["dy"], s["ids"], c["V"], scale=s["scale"], padding_idx=c["pad"],
                           out_rows=s["rows"], out_val=s["val"], out_count=s["count"], ws=ws)
    return {"rows": s["rows"], "val": s["val"], "count": s["count"]}


def _own_muon(s, c):
    import error_feedback_b200 as ef
    ws = _workspace(s, lambda: ef.muon_workspace_bytes(c["B"], c["m"], c["n"], TYPES[c["out"]]))
    ef.muon_update(s["g"], momentum=s["momentum"], mu=MU, nesterov=True, coefficients=COEF,
                   steps=STEPS, eps=EPS, scale=s["scale"], out=s["out"], ws=ws)
    return {"out": s["out"], "momentum": s["momentum"]}


_own = {"lookup": _own_lookup, "grad": _own_grad, "rows": _own_rows, "muon": _own_muon}


# --------------------------------------------------------------------- work

def _distinct(c):
    """Expected number of distinct tokens of T draws by Zipf's law."""
    h = math.log(c["V"] + 1.0)
    n, lo = 0.0, 1.0
    while lo < c["V"] + 1:
        hi = min(lo * 1.25 + 1, c["V"] + 1.0)
        k = hi - lo
        p = math.log(hi / lo) / h / k
        n += k * -math.expm1(c["T"] * math.log1p(-min(p, 0.999999)))
        lo = hi
    return min(n, c["T"], c["V"])


def work(c):
    size = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}
    if c["op"] == "muon":
        e = c["B"] * c["m"] * c["n"]
        p, q = min(c["m"], c["n"]), max(c["m"], c["n"])
        nbytes = e * (size[c["g"]] + size[c["out"]] + (8 if c["momentum"] else 0))
        # the two symmetric products by half
        return {"bytes": nbytes, "flops": c["B"] * STEPS * (p * p * q + p ** 3 + 2 * p * p * q)}
    T, V, D = c["T"], c["V"], c["D"]
    u = _distinct(c)
    if c["op"] == "lookup":
        return {"bytes": T * size[c["ids"]] + u * D * size[c["w"]] + T * D * size[c["out"]],
                "flops": T * D}
    nbytes = T * (D * size[c["dy"]] + size[c["ids"]])
    if c["op"] == "rows":
        nbytes += u * (D * size[c["out"]] + 4)
    else:
        nbytes += (2 * u if c["acc"] else V) * D * size[c["out"]]
    return {"bytes": nbytes, "flops": T * D}


# -------------------------------------------------------------- 64-bit values

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "lookup":
        return torch.index_select(s["w"], 0, s["ids"].long()).double() * s["scale"]
    if c["op"] == "muon":
        return _exact_muon(s, c)
    # sums over runs of equal sorted ids, as differences of running sums by column slabs
    ids = s["ids"].long()
    order = torch.argsort(ids, stable=True)
    order = order[ids[order] != c["pad"]]
    row, length = torch.unique_consecutive(ids[order], return_counts=True)
    end = torch.cumsum(length, 0)
    base = (s["out"].double() if c.get("acc") else
            torch.zeros(c["V"], c["D"], dtype=torch.float64, device="cuda")) if c["op"] == "grad" \
        else s["val"].double()
    for lo in range(0, c["D"], 512):
        run_sum = torch.cumsum(s["dy"][order, lo:lo + 512].double(), 0)
        run_sum = torch.cat([torch.zeros_like(run_sum[:1]), run_sum])
        part = (run_sum[end] - run_sum[end - length]) * s["scale"]
        if c["op"] == "grad":
            base[row, lo:lo + 512] += part
        else:
            base[:row.numel(), lo:lo + 512] = part
    if c["op"] == "grad":
        return base
    rows = s["rows"].clone()
    rows[:row.numel()] = row.int()
    return {"rows": rows, "val": base,
            "count": torch.tensor([row.numel()], dtype=torch.int32, device="cuda")}


def _exact_muon(s, c):
    u, mom = s["g"].double(), None
    if c["momentum"]:
        mom = s["momentum"].double() * MU + u
        u = u + MU * mom
    # the polynomial of each matrix by Horner's rule, on its shorter side
    a, b, d = COEF
    out = []
    for x in u:
        x = x / (torch.linalg.norm(x) + EPS)
        left = x.shape[0] <= x.shape[1]
        k = min(x.shape)
        eye = torch.eye(k, dtype=torch.float64, device="cuda")
        for _ in range(STEPS):
            g = torch.matmul(x, x.T) if left else torch.matmul(x.T, x)
            q = a * eye + torch.matmul(g, b * eye + d * g)
            x = torch.matmul(q, x) if left else torch.matmul(x, q)
        out.append(x * s["scale"])
    return {"out": torch.stack(out), "momentum": mom}
