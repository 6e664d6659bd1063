"""Layer norm, token log-probabilities and distillation: cases, inputs, plain forms, 64-bit values.

With ``own`` false ``run`` computes the operators with elementary torch
operations in 32 bits; with ``own`` true it calls ``error_feedback_b200``.
Operators ("op" of a case):

* ``norm``:      y = (x - mean) * rstd * w + b over each row, with mean and rstd
* ``norm_grad``: dx, and dw and db summed over the rows (added to what is there)
* ``logp``:      of each row of logits z and a token id: log softmax(scale z)[id],
  the entropy, the log of the sum, and the `top` largest logits (ids, log-probabilities;
  ties to the lowest id)
* ``logp_grad``: the gradient of the log-probabilities and entropies in the logits
* ``distill``:   weight * KL(softmax(scale teacher) || softmax(scale z)) where the
  teacher is a list of K ids and logits per row, and with ``grad`` its gradient in z
"""
import math

import torch

own = False

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one token of a decoding step: latency
        {"name": "norm 1 token", "op": "norm", "T": 1, "D": 4096, "x": "bf16", "out": "bf16",
         "w": "bf16"},
        # a training micro-batch (4 sequences of 4,096)
        {"name": "norm batch", "op": "norm", "T": 16384, "D": 4096, "x": "bf16", "out": "bf16",
         "w": "bf16"},
        # fp32 residual stream into bf16 activations, odd sizes, rows not 16-byte aligned
        {"name": "norm odd, f32 to bf16", "op": "norm", "T": 30011, "D": 1001, "x": "f32",
         "out": "bf16", "w": "f32"},
        # one short sequence whose weight gradients join those of earlier micro-batches
        {"name": "norm grad short, accumulate", "op": "norm_grad", "T": 500, "D": 1024,
         "x": "bf16", "w": "f32", "acc": True},
        # a training batch, weight gradients into the fp32 bucket
        {"name": "norm grad batch", "op": "norm_grad", "T": 32768, "D": 4096, "x": "bf16",
         "w": "bf16", "acc": False},
        # one token of a decoding step with 20 alternatives, fp32 logits
        {"name": "logp 1 token, top 20", "op": "logp", "T": 1, "V": 131072, "z": "f32", "top": 20,
         "mask": False, "pad": 0.0},
        # a teacher's pass over a batch: the 64 alternatives that a student learns from
        {"name": "logp batch, top 64", "op": "logp", "T": 4096, "V": 131072, "z": "bf16",
         "top": 64, "mask": False, "pad": 0.0},
        # odd sizes, forbidden tokens at -inf, padded positions
        {"name": "logp odd, masked", "op": "logp", "T": 1111, "V": 50021, "z": "f32", "top": 5,
         "mask": True, "pad": 0.1},
        # the loss of next tokens with an entropy term, backward
        {"name": "logp grad batch", "op": "logp_grad", "T": 2048, "V": 131072, "z": "bf16",
         "mask": False, "pad": 0.05, "entropy": True},
        # a short prompt's distillation loss alone (evaluation)
        {"name": "distill loss short", "op": "distill", "T": 64, "V": 32768, "z": "bf16", "K": 32,
         "pad": 0.0, "grad": False},
        # a distillation step: loss and gradient
        {"name": "distill batch", "op": "distill", "T": 2048, "V": 131072, "z": "bf16", "K": 64,
         "pad": 0.05, "grad": True},
        # odd sizes in fp32, a third of the positions padding
        {"name": "distill odd", "op": "distill", "T": 701, "V": 50021, "z": "f32", "K": 20,
         "pad": 0.33, "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "logp", "logp", "logp_grad", "distill", "distill"])
    kind = rng.choice(["f32", "bf16"])
    if op.startswith("norm"):
        T, D = _log(rng, 1, 131072), _log(rng, 32, 16384)
        if rng.random() < 0.6:          # most models' widths are multiples of 64
            D = max(64, D // 64 * 64)
        while T * D * SIZE[kind] > 1 << 27:
            T = max(1, T * 3 // 4)
        c = {"op": op, "T": T, "D": D, "x": kind, "w": rng.choice(["f32", "bf16"])}
        if op == "norm":
            c["out"] = rng.choice(["f32", "bf16"])
        else:
            c["acc"] = rng.random() < 0.5
        return c
    T, V = _log(rng, 1, 16384), _log(rng, 1000, 262144)
    if rng.random() < 0.5:
        V = V // 64 * 64
    while T * V * SIZE[kind] > 1 << 29:
        T = max(1, T * 3 // 4)
    c = {"op": op, "T": T, "V": V, "z": kind, "pad": rng.choice([0.0, 0.1, 0.4])}
    if op == "distill":
        c["K"], c["grad"] = _log(rng, 1, 128), rng.random() < 0.7
        return c
    c["mask"] = rng.random() < 0.3
    if op == "logp":
        c["top"] = rng.choice([0, 1, 5, _log(rng, 2, 128)])
    else:
        c["entropy"] = rng.random() < 0.5
    return c


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def empty(*shape, dtype=torch.float32):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    s = {"case": c}
    if c["op"].startswith("norm"):
        T, D = c["T"], c["D"]
        # a residual stream: columns of different size and offset
        x = randn(T, D).mul_(0.5 + rand(D)).add_(randn(D) * 0.3)
        s["x"] = x.to(TYPES[c["x"]])
        s["w"] = (1.0 + 0.1 * randn(D)).to(TYPES[c["w"]])
        s["b"] = (0.1 * randn(D)).to(TYPES[c["w"]])
        if c["op"] == "norm":
            s["out"] = empty(T, D, dtype=TYPES[c["out"]])
            s["mean"], s["rstd"] = empty(T), empty(T)
            return s
        # what the forward pass left
        x = s["x"].float()
        mean = x.mean(1)
        s["mean"], s["rstd"] = mean, ((x - mean[:, None]).square().mean(1) + EPS).rsqrt()
        s["dy"] = (randn(T, D) * 1e-2).to(TYPES[c["x"]])
        s["dx"] = empty(T, D, dtype=TYPES[c["x"]])
        s["dw"], s["db"] = (0.1 * randn(D), 0.1 * randn(D)) if c["acc"] else (empty(D), empty(D))
        return s

    T, V = c["T"], c["V"]
    z = randn(T, V).mul_(2.5)
    z += randn(T, 1)
    s["scale"] = 0.5 if c["op"] == "distill" else 1.0        # distillation at temperature 2
    pad = rand(T) < c["pad"]
    if c["op"] == "distill":
        K = min(c["K"], V)
        # the teacher's alternatives, best first, and a student that has learnt some of them
        k = torch.arange(K, device="cuda")
        start = (rand(T) * V).long().clamp_(max=V - 1)
        step = 1 + (rand(T) * (V // K - 1)).long()
        at = (start[:, None] + k * step[:, None]) % V
        s["teacher_ids"] = at.int()
        fall = 2.0 * torch.log1p(k.float())
        s["teacher_logits"] = 12.0 - fall + 0.3 * randn(T, K)
        z.scatter_(1, at, 11.0 - fall + 2.0 * randn(T, K))
        s["z"] = z.to(TYPES[c["z"]])
        s["weight"] = torch.where(pad, 0.0, 4.0 / T)         # the temperature's square, the mean
        s["loss"] = empty(T)
        s["dz"] = empty(T, V, dtype=s["z"].dtype) if c["grad"] else None
        return s
    ids = torch.exp(rand(T).double() * math.log(V + 1.0)).floor().long().sub_(1).clamp_(0, V - 1)
    # half of the tokens are ones that the model expects
    rows = torch.arange(T, device="cuda")
    z[rows, ids] = torch.where(rand(T) < 0.5, 13.0 + randn(T), z[rows, ids])
    if c["mask"]:
        keep = z[rows, ids]
        z.masked_fill_(rand(T, V) < 0.3, -math.inf)
        z[rows, ids] = keep
    s["z"] = z.to(TYPES[c["z"]])
    s["ids"] = torch.where(pad, -1, ids)
    if c["op"] == "logp":
        s["logprob"], s["entropy"], s["lse"] = empty(T), empty(T), empty(T)
        s["top_ids"] = empty(T, c["top"], dtype=torch.int32)
        s["top_logprobs"] = empty(T, c["top"])
        return s
    # what the forward pass left, and the loss's gradient in it
    s["lse"], s["entropy"] = _statistics(s["z"].float(), s["scale"])
    s["d_logprob"] = (-1.0 - 0.2 * rand(T)) / T
    s["d_entropy"] = (-0.01 - 0.01 * rand(T)) / T if c["entropy"] else None
    s["dz"] = empty(T, V, dtype=s["z"].dtype)
    return s


def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"]](s, c)


# ------------------------------------------------------------- plain forms

def _plain_norm(s, c):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    x = x - mean
    rstd = 1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + EPS)
    s["out"].copy_(x * rstd * s["w"].float() + s["b"].float())
    s["mean"].copy_(mean[:, 0])
    s["rstd"].copy_(rstd[:, 0])
    return {"out": s["out"], "mean": s["mean"], "rstd": s["rstd"]}


def _plain_norm_grad(s, c):
    x = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = g - g.mean(1, keepdim=True) - x * (g * x).mean(1, keepdim=True)
    s["dx"].copy_(dx * s["rstd"][:, None])
    dw, db = (dy * x).sum(0), dy.sum(0)
    if c["acc"]:
        s["dw"] += dw
        s["db"] += db
    else:
        s["dw"].copy_(dw)
        s["db"].copy_(db)
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def _statistics(z, scale):
    """(log of the sum, entropy) of the rows of softmax(scale z), in z's type."""
    z = z * scale
    m = z.amax(1, keepdim=True)
    z = z - m
    e = torch.exp(z)
    total = e.sum(1)
    spread = torch.where(e > 0, e * z, 0.0).sum(1) / total
    return m[:, 0] + torch.log(total), torch.log(total) - spread


def _plain_logp(s, c):
    z, ids = s["z"].float(), s["ids"]
    there = ids != -1
    lse, entropy = _statistics(z, s["scale"])
    logprob = z.gather(1, ids.clamp(min=0)[:, None])[:, 0] * s["scale"] - lse
    s["logprob"].copy_(torch.where(there, logprob, 0.0))
    s["entropy"].copy_(torch.where(there, entropy, 0.0))
    s["lse"].copy_(torch.where(there, lse, 0.0))
    if c["top"]:
        # whole numbers in the order of the logits, then of the ids from the last to the first
        b = (z + 0.0).view(torch.int32).long()
        key = torch.where(b < 0, b ^ 0x7FFFFFFF, b) * (1 << 32)
        key += torch.arange(c["V"] - 1, -1, -1, device="cuda")
        best = c["V"] - 1 - (torch.topk(key, min(c["top"], c["V"]), dim=1).values & 0xFFFFFFFF)
        value = z.gather(1, best) * s["scale"] - lse[:, None]
        s["top_ids"].copy_(torch.where(there[:, None], best, -1))
        s["top_logprobs"].copy_(torch.where(there[:, None], value, -math.inf))
    return {k: s[k] for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs")}


def _plain_logp_grad(s, c):
    z, ids = s["z"].float() * s["scale"], s["ids"]
    there = (ids != -1).float()
    logp = z - s["lse"][:, None]
    p = torch.exp(logp)
    g = (s["d_logprob"] * there * s["scale"])[:, None]
    dz = -g * p
    dz.scatter_add_(1, ids.clamp(min=0)[:, None], g)
    if c["entropy"]:
        h = (s["d_entropy"] * there * s["scale"])[:, None]
        dz -= h * torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0.0)
    s["dz"].copy_(dz)
    return s["dz"]


def _plain_distill(s, c):
    z, ids, w = s["z"].float() * s["scale"], s["teacher_ids"].long(), s["weight"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    t = s["teacher_logits"] * s["scale"]
    t = t - t.amax(1, keepdim=True)
    q = torch.exp(t)
    q_total = q.sum(1, keepdim=True)
    q = q / q_total
    logp = (z.gather(1, ids) - m) - torch.log(total)
    s["loss"].copy_(w * (q * (t - torch.log(q_total) - logp)).sum(1))
    if c["grad"]:
        dz = e / total
        dz.scatter_add_(1, ids, -q)
        s["dz"].copy_(dz * (w * s["scale"])[:, None])
    return {"loss": s["loss"], "dz": s["dz"]}


_plain = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "logp": _plain_logp,
          "logp_grad": _plain_logp_grad, "distill": _plain_distill}


# ------------------------------------------------- the framework's operators

def _workspace(s, nbytes):
    """The workspace that a user's program keeps beside its buffers."""
    ws = s.get("ws")
    if ws is None:
        ws = s["ws"] = torch.empty(nbytes(), dtype=torch.uint8, device="cuda")
    return ws


def _own_norm(s, c):
    import error_feedback_b200 as ef
    ef.layer_norm(s["x"], s["w"], s["b"], eps=EPS, out=s["out"], mean=s["mean"], rstd=s["rstd"])
    return {"out": s["out"], "mean": s["mean"], "rstd": s["rstd"]}


def _own_norm_grad(s, c):
    import error_feedback_b200 as ef
    ws = _workspace(s, lambda: ef.layer_norm_grad_workspace_bytes(c["T"], c["D"]))
    ef.layer_norm_grad(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], accumulate=c["acc"],
                       grad_x=s["dx"], grad_weight=s["dw"], grad_bias=s["db"], ws=ws)
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def _own_logp(s, c):
    import error_feedback_b200 as ef
    ws = _workspace(s, ef.token_logprobs_workspace_bytes)
    ef.token_logprobs(s["z"], s["ids"], scale=s["scale"], top=c["top"], padding_idx=-1,
                      logprob=s["logprob"], entropy=s["entropy"], lse=s["lse"],
                      top_ids=s["top_ids"], top_logprobs=s["top_logprobs"], ws=ws)
    return {k: s[k] for k in ("logprob", "entropy", "lse", "top_ids", "top_logprobs")}


def _own_logp_grad(s, c):
    import error_feedback_b200 as ef
    ws = _workspace(s, ef.token_logprobs_workspace_bytes)
    return ef.token_logprobs_grad(s["z"], s["ids"], s["lse"], grad_logprob=s["d_logprob"],
                                  entropy=s["entropy"], grad_entropy=s["d_entropy"],
                                  scale=s["scale"], padding_idx=-1, out=s["dz"], ws=ws)


def _own_distill(s, c):
    import error_feedback_b200 as ef
    ws = _workspace(s, ef.distill_loss_workspace_bytes)
    ef.distill_loss(s["z"], s["teacher_ids"], s["teacher_logits"], weight=s["weight"],
                    scale=s["scale"], loss=s["loss"], grad_logits=s["dz"], ws=ws)
    return {"loss": s["loss"], "dz": s["dz"]}


_own = {"norm": _own_norm, "norm_grad": _own_norm_grad, "logp": _own_logp,
        "logp_grad": _own_logp_grad, "distill": _own_distill}


# --------------------------------------------------------------------- work

def work(c):
    if c["op"].startswith("norm"):
        T, D, x, w = c["T"], c["D"], SIZE[c["x"]], SIZE[c["w"]]
        if c["op"] == "norm":
            return {"bytes": T * D * (x + SIZE[c["out"]]) + 2 * D * w + 8 * T, "flops": 8 * T * D}
        return {"bytes": T * D * 3 * x + D * w + 8 * T + D * (16 if c["acc"] else 8),
                "flops": 14 * T * D}
    T, V, z = c["T"], c["V"], SIZE[c["z"]]
    rows = T * (1.0 - c["pad"])                    # padding is not read
    if c["op"] == "logp":
        return {"bytes": int(rows * V * z) + T * (20 + 8 * c["top"]), "flops": int(7 * rows * V)}
    if c["op"] == "logp_grad":
        return {"bytes": int(rows * V * z) + T * V * z + T * 24,
                "flops": int((8 if c["entropy"] else 4) * rows * V)}
    return {"bytes": int(rows * V * z) + (T * V * z if c["grad"] else 0) + T * (8 + 8 * c["K"]),
            "flops": int((8 if c["grad"] else 4) * rows * V)}


# -------------------------------------------------------------- 64-bit values

SLAB = 1 << 26      # elements of the rows that are done at once


def _slabs(c):
    n = max(1, SLAB // (c["D"] if c["op"].startswith("norm") else c["V"]))
    return [slice(a, min(a + n, c["T"])) for a in range(0, c["T"], n)]


def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "logp": _exact_logp,
            "logp_grad": _exact_logp_grad, "distill": _exact_distill}[c["op"]](s, c)


def _joined(parts):
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_norm(s, c):
    parts = []
    for r in _slabs(c):
        x = s["x"][r].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = torch.rsqrt(var + EPS)
        y = torch.addcmul(s["b"].double(), (x - mean.unsqueeze(1)) * s["w"].double(),
                          rstd.unsqueeze(1))
        parts.append({"out": y, "mean": mean, "rstd": rstd})
    return _joined(parts)


def _exact_norm_grad(s, c):
    dw = s["dw"].double() if c["acc"] else torch.zeros(c["D"], dtype=torch.float64, device="cuda")
    db = s["db"].double() if c["acc"] else torch.zeros_like(dw)
    parts = []
    for r in _slabs(c):
        rstd = s["rstd"][r].double().unsqueeze(1)
        centred = s["x"][r].double() - s["mean"][r].double().unsqueeze(1)
        dy = s["dy"][r].double()
        db = db + torch.einsum("td->d", dy)
        dw = dw + torch.einsum("td,td,t->d", dy, centred, rstd[:, 0])
        g = dy * s["w"].double()
        along = torch.einsum("td,td->t", g, centred).unsqueeze(1) * rstd.pow(2) / c["D"]
        parts.append({"dx": rstd * (g - torch.mean(g, 1, True) - centred * along)})
    return {"dx": _joined(parts)["dx"], "dw": dw, "db": db}


def _exact_logp(s, c):
    parts = []
    for r in _slabs(c):
        z, ids = s["z"][r].double(), s["ids"][r]
        logp = torch.log_softmax(z * s["scale"], 1)
        out = {"logprob": logp[torch.arange(len(ids), device="cuda"), ids],
               "entropy": -torch.xlogy(torch.exp(logp), torch.exp(logp)).sum(1),
               "lse": torch.logsumexp(z * s["scale"], 1)}
        out = {k: v.masked_fill(ids == -1, 0.0) for k, v in out.items()}
        if c["top"]:
            order = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :c["top"]]
            skip = (ids == -1).unsqueeze(1)
            out["top_ids"] = order.int().masked_fill(skip, -1)
            out["top_logprobs"] = torch.take_along_dim(logp, order, 1).masked_fill(skip, -math.inf)
        else:
            out["top_ids"] = s["top_ids"][r]
            out["top_logprobs"] = s["top_logprobs"][r].double()
        parts.append(out)
    return _joined(parts)


def _exact_logp_grad(s, c):
    parts = []
    for r in _slabs(c):
        ids = s["ids"][r]
        logp = torch.log_softmax(s["z"][r].double() * s["scale"], 1)
        p = torch.exp(logp)
        d = torch.zeros_like(p)
        d[torch.arange(len(ids), device="cuda"), ids.clamp(min=0)] = 1.0
        d = (d - p) * s["d_logprob"][r].double().unsqueeze(1)
        if c["entropy"]:
            plogp = torch.xlogy(p, p)
            h = -plogp.sum(1, keepdim=True)
            d = d - (plogp + p * h) * s["d_entropy"][r].double().unsqueeze(1)
        parts.append({"dz": (d * s["scale"]).masked_fill((ids == -1).unsqueeze(1), 0.0)})
    return _joined(parts)["dz"]


def _exact_distill(s, c):
    parts = []
    for r in _slabs(c):
        logp = torch.log_softmax(s["z"][r].double() * s["scale"], 1)
        logq = torch.log_softmax(s["teacher_logits"][r].double() * s["scale"], 1)
        ids, w = s["teacher_ids"][r].long(), s["weight"][r].double()
        gap = logq - torch.take_along_dim(logp, ids, 1)
        out = {"loss": w * torch.einsum("tk,tk->t", torch.exp(logq), gap)}
        if c["grad"]:
            d = torch.exp(logp)
            d.scatter_add_(1, ids, -torch.exp(logq))
            out["dz"] = d * (w * s["scale"]).unsqueeze(1)
        parts.append(out)
    out = _joined(parts)
    return {"loss": out["loss"], "dz": out.get("dz")}
