"""A step of distillation made of the library's calls, as a program would run them: the
student's embedding lookup, layer norm and logits, the teacher's alternatives by
token_logprobs, the distillation loss with its gradient and the log-probabilities of the
next tokens with theirs, back through the norm (its weight gradients accumulated in the
flat bucket) and the embedding, then the error-feedback compress of the bucket and the
Muon update of the output matrix.  Every gradient in the bucket is checked against
autograd in 64 bits and one against a difference of the loss."""
import numpy as np
import pytest
import torch

import error_feedback_b200 as ef
import oracle
from gpu_util import same_bits

pytestmark = pytest.mark.gpu

V, D, K = 1500, 72, 24
LR = np.float32(0.5)
TAU, MIX, ENT = 2.0, 0.3, 0.01      # temperature, share of the tokens' own loss, entropy bonus


def _loss64(E, w, b, W, ids, target, tids, tl):
    x = E[ids]
    d = x - x.mean(1, keepdim=True)
    h = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt() * w + b
    z = h @ W
    q = torch.softmax(tl.double() / TAU, 1)
    kl = (q * (q.log() - torch.log_softmax(z / TAU, 1).gather(1, tids.long()))).sum(1)
    keep = (target >= 0).double()
    logp = torch.log_softmax(z, 1)
    ce = -(logp.gather(1, target.clamp(min=0)[:, None])[:, 0]) * keep
    ent = -(logp.exp() * logp).sum(1) * keep
    n = len(ids)
    return (kl * TAU**2 / n + MIX * ce / n - ENT * ent / n).sum()


@pytest.mark.parametrize("tokens", [9, 700])
def test_step(tokens):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    E = torch.randn(V, D, generator=g, device="cuda")
    w = 1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")
    b = 0.1 * torch.randn(D, generator=g, device="cuda")
    W = torch.randn(D, V, generator=g, device="cuda") * 0.2
    n_e = V * D
    ends = [0, n_e, n_e + D, n_e + 2 * D]
    ks = [n_e // 50, D // 4, D // 4]
    residual = torch.zeros(ends[-1], device="cuda")
    momentum = torch.zeros(D, V, device="cuda")
    ws_n = torch.empty(ef.layer_norm_grad_workspace_bytes(tokens, D), dtype=torch.uint8, device="cuda")
    ws_c = torch.empty(ef.topk_ef_batched_workspace_bytes(ends, ks), dtype=torch.uint8, device="cuda")
    ws_l = torch.empty(ef.token_logprobs_workspace_bytes(), dtype=torch.uint8, device="cuda")
    o = oracle.get()
    bucket = torch.zeros(ends[-1], device="cuda")
    want_bucket = torch.zeros(ends[-1], dtype=torch.float64, device="cuda")
    gW = torch.zeros(D, V, device="cuda")
    for micro in range(2):              # micro-batches into one bucket
        ids = torch.randint(0, V, (tokens,), generator=g, device="cuda")
        target = torch.randint(0, V, (tokens,), generator=g, device="cuda")
        target[:: 4] = -1               # positions without a next token
        # the teacher: its 24 alternatives, from logits in bf16
        tz = (torch.randn(tokens, V, generator=g, device="cuda") * 3).bfloat16()
        _, _, _, tids, tlp = ef.token_logprobs(tz, top=K, ws=ws_l)

        x = ef.embedding_lookup(E, ids)
        h, mean, rstd = ef.layer_norm(x, w, b)
        z = h @ W
        weight = torch.full((tokens,), TAU**2 / tokens, device="cuda")
        loss, dz = ef.distill_loss(z, tids, tlp, weight=weight, scale=1 / TAU, grad=True, ws=ws_l)
        logp, ent, lse, _, _ = ef.token_logprobs(z, target, padding_idx=-1, ws=ws_l)
        assert ef.topk_ef_last_device_status(ws_l) == 0
        keep = (target >= 0).float()
        dz += ef.token_logprobs_grad(z, target, lse, grad_logprob=-MIX / tokens * keep, entropy=ent,
                                     grad_entropy=-ENT / tokens * keep, padding_idx=-1, ws=ws_l)
        total = loss.double().sum() - (MIX * logp.double() + ENT * ent.double()).sum() / tokens
        dh = dz @ W.T
        gW += h.T @ dz
        dx, _, _ = ef.layer_norm_grad(dh, x, mean, rstd, w, accumulate=True, grad_weight=bucket[n_e:n_e + D],
                                      grad_bias=bucket[n_e + D:], ws=ws_n)
        assert ef.topk_ef_last_device_status(ws_n) == 0
        ef.embedding_grad(dx, ids, V, accumulate=True, out=bucket[:n_e].view(V, D))

        leaves = [t.double().requires_grad_() for t in (E, w, b)]
        want = _loss64(*leaves, W.double(), ids, target, tids, tlp)
        want.backward()
        # (lse and the sums of up to V terms in fp32, products of D terms: some hundred roundings)
        assert float(abs(total - want.detach())) < 1e-5 * float(want.detach().abs())
        want_bucket += torch.cat([t.grad.reshape(-1) for t in leaves])
        step = torch.randn(V, D, generator=g, device="cuda").double()
        eps = 1e-5
        diff = (_loss64(E.double() + eps * step, w.double(), b.double(), W.double(), ids, target, tids, tlp)
                - _loss64(E.double() - eps * step, w.double(), b.double(), W.double(), ids, target, tids, tlp)) / (2 * eps)
        have = ef.embedding_grad(dx, ids, V).double()
        assert float(abs(diff - (have * step).sum())) < 1e-4 * float(have.norm() * step.norm())
    for lo, hi in zip(ends[:-1], ends[1:]):
        off = (bucket[lo:hi].double() - want_bucket[lo:hi]).norm() / want_bucket[lo:hi].norm()
        assert float(off) < 1e-4, (lo, float(off))

    res0, b0 = residual.cpu().numpy(), bucket.cpu().numpy()
    gi, gv = ef.topk_ef_compress_batched(bucket, residual, ends, ks, LR, ws=ws_c)
    oi, ov = o.compress_batched(b0, res0, ends, ks, LR, 0)
    assert np.array_equal(gi.cpu().numpy(), oi) and same_bits(gv.cpu().numpy(), ov).all()
    assert same_bits(residual.cpu().numpy(), res0).all()
    update = ef.muon_update(gW, momentum=momentum, scale=0.1)
    assert update.isfinite().all()
