"""A data-parallel training step made of the library's calls, as a program
would run them: embedding lookup, the gradient of the table written into the
flat bucket beside a matrix's gradient, the error-feedback compress of the
bucket, the gTop-k merge of the workers' sets, their dense sum, and the Muon
update of the matrix.  Gradients are checked against autograd in 64 bits and
against differences of the loss, the sparse steps bit for bit against the
oracle."""
import numpy as np
import pytest
import torch

import error_feedback_b200 as ef
import oracle
from gpu_util import same_bits

pytestmark = pytest.mark.gpu

V, D, H, T, P = 400, 48, 72, 250, 2
LR = np.float32(0.5)


def _loss64(E, W, ids, target, scale):
    x = E.double()[ids] * scale
    return 0.5 * ((x @ W.double() - target.double()) ** 2).sum()


@pytest.mark.parametrize("tokens", [T, 3 * T])
def test_step(tokens):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    E = torch.randn(V, D, generator=g, device="cuda") * 0.3
    W = torch.randn(D, H, generator=g, device="cuda") * 0.2
    n_e, n_w = V * D, D * H
    offsets, ks = [0, n_e, n_e + n_w], [n_e // 50, n_w // 20]
    scale = D ** 0.5
    momentum = torch.zeros(D, H, device="cuda")
    residual = [torch.zeros(n_e + n_w, device="cuda") for _ in range(P)]
    ws_g = torch.empty(ef.embedding_grad_workspace_bytes(tokens, V, D), dtype=torch.uint8, device="cuda")
    ws_c = torch.empty(ef.topk_ef_batched_workspace_bytes(offsets, ks), dtype=torch.uint8, device="cuda")
    ws_u = torch.empty(ef.muon_workspace_bytes(1, D, H), dtype=torch.uint8, device="cuda")
    o = oracle.get()
    for step in range(3):
        idx, val, rows = [], [], []
        for p in range(P):
            ids = torch.randint(0, V, (tokens,), generator=g, device="cuda")
            target = torch.randn(tokens, H, generator=g, device="cuda")
            x = ef.embedding_lookup(E, ids, scale=scale)
            dh = x @ W - target
            bucket = torch.full((n_e + n_w,), 9.0, device="cuda")
            dx = dh @ W.T
            ef.embedding_grad(dx, ids, V, scale=scale, out=bucket[:n_e].view(V, D), ws=ws_g)
            assert ef.topk_ef_last_device_status(ws_g) == 0
            bucket[n_e:].view(D, H).copy_(x.T @ dh)
            # autograd in 64 bits
            E64, W64 = E.double().requires_grad_(), W.double().requires_grad_()
            loss = _loss64(E64, W64, ids, target, scale)
            loss.backward()
            want = torch.cat([E64.grad.reshape(-1), W64.grad.reshape(-1)])
            # (fp32 products of up to `tokens` terms on both sides: 2^-24 of a few thousand terms)
            assert float((bucket.double() - want).norm() / want.norm()) < 1e-5
            # a difference of the loss along a direction that touches the table alone
            d = torch.randn(V, D, generator=g, device="cuda").double()
            h = 1e-4
            with torch.no_grad():
                diff = (_loss64(E.double() + h * d, W, ids, target, scale)
                        - _loss64(E.double() - h * d, W, ids, target, scale)) / (2 * h)
            along = (bucket[:n_e].double() * d.reshape(-1)).sum()
            # (the loss is quadratic: the central difference has no error of its own)
            assert float(abs(diff - along)) <= 1e-5 * float(bucket[:n_e].double().norm() * d.norm())
            rows.append((ids, dx))

            res0, b0 = residual[p].cpu().numpy(), bucket.cpu().numpy()
            gi, gv = ef.topk_ef_compress_batched(bucket, residual[p], offsets, ks, LR, ws=ws_c)
            oi, ov = o.compress_batched(b0, res0, offsets, ks, LR, 0)
            assert np.array_equal(gi.cpu().numpy(), oi) and same_bits(gv.cpu().numpy(), ov).all()
            assert same_bits(residual[p].cpu().numpy(), res0).all()
            at = gi.clone()
            at[ks[0]:] += n_e                       # indices in the whole bucket
            idx.append(at)
            val.append(gv)
        k = sum(ks)
        mi, mv, mc = ef.gtopk_merge(torch.stack(idx), torch.stack(val), k, n_e + n_w)
        c = int(mc)
        update = ef.topk_allgather_sum(mi[:c].view(1, -1).contiguous(), mv[:c].view(1, -1).contiguous(), n_e + n_w)
        dense = np.zeros(n_e + n_w, np.float32)
        dense[mi[:c].cpu().numpy()] = mv[:c].cpu().numpy()
        assert same_bits(update.cpu().numpy(), dense).all()
        # the matrix's part of the merged update, orthogonalised in place
        mom0 = momentum.double()
        part = update[n_e:].view(D, H)
        u = part.double()
        ef.muon_update(part, momentum=momentum, scale=0.1, out=part, ws=ws_u)
        mu = float(torch.tensor(0.95))
        m1 = mom0 * mu + u
        assert torch.equal(momentum, m1.float())
        x64 = u + mu * momentum.double()
        x64 = x64 / (x64.norm() + 1e-7)
        for _ in range(5):
            a = x64 @ x64.T
            x64 = 3.4445 * x64 + (-4.7750 * a + 2.0315 * a @ a) @ x64
        # fp32 output: a few roundings of 2^-24 that five steps of slope 3.4 can grow 485 times
        assert float((part.double() - 0.1 * x64).norm() / (0.1 * x64).norm()) < 485 * 2.0**-24
        E -= update[:n_e].view(V, D)
        W -= part
        assert E.isfinite().all() and W.isfinite().all()

    # the row-sparse gradients of the workers, as index-sorted sets over the
    # table, add up to the sum of the dense ones
    sets = []
    for ids, dx in rows:
        r, v, cnt = ef.embedding_grad_rows(dx, ids, V, scale=scale, ws=ws_g)
        c = int(cnt)
        sets.append((r[:c, None] * D + torch.arange(D, dtype=torch.int32, device="cuda")).reshape(-1))
        sets.append(v[:c].reshape(-1))
    want = sum(ef.embedding_grad(dx, ids, V, scale=scale) for ids, dx in rows)
    got = torch.zeros(n_e, device="cuda")
    for i, v in zip(sets[::2], sets[1::2]):
        got += ef.topk_allgather_sum(i.view(1, -1), v.view(1, -1), n_e)
    assert torch.equal(got, want.reshape(-1))
