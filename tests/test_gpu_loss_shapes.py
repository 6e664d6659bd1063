"""Shapes that the losses take and refuse beside those of plain matrices."""
import pytest
import torch

import error_feedback_b200 as ef

pytestmark = pytest.mark.gpu


def test_tables_the_wrong_way_round():
    """As many elements as needed, in rows of another length: pairs of the wrong tokens."""
    z = torch.randn(4, 30, device="cuda")
    ids = torch.randint(0, 30, (4, 6), device="cuda", dtype=torch.int32)
    t = torch.randn(4, 6, device="cuda")
    for bad in (t.t().contiguous(), t.view(24), t.view(8, 3)):
        with pytest.raises(ValueError):
            ef.distill_loss(z, ids, bad)
    for kw in (dict(top_ids=ids.t().contiguous()), dict(top_logprobs=t.t().contiguous()), dict(top_ids=ids.view(24)),
               dict(top_logprobs=t.view(2, 12))):
        with pytest.raises(ValueError):
            ef.token_logprobs(z, top=6, **kw)
    want = ef.distill_loss(z, ids, t)[0]
    assert torch.equal(ef.distill_loss(z.view(2, 2, 30), ids.view(2, 2, 6), t.view(2, 2, 6))[0], want)
    assert torch.equal(ef.distill_loss(z[1], ids[1], t[1])[0], want[1:2])
    got = ef.token_logprobs(z.view(2, 2, 30), top=6, top_ids=ids.view(2, 2, 6), top_logprobs=t.view(2, 2, 6))
    assert torch.equal(got[3].view(4, 6), ef.token_logprobs(z, top=6)[3])


def test_rows_of_two_strides():
    """The first positions of each sequence: rows that no single stride reaches are refused, as a
    copy or one sequence at a time they work."""
    z = torch.randn(3, 5, 40, device="cuda")
    part = z[:, :-1]
    lse = torch.zeros(12, device="cuda")
    ids = torch.zeros(12, 2, dtype=torch.int32, device="cuda")
    for call in (lambda: ef.token_logprobs(part), lambda: ef.layer_norm(part), lambda: ef.layer_norm(z[:, :4].clone(), out=part),
                 lambda: ef.layer_norm_grad(part, z[:, :4].clone(), lse, lse),
                 lambda: ef.token_logprobs_grad(part, lse.long(), lse, grad_logprob=lse),
                 lambda: ef.distill_loss(part, ids, ids.float())):
        with pytest.raises(ValueError):
            call()
    want = ef.token_logprobs(part.contiguous())[2].view(3, 4)
    assert all(torch.equal(ef.token_logprobs(part[i])[2], want[i]) for i in range(3))
    # one stride: every second row of each sequence, columns of a wider buffer
    both = torch.randn(3, 4, 64, device="cuda")[:, ::2, 8:48]
    assert torch.equal(ef.token_logprobs(both)[2], ef.token_logprobs(both.contiguous())[2])
