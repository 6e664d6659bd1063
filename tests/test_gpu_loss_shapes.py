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
