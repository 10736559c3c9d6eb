"""GPU tests of the balance loss where a caller changes what it returned."""
import pytest
import torch

from combine_get_dispatch_layout_amd import moe
from test_gpu_balance import cu, inputs

pytestmark = pytest.mark.gpu


def test_counts_summed_in_place_before_backward():
    """As an all-reduce leaves them, which raises no version: the loss's gradient
    stays that of the call."""
    z, idx, mask, start = inputs(200, 64, 6, 4, 0.1)
    cfg = moe.BalanceConfig(64, 6, coefficient=0.3)
    lg = cu(z).requires_grad_()
    with torch.no_grad():
        o = moe.ep_balance_loss(cfg, lg, cu(idx), cu(mask), cu(start))
        want = moe.ep_balance_loss_backward(cfg, lg, o.counts, o.seq_tokens, torch.ones((), device="cuda"), cu(mask),
                                            cu(start))
    out = moe.ep_balance_loss(cfg, lg, cu(idx), cu(mask), cu(start))
    assert torch.equal(out.counts, o.counts) and torch.equal(out.seq_tokens, o.seq_tokens)
    out.counts.data.mul_(8)
    out.seq_tokens.data.mul_(8)
    out.score_sums.data.mul_(8)
    out.loss.backward()
    assert torch.equal(lg.grad, want)
