"""CPU-only checks of the balance loss under autograd, with stand-ins for the calls
of the library, and of what it and the router refuse there."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from combine_get_dispatch_layout_amd import moe


@pytest.fixture
def calls(monkeypatch):
    """A loss of 3 with counts of 5 and 7 tokens; what the backward call was given."""
    seen = []

    def loss(cfg, logits, *_):
        E = cfg.num_experts
        return moe.Balance(torch.tensor(3.0), torch.full((1, E), 5, dtype=torch.int32),
                           torch.full((1,), 7, dtype=torch.int32), torch.ones(1, E))

    def backward(cfg, logits, counts, seq_tokens, grad_loss, *_):
        seen.append((counts.clone(), seq_tokens.clone(), grad_loss.clone()))
        return torch.ones_like(logits)

    monkeypatch.setattr(moe, "ep_balance_loss", loss)
    monkeypatch.setattr(moe, "ep_balance_loss_backward", backward)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return seen


def test_backward_has_the_counts_of_its_call(calls):
    """Whatever the caller did to the returned ones, without raising their version
    as a collective does."""
    lg = torch.zeros((4, 16), requires_grad=True)
    idx = torch.zeros((4, 2), dtype=torch.int32)
    out = moe.Balance(*moe._BalanceLoss.apply(moe.BalanceConfig(16, 2), lg, idx, *[None] * 7))
    for t in (out.counts, out.seq_tokens):
        t.data.mul_(8)
    (2 * out.loss).backward()
    counts, tokens, g = calls[0]
    assert (counts == 5).all() and (tokens == 7).all() and float(g) == 2
    assert (lg.grad == 1).all()


@pytest.mark.parametrize("grad", [False, True])
def test_forward_mode_is_refused(grad):
    """Neither call has a tangent to give; none is lost without a word."""
    idx = torch.zeros((4, 2), dtype=torch.int32)
    with fwAD.dual_level():
        lg = fwAD.make_dual(torch.zeros((4, 16), requires_grad=grad), torch.ones(4, 16))
        with pytest.raises(RuntimeError, match="ep_balance_loss has no forward"):
            moe.ep_balance_loss(moe.BalanceConfig(16, 2), lg, idx)
        with pytest.raises(RuntimeError, match="ep_gate has no forward"):
            moe.ep_gate(moe.GateConfig(16, 2), lg)
        with torch.no_grad(), pytest.raises(RuntimeError, match="ep_gate has no forward"):
            moe.ep_gate(moe.GateConfig(16, 2), lg)
        with pytest.raises(ValueError, match="on the GPU"):        # without a tangent: as ever
            moe.ep_gate(moe.GateConfig(16, 2), torch.zeros(4, 16))
    with pytest.raises(ValueError, match="on the GPU"):
        moe.ep_gate(moe.GateConfig(16, 2), torch.zeros(4, 16))
