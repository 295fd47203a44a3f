"""GPU: operators without derivatives say so instead of dropping them."""
import pytest
import torch
from torch.autograd import forward_ad

from rnn_transducer_loss_gb300 import rnnt_distill_loss, rnnt_sample, rnnt_top_logits

pytestmark = pytest.mark.gpu


def test_top_logits():
    x = torch.randn(6, 29, device="cuda")
    want = rnnt_top_logits(x, 3)
    assert not any(t.requires_grad for t in want)
    leaf = x.clone().requires_grad_()
    got = rnnt_top_logits(leaf, 3)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert got[0].requires_grad and got[2].requires_grad and not got[1].requires_grad
    for t in (got[0], got[2]):
        with pytest.raises(RuntimeError, match="rnnt_top_logits is not differentiable"):
            (t.sum() + leaf.sum()).backward(retain_graph=True)
    n = torch.ones(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="detach"):                    # a teacher that is trained
        rnnt_distill_loss(x, *got[:2], 6 * n, 0 * n)
    with torch.no_grad():
        assert not any(t.requires_grad for t in rnnt_top_logits(leaf, 3))
    with forward_ad.dual_level():
        assert torch.equal(rnnt_top_logits(x, 3)[0], want[0])
        with pytest.raises(NotImplementedError):
            rnnt_top_logits(forward_ad.make_dual(x, x), 3)


def test_sample():
    x, s, u = torch.randn(2, 3, 29, device="cuda"), torch.zeros(2, 3, device="cuda"), torch.rand(2, 3, device="cuda")
    want = rnnt_sample(x, s, u)
    assert not want[0].requires_grad
    for a, b in ((x.clone().requires_grad_(), s), (x, s.clone().requires_grad_()),
                 (x.clone().requires_grad_(), s.clone().requires_grad_())):
        got = rnnt_sample(a, b, u)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert got[0].requires_grad and not got[1].requires_grad
        with pytest.raises(RuntimeError, match="rnnt_sample is not differentiable"):
            got[0].sum().backward()
    with forward_ad.dual_level(), pytest.raises(NotImplementedError):
        rnnt_sample(x, forward_ad.make_dual(s, s), u)
