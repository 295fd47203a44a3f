"""GPU: tensors that rnnt_beam_reorder writes to count as changed in place."""
import pytest
import torch

from rnn_transducer_loss_gb300 import rnnt_beam_reorder

pytestmark = pytest.mark.gpu


def test_saved_results_are_noticed():
    """A backward pass that saved an `out` tensor raises once the tensor was written to again."""
    x = torch.randn(2, 3, 5, device="cuda")
    p = torch.tensor([[2, 1, 0], [0, 0, 1]], dtype=torch.int32, device="cuda")
    y = torch.empty(2, 3, 5, device="cuda")
    w = torch.ones(5, device="cuda", requires_grad=True)
    rnnt_beam_reorder([x], p, out=[y])
    want = y.sum((0, 1))
    (w * y).sum().backward()
    assert torch.allclose(w.grad, want)
    loss = (w * y).sum()
    rnnt_beam_reorder([2 * x], p, out=[y])
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.backward()
    loss = (w * y).sum()
    rnnt_beam_reorder([x], p)                       # new results: nothing of y changes
    loss.backward()


def test_inference_tensors():
    x = torch.randn(2, 3, 5, device="cuda")
    p = torch.tensor([[2, 1, 0], [0, 0, 1]], dtype=torch.int32, device="cuda")
    want, = rnnt_beam_reorder([x], p)
    with torch.inference_mode():
        y = torch.empty(2, 3, 5, device="cuda")
        rnnt_beam_reorder([x], p, out=[y])
        assert torch.equal(y, want)
        y.zero_()
    rnnt_beam_reorder([x], p, out=[y])
    assert torch.equal(y, want)
