"""GPU: tensors that are negative views, whose memory holds other values than they do."""
import pytest
import torch

from rnn_transducer_loss_gb300 import rnnt_beam_select, rnnt_embed, rnnt_embed_grad

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def views(*shape):
    """Negative views of different strides."""
    z = torch.randn(*shape, device="cuda", dtype=torch.complex64)
    x = torch.randn(*shape, device="cuda")
    for v in (z.conj().imag, torch._neg_view(x), torch._neg_view(x.half())):
        assert v.is_neg()
        yield v


@pytest.mark.parametrize("D", [1, 6])
def test_embed(D):
    tokens = i32([[1, 4, 4], [0, 2, -1]])
    for w in views(5, D):
        want = rnnt_embed(w.resolve_neg().contiguous(), tokens, scale=2.0)
        assert torch.equal(rnnt_embed(w, tokens, scale=2.0), want)
        leaf = w.clone().requires_grad_()
        assert torch.equal(rnnt_embed(torch._neg_view(-leaf), tokens, scale=2.0), want)


@pytest.mark.parametrize("B,D", [(1, 1), (1, 6), (2, 6)])
def test_embed_grad(B, D):
    tokens = i32([[1], [4]][:B])
    for go in views(B, 1, D):
        want = rnnt_embed_grad(go.resolve_neg().contiguous(), tokens, 5)
        assert torch.equal(rnnt_embed_grad(go, tokens, 5), want)
        w = torch.zeros(5, D, device="cuda", dtype=go.dtype).requires_grad_()
        assert torch.equal(torch.autograd.grad(rnnt_embed(w, tokens), w, go)[0], want)


@pytest.mark.parametrize("K,V", [(1, 1), (1, 7), (3, 1), (3, 40)])
def test_select(K, V):
    s = torch.randn(1, K, device="cuda")
    for x in views(1, K, V):
        for scores in (s, *list(views(1, K))[:2]):
            want = rnnt_beam_select(x.resolve_neg().contiguous(), scores.resolve_neg().contiguous(),
                                    4, fused_log_softmax=False)
            got = rnnt_beam_select(x, scores, 4, fused_log_softmax=False)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
