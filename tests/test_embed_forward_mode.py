"""Forward-mode derivatives of the lookup and its gradient: there are none, and asking for one
raises instead of dropping it."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

from rnn_transducer_loss_gb300 import RNNTEmbedding, embedding, rnnt_embed, rnnt_embed_grad


def raises():
    return pytest.raises(NotImplementedError, match="jvp")


def refusals(device):
    w, t = torch.randn(5, 3, device=device), torch.randn(5, 3, device=device)
    go, s = torch.randn(2, 4, 3, device=device), torch.randn(2, 4, 3, device=device)
    tokens = torch.tensor([[1, 2, 0, 4], [3, 3, 1, 0]], dtype=torch.int32, device=device)
    plain, back = rnnt_embed(w, tokens), rnnt_embed_grad(go, tokens, 5)
    with fwd.dual_level():
        for leaf in (w, w.clone().requires_grad_()):
            with raises():
                rnnt_embed(fwd.make_dual(leaf, t), tokens)
        with raises(), torch.no_grad():
            rnnt_embed(fwd.make_dual(w, t), tokens)
        with raises():
            rnnt_embed_grad(fwd.make_dual(go, s), tokens, 5)
        mod = RNNTEmbedding(5, 3, device=device)
        out = mod(tokens)
        with raises():                              # forward over reverse
            torch.autograd.grad(out, mod.weight, fwd.make_dual(go, s))
        # without a tangent nothing changes
        assert torch.equal(rnnt_embed(w, tokens), plain)
        assert torch.equal(rnnt_embed_grad(go, tokens, 5), back)
        assert torch.equal(torch.autograd.grad(mod(tokens), mod.weight, go)[0], back)
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: rnnt_embed(x, tokens), (w,), (t,))


def test_refused_on_cpu(monkeypatch):
    """The kernels' part as torch operations."""
    def forward(weight, tokens, lengths, start, scale, check):
        return weight[tokens.long()] * scale

    def gradient(grad_out, tokens, V, lengths, start, scale, check):
        rows = (grad_out * scale).reshape(-1, grad_out.shape[2])
        return torch.zeros(V, grad_out.shape[2]).index_add(0, tokens.long().reshape(-1), rows)

    monkeypatch.setattr(embedding, "_forward", forward)
    monkeypatch.setattr(embedding, "_gradient", gradient)
    refusals("cpu")


@pytest.mark.gpu
def test_refused():
    refusals("cuda")
