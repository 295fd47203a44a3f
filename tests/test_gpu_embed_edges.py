"""GPU: the label embedding and its gradient where they can go wrong."""
import pytest
import torch

from rnn_transducer_loss_gb300 import rnnt_embed, rnnt_embed_grad

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B", [1, 3, 5000])
@pytest.mark.parametrize("bad", [-1, 1, 5, -2 ** 31, 2 ** 31 - 1])
def test_lengths_of_no_tokens(B, bad):
    """Sequences of the start symbol alone: a length that is not 0 is reported, and the start symbol
    stays, by each of the gradient's ways (up to 4096 places, and more)."""
    V, D = 9, 4
    w = torch.randn(V, D, device="cuda")
    go = torch.randn(B, 1, D, device="cuda")
    tokens, good = torch.empty(B, 0, dtype=torch.int32, device="cuda"), i32([0] * B)
    lengths = good.clone()
    lengths[B // 2] = bad
    want = w[2].expand(B, 1, D)
    assert torch.equal(rnnt_embed(w, tokens, good, start=2), want)
    total = rnnt_embed_grad(go, tokens, V, good, start=2)
    with pytest.raises(ValueError):
        rnnt_embed(w, tokens, lengths, start=2)
    with pytest.raises(ValueError):
        rnnt_embed_grad(go, tokens, V, lengths, start=2)
    assert torch.equal(rnnt_embed(w, tokens, lengths, start=2, check=False), want)
    assert torch.equal(rnnt_embed_grad(go, tokens, V, lengths, start=2, check=False), total)


@pytest.mark.parametrize("S", [1, 7, 3000])
def test_start_of_bad_lengths(S):
    """With tokens, a length below 0 counts as 0 and one past S as S; the start symbol stays."""
    w = torch.randn(9, 4, device="cuda")
    tokens = torch.randint(0, 9, (3, S), device="cuda", dtype=torch.int32)
    lengths, near = i32([-7, S + 9, 1]), i32([0, S, 1])
    go = torch.randn(3, S + 1, 4, device="cuda")
    with pytest.raises(ValueError):
        rnnt_embed(w, tokens, lengths, start=8)
    assert torch.equal(rnnt_embed(w, tokens, lengths, start=8, check=False),
                       rnnt_embed(w, tokens, near, start=8))
    assert torch.equal(rnnt_embed_grad(go, tokens, 9, lengths, start=8, check=False),
                       rnnt_embed_grad(go, tokens, 9, near, start=8))
