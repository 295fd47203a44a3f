"""Label embedding: ``rnnt_embed`` (lookup with scaling, differentiable), its gradient
``rnnt_embed_grad``, and the module ``RNNTEmbedding``.

The prediction network of a transducer reads the labels the loss takes, behind
a start symbol: ``rnnt_embed(weight, targets, target_lengths, start=blank)``
gives its (B, S + 1, D) input from the loss's own ``targets`` and
``target_lengths``; in decoding the (B, K) tokens of ``rnnt_beam_select`` are
looked up as they are.
"""
from __future__ import annotations

import torch

from . import _native as N
from ._host import DTYPES as _DT
from ._host import call, finish, int32, status_word, stream_of


def _places(tokens, lengths, start, device):
    """Checked (tokens, lengths, B, S, has_start, start); tokens may be None-like empty."""
    int32("tokens", tokens, device)
    if tokens.dim() != 2:
        raise ValueError("tokens must be (B, S)")
    B, S = tokens.shape
    if S > 1 and tokens.stride(1) != 1 or B > 1 and tokens.stride(0) < S:
        tokens = tokens.contiguous()
    if lengths is not None:
        int32("lengths", lengths, device)
        if lengths.dim() != 1 or lengths.shape[0] != B:
            raise ValueError("lengths must be (B,)")
        lengths = lengths.contiguous()
    return tokens, lengths, B, S


def _check_start(start, V):
    if start is not None and not -V <= start < V:
        raise ValueError(f"start must be in [{-V}, {V - 1}]")
    return (0, 0) if start is None else (1, int(start))


def _forward(weight, tokens, lengths, start, scale, check):
    if not weight.is_cuda:
        raise ValueError("weight must be a CUDA tensor")
    if weight.dtype not in _DT:
        raise ValueError(f"weight must be float32, float16 or bfloat16, got {weight.dtype}")
    if weight.dim() != 2 or weight.shape[0] < 1 or weight.shape[1] < 1:
        raise ValueError("weight must be (V, D)")
    dev = weight.device
    V, D = weight.shape
    if D > 1 and weight.stride(1) != 1 or V > 1 and weight.stride(0) < D:
        weight = weight.contiguous()
    tokens, lengths, B, S = _places(tokens, lengths, start, dev)
    has, first = _check_start(start, V)
    out = torch.empty((B, S + has, D), dtype=weight.dtype, device=dev)
    if out.numel() == 0:
        return out
    status = status_word(check, dev)
    call("rnnt_embed", dev, N.rnnt_embed, weight.data_ptr(), _DT[weight.dtype], V, D,
         max(weight.stride(0), D), tokens.data_ptr(), max(tokens.stride(0), S),
         None if lengths is None else lengths.data_ptr(), B, S, has, first, scale, out.data_ptr(),
         None if status is None else status.data_ptr(), stream_of(dev))
    finish("rnnt_embed", status, "tokens below the vocabulary size, lengths in [0, tokens.shape[1]]")
    return out


def rnnt_embed_grad(grad_out: torch.Tensor, tokens: torch.Tensor, num_embeddings: int,
                    lengths: torch.Tensor | None = None, start: int | None = None,
                    scale: float = 1.0, check: bool = True) -> torch.Tensor:
    """Gradient of :func:`rnnt_embed` with respect to its weight, (num_embeddings, D).

    ``grad_out`` is (B, P, D), P = S + 1 with a start symbol and S without.
    Rows of ids that do not occur are zero; ``grad_out`` at padding is not read.
    The places are sorted by id and added in float32 in an order that depends on
    the tokens alone: the same inputs give the same bits.
    """
    if not grad_out.is_cuda:
        raise ValueError("grad_out must be a CUDA tensor")
    if grad_out.dtype not in _DT:
        raise ValueError(f"grad_out must be float32, float16 or bfloat16, got {grad_out.dtype}")
    dev = grad_out.device
    tokens, lengths, B, S = _places(tokens, lengths, start, dev)
    V = int(num_embeddings)
    if V < 1:
        raise ValueError("num_embeddings must be at least 1")
    has, first = _check_start(start, V)
    if grad_out.dim() != 3 or grad_out.shape[0] != B or grad_out.shape[1] != S + has:
        raise ValueError(f"grad_out must be ({B}, {S + has}, D)")
    D = grad_out.shape[2]
    if grad_out.numel() == 0:
        return torch.zeros((V, D), dtype=grad_out.dtype, device=dev)
    grad_out = grad_out.contiguous()
    scale = float(scale)
    grad = torch.empty((V, D), dtype=grad_out.dtype, device=dev)
    nbytes = N.rnnt_embed_grad_workspace_size(B, S, has, V, D)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    status = status_word(check, dev)
    call("rnnt_embed_grad", dev, N.rnnt_embed_grad, grad_out.data_ptr(), _DT[grad_out.dtype],
         tokens.data_ptr(), max(tokens.stride(0), S),
         None if lengths is None else lengths.data_ptr(), B, S, has, first, V, D, scale,
         grad.data_ptr(), ws.data_ptr(), nbytes, None if status is None else status.data_ptr(),
         stream_of(dev))
    finish("rnnt_embed_grad", status,
           "tokens below the vocabulary size, lengths in [0, tokens.shape[1]]")
    return grad


class _EmbedFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, tokens, lengths, start, scale, check):
        ctx.save_for_backward(tokens, lengths)
        ctx.args = (weight.shape[0], start, scale)
        return _forward(weight, tokens, lengths, start, scale, check)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        tokens, lengths = ctx.saved_tensors
        V, start, scale = ctx.args
        # what the device could object to, it objected to in the forward call
        return (rnnt_embed_grad(grad_out, tokens, V, lengths, start, scale, check=False),
                None, None, None, None, None)


def rnnt_embed(weight: torch.Tensor, tokens: torch.Tensor, lengths: torch.Tensor | None = None,
               start: int | None = None, scale: float = 1.0, check: bool = True) -> torch.Tensor:
    """``scale * weight[tokens]`` as (B, P, D), differentiable once with respect to ``weight``.

    ``weight`` is (V, D) float32, float16 or bfloat16; ``tokens`` (B, S) int32,
    ``lengths`` (B,) int32 or None.  With ``start`` (an id in [-V, V-1], negative
    counting from the end; the blank, as a rule) every sequence begins with that
    id and P = S + 1; without it P = S.  Negative tokens, and tokens at or past
    ``lengths[b]`` (which are not read), are padding: zeros, and no gradient.
    Each element is multiplied in float32 and rounded once.  ``check`` reads the
    device status word after the call (one synchronisation) and raises on tokens
    outside the vocabulary and lengths outside [0, S]; without it such a token
    is padding and such a length the nearer bound.
    """
    scale = float(scale)
    if torch.is_grad_enabled() and weight.requires_grad:
        return _EmbedFunction.apply(weight, tokens, lengths, start, scale, check)
    return _forward(weight, tokens, lengths, start, scale, check)


class RNNTEmbedding(torch.nn.Module):
    """Module form of :func:`rnnt_embed`: a (num_embeddings, embedding_dim) table drawn
    from N(0, 1), looked up and multiplied by ``scale``."""

    def __init__(self, num_embeddings: int, embedding_dim: int, start: int | None = None,
                 scale: float = 1.0, check: bool = True, device=None, dtype=None):
        super().__init__()
        self.start, self.scale, self.check = start, scale, check
        self.weight = torch.nn.Parameter(torch.empty(num_embeddings, embedding_dim, device=device,
                                                     dtype=dtype))
        torch.nn.init.normal_(self.weight)

    def forward(self, tokens, lengths=None):
        return rnnt_embed(self.weight, tokens, lengths, self.start, self.scale, self.check)
