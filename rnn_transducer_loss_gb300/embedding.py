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
from ._host import call, differentiated, finish, int32, status_word

_INT32 = torch.int32
_WANTED = "tokens below the vocabulary size, lengths in [0, tokens.shape[1]]"


def _places(tokens, lengths, device):
    """(tokens, row stride of tokens, B, S) with tokens' rows as the kernels read them; raises
    unless tokens is (B, S) and lengths None or (B,), int32 on the device."""
    if tokens.dtype is not _INT32 or tokens.device != device:
        int32("tokens", tokens, device)
    if tokens.dim() != 2:
        raise ValueError("tokens must be (B, S)")
    B, S = tokens.shape
    if lengths is not None:
        if lengths.dtype is not _INT32 or lengths.device != device:
            int32("lengths", lengths, device)
        if lengths.shape != (B,):
            raise ValueError("lengths must be (B,)")
    row, step = tokens.stride()
    if S > 1 and step != 1 or B > 1 and row < S:
        tokens, row = tokens.contiguous(), S
    return tokens, row if row > S else S, B, S


def _start(start, V):
    """(has_start, start) of the C entry points."""
    if start is None:
        return 0, 0
    if not -V <= start < V:
        raise ValueError(f"start must be in [{-V}, {V - 1}]")
    return 1, int(start)


def _forward(weight, tokens, lengths, start, scale, check):
    dt = _DT.get(weight.dtype)
    device = weight.device
    if device.type != "cuda":
        raise ValueError("weight must be a CUDA tensor")
    if dt is None:
        raise ValueError(f"weight must be float32, float16 or bfloat16, got {weight.dtype}")
    if weight.dim() != 2:
        raise ValueError("weight must be (V, D)")
    V, D = weight.shape
    if V < 1 or D < 1:
        raise ValueError("weight must be (V, D)")
    tokens, row, B, S = _places(tokens, lengths, device)
    has, first = _start(start, V)
    out = torch.empty((B, S + has, D), dtype=weight.dtype, device=device)
    if not B or not S + has:
        return out
    if weight.is_neg():                     # its memory holds the negatives
        weight = weight.resolve_neg()
    wrow, step = weight.stride()
    if D > 1 and step != 1 or V > 1 and wrow < D:
        weight, wrow = weight.contiguous(), D
    if lengths is not None:
        lengths = lengths.contiguous()
    status = status_word(device) if check else None
    call("rnnt_embed", device, N.rnnt_embed, weight.data_ptr(), dt, V, D,
         wrow if wrow > D else D, tokens.data_ptr(), row,
         None if lengths is None else lengths.data_ptr(), B, S, has, first, scale, out.data_ptr(),
         None if status is None else status.data_ptr())
    if check:
        finish("rnnt_embed", status, _WANTED)
    return out


def _gradient(grad_out, tokens, V, lengths, start, scale, check):
    dt = _DT.get(grad_out.dtype)
    device = grad_out.device
    if device.type != "cuda":
        raise ValueError("grad_out must be a CUDA tensor")
    if dt is None:
        raise ValueError(f"grad_out must be float32, float16 or bfloat16, got {grad_out.dtype}")
    if V < 1:
        raise ValueError("num_embeddings must be at least 1")
    tokens, row, B, S = _places(tokens, lengths, device)
    has, first = _start(start, V)
    if grad_out.dim() != 3 or grad_out.shape[:2] != (B, S + has):
        raise ValueError(f"grad_out must be ({B}, {S + has}, D)")
    D = grad_out.shape[2]
    if not B or not S + has or not D:
        return torch.zeros((V, D), dtype=grad_out.dtype, device=device)
    if grad_out.is_neg():                   # its memory holds the negatives
        grad_out = grad_out.resolve_neg()
    grad_out = grad_out.contiguous()
    if lengths is not None:
        lengths = lengths.contiguous()
    grad = torch.empty((V, D), dtype=grad_out.dtype, device=device)
    nbytes = N.rnnt_embed_grad_workspace_size(B, S, has, V, D)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    status = status_word(device) if check else None
    call("rnnt_embed_grad", device, N.rnnt_embed_grad, grad_out.data_ptr(), dt,
         tokens.data_ptr(), row, None if lengths is None else lengths.data_ptr(), B, S, has, first,
         V, D, scale, grad.data_ptr(), ws.data_ptr() if nbytes else None, nbytes,
         None if status is None else status.data_ptr())
    if check:
        finish("rnnt_embed_grad", status, _WANTED)
    return grad


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, weight, tokens, lengths, start, scale, check):
        ctx.save_for_backward(tokens, lengths)
        ctx.args = (weight.shape[0], start, scale)
        return _forward(weight, tokens, lengths, start, scale, check)

    @staticmethod
    def backward(ctx, grad_out):
        tokens, lengths = ctx.saved_tensors
        V, start, scale = ctx.args
        # what the device could object to, it objected to in the forward call
        if differentiated(grad_out):
            grad = _EmbedGrad.apply(grad_out, tokens, V, lengths, start, scale, False)
        else:
            grad = _gradient(grad_out, tokens, V, lengths, start, scale, False)
        return grad, None, None, None, None, None


class _EmbedGrad(torch.autograd.Function):
    """The gradient is linear in grad_out, and its own gradient is the lookup."""

    @staticmethod
    def forward(ctx, grad_out, tokens, V, lengths, start, scale, check):
        ctx.save_for_backward(tokens, lengths)
        ctx.args = (start, scale)
        return _gradient(grad_out, tokens, V, lengths, start, scale, check)

    @staticmethod
    def backward(ctx, grad):
        tokens, lengths = ctx.saved_tensors
        start, scale = ctx.args
        return (rnnt_embed(grad, tokens, lengths, start, scale, False),
                None, None, None, None, None, None)


def rnnt_embed(weight: torch.Tensor, tokens: torch.Tensor, lengths: torch.Tensor | None = None,
               start: int | None = None, scale: float = 1.0, check: bool = True) -> torch.Tensor:
    """``scale * weight[tokens]`` as (B, P, D), differentiable with respect to ``weight``.

    ``weight`` is (V, D) float32, float16 or bfloat16; ``tokens`` (B, S) int32,
    ``lengths`` (B,) int32 or None.  With ``start`` (an id in [-V, V-1], negative
    counting from the end; the blank, as a rule) every sequence begins with that
    id and P = S + 1; without it P = S.  Negative tokens, and tokens at or past
    ``lengths[b]`` (which are not read), are padding: zeros, and no gradient.
    Each element is multiplied in float32 and rounded once.  ``check`` reads the
    device status word after the call (one synchronisation) and raises on tokens
    outside the vocabulary and lengths outside [0, S]; without it such a token
    is padding and such a length the nearer bound.  A backward pass is captured
    into a CUDA graph with ``check=False`` and with no eager graph of the same
    weight alive (autograd would make the capture wait for that one's stream).
    Forward-mode derivatives raise.
    """
    if differentiated(weight):
        return _Embed.apply(weight, tokens, lengths, start, float(scale), check)
    return _forward(weight, tokens, lengths, start, float(scale), check)


def rnnt_embed_grad(grad_out: torch.Tensor, tokens: torch.Tensor, num_embeddings: int,
                    lengths: torch.Tensor | None = None, start: int | None = None,
                    scale: float = 1.0, check: bool = True) -> torch.Tensor:
    """Gradient of :func:`rnnt_embed` with respect to its weight, (num_embeddings, D).

    ``grad_out`` is (B, P, D), P = S + 1 with a start symbol and S without.
    Rows of ids that do not occur are zero; ``grad_out`` at padding is not read.
    The places are sorted by id and added in float32 in an order that depends on
    the tokens alone: the same inputs give the same bits.  Differentiable with
    respect to ``grad_out`` (in backward mode; forward-mode derivatives raise).
    """
    if differentiated(grad_out):
        return _EmbedGrad.apply(grad_out, tokens, int(num_embeddings), lengths, start,
                                float(scale), check)
    return _gradient(grad_out, tokens, int(num_embeddings), lengths, start, float(scale), check)


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
