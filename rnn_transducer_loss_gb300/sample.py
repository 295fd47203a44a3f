"""Drawing labels from the joiner's outputs: ``rnnt_sample``, the stochastic counterpart of
``rnnt_beam_select``."""
from __future__ import annotations

import torch

from . import _native as N
from ._host import DTYPES as _DT
from ._host import call, finish, status_word, without_gradient

_F32, _I32 = torch.float32, torch.int32


def rnnt_sample(logits: torch.Tensor, scores: torch.Tensor, random: torch.Tensor,
                temperature: float = 1.0, top_k: int | None = None, top_p: float = 1.0,
                min_p: float = 0.0, finished: torch.Tensor | None = None,
                fused_log_softmax: bool = True, check: bool = True):
    """One step of drawing, one extension of every hypothesis: (scores, tokens), each (B, K).

    ``logits`` (B, K, V) float32, float16 or bfloat16 are the joiner's outputs
    (log-probabilities with ``fused_log_softmax=False``), ``scores`` (B, K) float32 the
    hypotheses' log-probabilities so far, ``random`` (B, K) float32 a number in
    [0, 1) each (``torch.rand``).  With e = exp(logits / ``temperature``) the outputs kept
    are, in descending order (ties: the lowest token first), the first ``top_k``, of these
    the fewest whose sum of e is at least ``top_p`` of theirs, and of these the ones with
    e >= ``min_p`` times the largest; logits of -inf are never kept.  The token is the
    first kept one at which the running sum of e, by token, is above ``random`` times
    the whole.  Sums decide as if held to 40 bits, so equal inputs draw equal
    tokens wherever they lie.  A returned score is the old one plus the token's
    log-probability among all outputs at temperature 1, within 5e-6 and one float32
    rounding.  A hypothesis that is ``finished`` ((B, K) bool or uint8) keeps its score and
    gets token -1, whatever its logits hold; one of score -inf, or without a finite logit, gets
    score -inf and token -1.  ``check`` reads the device status word (one
    synchronisation) and raises on scores or logits that are NaN or +inf and on random
    numbers outside [0, 1); without it such a hypothesis gets score -inf and token -1.
    Not differentiable: a backward pass through the scores raises, and so does a forward-mode
    derivative.
    """
    return without_gradient("rnnt_sample", (logits, scores),
                            _sample(logits, scores, random, temperature, top_k, top_p, min_p, finished,
                                    fused_log_softmax, check))


def _sample(logits, scores, random, temperature, top_k, top_p, min_p, finished, fused_log_softmax, check):
    dt = _DT.get(logits.dtype)
    device = logits.device
    if device.type != "cuda":
        raise ValueError("logits must be a CUDA tensor")
    if dt is None:
        raise ValueError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
    if logits.dim() != 3:
        raise ValueError("logits must be (B, K, V)")
    B, K, V = shape = logits.shape
    if not 1 <= V <= N.MAX_TOP_VOCAB or K < 1:
        raise ValueError(f"logits must have a hypothesis and 1 to {N.MAX_TOP_VOCAB} outputs")
    for name, t in (("scores", scores), ("random", random)):
        if t.dtype is not _F32 or t.shape != shape[:2] or t.device != device:
            raise ValueError(f"{name} must be float32 ({B}, {K}) on {device}")
    if finished is not None:
        if finished.dtype not in (torch.bool, torch.uint8) or finished.shape != shape[:2] \
                or finished.device != device:
            raise ValueError(f"finished must be bool or uint8 ({B}, {K}) on {device}")
        finished = finished.contiguous()
    temperature, top_p, min_p = float(temperature), float(top_p), float(min_p)
    if top_k is not None and int(top_k) < 1:
        raise ValueError("top_k must be at least 1, or None")
    top_k = 0 if top_k is None else min(int(top_k), V)
    if not (1e-4 <= temperature <= 1e4 and 0.0 < top_p <= 1.0 and 0.0 <= min_p <= 1.0):
        raise ValueError("wanted: temperature in [1e-4, 1e4], top_p in (0, 1], min_p in [0, 1]")
    if logits.is_neg() or scores.is_neg() or random.is_neg():   # their memory holds the negatives
        logits, scores, random = (t.resolve_neg() for t in (logits, scores, random))
    scores, random = scores.contiguous(), random.contiguous()
    out = torch.empty((B, K), dtype=_F32, device=device)
    tokens = torch.empty((B, K), dtype=_I32, device=device)
    if not B:
        return out, tokens
    item, row, step = logits.stride()
    if V > 1 and step != 1:
        logits = logits.contiguous()
        item, row, step = logits.stride()
    status = status_word(device) if check else None
    call("rnnt_sample", device, N.rnnt_sample, logits.data_ptr(), dt, B, K, V, item, row,
         scores.data_ptr(), random.data_ptr(), None if finished is None else finished.data_ptr(),
         temperature, top_k, top_p, min_p, 1 if fused_log_softmax else 0, out.data_ptr(),
         tokens.data_ptr(), None if status is None else status.data_ptr())
    if check:
        finish("rnnt_sample", status, "finite scores or -inf, logits below +inf and not NaN, "
                                      "random numbers in [0, 1)")
    return out, tokens
