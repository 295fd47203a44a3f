"""Beam search on the joiner's outputs: ``rnnt_beam_select`` (the best extensions of a batch's
hypotheses) and ``rnnt_beam_reorder`` (the states of the selected ones)."""
from __future__ import annotations

import torch

from . import _native as N
from ._host import DTYPES as _DT
from ._host import call, finish, int32, status_word, stream_of


def rnnt_beam_select(logits: torch.Tensor, scores: torch.Tensor, beam: int | None = None,
                     finished: torch.Tensor | None = None, fused_log_softmax: bool = True,
                     check: bool = True):
    """One step of beam search: (scores, tokens, parents), each (B, beam), best first.

    ``logits`` (B, K, V) float32, float16 or bfloat16 are the joiner's outputs
    for K hypotheses of each item (log-probabilities with
    ``fused_log_softmax=False``), ``scores`` (B, K) float32 their
    log-probabilities so far, ``beam`` (default K) how many to keep.  A
    hypothesis offers its score plus the log-probability of every output whose
    logit is above -inf; one that is ``finished`` ((B, K) bool or uint8) offers
    itself alone, with its score unchanged and token -1, and its logits are not
    read; one of score -inf offers nothing.  Values are compared in 64 bits,
    ties go to the lowest hypothesis, then the lowest token.  ``parents`` says
    which hypothesis each result extends (for :func:`rnnt_beam_reorder`); places
    left over get score -inf, token -1, parent -1.  ``check`` reads the device
    status word (one synchronisation) and raises on scores or logits that are
    NaN or +inf; without it a hypothesis that holds one offers nothing.
    """
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dtype not in _DT:
        raise ValueError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
    if logits.dim() != 3:
        raise ValueError("logits must be (B, K, V)")
    dev = logits.device
    B, K, V = logits.shape
    if K < 1 or K > N.MAX_BEAM or V < 1 or V > N.MAX_BEAM_VOCAB:
        raise ValueError(f"logits must have 1 to {N.MAX_BEAM} hypotheses and 1 to "
                         f"{N.MAX_BEAM_VOCAB} outputs")
    beam = K if beam is None else int(beam)
    if beam < 1 or beam > N.MAX_BEAM:
        raise ValueError(f"beam must be in [1, {N.MAX_BEAM}]")
    if scores.dtype != torch.float32 or scores.shape != (B, K) or scores.device != dev:
        raise ValueError(f"scores must be float32 ({B}, {K}) on {dev}")
    if finished is not None:
        if finished.dtype not in (torch.bool, torch.uint8) or finished.shape != (B, K) \
                or finished.device != dev:
            raise ValueError(f"finished must be bool or uint8 ({B}, {K}) on {dev}")
        finished = finished.contiguous()
    if V > 1 and logits.stride(2) != 1:
        logits = logits.contiguous()
    scores = scores.contiguous()
    out_scores = torch.empty((B, beam), dtype=torch.float32, device=dev)
    out = torch.empty((2, B, beam), dtype=torch.int32, device=dev)
    tokens, parents = out.unbind(0)
    if B == 0:
        return out_scores, tokens, parents
    dt = _DT[logits.dtype]
    nbytes = N.rnnt_beam_workspace_size(B, K, V, beam, dt)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    status = status_word(check, dev)
    call("rnnt_beam_select", dev, N.rnnt_beam_select, logits.data_ptr(), dt, B, K, V,
         logits.stride(0), logits.stride(1), scores.data_ptr(),
         None if finished is None else finished.data_ptr(), beam, 1 if fused_log_softmax else 0,
         out_scores.data_ptr(), tokens.data_ptr(), parents.data_ptr(), ws.data_ptr(), nbytes,
         None if status is None else status.data_ptr(), stream_of(dev))
    finish("rnnt_beam_select", status, "finite scores or -inf, logits below +inf and not NaN")
    return out_scores, tokens, parents


def _describe(state, x, out, d, src, dst):
    """Fills a State with the rows of x and out: the batch axis d, the beam axis d + 1, the
    trailing axes that are adjacent in both as a row, and up to three further axes."""
    size = x.element_size()
    xs, os, shape = x.stride(), out.stride(), x.shape
    row, last = 1, len(shape) - 1
    while last > d + 1 and (shape[last] == 1 or xs[last] == row and os[last] == row):
        row *= shape[last]
        last -= 1
    axes = []
    for i in range(last, -1, -1):
        if i == d or i == d + 1 or shape[i] == 1:
            continue
        n, a, b = shape[i], xs[i], os[i]
        if axes and (i < d) == axes[-1][3] and a == axes[-1][0] * axes[-1][1] \
                and b == axes[-1][0] * axes[-1][2]:
            axes[-1] = (axes[-1][0] * n, axes[-1][1], axes[-1][2], i < d)
        else:
            axes.append((n, a, b, i < d))
    if len(axes) > 3:
        raise ValueError("a state has more than three axes that are not adjacent in memory; "
                         "make it contiguous")
    state.src, state.dst, state.row_bytes = src, dst, row * size
    for j in range(3):
        n, a, b = axes[j][:3] if j < len(axes) else (1, 0, 0)
        state.n[j], state.src_stride[j], state.dst_stride[j] = n, a * size, b * size
    state.src_batch, state.src_beam = xs[d] * size, xs[d + 1] * size
    state.dst_batch, state.dst_beam = os[d] * size, os[d + 1] * size


def rnnt_beam_reorder(states, parents: torch.Tensor, batch_dim=0, out=None, check: bool = True):
    """The states of the selected hypotheses: ``new[.., b, k, ..] = old[.., b, parents[b, k], ..]``.

    ``states`` is a sequence of CUDA tensors of any type, each with a batch axis
    of size B and, behind it, a beam axis of size K: ``batch_dim`` says where
    (one number, or one per state; a recurrent state (layers, B, K, width) has
    batch_dim 1).  ``parents`` (B, K') int32 is what
    :func:`rnnt_beam_select` returned; the results have K' in the place of K,
    and zeros where the parent is -1.  ``out`` gives tensors to write to (they
    must not share memory with ``states``: keep two sets and swap them);
    without it the results are new contiguous tensors.  Views are read with
    their strides: the filled part of a cache need not be copied out first.
    ``check`` reads the device status word (one synchronisation) and raises on
    parents outside [-1, K); without it such a parent counts as -1.
    """
    states = list(states)
    if not states:
        return []
    dev = states[0].device
    if not states[0].is_cuda:
        raise ValueError("states must be CUDA tensors")
    int32("parents", parents, dev)
    if parents.dim() != 2 or parents.shape[1] < 1:
        raise ValueError("parents must be (B, K') with K' >= 1")
    B, Ko = parents.shape
    dims = [batch_dim] * len(states) if isinstance(batch_dim, int) else list(batch_dim)
    if len(dims) != len(states):
        raise ValueError("batch_dim must be one number, or one per state")
    K = None
    for i, (x, d) in enumerate(zip(states, dims)):
        if x.device != dev:
            raise ValueError(f"states must be on {dev}")
        d = dims[i] = d + x.dim() if d < 0 else d
        if not 0 <= d < x.dim() - 1:
            raise ValueError("batch_dim must leave a beam axis behind it")
        if K is None:
            K = x.shape[d + 1]
        if x.shape[d] != B or x.shape[d + 1] != K or K < 1:
            raise ValueError(f"states must have a batch axis of {B} and, behind it, a beam axis "
                             "of the same size, at least 1")
    parents = parents.contiguous()
    shapes = [x.shape[:d + 1] + (Ko,) + x.shape[d + 2:] for x, d in zip(states, dims)]
    if out is None:
        out = [torch.empty(s, dtype=x.dtype, device=dev) for s, x in zip(shapes, states)]
    else:
        out = list(out)
        if len(out) != len(states):
            raise ValueError("out must have one tensor per state")
        for o, x, s in zip(out, states, shapes):
            if o.device != dev or o.dtype != x.dtype or o.shape != s:
                raise ValueError(f"out must be {x.dtype} {tuple(s)} on {dev}")
            if any(n > 1 and a == 0 for n, a in zip(o.shape, o.stride())):
                raise ValueError("out must not be an expanded tensor")
    todo = [(x, o, d) for x, o, d in zip(states, out, dims) if o.numel()]
    status = status_word(check, dev) if todo else None
    for i in range(0, len(todo), N.MAX_STATES):
        part = todo[i:i + N.MAX_STATES]
        array = (N.State * len(part))()
        for s, (x, o, d) in zip(array, part):
            _describe(s, x, o, d, x.data_ptr(), o.data_ptr())
        call("rnnt_beam_reorder", dev, N.rnnt_beam_reorder, array, len(part), parents.data_ptr(),
             B, K, Ko, None if status is None or i else status.data_ptr(), stream_of(dev))
    finish("rnnt_beam_reorder", status, f"parents in [-1, {K})")
    return out
