"""Beam search on the joiner's outputs: ``rnnt_beam_select`` (the best extensions of a batch's
hypotheses) and ``rnnt_beam_reorder`` (the states of the selected ones)."""
from __future__ import annotations

import struct
from functools import lru_cache

import torch

from . import _native as N
from ._host import DTYPES as _DT
from ._host import call, finish, int32, status_word

_F32, _I32 = torch.float32, torch.int32


@lru_cache(maxsize=256)
def _workspace_size(B, K, V, beam, dt, index):
    with torch.cuda.device(index):
        return N.rnnt_beam_workspace_size(B, K, V, beam, dt)


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
    itself alone, with its score unchanged and token -1, whatever its logits
    hold; one of score -inf offers nothing.  The order is that of the exact
    values to 40 bits (a returned score is within 5e-6 of its value and one
    float32 rounding; a candidate below float32's range keeps its place, its token
    and its parent, and has score -inf), ties go to the lowest hypothesis, then the
    lowest token.
    ``parents`` says which hypothesis each result extends (for
    :func:`rnnt_beam_reorder`); places left over get score -inf, token -1,
    parent -1.  ``check`` reads the device status word (one synchronisation) and
    raises on scores or logits that are NaN or +inf; without it a hypothesis
    that holds one offers nothing.  Not differentiable.
    """
    dt = _DT.get(logits.dtype)
    device = logits.device
    if device.type != "cuda":
        raise ValueError("logits must be a CUDA tensor")
    if dt is None:
        raise ValueError(f"logits must be float32, float16 or bfloat16, got {logits.dtype}")
    if logits.dim() != 3:
        raise ValueError("logits must be (B, K, V)")
    B, K, V = shape = logits.shape
    if not 1 <= K <= N.MAX_BEAM or not 1 <= V <= N.MAX_BEAM_VOCAB:
        raise ValueError(f"logits must have 1 to {N.MAX_BEAM} hypotheses and 1 to "
                         f"{N.MAX_BEAM_VOCAB} outputs")
    beam = K if beam is None else int(beam)
    if not 1 <= beam <= N.MAX_BEAM:
        raise ValueError(f"beam must be in [1, {N.MAX_BEAM}]")
    if scores.dtype is not _F32 or scores.shape != shape[:2] or scores.device != device:
        raise ValueError(f"scores must be float32 ({B}, {K}) on {device}")
    if finished is not None:
        if finished.dtype not in (torch.bool, torch.uint8) or finished.shape != shape[:2] \
                or finished.device != device:
            raise ValueError(f"finished must be bool or uint8 ({B}, {K}) on {device}")
        finished = finished.contiguous()
    if logits.is_neg() or scores.is_neg():  # their memory holds the negatives
        logits, scores = logits.resolve_neg(), scores.resolve_neg()
    scores = scores.contiguous()
    # three allocations: the code of the second and third is in the caches, while that of the views
    # that would share one is not (7 us instead of 11)
    out_scores = torch.empty((B, beam), dtype=_F32, device=device)
    tokens = torch.empty((B, beam), dtype=_I32, device=device)
    parents = torch.empty((B, beam), dtype=_I32, device=device)
    if not B:
        return out_scores, tokens, parents
    item, row, step = logits.stride()
    if V > 1 and step != 1:
        logits = logits.contiguous()
        item, row, step = logits.stride()
    nbytes = _workspace_size(B, K, V, beam, dt, device.index)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    status = status_word(device) if check else None
    call("rnnt_beam_select", device, N.rnnt_beam_select, logits.data_ptr(), dt, B, K, V,
         item, row, scores.data_ptr(), None if finished is None else finished.data_ptr(), beam,
         1 if fused_log_softmax else 0, out_scores.data_ptr(), tokens.data_ptr(),
         parents.data_ptr(), ws.data_ptr() if nbytes else None, nbytes,
         None if status is None else status.data_ptr())
    if check:
        finish("rnnt_beam_select", status, "finite scores or -inf, logits below +inf and not NaN")
    return out_scores, tokens, parents


@lru_cache(maxsize=256)
def _describe(shape, xs, os, size, d):
    """(row bytes, n, strides of x, strides of out, batch and beam strides) of a state's rows: its
    batch axis is d, its beam axis d + 1, the trailing axes that are adjacent in both tensors
    are a row, and up to three axes are left.  Strides go in as elements and come out as bytes."""
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
    axes += [(1, 0, 0, False)] * (3 - len(axes))
    return (row * size, tuple(a[0] for a in axes), tuple(a[1] * size for a in axes),
            tuple(a[2] * size for a in axes), xs[d] * size, xs[d + 1] * size, os[d] * size,
            os[d + 1] * size)


# rnnt_state_t behind its two pointers (row_bytes, n, padding, strides, batch and beam strides)
_ROWS = struct.Struct("=q3i4x3q3q4q")
_POINTERS = struct.Struct("=QQ")


def _pack(rows):
    r = rows
    return _ROWS.pack(r[0], *r[1], *r[2], *r[3], *r[4:])


@lru_cache(maxsize=1024)
def _plan(shape, strides, dtype, d, B, K, Ko):
    """(shape of a new result, packed rows or None if there are none) of a state by its layout;
    raises if it is no state of (B, K)."""
    shape = tuple(shape)
    if d < 0:
        d += len(shape)
    if not 0 <= d < len(shape) - 1:
        raise ValueError("batch_dim must leave a beam axis behind it")
    if shape[d] != B or shape[d + 1] != K or K < 1:
        raise ValueError(f"states must have a batch axis of {B} and, behind it, a beam axis "
                         "of the same size, at least 1")
    new = shape[:d + 1] + (Ko,) + shape[d + 2:]
    out, n = [], 1
    for m in reversed(new):
        out.append(n)
        n *= max(m, 1)
    out = tuple(reversed(out))
    return new, None if 0 in new else _pack(_describe(shape, strides, out, dtype.itemsize, d))


def _apart(states, out):
    """Raises where a result shares memory with a state or is given twice, as one C call does by
    itself: for more states than it takes, of which an early one's result could be a late one's
    source."""
    def span(x):
        at = x.data_ptr()
        return at, at + x.element_size() * (1 + sum((n - 1) * a for n, a in zip(x.shape, x.stride())))

    src = [span(x) for x in states if x.numel()]
    dst = [span(y) for y in out if y.numel()]
    if len({a for a, _ in dst}) < len(dst):
        raise ValueError("out holds a tensor twice")
    if any(a < d and c < b for a, b in dst for c, d in src):
        raise ValueError("out must not share memory with states")


def rnnt_beam_reorder(states, parents: torch.Tensor, batch_dim=0, out=None, check: bool = True):
    """The states of the selected hypotheses: ``new[.., b, k, ..] = old[.., b, parents[b, k], ..]``.

    ``states`` is a sequence of CUDA tensors of any type, each with a batch axis
    of size B and, behind it, a beam axis of size K: ``batch_dim`` says where
    (one number, or one per state; a recurrent state (layers, B, K, width) has
    batch_dim 1).  ``parents`` (B, K') int32 is what
    :func:`rnnt_beam_select` returned; the results have K' in the place of K,
    and zeros where the parent is -1.  ``out`` gives tensors to write to (they
    must not share memory with ``states`` or one another: keep two sets and swap them);
    without it the results are new contiguous tensors.  Views are read with
    their strides: the filled part of a cache need not be copied out first.
    ``check`` reads the device status word (one synchronisation) and raises on
    parents outside [-1, K); without it such a parent counts as -1.  Not
    differentiable.
    """
    states = list(states)
    if not states:
        return []
    device = states[0].device
    if device.type != "cuda":
        raise ValueError("states must be CUDA tensors")
    if parents.dtype is not _I32 or parents.device != device:
        int32("parents", parents, device)
    if parents.dim() != 2 or parents.shape[1] < 1:
        raise ValueError("parents must be (B, K') with K' >= 1")
    B, Ko = parents.shape
    dims = [batch_dim] * len(states) if isinstance(batch_dim, int) else batch_dim
    if len(dims) != len(states):
        raise ValueError("batch_dim must be one number, or one per state")
    first = states[0].shape
    d = dims[0] + len(first) if dims[0] < 0 else dims[0]
    if not 0 <= d < len(first) - 1:
        raise ValueError("batch_dim must leave a beam axis behind it")
    K = first[d + 1]
    if out is not None:
        out = list(out)
        if len(out) != len(states):
            raise ValueError("out must have one tensor per state")
        if len(out) > N.MAX_STATES:
            _apart(states, out)
    results, rows = [], []
    for i, x in enumerate(states):
        if x.device != device:
            raise ValueError(f"states must be on {device}")
        if x.is_conj() or x.is_neg():
            states[i] = x = x.resolve_conj().resolve_neg()
        dtype = x.dtype
        new, packed = _plan(x.shape, x.stride(), dtype, dims[i], B, K, Ko)
        if out is None:
            y = torch.empty(new, dtype=dtype, device=device)
        else:
            y = out[i]
            if y.device != device or y.dtype != dtype or y.shape != new:
                raise ValueError(f"out must be {dtype} {new} on {device}")
            if y.is_conj() or y.is_neg():
                raise ValueError("out must not be a conjugate or negative view")
            if any(n > 1 and a == 0 for n, a in zip(new, y.stride())):
                raise ValueError("out must not be an expanded tensor")
            if packed is not None:
                d = dims[i] + x.dim() if dims[i] < 0 else dims[i]
                packed = _pack(_describe(tuple(x.shape), x.stride(), y.stride(), x.element_size(), d))
        results.append(y)
        if packed is not None:
            rows.append(_POINTERS.pack(x.data_ptr(), y.data_ptr()) + packed)
    if not rows:
        return results
    parents = parents.contiguous()
    status = status_word(device) if check else None
    for i in range(0, len(rows), N.MAX_STATES):
        part = rows[i:i + N.MAX_STATES]
        call("rnnt_beam_reorder", device, N.rnnt_beam_reorder, b"".join(part), len(part),
             parents.data_ptr(), B, K, Ko, None if status is None or i else status.data_ptr())
    if out is not None:                     # what autograd saved of them is no longer so
        torch.autograd.graph.increment_version([y for y in results if not y.is_inference()])
    if status is not None:
        finish("rnnt_beam_reorder", status, f"parents in [-1, {K})")
    return results
