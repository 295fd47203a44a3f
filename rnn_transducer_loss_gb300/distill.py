"""Learning from a teacher: ``rnnt_top_logits`` (the largest logits of a teacher's lattice rows and
what remains) and ``rnnt_distill_loss`` (the divergence of a student's rows from them, with its
gradient); ``RNNTDistillLoss`` is its module form.

The student's logits, lengths and reductions are those of ``rnnt_loss``; a teacher's rows are kept
as k logits, k ids and one number instead of the whole vocabulary:
``rnnt_distill_loss(student, *rnnt_top_logits(teacher, k)[:2], T, U)``.
"""
from __future__ import annotations

import torch

from . import _native as N
from ._host import DTYPES as _DT
from ._host import call, differentiated, finish, int32, status_word, without_gradient

_F32, _I32 = torch.float32, torch.int32


def _logits(name, t):
    dt = _DT.get(t.dtype)
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if dt is None:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    if t.dim() not in (2, 4):
        raise ValueError(f"{name} must be 2-D (sum_b T_b*(U_b+1), V) or 4-D "
                         "(B, max_T, max_U+1, V)")
    if not 1 <= t.shape[-1] <= N.MAX_TOP_VOCAB:
        raise ValueError(f"{name} must have 1 to {N.MAX_TOP_VOCAB} outputs")
    return dt


def _lengths(logit_lengths, target_lengths, device, B):
    for name, t in (("logit_lengths", logit_lengths), ("target_lengths", target_lengths)):
        if t.dtype is not _I32 or t.device != device:
            int32(name, t, device)
        if t.dim() != 1 or t.shape[0] != (logit_lengths.shape[0] if B is None else B):
            raise ValueError("lengths must be (B,), B the batch size")
    return logit_lengths.contiguous(), target_lengths.contiguous()


def _temperature(temperature):
    temperature = float(temperature)
    if not 1e-4 <= temperature <= 1e4:
        raise ValueError("temperature must be in [1e-4, 1e4]")
    return temperature


def rnnt_top_logits(logits: torch.Tensor, k: int, logit_lengths: torch.Tensor | None = None,
                    target_lengths: torch.Tensor | None = None, temperature: float = 1.0,
                    check: bool = True):
    """What a student needs of a teacher's rows: (values, ids, rest).

    ``logits`` is the compact (N, V) matrix or the padded (B, max_T, max_U+1, V)
    tensor of ``rnnt_loss``, float32, float16 or bfloat16.  ``values`` (..., k) of
    its type are the k largest logits above -inf of every row, best first, equal ones by
    id; ``ids`` (..., k) int32 say which outputs they are; places left over hold
    -inf and -1.  ``rest`` (...) float32 is the log-sum-exp of the remaining logits /
    ``temperature``, -inf where there are none.  With padded logits the (B,) int32
    lengths leave rows outside their sequence unused, and empty.  ``check``
    reads the device status word (one synchronisation) and raises on rows that hold
    NaN or +inf and on lengths outside the tensor; without it such a row is empty and such
    a length the nearer bound.  Not differentiable: a backward pass through the results raises, and
    so does a forward-mode derivative.
    """
    return without_gradient("rnnt_top_logits", (logits,),
                            _top_logits(logits, k, logit_lengths, target_lengths, temperature, check))


def _top_logits(logits, k, logit_lengths, target_lengths, temperature, check):
    dt = _logits("logits", logits)
    device, V = logits.device, logits.shape[-1]
    k = int(k)
    if not 1 <= k <= min(V, N.MAX_TOP):
        raise ValueError(f"k must be in [1, {min(V, N.MAX_TOP)}]")
    temperature = _temperature(temperature)
    B = T = U = 0
    if (logit_lengths is None) != (target_lengths is None):
        raise ValueError("logit_lengths and target_lengths go together")
    if logit_lengths is not None:
        if logits.dim() != 4:
            raise ValueError("lengths go with padded (4-D) logits; compact ones have no other rows")
        B, T, U = logits.shape[0], logits.shape[1], logits.shape[2] - 1
        logit_lengths, target_lengths = _lengths(logit_lengths, target_lengths, device, B)
    if logits.is_neg():                     # its memory holds the negatives
        logits = logits.resolve_neg()
    logits = logits.contiguous()
    lead = logits.shape[:-1]
    values = torch.empty((*lead, k), dtype=logits.dtype, device=device)
    ids = torch.empty((*lead, k), dtype=_I32, device=device)
    rest = torch.empty(lead, dtype=_F32, device=device)
    rows = rest.numel()
    if not rows:
        return values, ids, rest
    status = status_word(device) if check else None
    call("rnnt_top_logits", device, N.rnnt_top_logits, logits.data_ptr(), dt, rows, V,
         None if logit_lengths is None else logit_lengths.data_ptr(),
         None if target_lengths is None else target_lengths.data_ptr(), B, T, U, k, temperature,
         values.data_ptr(), ids.data_ptr(), rest.data_ptr(),
         None if status is None else status.data_ptr())
    if check:
        finish("rnnt_top_logits", status, "logits below +inf and not NaN, lengths in the layout")
    return values, ids, rest


def rnnt_distill_loss_forward(logits, teacher_logits, teacher_ids, logit_lengths, target_lengths,
                              teacher_rest=None, temperature=1.0, weight=1.0, reduction="mean",
                              want_grad=True, check=True):
    """One call: (loss[B] float32, reduced float32 scalar, grad or None, workspace)."""
    dt = _logits("logits", logits)
    device, V = logits.device, logits.shape[-1]
    lead = logits.shape[:-1]
    if reduction not in N.REDUCTIONS:
        raise ValueError(f"reduction must be one of {tuple(N.REDUCTIONS)}")
    teacher_dt = _DT.get(teacher_logits.dtype)
    if teacher_dt is None or teacher_logits.device != device:
        raise ValueError(f"teacher_logits must be float32, float16 or bfloat16 on {device}")
    k = teacher_logits.shape[-1] if teacher_logits.dim() else 0
    if teacher_logits.shape[:-1] != lead or not 1 <= k <= N.MAX_TOP:
        raise ValueError(f"teacher_logits must be {(*lead, 'k')}, k in [1, {N.MAX_TOP}]")
    if teacher_ids.dtype is not _I32 or teacher_ids.device != device:
        int32("teacher_ids", teacher_ids, device)
    if teacher_ids.shape != teacher_logits.shape:
        raise ValueError("teacher_ids must have the shape of teacher_logits")
    if teacher_rest is not None and (teacher_rest.dtype is not _F32 or teacher_rest.shape != lead
                                     or teacher_rest.device != device):
        raise ValueError(f"teacher_rest must be float32 {tuple(lead)} on {device}")
    padded = logits.dim() == 4
    logit_lengths, target_lengths = _lengths(logit_lengths, target_lengths, device,
                                             lead[0] if padded else None)
    B = logit_lengths.shape[0]
    temperature, weight = _temperature(temperature), float(weight)
    if not -1e30 < weight < 1e30:
        raise ValueError("weight must be finite and below 1e30")
    if not B:
        raise ValueError("the batch must not be empty")
    T, U = (lead[1], lead[2] - 1) if padded else (0, 0)

    def plain(t):
        return (t.resolve_neg() if t.is_neg() else t).contiguous()

    logits, teacher_logits = plain(logits), plain(teacher_logits)
    if logits.data_ptr() % 16:              # a contiguous view that begins between two vectors
        logits = logits.clone()
    teacher_ids = teacher_ids.contiguous()
    if teacher_rest is not None:
        teacher_rest = plain(teacher_rest)
    loss = torch.empty(B, dtype=_F32, device=device)
    reduced = torch.empty((), dtype=_F32, device=device)
    grad = torch.empty_like(logits) if want_grad else None
    rows = logits.numel() // V
    if not rows:
        raise ValueError("logits must have rows")
    nbytes = N.rnnt_distill_workspace_size(B, rows)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    status = status_word(device) if check else None
    call("rnnt_distill_loss", device, N.rnnt_distill_loss, logits.data_ptr(), dt, rows, V,
         teacher_logits.data_ptr(), teacher_dt, teacher_ids.data_ptr(),
         None if teacher_rest is None else teacher_rest.data_ptr(), k, logit_lengths.data_ptr(),
         target_lengths.data_ptr(), B, 1 if padded else 0, T, U, temperature, weight,
         N.REDUCTIONS[reduction], loss.data_ptr(), reduced.data_ptr(),
         grad.data_ptr() if want_grad else None, ws.data_ptr(), nbytes,
         None if status is None else status.data_ptr())
    if check:
        finish("rnnt_distill_loss", status,
               "T_b >= 0, U_b >= 0 within the layout, sum T_b*(U_b+1) rows of compact logits, "
               "different teacher_ids below V in a row, logits and rest below +inf and not NaN")
    return loss, reduced, grad, ws


class _Distill(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, teacher_logits, teacher_ids, logit_lengths, target_lengths,
                teacher_rest, temperature, weight, reduction, check):
        loss, reduced, ctx.grad, ctx.ws = rnnt_distill_loss_forward(
            logits, teacher_logits, teacher_ids, logit_lengths, target_lengths, teacher_rest,
            temperature, weight, reduction, ctx.needs_input_grad[0], check)
        ctx.per_sample = reduction == "none"
        ctx.used = False
        ctx.batch = logit_lengths.shape[0]
        return loss if ctx.per_sample else reduced

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out):
        if ctx.used:
            # The saved gradient was scaled in place by the first backward.
            raise RuntimeError("rnnt_distill_loss: backward can run only once per forward call "
                               "(the gradient buffer is scaled in place); recompute the loss "
                               "to differentiate again")
        grad, ws = ctx.grad, ctx.ws
        if grad is None:
            return (None,) * 10
        ctx.used, ctx.grad, ctx.ws = True, None, None
        factors = grad_out.detach().to(_F32).contiguous()
        V = grad.shape[-1]
        each = grad.shape[1] * grad.shape[2] if grad.dim() == 4 else 0
        call("rnnt_distill_grad_scale", grad.device, N.rnnt_distill_grad_scale, grad.data_ptr(),
             _DT[grad.dtype], grad.numel() // V, V, ctx.batch, each, ws.data_ptr(), ws.numel(),
             factors.data_ptr(), 1 if ctx.per_sample else 0)
        return (grad,) + (None,) * 9


def rnnt_distill_loss(logits: torch.Tensor, teacher_logits: torch.Tensor,
                      teacher_ids: torch.Tensor, logit_lengths: torch.Tensor,
                      target_lengths: torch.Tensor, teacher_rest: torch.Tensor | None = None,
                      temperature: float = 1.0, weight: float = 1.0, reduction: str = "mean",
                      check: bool = True) -> torch.Tensor:
    """Divergence of a student's lattice rows from a teacher's, differentiable in ``logits``.

    ``logits`` and the (B,) int32 lengths are those of ``rnnt_loss``: compact
    (sum_b T_b*(U_b+1), V) or padded (B, max_T, max_U+1, V), float32, float16 or bfloat16;
    ``teacher_logits`` and ``teacher_ids`` (int32) have k <= 64 places in the place of V,
    as ``rnnt_top_logits`` gives them (a negative id is an empty place).  Every row adds
    ``weight * temperature**2 * KL(p || q)``, p the softmax of the teacher's logits /
    ``temperature`` over the places, q that of the student's over the vocabulary.  With
    ``teacher_rest`` (float32, one number a row: the log-sum-exp of the teacher's
    remaining logits / ``temperature``) the outputs without a place are one more class of
    both.  A row whose teacher holds nothing adds nothing.  Returns float32
    per-sample sums (reduction="none") or their float32 sum or mean.

    The gradient is computed with the loss, in the type of ``logits``; backward multiplies
    it in place by the upstream gradient (nothing to do where that is 1: give the term's
    ``weight`` here), so it runs once per call.  A float16 gradient has then been rounded
    before a gradient scaler's factor: what the scaler is there to save may be 0 already, and
    the second pass reads and writes the whole gradient.  With a scaler, its scale belongs
    into the weight and the term behind the scaler:
    ``scaler.scale(loss) + rnnt_distill_loss(..., weight=w * scaler.get_scale())``.
    ``check`` reads the device status word (one
    synchronisation) and raises on lengths that do not fit, ids at or above V or twice in a
    row, and NaN or +inf; without it such an id's place counts as empty.  A step is captured
    into a CUDA graph with ``check=False`` and with no eager graph of the same leaf alive.
    The teacher is not differentiated, and forward-mode derivatives raise.
    """
    if torch.is_grad_enabled() and (teacher_logits.requires_grad or teacher_rest is not None
                                    and teacher_rest.requires_grad):
        raise ValueError("the teacher is not differentiated: detach teacher_logits and "
                         "teacher_rest")
    if differentiated(logits):
        return _Distill.apply(logits, teacher_logits, teacher_ids, logit_lengths, target_lengths,
                              teacher_rest, temperature, weight, reduction, check)
    loss, reduced, _, _ = rnnt_distill_loss_forward(
        logits, teacher_logits, teacher_ids, logit_lengths, target_lengths, teacher_rest,
        temperature, weight, reduction, False, check)
    return loss if reduction == "none" else reduced


class RNNTDistillLoss(torch.nn.Module):
    """Module form of :func:`rnnt_distill_loss`."""

    def __init__(self, temperature: float = 1.0, weight: float = 1.0, reduction: str = "mean",
                 check: bool = True):
        super().__init__()
        self.temperature, self.weight = temperature, weight
        self.reduction, self.check = reduction, check

    def forward(self, logits, teacher_logits, teacher_ids, logit_lengths, target_lengths,
                teacher_rest=None):
        return rnnt_distill_loss(logits, teacher_logits, teacher_ids, logit_lengths,
                                 target_lengths, teacher_rest, self.temperature, self.weight,
                                 self.reduction, self.check)
