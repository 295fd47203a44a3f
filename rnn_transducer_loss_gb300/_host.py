"""What the label-side entry points share: argument checks, the current stream, the status word.

A small call's time is the host's (a Python call, the checks, one ctypes call, a launch), so
these take few steps: one combined test of the arguments, whose parts are looked at again
only to say what is wrong.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import _native as N

DTYPES = {torch.float32: N.RNNT_F32, torch.float16: N.RNNT_F16, torch.bfloat16: N.RNNT_BF16}

current_device = torch._C._cuda_getDevice
stream_of = torch._C._cuda_getCurrentRawStream      # of a device index, as an integer


def differentiated(t):
    """Whether autograd has to see a call on t: for its backward pass, or, where a forward-mode
    level is open, for the error that a tangent meets (a call past autograd would drop it)."""
    return t.requires_grad and torch.is_grad_enabled() or forward_ad._current_level >= 0


def int32(name, t, device):
    if t.dtype != torch.int32:
        raise ValueError(f"{name} must be int32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")


def status_word(device):
    """The device word a checked call reports to (the call itself resets it)."""
    return torch.empty(1, dtype=torch.int32, device=device)


def call(where, device, fn, *args):
    """fn(*args, stream) with `device` current."""
    index = device.index
    if current_device() == index:
        rc = fn(*args, stream_of(index))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream_of(index))
    if rc:
        raise N.RNNTError(rc, where)


def finish(where, status, wanted):
    code = int(status.item())
    if code == N.RNNT_INVALID_VALUE:
        raise ValueError(f"{where}: {N.status_string(code)} (wanted: {wanted})")
    if code != N.RNNT_OK:
        raise N.RNNTError(code, where)
