"""What the label-side entry points share: argument checks, the current stream, the status word."""
from __future__ import annotations

import torch

from . import _native as N

DTYPES = {torch.float32: N.RNNT_F32, torch.float16: N.RNNT_F16, torch.bfloat16: N.RNNT_BF16}


def int32(name, t, device):
    if t.dtype != torch.int32:
        raise ValueError(f"{name} must be int32, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")


def stream_of(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def status_word(check, device):
    """The device word a checked call reports to (the call itself resets it)."""
    return torch.empty(1, dtype=torch.int32, device=device) if check else None


def call(where, device, fn, *args):
    if torch.cuda.current_device() == device.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc != N.RNNT_OK:
        raise N.RNNTError(rc, where)


def finish(where, status, wanted):
    if status is None:
        return
    code = int(status.item())
    if code == N.RNNT_INVALID_VALUE:
        raise ValueError(f"{where}: {N.status_string(code)} (wanted: {wanted})")
    if code != N.RNNT_OK:
        raise N.RNNTError(code, where)
