"""The selection's kernels on the CPU: their source, compiled as plain C++ (``cuda_on_cpu.h``), a
fiber for each CUDA thread.  What a GPU must never be given (an invariant broken on purpose) and
what should fail before it is run there can be looked at here."""
import os
import re
import subprocess

import numpy as np
import torch

from rnn_transducer_loss_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
NO_MINIMUM = "no_minimum"


def device_source():
    """The kernels of rnnt_beam.cu and what chooses their splits, inline assembly as C++."""
    s = open(os.path.join(B.CSRC, "rnnt_beam.cu")).read()
    s = s[s.index("// ------------------------------------------------- order-preserving integers"):
          s.index("bool select_ok(")]

    def body(name, text):
        nonlocal s
        s, n = re.subn(r"__device__ __forceinline__ " + name + r"\([^)]*\) \{.*?\n\}\n",
                       lambda m: m.group(0).split("{")[0] + "{ return " + text + "; }\n", s,
                       flags=re.S)
        assert n == 1, name

    body("float ex2", "std::exp2(x)")
    body("float2 fma2", "make_float2(std::fma(a.x, b.x, c.x), std::fma(a.y, b.y, c.y))")
    body("float2 add2", "make_float2(a.x + b.x, a.y + b.y)")
    body("uint4 load_stream", "*at")
    s, n = re.subn(r"extern __shared__ (?:__align__\(16\) )?(\w+) (\w+)\[\];",
                   r"\1* \2 = reinterpret_cast<\1*>(g_fiber->cta->dynamic);", s)
    assert n == 2 and "asm" not in s
    return re.sub(r"#pragma unroll.*", "", s)


def build(folder):
    with open(os.path.join(folder, "device.inc"), "w") as f:
        f.write(device_source())
    out = os.path.join(folder, "beam_on_cpu")
    subprocess.run(["g++", "-std=c++20", "-O1", "-ffp-contract=off", "-fno-strict-aliasing", "-w",
                    "-I", folder, "-I", HERE, "-I", os.path.join(B.ROOT, "include"),
                    os.path.join(HERE, "beam_on_cpu.cpp"), "-o", out], check=True)
    return out


def select(program, logits, scores, beam, finished=None, fused=True, splits=0, skip=0, plant=None):
    """(scores, tokens, parents, status) of one item: logits (K, V) of a torch type, scores (K,).
    `splits`: of a row in the two-launch kernels, 0 for what the host
    chooses, -1 for what it does where no cluster has more than 8 blocks; `skip`: elements
    between a 16-byte boundary and the first row."""
    K, V = logits.shape
    dt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[logits.dtype]
    raw = logits.contiguous().view(torch.int32 if dt == 0 else torch.int16).numpy()
    head = np.array([dt, K, V, beam, fused, splits, skip, finished is not None,
                     plant == NO_MINIMUM], dtype=np.int32)
    fin = np.zeros(K, np.uint8) if finished is None else np.asarray(finished, np.uint8)
    data = (head.tobytes() + np.asarray(scores, np.float32).tobytes() + fin.tobytes() +
            np.zeros(skip, raw.dtype).tobytes() + raw.tobytes())
    r = subprocess.run([program], input=data, stdout=subprocess.PIPE, timeout=600, check=True)
    status = np.frombuffer(r.stdout, np.int32, 2)
    assert status[1] == 1, "threads wait for others that never come"
    at = 8
    parts = []
    for t in (np.float32, np.int32, np.int32):
        parts.append(np.frombuffer(r.stdout, t, beam, at))
        at += 4 * beam
    return (*parts, int(status[0]))
