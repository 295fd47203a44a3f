"""The drawing kernel on the CPU, as ``tests.on_cpu`` does it for the beam selection: its source as plain
C++, a fiber for each CUDA thread, every access checked for its alignment and its array's bounds."""
import os
import re
import subprocess

import numpy as np
import torch

from rnn_transducer_loss_gb300 import build as B

HERE = os.path.dirname(os.path.abspath(__file__))


def device_source():
    """What the kernel needs of rnnt_rows.cuh, and rnnt_sample.cu up to its launches; inline assembly
    as C++."""
    rows = open(os.path.join(B.CSRC, "rnnt_rows.cuh")).read()
    rows = rows[rows.index("constexpr unsigned kAll"):rows.index("// Device-side memory limits")]
    rows = re.sub(r"__device__ __forceinline__ uint32_t shared_at.*?(?=// A row in a stage)",
                  "", rows, flags=re.S)        # copies: in the harness
    s = open(os.path.join(B.CSRC, "rnnt_sample.cu")).read()
    s = rows + s[s.index("// ------------------------------------------------------------ pairs of floats"):
                 s.index("template <typename T>\nvoid launch_sample")]

    def body(name, text):
        nonlocal s
        s, n = re.subn(r"__device__ __forceinline__ " + name + r"\([^)]*\) \{.*?\n\}\n",
                       lambda m: m.group(0).split("{")[0] + "{ return " + text + "; }\n", s, flags=re.S)
        assert n == 1, name

    body("float ex2", "std::exp2(x)")
    body("float max_nan", "a != a ? a : b != b ? b : a > b ? a : b")
    body("float warp_max", "warp_reduced(x, [](float a, float b) { return fmaxf(a, b); })")
    body("float warp_max_nan", "warp_reduced(x, max_nan)")
    body("float reciprocal", "1.0f / x")
    body("float2 fma2", "make_float2(std::fma(a.x, b.x, c.x), std::fma(a.y, b.y, c.y))")
    body("float2 mul2", "make_float2(a.x * b.x, a.y * b.y)")
    body("float2 add2", "make_float2(a.x + b.x, a.y + b.y)")
    s = re.sub(r"__device__ __forceinline__ void pack\(.*?\n\}\n", "", s, flags=re.S)      # of results
    s, n = re.subn(r"extern __shared__ uint4 stage\[\];",
                   "uint4* stage = reinterpret_cast<uint4*>(g_fiber->cta->dynamic);", s)
    assert n == 1 and "asm" not in s
    return re.sub(r"#pragma unroll.*", "", s)


def build(folder):
    with open(os.path.join(folder, "sample_device.inc"), "w") as f:
        f.write(device_source())
    out = os.path.join(folder, "sample_on_cpu")
    subprocess.run(["g++", "-std=c++20", "-O1", "-ffp-contract=off", "-fno-strict-aliasing", "-w",
                    "-fsanitize=alignment,bounds", "-fno-sanitize-recover=all",
                    "-I", folder, "-I", HERE, "-I", os.path.join(B.ROOT, "include"),
                    os.path.join(HERE, "sample_on_cpu.cpp"), "-o", out], check=True)
    return out


def sample(program, logits, scores, random, tau=1.0, top_k=0, top_p=1.0, min_p=0.0, fused=True, skip=0,
           threads=None, here=True):
    """(scores, tokens, status) of logits (B, K, V) of a torch type; `skip`: elements between a 16-byte
    boundary and the first row; `threads`, `here`: the kernel's form, as the host chooses by default."""
    n, K, V = logits.shape
    dt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}[logits.dtype]
    raw = logits.contiguous().view(torch.int32 if dt == 0 else torch.int16).numpy()
    if threads is None:
        size = V * (4 if dt == 0 else 2)
        threads = 128 if size <= 4 << 10 else 256 if size <= 32 << 10 else 512
    head = np.array([dt, n, K, V, top_k or 0, fused, skip, threads, here], dtype=np.int32)
    data = (head.tobytes() + np.array([tau, top_p, min_p]).tobytes() + np.asarray(scores, np.float32).tobytes() +
            np.asarray(random, np.float32).tobytes() + np.zeros(skip, raw.dtype).tobytes() + raw.tobytes())
    r = subprocess.run([program], input=data, stdout=subprocess.PIPE, timeout=900, check=True)
    status = np.frombuffer(r.stdout, np.int32, 2)
    assert status[1] == 1, "threads wait for others that never come"
    out = np.frombuffer(r.stdout, np.float32, n * K, 8).reshape(n, K)
    return out, np.frombuffer(r.stdout, np.int32, n * K, 8 + 4 * n * K).reshape(n, K), int(status[0])
