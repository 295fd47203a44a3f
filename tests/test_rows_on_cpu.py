"""Rows of a tensor in shared memory: what the copies read, and what they leave (``on_cpu/rows_on_cpu.cpp``)."""
import os
import subprocess

import pytest

from on_cpu import drawing as D
from rnn_transducer_loss_gb300 import build as B


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    folder = str(tmp_path_factory.mktemp("rows"))
    with open(os.path.join(folder, "sample_device.inc"), "w") as f:
        f.write(D.device_source())
    out = os.path.join(folder, "rows_on_cpu")
    subprocess.run(["g++", "-std=c++20", "-O1", "-ffp-contract=off", "-fno-strict-aliasing", "-w",
                    "-fsanitize=alignment,bounds", "-fno-sanitize-recover=all",
                    "-I", folder, "-I", D.HERE, "-I", os.path.join(B.ROOT, "include"),
                    os.path.join(D.HERE, "rows_on_cpu.cpp"), "-o", out], check=True)
    return out


@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 8, 9, 17, 40])
@pytest.mark.parametrize("dtype", [0, 1, 2], ids=["f32", "f16", "bf16"])
def test_copies_stay_in_the_tensor(program, dtype, V):
    """Rows shorter than a 16-byte unit share the tensor's first and last one."""
    for skip in range(4 if dtype == 0 else 8):
        for rows in (1, 2, 5, 16):
            r = subprocess.run([program, str(dtype), str(V), str(rows), str(skip)])
            assert r.returncode == 0, (skip, rows, r.returncode)
