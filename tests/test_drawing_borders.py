"""Draws whose borders lie next to running sums, on the CPU (``on_cpu/drawing.py``): tokens are those of the
float64 form."""
import numpy as np
import pytest
import torch

import sample_ref as R
from on_cpu import drawing as D

MOST = 1 - 2.0 ** -24


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return D.build(str(tmp_path_factory.mktemp("borders")))


def check(program, x, random, kw, **form):
    """A row drawn with each of the numbers."""
    random = np.asarray(random, np.float32)[None]
    x = x[None, None].expand(1, random.size, -1)
    out, tokens, status = D.sample(program, x, np.zeros_like(random), random, **kw, **form)
    args = (x.double().numpy(), np.zeros(random.shape), random.astype(np.float64))
    ok = R.sample(*args, **kw)[1] == tokens
    for nudge in ((0, R.NEAR), (0, -R.NEAR), (R.NEAR, 0), (-R.NEAR, 0)):
        ok |= R.sample(*args, nudge=nudge, **kw)[1] == tokens
    assert ok.all() and status == 0, (tokens, R.sample(*args, **kw)[1])


@pytest.mark.parametrize("top_p", [1 - 2.910e-7, 1 - 2.0e-7, 1 - 3.9e-7])
def test_border_in_a_tail_of_tiny_masses(program, top_p):
    """Masses below 2^-32 of the whole count as nothing in a histogram, so that its bin lies beside the
    border: a bisection by sums of pairs, towards a target that is one too."""
    head = torch.cat([torch.zeros(3000), torch.full((7000,), -0.8016451)])
    tail = torch.full((5000,), float(np.log(2.0 ** -33 * float(head.double().exp().sum()))))
    check(program, torch.cat([head, tail]), [MOST], dict(top_p=top_p), threads=512)


def test_border_in_a_crowd(program):
    """Equal masses are all rounded the same way, in rows that are read from the cache."""
    x = torch.full((100000,), -22.3)
    x[:4] = torch.tensor([0.0, -0.37, -0.91, -0.53])
    check(program, x, [MOST], dict(top_p=0.999995), threads=512, here=False)
