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


def few_values(V, values, dtype):
    """A row of few values, the larger ones first: all terms of a value share one error."""
    x = torch.empty(V)
    for i, v in enumerate(sorted(values, reverse=True)):
        x[i * V // len(values):] = v
    return x.to(dtype)


def beside(sums, whole, seed, n):
    """float32 numbers at and next to some of the running sums' shares of the whole."""
    at = np.random.default_rng(seed).integers(0, len(sums) - 1, size=n)
    u = (sums[at] / whole).astype(np.float32)
    u = np.concatenate([u, np.nextafter(u, np.float32(0)), np.nextafter(u, np.float32(1))])
    return u[u < 1]


VALUES = [(-0.9375, 0.0), (-6.5625, -5.625, 0.0), (-3.03125, -2.0, -1.046875, -0.09765625)]


def test_draw_in_equal_logits(program):
    """25000 equal terms on either side of a step: their errors add up."""
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.full((50000,), -6.5625)
        x[25000:], x[-1] = -5.625, 0.0
        check(program, x.to(dtype), [0.2791885435581207], dict())


@pytest.mark.parametrize("values", VALUES, ids=str)
def test_draws_beside_running_sums(program, values):
    for V, dtype in ((29, torch.float32), (203, torch.bfloat16), (1001, torch.float16), (20011, torch.bfloat16)):
        x = few_values(V, values, dtype)
        sums = np.cumsum(np.exp(x.double().numpy()))
        check(program, x, beside(sums, sums[-1], V, 3), dict())


@pytest.mark.parametrize("values", VALUES, ids=str)
def test_top_p_beside_running_sums(program, values):
    """The last id drawn is the last one kept."""
    for V, places in ((29, (0, 5, 13, 26, 27)), (1001, (3, 250, 499, 750, 998)), (5003, (1200, 2500, 4100))):
        x = few_values(V, values, torch.bfloat16)
        sums = np.cumsum(np.exp(x.double().numpy()))
        for at in places:
            for off in (-2e-8, -3e-9, 3e-9, 2e-8):
                check(program, x, [MOST], dict(top_p=sums[at] / sums[-1] + off))
