"""GPU: draws whose borders lie next to running sums: tokens are those of the float64 form."""
import numpy as np
import pytest
import torch

import sample_ref as R
from rnn_transducer_loss_gb300 import rnnt_sample

pytestmark = pytest.mark.gpu
MOST = 1 - 2.0 ** -24
NUDGES = [(0, R.NEAR), (0, -R.NEAR), (R.NEAR, 0), (-R.NEAR, 0)]


def check(x, random, **kw):
    """A row drawn with each of the numbers."""
    random = np.asarray(random, np.float32)[None]
    x = x[None, None].expand(1, random.size, -1)
    _, tokens = rnnt_sample(x.cuda(), torch.zeros(random.shape, device="cuda"), torch.tensor(random, device="cuda"),
                            temperature=kw.get("tau", 1.0), top_p=kw.get("top_p", 1.0))
    tokens = tokens.cpu().numpy()
    args = (x.double().numpy(), np.zeros(random.shape), random.astype(np.float64))
    want = R.sample(*args, **kw)[1]
    ok = want == tokens
    for nudge in NUDGES:
        if not ok.all():
            ok |= R.sample(*args, nudge=nudge, **kw)[1] == tokens
    assert ok.all(), (tokens[~ok], want[~ok], random[~ok])


@pytest.mark.parametrize("top_p", [1 - 2.910e-7, 1 - 2.0e-7, 1 - 3.9e-7])
def test_border_in_a_tail_of_tiny_masses(top_p):
    head = torch.cat([torch.zeros(3000), torch.full((7000,), -0.8016451)])
    tail = torch.full((5000,), float(np.log(2.0 ** -33 * float(head.double().exp().sum()))))
    check(torch.cat([head, tail]), [MOST], top_p=top_p)


def test_border_in_a_crowd():
    x = torch.full((100000,), -22.3)
    x[:4] = torch.tensor([0.0, -0.37, -0.91, -0.53])
    check(x, [MOST], top_p=0.999995)


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


def test_draw_in_equal_logits():
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.full((50000,), -6.5625)
        x[25000:], x[-1] = -5.625, 0.0
        check(x.to(dtype), [0.2791885435581207])


@pytest.mark.parametrize("V", [29, 1024, 5000, 50000, 400000])
@pytest.mark.parametrize("values", VALUES, ids=str)
def test_draws_beside_running_sums(values, V):
    for tau in (1.0, 0.7):
        for dtype in (torch.float16, torch.bfloat16, torch.float32):
            x = few_values(V, values, dtype)
            sums = np.cumsum(np.exp(x.double().numpy() / tau))
            check(x, beside(sums, sums[-1], V, 20 if V < 100000 else 4), tau=tau)


@pytest.mark.parametrize("V", [29, 1024, 5000, 50000, 400000])
@pytest.mark.parametrize("values", VALUES, ids=str)
def test_top_p_beside_running_sums(values, V):
    """The last id drawn is the last one kept."""
    x = few_values(V, values, torch.bfloat16)
    sums = np.cumsum(np.exp(x.double().numpy()))
    for at in np.random.default_rng(V).integers(0, V - 1, size=4):
        for off in (-2e-8, -3e-9, 3e-9, 2e-8):
            check(x, [MOST, 0.5], top_p=sums[at] / sums[-1] + off)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_largest_vocabulary(dtype):
    V = 1 << 20
    x = torch.randn(V, generator=torch.Generator().manual_seed(3)) * 2
    x = x.to(dtype)
    for kw in (dict(), dict(top_p=0.9), dict(tau=0.5, top_p=0.99)):
        check(x, [0.0, 0.3, 0.77, MOST], **kw)
    check(few_values(V, VALUES[1], dtype), [0.0, 0.3, 0.77, MOST], top_p=0.9)
    # and between two 16-byte units
    u = torch.tensor([[0.4]], device="cuda")
    a, b = (rnnt_sample(t[None, None], u * 0, u, top_p=0.8)[1] for t in (x.cuda(), torch.cat([x[:1], x]).cuda()[1:]))
    assert torch.equal(a, b)
