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
