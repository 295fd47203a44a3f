"""Drawing labels, what needs no GPU: refusals at the C boundary."""
import pytest
import torch

import rnn_transducer_loss_gb300 as pkg
from rnn_transducer_loss_gb300 import _native as N
from rnn_transducer_loss_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return N.load()


def sample(**kw):
    a = dict(logits=1 << 20, dt=N.RNNT_F32, B=2, K=4, V=30, batch_stride=120, beam_stride=30, scores=4096,
             random=4352, finished=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, fused=1,
             out_scores=8192, out_tokens=8448, status_dev=None, stream=None)
    a.update(kw)
    return N.rnnt_sample(*a.values())


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(scores=None), dict(random=None), dict(out_scores=None), dict(out_tokens=None),
    dict(dt=3), dict(B=0), dict(K=0), dict(V=0), dict(V=(1 << 20) + 1), dict(B=1 << 16, K=1 << 16),
    dict(batch_stride=-1), dict(beam_stride=-1), dict(batch_stride=1 << 61), dict(beam_stride=1 << 60),
    dict(temperature=0.0), dict(temperature=float("nan")), dict(temperature=1e5), dict(top_k=-1),
    dict(top_p=0.0), dict(top_p=1.5), dict(top_p=float("nan")), dict(min_p=-1.0), dict(min_p=2.0),
    dict(logits=(1 << 20) + 1), dict(scores=4097), dict(random=4354), dict(out_scores=8193), dict(out_tokens=8450),
    dict(status_dev=1), dict(out_scores=4096), dict(out_tokens=8192), dict(out_tokens=(1 << 20) + 512),
    dict(finished=8192),
], ids=str)
def test_sample_refuses(bad):
    assert sample(**bad) == N.RNNT_INVALID_VALUE


def test_no_cpu_form():
    x = torch.zeros(2, 3, 10)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rnnt_sample(x, x[:, :, 0], x[:, :, 0])
