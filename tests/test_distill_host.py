"""Learning from a teacher, what needs no GPU: refusals at the C boundary, workspace sizes."""
import pytest
import torch

import rnn_transducer_loss_gb300 as pkg
from rnn_transducer_loss_gb300 import _native as N
from rnn_transducer_loss_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()
    return N.load()


def top(**kw):
    a = dict(logits=1 << 20, dt=N.RNNT_F32, rows=12, V=30, logit_lengths=4096, target_lengths=4352,
             B=2, max_T=3, max_U=1, k=4, temperature=1.0, values=1 << 21, ids=1 << 22, rest=1 << 23,
             status_dev=None, stream=None)
    a.update(kw)
    return N.rnnt_top_logits(*a.values())


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(values=None), dict(ids=None), dict(rest=None), dict(dt=3), dict(V=0),
    dict(V=(1 << 20) + 1), dict(rows=0), dict(k=0), dict(k=31), dict(V=100, k=65),
    dict(logit_lengths=None), dict(target_lengths=None), dict(B=0), dict(rows=11), dict(max_T=0),
    dict(max_U=-1), dict(temperature=0.0), dict(temperature=float("nan")), dict(temperature=2e4),
    dict(values=1 << 20), dict(ids=(1 << 21) + 16), dict(rest=(1 << 22) + 4), dict(logits=(1 << 20) + 2),
    dict(ids=(1 << 22) + 2), dict(rest=(1 << 23) + 1), dict(logit_lengths=4097), dict(status_dev=4098),
    dict(rows=1 << 62, logit_lengths=None, target_lengths=None),
    dict(B=2 ** 31 - 1, max_T=2 ** 31 - 1, max_U=2 ** 31 - 2, rows=1 << 60),
], ids=str)
def test_top_refuses(bad):
    assert top(**bad) == N.RNNT_INVALID_VALUE


def distill(**kw):
    a = dict(logits=1 << 20, dt=N.RNNT_F16, rows=12, V=30, teacher=1 << 21, teacher_dt=N.RNNT_F32,
             ids=1 << 22, rest=1 << 23, k=4, logit_lengths=4096, target_lengths=4352, B=2, padded=1,
             max_T=3, max_U=1, temperature=1.0, weight=1.0, reduction=1, loss=8192, reduced=8448,
             grad=1 << 24, workspace=1 << 25, workspace_bytes=1 << 20, status_dev=None, stream=None)
    a.update(kw)
    return N.rnnt_distill_loss(*a.values())


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(teacher=None), dict(ids=None), dict(logit_lengths=None),
    dict(target_lengths=None), dict(loss=None), dict(workspace=None), dict(dt=-1), dict(teacher_dt=7),
    dict(V=0), dict(V=(1 << 20) + 1), dict(rows=0), dict(rows=13), dict(k=0), dict(k=65), dict(B=0),
    dict(max_T=0), dict(max_U=-1), dict(temperature=-1.0), dict(temperature=float("inf")),
    dict(weight=float("nan")), dict(weight=1e30), dict(reduction=3), dict(reduction=-1),
    dict(logits=(1 << 20) + 8), dict(grad=(1 << 24) + 2), dict(grad=1 << 20), dict(grad=(1 << 20) + 64),
    dict(grad=(1 << 21) - 64), dict(workspace=(1 << 25) + 16), dict(workspace=1 << 24),
    dict(teacher=(1 << 21) + 2), dict(ids=(1 << 22) + 1), dict(rest=(1 << 23) + 2), dict(loss=8193),
    dict(reduced=8196), dict(loss=1 << 23), dict(reduced=4356), dict(status_dev=2),
    dict(padded=0, rows=1 << 61),
], ids=str)
def test_distill_refuses(bad):
    assert distill(**bad) == N.RNNT_INVALID_VALUE


def test_distill_workspace():
    n = N.rnnt_distill_workspace_size(2, 12)
    assert n > 0 and n % 256 == 0
    assert distill(workspace_bytes=n - 1) == N.RNNT_WORKSPACE_TOO_SMALL
    big = N.rnnt_distill_workspace_size(16, 500_000)
    assert 4 * 500_000 <= big <= 4 * 500_000 + 4096
    for args in ((0, 12), (2, 0), (-1, 5)):
        with pytest.raises(N.RNNTError):
            N.rnnt_distill_workspace_size(*args)


def scale(**kw):
    a = dict(grad=1 << 20, dt=N.RNNT_BF16, rows=12, V=30, B=2, rows_each=6, workspace=1 << 21,
             workspace_bytes=1 << 20, factors=4096, per_sample=1, stream=None)
    a.update(kw)
    return N.rnnt_distill_grad_scale(*a.values())


@pytest.mark.parametrize("bad", [
    dict(grad=None), dict(workspace=None), dict(factors=None), dict(dt=3), dict(rows=0), dict(V=0),
    dict(B=0), dict(rows_each=-1), dict(rows_each=5), dict(rows_each=4), dict(rows_each=24),
    dict(grad=(1 << 20) + 4), dict(workspace=(1 << 21) + 128), dict(factors=4098),
], ids=str)
def test_scale_refuses(bad):
    assert scale(**bad) == N.RNNT_INVALID_VALUE


def test_scale_workspace():
    assert scale(workspace_bytes=64) == N.RNNT_WORKSPACE_TOO_SMALL


def test_limits_match_the_header():
    hdr = open(B.HDR).read()
    assert f"#define RNNT_MAX_TOP {N.MAX_TOP}\n" in hdr
    assert "#define RNNT_MAX_TOP_VOCAB (1 << 20)" in hdr and N.MAX_TOP_VOCAB == 1 << 20


def test_no_cpu_form():
    x = torch.zeros(4, 10)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    n = torch.ones(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rnnt_top_logits(x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.rnnt_distill_loss(x, x[:, :2], ids, n, n * 0)
    with pytest.raises(ValueError, match="CUDA"):
        pkg.RNNTDistillLoss()(x.requires_grad_(), x[:, :2].detach(), ids, n, n * 0)
