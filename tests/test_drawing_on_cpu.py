"""The drawing kernel's source on the CPU (``on_cpu/drawing.py``), every access checked for its alignment
and its array's bounds, against the float64 form."""
import numpy as np
import pytest
import torch

import sample_ref as R
from on_cpu import drawing as D

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    return D.build(str(tmp_path_factory.mktemp("drawing")))


def logits(kind, K, V, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(1, K, V, generator=g) * 2
    x[..., 0] += 4
    if kind == "masked":
        x[torch.rand(1, K, V, generator=g) < 0.7] = -float("inf")
        x[0, 0] = -float("inf")
    if kind == "lowest":
        x[torch.rand(1, K, V, generator=g) < 0.7] = torch.finfo(dtype).min
    if kind == "ties":
        x = (x * 0.8).round()
    if kind == "equal":
        x.fill_(-2.5)
    random = torch.rand(1, K, generator=g)
    random[0, :3] = torch.tensor([0.0, 1 - 2.0 ** -24, 0.5])[:K]
    return x.to(dtype), -20 * torch.rand(1, K, generator=g), random


def same(program, x, scores, random, kw, **form):
    out, tokens, status = D.sample(program, x, scores, random, **kw, **form)
    args = (x.double().numpy(), scores.double().numpy(), random.double().numpy())
    ok = R.sample(*args, **kw)[1] == tokens
    for nudge in ((0, R.NEAR), (0, -R.NEAR), (R.NEAR, 0), (-R.NEAR, 0)):       # draws next to a border
        ok |= R.sample(*args, nudge=nudge, **kw)[1] == tokens
    assert ok.all() and status == 0


FILTERS = [dict(), dict(tau=0.7, top_k=40), dict(tau=0.8, top_p=0.95), dict(top_p=0.9, min_p=0.002),
           dict(tau=0.5, top_k=200, top_p=0.99, min_p=0.001), dict(top_k=1)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", ["plain", "masked", "lowest", "ties", "equal"])
@pytest.mark.parametrize("V,threads,here", [(2, None, True), (29, None, True), (700, 128, True)])
def test_rows(program, V, threads, here, kind, dtype):
    x, scores, random = logits(kind, 3, V, DT[dtype], V)
    for kw in FILTERS:
        same(program, x, scores, random, kw, skip=3 * V % 8, threads=threads, here=here)


@pytest.mark.parametrize("here", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_rows(program, dtype, here):
    """Histograms in more than one turn (more equal elements than a list holds), and rows that are read
    from the cache."""
    for kind in ("plain", "equal"):
        x, scores, random = logits(kind, 1, 3001, DT[dtype], 5)
        for kw in (dict(top_p=0.9), dict(top_k=700)):
            same(program, x, scores, random, kw, threads=512, here=here)
