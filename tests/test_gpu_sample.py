"""GPU: drawing labels against the float64 form: equal tokens, scores within one rounding."""
import numpy as np
import pytest
import torch

import label_ref as L
import sample_ref as R
from rnn_transducer_loss_gb300 import (rnnt_beam_reorder, rnnt_beam_select, rnnt_embed, rnnt_sample,
                                       rnnt_top_logits)

pytestmark = pytest.mark.gpu
DT = L.DTYPES
LEAST, MOST = 0.0, 1.0 - 2.0 ** -24
NUDGES = [(a * R.NEAR, b * R.NEAR) for a, b in ((0, 1), (0, -1), (1, 0), (-1, 0), (1, 1), (1, -1), (-1, 1), (-1, -1))]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make(kind, B, K, V, dtype, seed):
    g = gen(seed)
    x = torch.randn(B, K, V, device="cuda", generator=g) * 2
    x[..., 0] += 4
    if kind == "masked":
        x[torch.rand(B, K, V, device="cuda", generator=g) < 0.7] = -float("inf")
        x[0, 0] = -float("inf")
    if kind == "lowest":
        x[torch.rand(B, K, V, device="cuda", generator=g) < 0.7] = torch.finfo(dtype).min
        x[0, 0] = torch.finfo(dtype).min
    if kind == "ties":
        x = (x * 0.8).round()
    if kind == "equal":
        x.fill_(-2.5)
    if kind == "one":
        x.fill_(-30.0)
        x[..., V // 3] = 5.0
    if kind == "wide":
        x *= 30
    if kind == "sorted":
        x = x.sort(dim=2, descending=bool(seed % 2)).values
    x = x.to(dtype)
    scores = -20 * torch.rand(B, K, device="cuda", generator=g)
    random = torch.rand(B, K, device="cuda", generator=g)
    flat = random.view(-1)
    flat[:1] = LEAST
    if flat.numel() > 1:
        flat[1:2] = MOST
        flat[2:3] = 0.5
    return x, scores, random


def check(x, scores, random, finished=None, fused=True, **kw):
    got = rnnt_sample(x, scores, random, finished=finished, fused_log_softmax=fused,
                      temperature=kw.get("tau", 1.0), top_k=kw.get("top_k"), top_p=kw.get("top_p", 1.0),
                      min_p=kw.get("min_p", 0.0), check=kw.get("check", True))
    kw.pop("check", None)
    args = (L.f64(x), L.f64(scores), L.f64(random))
    want = R.sample(*args, finished=finished, fused=fused, **kw)
    assert got[0].dtype == torch.float32 and got[1].dtype == torch.int32
    tokens = got[1].cpu().numpy()
    for nudge in NUDGES:                    # of draws next to a border
        off = tokens != want[1]
        if not off.any():
            break
        other = R.sample(*args, finished=finished, fused=fused, nudge=nudge, **kw)
        for w, o in zip(want, other):
            w[off] = o[off]
    assert np.array_equal(tokens, want[1]), (np.argwhere(tokens != want[1])[:5],
                                             tokens[tokens != want[1]][:5], want[1][tokens != want[1]][:5])
    out = L.f64(got[0])
    assert np.array_equal(np.isneginf(out), np.isneginf(want[0]) | (want[0] < torch.finfo(torch.float32).min))
    some = np.isfinite(out)
    out, exact = out[some], want[0][some]
    assert (np.abs(out - exact) <= np.abs(exact) * L.U32 * 1.001 + (5e-6 if fused else 0)).all()
    return got


SHAPES = [(1, 1, 1), (1, 4, 2), (2, 3, 16), (32, 10, 29), (3, 5, 130), (1, 4, 1024), (16, 2, 1001),
          (2, 8, 2056), (4, 8, 5000), (2, 3, 9001), (1, 2, 16384), (2, 4, 50000), (1, 2, 50001), (1, 1, 70000)]
FILTERS = [dict(), dict(tau=0.7, top_k=40), dict(tau=0.8, top_p=0.95), dict(top_p=0.9, min_p=0.002),
           dict(tau=1.3, top_k=7, top_p=0.5), dict(min_p=0.1), dict(tau=0.5, top_k=200, top_p=0.99, min_p=0.001),
           dict(top_k=1), dict(tau=3.0, top_p=0.999), dict(tau=0.05), dict(tau=100.0, top_k=300)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sample(shape, dtype):
    kinds = ("plain", "masked", "lowest", "ties", "equal", "one", "wide", "sorted")
    for i, kind in enumerate(kinds):
        x, scores, random = make(kind, *shape, DT[dtype], 7 * i + shape[2])
        for kw in FILTERS:
            check(x, scores, random, **kw)


def test_sample_log_probabilities():
    x, scores, random = make("plain", 6, 4, 5000, torch.float32, 1)
    check(torch.log_softmax(x, -1), scores, random, fused=False, tau=0.8, top_p=0.9)
    check(torch.log_softmax(x, -1).bfloat16(), scores, random, fused=False, top_k=12)


@pytest.mark.parametrize("V", [29, 1024, 50000])
def test_sample_every_token_by_its_share(V):
    """Equally spaced numbers draw each token as often as its probability says, to one draw."""
    n = 4096
    x = torch.randn(1, 1, V, device="cuda", generator=gen(2)).expand(1, n, V)
    random = (torch.arange(n, device="cuda") / n)[None]
    for kw in (dict(), dict(top_k=5), dict(top_p=0.7), dict(temperature=0.3, min_p=0.05)):
        _, tokens = rnnt_sample(x, torch.zeros(1, n, device="cuda"), random, **kw)
        e = np.exp(L.f64(x)[0, 0] / kw.get("temperature", 1.0))
        order = np.argsort(-e, kind="stable")
        if "top_k" in kw:
            e[order[5:]] = 0
        if "top_p" in kw:
            s = e[order]
            e[order[np.cumsum(s) - s >= 0.7 * s.sum()]] = 0
        if "min_p" in kw:
            e[e < 0.05 * e.max()] = 0
        share = np.bincount(tokens[0].cpu().numpy(), minlength=V) / n
        assert (np.abs(share - e / e.sum()) <= 1.0 / n + 1e-9).all()


def test_sample_borders():
    """Numbers and masses that fall exactly on a border."""
    for V in (4, 16, 1024, 4096, 32768):
        x = torch.zeros(1, 9, V, device="cuda")
        scores = torch.zeros(1, 9, device="cuda")
        random = torch.tensor([[0.0, 0.25, 0.5, 0.75, 2.0 ** -24, 1 - 2.0 ** -24, 0.125, 0.375, 0.3]], device="cuda")
        for kw in (dict(), dict(top_p=0.5), dict(top_p=0.25, top_k=V // 2), dict(min_p=1.0), dict(top_k=V),
                   dict(top_k=2 ** 31 - 1), dict(top_k=V - 1)):
            check(x, scores, random, **kw)


def test_sample_finished_and_lost():
    x, scores, random = make("plain", 4, 6, 1024, torch.float16, 3)
    finished = torch.rand(4, 6, device="cuda", generator=gen(4)) < 0.4
    finished[0, 0], finished[0, 1] = True, False
    scores[0, 1] = -float("inf")
    x[finished] = float("nan")
    random = random.clone()
    random[finished] = float("nan")
    want = R.sample(np.nan_to_num(L.f64(x)), L.f64(scores), np.nan_to_num(L.f64(random)), finished=finished)
    for f in (finished, finished.to(torch.uint8) * 3):
        got = rnnt_sample(x, scores, random, finished=f)
        assert np.array_equal(got[1].cpu().numpy(), want[1])
        assert torch.equal(got[0][finished], scores[finished])
        assert got[0][0, 1] == -float("inf") and got[1][0, 1] == -1


@pytest.mark.parametrize("V", [29, 1024, 5000, 50000])
def test_sample_checks(V):
    x, scores, random = make("plain", 2, 3, V, torch.float32, 5)
    base = rnnt_sample(x, scores, random)

    def changed(t, at, value):
        t = t.clone()
        t[at] = value
        return t

    nan, inf = float("nan"), float("inf")
    for args in ((changed(x, (1, 1, V - 1), nan), scores, random), (changed(x, (1, 1, 0), inf), scores, random),
                 (x, changed(scores, (1, 1), nan), random), (x, changed(scores, (1, 1), inf), random),
                 (x, scores, changed(random, (1, 1), 1.0)), (x, scores, changed(random, (1, 1), -0.5)),
                 (x, scores, changed(random, (1, 1), nan))):
        with pytest.raises(ValueError, match="wanted"):
            rnnt_sample(*args)
        got = rnnt_sample(*args, check=False)
        assert got[1][1, 1] == -1 and got[0][1, 1] == -inf
        same = torch.ones(2, 3, dtype=torch.bool)
        same[1, 1] = False
        assert torch.equal(got[0].cpu()[same], base[0].cpu()[same])
        assert torch.equal(got[1].cpu()[same], base[1].cpu()[same])


def same(got, want):
    """Equal tokens; scores that are both within 5e-6 and half a step of the exact ones, so within twice
    that of one another (the terms of a row's sum are grouped by where it lies in memory)."""
    a, b = L.f64(got[0]), L.f64(want[0])
    return torch.equal(got[1], want[1]) and (np.abs(a - b) <= 2 * (5e-6 + np.abs(b) * L.U32 * 1.001)).all()


def test_sample_views():
    """Rows anywhere in a 16-byte unit, other strides, expanded and negative views."""
    for dtype in DT.values():
        x, scores, random = make("plain", 4, 5, 301, dtype, 6)
        kw = dict(temperature=0.9, top_p=0.9)
        want = rnnt_sample(x, scores, random, **kw)
        wide = torch.zeros(4, 7, 333, device="cuda", dtype=dtype)
        wide[:, 1:6, 5:306] = x
        for y in (wide[:, 1:6, 5:306], x.transpose(0, 1).contiguous().transpose(0, 1),
                  x.transpose(1, 2).contiguous().transpose(1, 2), torch.stack([x, x], 3)[..., 1]):
            assert same(rnnt_sample(y, scores, random, **kw), want)
    n = torch.complex(x.float(), x.float()).conj().imag
    a = rnnt_sample(n, torch.complex(scores, scores).conj().imag, random)
    b = rnnt_sample(-x.float(), -scores, random)
    assert same(a, b)
    one = rnnt_sample(x[:1, :1].expand(4, 5, 301), scores, random)
    two = rnnt_sample(x[:1, :1].repeat(4, 5, 1), scores, random)
    assert same(one, two)


def test_sample_refusals():
    x, scores, random = make("plain", 2, 3, 20, torch.float32, 7)
    for kw in (dict(logits=x[0]), dict(logits=x.double()), dict(logits=x.cpu()), dict(scores=scores[:1]),
               dict(scores=scores.half()), dict(random=random.double()), dict(random=random.cpu()),
               dict(random=random[:, :2]), dict(finished=torch.zeros(2, 3, device="cuda")),
               dict(temperature=0.0), dict(temperature=float("nan")), dict(top_k=0), dict(top_k=-1), dict(top_p=0.0),
               dict(top_p=1.1), dict(min_p=-0.1), dict(min_p=1.5), dict(min_p=float("nan"))):
        with pytest.raises(ValueError):
            rnnt_sample(**{**dict(logits=x, scores=scores, random=random), **kw})
    empty = rnnt_sample(x[:0], scores[:0], random[:0])
    assert empty[0].shape == (0, 3) and empty[1].shape == (0, 3)


def test_sample_captured():
    x, scores, random = make("plain", 4, 4, 1024, torch.float16, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rnnt_sample(x, scores, random, check=False)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = rnnt_sample(x, scores, random, temperature=0.8, top_p=0.9, check=False)
    torch.cuda.synchronize()
    for seed in range(3):
        random.copy_(torch.rand(4, 4, device="cuda", generator=gen(seed)))
        g.replay()
        want = rnnt_sample(x, scores, random, temperature=0.8, top_p=0.9)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_sample_far_rows():
    """Hypotheses beyond 2^31 elements."""
    V = 1024
    x = torch.zeros(1, (1 << 21) + 64, V, device="cuda", dtype=torch.float16)
    K = x.shape[1]
    x[0, -64:] = torch.randn(64, V, device="cuda", generator=gen(9)).half()
    scores, random = torch.zeros(1, K, device="cuda"), torch.rand(1, K, device="cuda", generator=gen(10))
    got = rnnt_sample(x, scores, random, top_k=50)
    want = rnnt_sample(x[:, -64:].clone(), scores[:, -64:], random[:, -64:], top_k=50)
    assert all(torch.equal(a[:, -64:], b) for a, b in zip(got, want))


def test_drawing_loop():
    """Drawn label sequences, step by step: embedding, a recurrent joiner, the draw, states in the order
    of the beam selection that may follow; the log-probabilities add up to the sequences'."""
    B, K, V, D, steps = 2, 3, 29, 16, 6
    g = gen(11)
    emb = torch.randn(V, D, device="cuda", generator=g)
    joint = torch.randn(V, D, device="cuda", generator=g)
    tokens = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    scores = torch.zeros(B, K, device="cuda")
    total, finished = np.zeros((B, K)), torch.zeros(B, K, dtype=torch.bool, device="cuda")
    history = torch.zeros(B, K, steps, dtype=torch.int32, device="cuda")
    for step in range(steps):
        h = rnnt_embed(emb, tokens).tanh()
        logits = h @ joint.t()
        random = torch.rand(B, K, device="cuda", generator=g)
        want = R.sample(L.f64(logits), L.f64(scores), L.f64(random), 0.9, None, 0.95, 0.0, finished)
        scores, tokens = rnnt_sample(logits, scores, random, 0.9, top_p=0.95, finished=finished)
        assert np.array_equal(tokens.cpu().numpy(), want[1])
        total = want[0]
        history[:, :, step] = tokens
        finished = finished | (tokens == 0)
    assert (np.abs(L.f64(scores) - total) <= 1e-4).all()
    _, _, parents = rnnt_beam_select(torch.zeros(B, K, 1, device="cuda"), scores, finished=torch.ones_like(finished))
    best, = rnnt_beam_reorder([history], parents)
    order = scores.argsort(dim=1, descending=True, stable=True)
    assert torch.equal(best, torch.take_along_dim(history, order[:, :, None], 1))
    assert rnnt_top_logits(logits.view(-1, V), 4)[1][0, 0] == logits.view(-1, V)[0].argmax()
