"""GPU: label embedding, its gradient, beam selection and reordering against float64 forms."""
import numpy as np
import pytest
import torch

import label_ref as R
from rnn_transducer_loss_gb300 import (RNNTEmbedding, rnnt_beam_reorder, rnnt_beam_select,
                                       rnnt_embed, rnnt_embed_grad, rnnt_loss)

pytestmark = pytest.mark.gpu
DT = R.DTYPES


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make_tokens(B, S, V, seed, pad=True):
    """(tokens, lengths): some ids -1, lengths from 0 to S, values past them out of range."""
    rng = np.random.default_rng(seed)
    tokens = rng.integers(0, V, size=(B, S))
    if pad and S > 2:
        tokens[rng.random((B, S)) < 0.1] = -1
    lengths = rng.integers(0, S + 1, size=B)
    lengths[0] = S
    if B > 1:
        lengths[1] = 0
    for b in range(B):
        tokens[b, lengths[b]:] = V + 7 + b
    return tokens, lengths


EMBED = [  # B, S, V, D, start, with lengths, scale
    (1, 1, 1, 1, None, False, 1.0), (1, 1, 29, 8, None, False, 2.5), (3, 5, 29, 301, 0, True, 17.35),
    (2, 0, 7, 16, -1, False, 1.0), (4, 33, 1000, 64, 5, True, 0.1), (2, 9, 50, 2048, None, True, 3.0),
    (2, 3, 11, 8200, -11, True, 1.0), (300, 4, 64, 6, None, True, -0.7), (5, 100, 513, 130, 2, True, 8.0),
    (64, 16, 5000, 512, 0, True, 22.6),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", EMBED, ids=str)
def test_embed(case, dtype):
    B, S, V, D, start, some, scale = case
    tokens, lengths = make_tokens(B, S, V, 3) if some else (
        np.random.default_rng(3).integers(0, V, size=(B, S)), None)
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(V, D, device="cuda", dtype=DT[dtype], generator=g)
    got = rnnt_embed(w, i32(tokens), None if lengths is None else i32(lengths), start=start,
                     scale=scale)
    ids = R.place_ids(tokens, lengths, start, V)
    want = R.embed(R.f64(w), ids, scale)
    assert got.dtype == w.dtype and tuple(got.shape) == want.shape
    assert (np.abs(R.f64(got) - want) <= R.embed_bound(want, w.dtype)).all()
    assert (R.f64(got)[ids < 0] == 0).all()


GRAD = EMBED + [
    (2, 1023, 3, 24, 1, False, 1.5),        # few ids, each of them over many tiles
    (1, 4000, 1, 5, None, False, 1.0),      # one id
    (9, 1000, 2500, 32, 0, True, 1.0),      # two digits, two blocks
    (1, 2048, 700, 40, None, False, 1.0), (1, 2049, 700, 40, None, False, 1.0),
    (1, 4096, 700, 40, None, False, 1.0),   # the most places of the one-launch kernel
    (1, 4097, 700, 40, None, False, 1.0),   # and one more
    (1, 5000, 1, 5, None, False, 1.0),      # one id, over tiles
    (5, 1000, 3, 24, 1, False, 1.5),        # few ids, each of them over many tiles
    (9, 1000, 40, 301, None, False, 1.0),   # ids of 5 to 9 tiles, odd rows
    (16, 290, 9000, 260, 3, True, 2.0),     # ids of one place or none
    (2, 1023, 1, 33, 0, False, 0.5), (7, 290, 9000, 260, 3, True, 2.0),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", GRAD, ids=str)
def test_embed_grad(case, dtype):
    B, S, V, D, start, some, scale = case
    tokens, lengths = make_tokens(B, S, V, 4) if some else (
        np.random.default_rng(4).integers(0, V, size=(B, S)), None)
    ids = R.place_ids(tokens, lengths, start, V)
    g = torch.Generator(device="cuda").manual_seed(6)
    go = torch.randn(*ids.shape, D, device="cuda", dtype=DT[dtype], generator=g)
    go[torch.as_tensor(ids < 0, device="cuda")] = float("nan")      # padding is not read
    args = (go, i32(tokens), V, None if lengths is None else i32(lengths))
    got = rnnt_embed_grad(*args, start=start, scale=scale)
    want, mass, n = R.embed_grad(np.nan_to_num(R.f64(go)), ids, V, scale)
    assert got.dtype == go.dtype and tuple(got.shape) == (V, D)
    err = np.abs(R.f64(got) - want)
    assert (err <= R.grad_bound(want, mass, n, go.dtype)).all(), np.nanmax(err)
    assert (R.f64(got)[n == 0] == 0).all()
    again = rnnt_embed_grad(*args, start=start, scale=scale)
    assert torch.equal(got, again)


@pytest.mark.parametrize("V,D,N", [(5_000_000, 2, 3000), (5_000_000, 2, 5000), (70, 4, 200_000), (9000, 4, 150_000)])
def test_embed_grad_many(V, D, N):
    """Two digits of one launch's sort, three of the cluster's; more places than its threads hold at
    a time."""
    g = torch.Generator(device="cuda").manual_seed(N)
    tokens = torch.randint(0, V, (1, N), device="cuda", dtype=torch.int32, generator=g)
    go = torch.randint(-8, 9, (1, N, D), device="cuda", generator=g).float()
    got = rnnt_embed_grad(go, tokens, V)
    want = np.zeros((V, D))
    np.add.at(want, tokens[0].cpu().numpy(), R.f64(go)[0])
    assert np.array_equal(R.f64(got), want)           # small integers: every sum is exact


def test_embed_views():
    """A column slice of a table, a transposed one, strided and expanded tokens, strided lengths."""
    g = torch.Generator(device="cuda").manual_seed(9)
    big = torch.randn(40, 103, device="cuda", generator=g)
    tokens = torch.randint(0, 40, (6, 20), device="cuda", dtype=torch.int32, generator=g)
    lengths = torch.randint(0, 10, (12,), device="cuda", dtype=torch.int32, generator=g)
    for w in (big[:, 3:67], big[:, :64], big[1::2, 5:70], big.half().t()[:, ::2][:60, :20]):
        t = tokens % w.shape[0]
        for tok in (t, t[:, ::2], t[:1].expand(6, 20), t[:, 3:13]):
            n = lengths[::2].clamp(max=tok.shape[1])
            got = rnnt_embed(w, tok, n, start=-1, scale=2.0)
            want = rnnt_embed(w.contiguous(), tok.contiguous(), n.contiguous(), start=-1, scale=2.0)
            assert torch.equal(got, want)
            go = torch.randn(want.shape, device="cuda", generator=g).to(w.dtype)
            a = rnnt_embed_grad(go, tok, w.shape[0], n, start=-1)
            b = rnnt_embed_grad(go.transpose(0, 1).contiguous().transpose(0, 1), tok.contiguous(),
                                w.shape[0], n.contiguous(), start=-1)
            assert torch.equal(a, b)


def test_embed_refuses_on_device():
    w = torch.randn(10, 4, device="cuda")
    for tokens, lengths in (([[3, 10]], None), ([[3, 4]], [3]), ([[3, 4]], [-1])):
        n = None if lengths is None else i32(lengths)
        with pytest.raises(ValueError):
            rnnt_embed(w, i32(tokens), n)
        with pytest.raises(ValueError):
            rnnt_embed_grad(torch.ones(1, 2, 4, device="cuda"), i32(tokens), 10, n)
    got = rnnt_embed(w, i32([[3, 10]]), check=False)
    assert torch.equal(got[0, 0], w[3]) and (got[0, 1] == 0).all()
    rnnt_embed(w, i32([[9, -5]]))


def test_embed_autograd():
    """Against the formula and, the lookup being linear, against differences."""
    V, D = 17, 12
    mod = RNNTEmbedding(V, D, start=0, scale=D ** 0.5, device="cuda")
    tokens, lengths = make_tokens(4, 7, V, 11)
    c = torch.randn(4, 8, D, device="cuda")
    out = mod(i32(tokens), i32(lengths))
    (out * c).sum().backward()
    ids = R.place_ids(tokens, lengths, 0, V)
    want, mass, n = R.embed_grad(R.f64(c), ids, V, D ** 0.5)
    assert (np.abs(R.f64(mod.weight.grad) - want) <= R.grad_bound(want, mass, n, c.dtype)).all()
    w = R.f64(mod.weight)
    for v, d in ((0, 0), (5, 3), (16, 11)):
        up, down = w.copy(), w.copy()
        up[v, d] += 0.5
        down[v, d] -= 0.5
        diff = ((R.embed(up, ids, D ** 0.5) - R.embed(down, ids, D ** 0.5)) * R.f64(c)).sum()
        assert abs(diff - R.f64(mod.weight.grad)[v, d]) <= 1e-5 * max(1.0, mass[v, d])
    mod.weight.grad = None                      # an expanded upstream gradient
    mod(i32(tokens), i32(lengths)).sum().backward()
    ones, mass, n = R.embed_grad(np.ones((4, 8, D)), ids, V, D ** 0.5)
    assert (np.abs(R.f64(mod.weight.grad) - ones) <= R.grad_bound(ones, mass, n, c.dtype)).all()
    with torch.no_grad():
        assert not mod(i32(tokens)[:, :0]).requires_grad
    # twice: the gradient is linear in the upstream one, and its gradient is the lookup
    c.requires_grad_(True)
    g, = torch.autograd.grad(mod(i32(tokens), i32(lengths)), mod.weight, c, create_graph=True)
    a = torch.randn(V, D, device="cuda")
    back, = torch.autograd.grad(g, c, a)
    want = R.embed(R.f64(a), ids, D ** 0.5)
    assert (np.abs(R.f64(back) - want) <= R.embed_bound(want, a.dtype)).all()
    g2 = rnnt_embed_grad(c, i32(tokens), V, i32(lengths), start=0, scale=D ** 0.5)
    assert torch.equal(g2, g) and torch.equal(torch.autograd.grad(g2, c, a)[0], back)


def logits_of(B, K, V, dtype, seed, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, K, V, device="cuda", generator=g) * scale
    scores = -20.0 + 10.0 * torch.randn(B, K, device="cuda", generator=g).sort(1, True).values
    return x.to(DT[dtype]), scores


def check_select(x, scores, beam, finished=None, fused=True):
    got = rnnt_beam_select(x, scores, beam, finished, fused)
    want = R.select(R.f64(x), R.f64(scores), got[0].shape[1],
                    None if finished is None else finished.cpu().numpy(), fused)
    np.testing.assert_array_equal(got[2].cpu().numpy(), want[2])
    np.testing.assert_array_equal(got[1].cpu().numpy(), want[1])
    s = R.f64(got[0])
    empty = np.isinf(want[0])
    assert (s[empty] == -np.inf).all()
    with np.errstate(invalid="ignore"):
        assert (np.abs(s - want[0])[~empty] <= R.score_bound(want[0], fused)[~empty]).all()


SELECT = [  # B, K, V, beam
    (1, 1, 1, 1), (1, 1, 5, 8), (2, 3, 29, 3), (1, 4, 1024, 4), (3, 10, 1001, 7), (2, 64, 70, 64),
    (5, 1, 333, 1), (2, 5, 5003, 16), (1, 2, 20000, 64), (1, 3, 50021, 9), (40, 2, 64, 2),
]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", SELECT, ids=str)
def test_select(case, dtype, fused):
    B, K, V, beam = case
    x, scores = logits_of(B, K, V, dtype, V + K)
    if not fused:
        x = torch.log_softmax(x.float(), -1).to(x.dtype)
    check_select(x, scores, beam, None, fused)


@pytest.mark.parametrize("K", list(range(1, 20)))
def test_select_beams(K):
    """Every number of hypotheses about the largest cluster, with a narrower and a wider result."""
    x, scores = logits_of(3, K, 517, "f16", K)
    for beam in (1, K, 2 * K):
        check_select(x, scores, beam)


@pytest.mark.parametrize("K", [1, 2, 17])
@pytest.mark.parametrize("fused", [True, False])
def test_select_small_vocabularies(K, fused):
    """As many results as there are candidates, one less and one more, and lists of every length."""
    for V in (1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 17):
        x, scores = logits_of(2, K, V, "f32", V + 100 * K)
        if not fused:
            x = torch.log_softmax(x, -1)
        for beam in sorted({1, 2, max(V - 1, 1), V, V + 1, min(K * V, 64), min(K * V + 1, 64)}):
            check_select(x, scores, beam, None, fused)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [31, 4099])
def test_select_ties(dtype, V):
    """Equal logits and equal rows: the lowest hypothesis, then the lowest token; -0 equals 0."""
    x, scores = logits_of(3, 6, V, dtype, 2)
    x = (x * 0.5).round()
    x[0] = 0.0
    x[0, :, 1::2] = -0.0
    x[1] = x[1, :1]
    scores[:] = scores[:, :1]
    check_select(x, scores, 13)
    check_select(x, scores, 64)


@pytest.mark.parametrize("V", [3, 600, 17000])
def test_select_masked(V):
    """Masked outputs, rows that leave nothing, dead and finished hypotheses with NaN behind them."""
    x, scores = logits_of(4, 5, V, "f32", 8)
    x[:, :, V // 2:] = float("-inf")
    x[0, 1] = float("-inf")
    x[1] = float("-inf")
    finished = torch.zeros(4, 5, dtype=torch.bool, device="cuda")
    finished[0, 0] = finished[2] = True
    scores[3, 1:] = float("-inf")
    scores[2, 4] = float("-inf")
    x[0, 0] = x[2] = x[3, 1:] = float("nan")
    for beam in (1, 5, 64):
        check_select(x, scores, beam, finished)
        check_select(x, scores, beam, finished.to(torch.uint8) * 3)
        check_select(x, scores, beam, finished, fused=False)
    low = torch.finfo(torch.float32).min            # a mask of the type's lowest value
    x, scores = logits_of(2, 3, V, "f32", 9)
    x[:, :, 1:] = low
    x[1, 2] = low
    check_select(x, scores, 3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_select_crowded(dtype):
    """The best elements in few threads' hands, rising, falling and constant rows."""
    V = 16384
    x = torch.zeros(1, 4, V, device="cuda")
    x[0, 0] = torch.arange(V, device="cuda") / V
    x[0, 1] = -torch.arange(V, device="cuda") / V
    x[0, 2, ::2048] = 5.0
    x[0, 2, 1::2048] = 5.5
    x = x.to(DT[dtype])
    check_select(x, torch.tensor([[-1.0, -1.5, -2.0, -2.5]], device="cuda"), 64)


def test_select_close():
    """Candidates of different hypotheses a few units of 1e-7 apart."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(8, 1, 900, device="cuda", generator=g).expand(8, 6, 900).clone()
    x[:, 1:] += torch.randn(8, 5, 900, device="cuda", generator=g) * 1e-6
    scores = torch.full((8, 6), -0.5, device="cuda")
    scores += torch.randn(8, 6, device="cuda", generator=g) * 1e-7
    check_select(x, scores, 24)
    perm = torch.stack([torch.randperm(900, device="cuda", generator=g) for _ in range(6)])
    check_select(x.gather(2, perm.expand(8, 6, 900)), scores, 24)


def test_select_views():
    """Strided logits: every alignment of a row, hypotheses and items in other orders."""
    x, scores = logits_of(3, 4, 1100, "f16", 5)
    for n, y in enumerate((x[:, :, 1:1000], x[:, ::2, 7:], x[1:, :, :29],
                           x.transpose(0, 1)[:3, :, 2:900], x[:1].expand(3, 4, 1100),
                           x[:, :, ::3])):
        s = scores[:y.shape[0], :y.shape[1]]
        check_select(y, s.t().contiguous().t() if n % 2 else s, 5)


def test_select_refuses_on_device():
    x, scores = logits_of(2, 3, 40, "f32", 5)
    for bad in (float("nan"), float("inf")):
        y, s = x.clone(), scores.clone()
        y[1, 2, 39] = bad
        with pytest.raises(ValueError):
            rnnt_beam_select(y, scores)
        with pytest.raises(ValueError):
            rnnt_beam_select(y, scores, fused_log_softmax=False)
        s[0, 1] = bad
        with pytest.raises(ValueError):
            rnnt_beam_select(x, s)
        got = rnnt_beam_select(y, scores, check=False)
        want = R.select(R.f64(y), R.f64(scores), 3)
        np.testing.assert_array_equal(got[1].cpu().numpy(), want[1])
        np.testing.assert_array_equal(got[2].cpu().numpy(), want[2])


def plain_reorder(x, parents, d):
    rows = torch.arange(parents.shape[0], device=x.device)[:, None]
    at = parents.long()
    got = x.movedim((d, d + 1), (0, 1))[rows, at.clamp_min(0)]
    got[at < 0] = 0
    return got.movedim((0, 1), (d, d + 1))


STATES = [  # shape, batch_dim, type
    ((3, 4), 0, torch.float32), ((3, 4, 7), 0, torch.int32), ((2, 3, 4, 640), 1, torch.float16),
    ((3, 4, 2, 5, 33), 0, torch.bfloat16), ((3, 4, 5000), -3, torch.float64),
    ((2, 3, 3, 4, 6), 2, torch.uint8), ((3, 4, 3), 0, torch.bool), ((3, 4, 70001), 0, torch.int8),
]


def make_states():
    g = torch.Generator(device="cuda").manual_seed(2)
    return [torch.randint(0, 2 if t == torch.bool else 100, s, device="cuda", generator=g).to(t)
            for s, _, t in STATES]


@pytest.mark.parametrize("parents", [[[0, 1, 2, 3]] * 3, [[3, 3, -1], [0, 0, 0], [-1, -1, 2]],
                                     [[1], [2], [0]], [[2] * 9, [1] * 9, [0] * 9]])
def test_reorder(parents):
    states, p = make_states(), i32(parents)
    dims = [d for _, d, _ in STATES]
    got = rnnt_beam_reorder(states * 3, p, dims * 3)           # more than one launch
    for x, d, y in zip(states * 3, dims * 3, got):
        assert torch.equal(y, plain_reorder(x, p, d + x.dim() if d < 0 else d))
        assert y.is_contiguous()


def test_reorder_views():
    """Filled parts of caches, strided outputs and two sets in one tensor."""
    g = torch.Generator(device="cuda").manual_seed(3)
    cache = torch.randn(2, 3, 4, 2, 50, 16, device="cuda", generator=g)
    p = i32([[1, 1, -1], [3, 0, 2], [2, 3, 3]])
    for n in (0, 1, 17, 49):
        x = cache[0, :, :, :, :n]
        y, = rnnt_beam_reorder([x], p)
        assert torch.equal(y, plain_reorder(x, p, 0))
    x = cache[0, ..., 1:6]                                      # rows of 20 bytes, off 16
    y, = rnnt_beam_reorder([x], p)
    assert torch.equal(y, plain_reorder(x, p, 0))
    x = cache[0].transpose(3, 4)                                # nothing adjacent
    y, = rnnt_beam_reorder([x], p)
    assert torch.equal(y, plain_reorder(x, p, 0))
    to = torch.full((3, 3, 2, 50, 16), 7.0, device="cuda")
    want = plain_reorder(cache[0, :, :, :, 5:20], p, 0)
    got = rnnt_beam_reorder([cache[0, :, :, :, 5:20]], p, out=[to[:, :, :, 20:35]])
    assert got[0].data_ptr() == to[:, :, :, 20:35].data_ptr() and torch.equal(got[0], want)
    assert (to[:, :, :, :20] == 7).all() and (to[:, :, :, 35:] == 7).all()
    q = i32([[3, 2, 1, 0]] * 3)
    want = plain_reorder(cache[0], q, 0)
    rnnt_beam_reorder([cache[0]], q, out=[cache[1]])
    assert torch.equal(cache[1], want)


def test_reorder_refuses():
    x = torch.randn(3, 4, 8, device="cuda")
    for bad in (4, -2):
        p = i32([[0, 1], [bad, 0], [1, 1]])
        with pytest.raises(ValueError):
            rnnt_beam_reorder([x], p)
        y, = rnnt_beam_reorder([x], p, check=False)
        assert (y[1, 0] == 0).all() and torch.equal(y[0], x[0, :2])
    p = i32([[0, 1, 2, 3]] * 3)
    from rnn_transducer_loss_gb300 import _native as N
    with pytest.raises(N.RNNTError):
        rnnt_beam_reorder([x], p, out=[x])
    with pytest.raises(ValueError):
        rnnt_beam_reorder([x], p, out=[x[:, :, :1].expand(3, 4, 8)])
    y = torch.empty_like(x)
    with pytest.raises(N.RNNTError):                # one result for two states
        rnnt_beam_reorder([x, x], p, out=[y, y])
    a, b = rnnt_beam_reorder([x, x], p)             # one state twice
    assert torch.equal(a, b) and a.data_ptr() != b.data_ptr()
    assert rnnt_beam_reorder([], p) == []


def test_reorder_many_refuses():
    """More states than one launch takes: an early result must not be a late one's source."""
    x = [torch.randn(2, 3, 5, device="cuda") for _ in range(20)]
    y = [torch.empty_like(t) for t in x]
    p = i32([[2, 1, 0], [0, 0, -1]])
    for a, b in zip(x, rnnt_beam_reorder(x, p, out=y)):
        assert torch.equal(b, plain_reorder(a, p, 0))
    for bad in (y[:1] + y[2:] + y[:1], [x[18]] + y[1:], x):
        with pytest.raises(ValueError):
            rnnt_beam_reorder(x, p, out=bad)


def test_reorder_lazy_views():
    """Conjugate and negative views, whose memory holds other values than they do."""
    z = torch.randn(2, 3, 5, device="cuda", dtype=torch.complex64)
    p = i32([[2, 1, 0], [0, 0, 1]])
    a, b = rnnt_beam_reorder([z.conj(), z.conj().imag], p)
    rows = torch.arange(2, device="cuda")[:, None]
    assert torch.equal(a, z.conj().resolve_conj()[rows, p.long()])
    assert torch.equal(b, -z.imag[rows, p.long()])
    with pytest.raises(ValueError):
        rnnt_beam_reorder([z], p, out=[torch.empty_like(z).conj()])


def test_streams_and_graphs():
    """Another stream than the tensors' first one; two graphs, replayed in turn with new inputs."""
    w = torch.randn(60, 32, device="cuda")
    x, scores = logits_of(2, 4, 60, "f32", 4)
    states = [torch.randn(2, 2, 4, 32, device="cuda")]

    def step():
        s, t, p = rnnt_beam_select(x, scores, check=False)
        h, = rnnt_beam_reorder(states, p, 1, check=False)
        e = rnnt_embed(w, t, scale=2.0, check=False)
        return s, t, p, h, e, rnnt_embed_grad(e, t, 60, check=False)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(step(), on_side):
        assert torch.equal(a, b)
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for seed in (5, 6, 7):
        y, s = logits_of(2, 4, 60, "f32", seed)
        x.copy_(y)
        scores.copy_(s)
        w.normal_()
        want = step()
        for graph, out in zip(graphs, outs):
            graph.replay()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls that overlap on the device share nothing."""
    jobs = []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        tokens = torch.randint(0, 900, (4, 1100), device="cuda", dtype=torch.int32, generator=g)
        go = torch.randn(4, 1101, 64, device="cuda", generator=g)
        x, scores = logits_of(3, 20, 30000, "f16", seed)
        jobs.append((tokens, go, x, scores))

    def run(job):
        tokens, go, x, scores = job
        return (rnnt_embed_grad(go, tokens, 900, start=0, check=False),
                *rnnt_beam_select(x, scores, check=False))

    want = [run(j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, (st, job) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(st):
                got[i].append(run(job))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


@pytest.mark.parametrize("B", [2, 9])
def test_captured_training(B):
    """A forward and backward pass in a graph, by one launch and by three, replayed with new labels."""
    g = torch.Generator(device="cuda").manual_seed(B)
    w = torch.randn(300, 48, device="cuda", generator=g).requires_grad_()
    tokens = torch.zeros(B, 600, device="cuda", dtype=torch.int32)
    lengths = torch.full((B,), 600, device="cuda", dtype=torch.int32)
    go = torch.randn(B, 601, 48, device="cuda", generator=g)

    def step():
        out = rnnt_embed(w, tokens, lengths, start=0, scale=3.0, check=False)
        return out.detach(), torch.autograd.grad(out, w, go)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                            # nothing of it lives on: no eager graph of the same leaf
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for low in (600, 40, 0):
        tokens.copy_(torch.randint(0, 300, tokens.shape, device="cuda", generator=g))
        lengths.copy_(torch.randint(low, 601, lengths.shape, device="cuda", generator=g))
        graph.replay()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_far_offsets():
    """Tables, logits and states whose last elements lie behind 2^31 elements."""
    V, D = 1_100_000, 2048
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    w[-1], w[-2] = 3.0, 5.0
    tokens = i32([[V - 1, V - 2, 0, -1]])
    out = rnnt_embed(w, tokens, scale=2.0)
    assert [float(out[0, i, 7]) for i in range(4)] == [6.0, 10.0, 0.0, 0.0]
    del w
    go = torch.ones(1, 4, D, dtype=torch.bfloat16, device="cuda")
    for places in (go, torch.ones(1, 4000, D, dtype=torch.bfloat16, device="cuda")):
        t = tokens if places is go else tokens.repeat(1, 1000)
        g = rnnt_embed_grad(places, t, V)
        n = places.shape[1] // 4
        assert (g[[V - 1, V - 2, 0]] == n).all() and not g[1:V - 2].any()
        del g
    x = torch.zeros(33, 64, 1 << 20, dtype=torch.bfloat16, device="cuda")
    x[32, 63, 1_000_001] = 8.0
    x[32, 62, 17] = 7.0
    scores = torch.zeros(33, 64, device="cuda")
    s, tok, par = rnnt_beam_select(x, scores, 2)
    assert tok[32].tolist() == [1_000_001, 17] and par[32].tolist() == [63, 62]
    assert tok[5].tolist() == [0, 1] and par[5].tolist() == [0, 0]
    del x
    big = torch.zeros(2, 3, 1_000_000_007, dtype=torch.int8, device="cuda")
    big[1, 2, -1] = 9
    y, = rnnt_beam_reorder([big], i32([[0, 0, 1], [2, 1, 2]]))
    assert y[1, :, -1].tolist() == [9, 0, 9] and not y[0].any()


def test_training_step():
    """Embedding -> prediction network -> joiner -> loss: the table's gradient against
    differences of the loss."""
    torch.manual_seed(0)
    V, D, H = 12, 8, 6
    T, U = i32([5, 7, 4]), i32([3, 1, 0])
    y = i32([[1, 2, 3], [4, 5, 6], [7, 8, 9]])
    emb = RNNTEmbedding(V, D, start=0, scale=D ** 0.5, device="cuda")
    enc = torch.randn(3, 7, H, device="cuda")
    a, b = torch.randn(D, H, device="cuda") * 0.3, torch.randn(H, V, device="cuda") * 0.5

    def loss():
        pred = emb(y, U) @ a
        z = torch.tanh(enc[:, :, None] + pred[:, None]) @ b
        rows = [z[i, :int(T[i]), :int(U[i]) + 1].reshape(-1, V) for i in range(3)]
        return rnnt_loss(torch.cat(rows), y, T, U, blank=0, reduction="sum")

    loss().backward()
    g = emb.weight.grad.clone()
    assert (g[10:] == 0).all() and (g[4] != 0).any() and (g[5:10] == 0).all()
    with torch.no_grad():
        for v, d in ((0, 1), (1, 0), (3, 7), (4, 2)):
            w, h = emb.weight[v, d].item(), 0.01
            up, down = [], []
            for to, sign in ((up, 1), (down, -1)):
                emb.weight[v, d] = w + sign * h
                to.append(float(loss()))
            emb.weight[v, d] = w
            # the loss (about 40) is rounded to 2e-6 and its differences are divided by 0.02;
            # the third derivative's part is of the order of h^2
            assert abs((up[0] - down[0]) / (2 * h) - float(g[v, d])) <= 5e-3 * max(1.0, abs(float(g[v, d])))


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_decoding_loop(dtype):
    """Frames of selection, reorder, lookup and state update against the same search in float64."""
    B, K, V, D, T = 3, 4, 40, 16, 12
    g = torch.Generator(device="cuda").manual_seed(12)
    dt = DT[dtype]
    table = torch.randn(V, D, device="cuda", generator=g).to(dt)
    frames = (torch.randn(B, T, V, device="cuda", generator=g) * 2).to(dt)
    lengths = [12, 7, 9]
    scores = torch.full((B, K), float("-inf"), device="cuda")
    scores[:, 0] = 0.0
    state = torch.zeros(B, K, V, device="cuda", dtype=dt)     # what a hypothesis adds to the logits
    history = torch.full((B, K, T), -1, device="cuda", dtype=torch.int32)
    proj = torch.randn(D, V, device="cuda", generator=g).to(dt)
    ref = [[(0.0, np.zeros(V), [])] for _ in range(B)]
    rounded = lambda t: R.f64(t.to(dt))  # noqa: E731
    for t in range(T):
        done = torch.tensor([[t >= n] * K for n in lengths], device="cuda")
        x = frames[:, t, None] + state
        scores, tokens, parents = rnnt_beam_select(x, scores, K, done)
        state, history = rnnt_beam_reorder([state, history], parents)
        history[:, :, t] = tokens
        e = rnnt_embed(table, tokens, scale=0.5)
        label = (tokens > 0)[:, :, None]                       # 0: blank, -1: nothing
        state = torch.where(label, (e.double() @ proj.double() * 0.1).to(dt), state)
        for b in range(B):
            hyps = ref[b]
            xs = np.stack([rounded((frames[b, t] + torch.as_tensor(h[1], device="cuda").to(dt)))
                           for h in hyps])[None]
            fin = np.full((1, len(hyps)), t >= lengths[b])
            s, tok, par = R.select(xs, np.array([[h[0] for h in hyps]]), K, fin)
            new = []
            for r in range(K):
                if par[0, r] < 0:
                    continue
                old, v = hyps[par[0, r]], int(tok[0, r])
                st = old[1]
                if v > 0:
                    e64 = rounded(torch.as_tensor(R.f64(table)[v] * 0.5, device="cuda"))
                    st = rounded(torch.as_tensor(e64 @ R.f64(proj) * 0.1, device="cuda"))
                new.append((s[0, r], st, old[2] + [v]))
            ref[b] = new
    for b in range(B):
        for r, (s, _, seq) in enumerate(ref[b]):
            assert history[b, r].tolist() == seq
            # every step rounds the score (below 64 in size: 2^-19 at most) and its log-sum-exp
            assert abs(float(scores[b, r]) - s) <= T * (2.0 ** -19 + 4e-6)
