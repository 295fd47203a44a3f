"""GPU: a teacher's top logits and the distillation loss against float64 forms."""
import numpy as np
import pytest
import torch

import distill_ref as R
import label_ref as L
from rnn_transducer_loss_gb300 import (RNNTDistillLoss, rnnt_distill_loss, rnnt_loss,
                                       rnnt_top_logits)

pytestmark = pytest.mark.gpu
DT = L.DTYPES


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_rows(kind, N, V, dtype, seed):
    g = gen(seed)
    x = torch.randn(N, V, device="cuda", generator=g) * 2
    if kind == "masked":                  # outputs ruled out, whole rows among them
        x[torch.rand(N, V, device="cuda", generator=g) < 0.6] = -float("inf")
        x[N // 2] = -float("inf")
    if kind == "lowest":                  # ruled out by the type's lowest value
        x[torch.rand(N, V, device="cuda", generator=g) < 0.6] = torch.finfo(dtype).min
        x[N // 2] = torch.finfo(dtype).min
    if kind == "ties":
        x = (x * 1.5).round()
    if kind == "equal":
        x.fill_(-3.5)
        x[:, V // 2] = 1.0
    if kind == "far":
        x *= 200 if dtype == torch.float16 else 1e4
    if kind == "sorted":
        x = x.sort(dim=1, descending=bool(seed % 2)).values
    return x.to(dtype)


TOP = [  # rows, V, k
    (1, 1, 1), (3, 2, 2), (7, 16, 4), (50, 29, 8), (33, 29, 29), (9, 64, 64), (70, 130, 64), (40, 256, 32),
    (40, 1024, 8), (5, 1024, 64), (12, 1000, 33), (9, 1001, 7), (6, 2048, 16), (5, 2056, 31), (4, 4099, 40),
    (4, 5000, 32), (3, 9001, 64), (3, 16384, 64), (2, 50000, 17), (2, 50001, 64), (1, 70000, 3),
]


def check_top(x, k, tau, got, live=None):
    want = R.top(L.f64(x).reshape(-1, x.shape[-1]), k, tau)
    values, ids, rest = (L.f64(t).reshape(w.shape) for t, w in zip(got, want))
    wv, wi, wr, bound = want
    if live is not None:
        wv[~live], wi[~live], wr[~live], bound[~live] = -np.inf, -1, -np.inf, 0
    assert np.array_equal(ids, wi)
    assert np.array_equal(values, wv)
    none = np.isneginf(wr)
    assert np.array_equal(np.isneginf(rest), none)
    err = np.abs(rest[~none] - wr[~none])
    assert (err <= bound[~none]).all(), (err / np.maximum(bound[~none], 1e-300)).max()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", TOP, ids=str)
def test_top(case, dtype):
    N, V, k = case
    for i, kind in enumerate(("plain", "masked", "lowest", "ties", "equal", "sorted", "far")):
        x = make_rows(kind, N, V, DT[dtype], 11 * i + V)
        tau = (1.0, 2.0, 0.7)[(i + V) % 3]
        check_top(x, k, tau, rnnt_top_logits(x, k, temperature=tau))


def test_top_alignments():
    """Rows that begin anywhere in a 16-byte unit, non-contiguous and negative views."""
    big = torch.randn(40 * 301 + 16, device="cuda", generator=gen(1))
    for dtype in DT.values():
        for skip in (0, 1, 3, 7):
            x = big.to(dtype)[skip:skip + 40 * 301].view(40, 301)
            check_top(x, 9, 1.0, rnnt_top_logits(x, 9))
    x = big[:12000].view(40, 300)
    for y in (x[:, ::2], x.t(), x[::3], x[:1].expand(5, 300), torch.complex(x, x).conj().imag):
        check_top(y, 5, 1.0, rnnt_top_logits(y, 5))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V,k", [(29, 8), (1024, 8), (5000, 32)])
def test_top_padded(V, k, dtype):
    T, U = [5, 0, 3, 4], [2, 3, 0, 1]
    x = torch.randn(4, 5, 4, V, device="cuda", generator=gen(2)).to(DT[dtype])
    _, live = R.rows_of(T, U, True)
    x.view(-1, V)[torch.as_tensor(~live, device="cuda")] = float("nan")        # not read
    got = rnnt_top_logits(x, k, i32(T), i32(U))
    assert got[0].shape == (4, 5, 4, k) and got[2].shape == (4, 5, 4)
    check_top(torch.nan_to_num(x), k, 1.0, got, live)


@pytest.mark.parametrize("V", [29, 1024, 5000, 50000])
def test_top_bad_rows(V):
    for value in (float("nan"), float("inf")):
        for at in (0, V // 2, V - 1):
            x = torch.randn(4, V, device="cuda", generator=gen(3))
            x[2, at] = value
            with pytest.raises(ValueError, match="NaN"):
                rnnt_top_logits(x, 3)
            check_top(x, 3, 1.0, rnnt_top_logits(x, 3, check=False))
    x = torch.randn(2, 3, 2, V, device="cuda", generator=gen(3))
    with pytest.raises(ValueError, match="lengths"):
        rnnt_top_logits(x, 3, i32([3, 4]), i32([1, 1]))
    got = rnnt_top_logits(x, 3, i32([3, 4]), i32([1, -1]), check=False)
    check_top(x, 3, 1.0, got, np.array([True] * 6 + [False] * 6))


# ------------------------------------------------------------------ distillation
def make_teacher(x, k, tau, kind, seed, dtype=None):
    """(values, ids, rest) of rows that resemble the student's: places empty or of no weight, rows
    with nothing in them."""
    N, V = x.shape
    rng = np.random.default_rng(seed)
    t = torch.nan_to_num(x.float(), neginf=-30.0) + torch.randn(N, V, device="cuda", generator=gen(seed))
    values, ids, rest = rnnt_top_logits(t, k, temperature=tau)
    if kind == "gaps":
        gap = torch.as_tensor(rng.random((N, k)) < 0.3, device="cuda")
        ids[gap] = -1 - (torch.arange(k, device="cuda", dtype=torch.int32)[None] % 3).expand(N, k)[gap]
        values[torch.as_tensor(rng.random((N, k)) < 0.2, device="cuda")] = -float("inf")
        rest[torch.as_tensor(rng.random(N) < 0.3, device="cuda")] = -float("inf")
        ids[N // 3], rest[N // 3] = -1, -float("inf")             # nothing
        ids[N // 2] = -1                                            # the rest alone
        order = torch.as_tensor(rng.permutation(k), device="cuda")
        values, ids = values[:, order].contiguous(), ids[:, order].contiguous()
    return values.to(dtype or torch.float32), ids, rest


def expected(x, values, ids, rest, tau, owner, live, B, weight, reduction):
    loss, grad, err, part = R.distill(L.f64(x), L.f64(values), ids.cpu().numpy(),
                                      None if rest is None else L.f64(rest), tau)
    loss[~live], grad[~live], err[~live], part[~live] = 0, 0, 0, 0
    total, bound = np.zeros(B), np.zeros(B)
    np.add.at(total, owner, loss * weight)
    np.add.at(bound, owner, err * abs(weight))
    scale = weight / (B if reduction == "mean" else 1)
    if reduction != "none":
        total, bound = total.sum(), bound.sum()
        if reduction == "mean":
            total, bound = total / B, bound / B
    return total, grad * scale, bound + np.abs(total) * L.U32 * 1.01 + 1e-40, part * abs(scale)


def check_distill(x, got_loss, got_grad, want, dtype):
    total, grad, bound, part = want
    loss = L.f64(got_loss)
    assert np.array_equal(np.isinf(loss), np.isinf(total))
    fine = np.isfinite(total)
    err = np.abs(np.where(fine, loss, 0) - np.where(fine, total, 0))
    assert (err <= np.where(fine, bound, 0)).all(), (err, bound)
    if got_grad is not None:
        g = L.f64(got_grad).reshape(grad.shape)
        limit = R.grad_bound(grad, part, 1.0, dtype)
        bad = ~(np.abs(g - grad) <= limit)
        assert not bad.any(), (np.argwhere(bad)[:5], g[bad][:5], grad[bad][:5], limit[bad][:5])


DISTILL = [  # T, U, V, k, tau, weight, reduction
    ([1], [0], 1, 1, 1.0, 1.0, "none"), ([8, 6], [3, 2], 16, 4, 1.0, 1.0, "none"),
    ([5, 1, 7], [2, 0, 3], 29, 8, 2.0, 0.5, "mean"), ([4, 0, 9], [1, 2, 2], 29, 29, 1.0, 1.0, "sum"),
    ([3, 2], [4, 0], 130, 64, 0.5, -2.0, "mean"), ([6, 3], [2, 5], 301, 7, 1.0, 1.0, "mean"),
    ([9, 4], [3, 1], 1024, 8, 2.0, 0.1, "sum"), ([4, 3], [2, 1], 1000, 33, 1.0, 1.0, "none"),
    ([2, 3], [1, 2], 1025, 1, 1.0, 3.0, "mean"), ([3, 2], [1, 1], 2048, 16, 4.0, 1.0, "mean"),
    ([2, 1], [2, 1], 4099, 40, 1.0, 1.0, "sum"), ([2, 1], [1, 2], 5000, 32, 1.0, 1.0, "mean"),
    ([2], [1], 9001, 64, 1.0, 1.0, "none"), ([2], [0], 50000, 20, 1.0, 1.0, "mean"),
    ([1], [1], 50001, 64, 2.0, 1.0, "mean"), ([1], [0], 70000, 5, 1.0, 1.0, "sum"),
]


@pytest.mark.parametrize("padded", [False, True], ids=["compact", "padded"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", DISTILL, ids=str)
def test_distill(case, dtype, padded):
    T, U, V, k, tau, weight, reduction = case
    B, dt = len(T), DT[dtype]
    owner, live = R.rows_of(T, U, padded)
    N = len(owner)
    for i, (kind, places, with_rest) in enumerate((
            ("plain", "plain", True), ("plain", "gaps", False), ("lowest", "gaps", True), ("ties", "plain", False))):
        x = make_rows(kind, N, V, dt, 5 * i + V)
        values, ids, rest = make_teacher(x, k, tau, places, i + V, list(DT.values())[(i + V) % 3])
        rest = rest if with_rest else None
        want = expected(x, values, ids, rest, tau, owner, live, B, weight, reduction)
        if padded:
            dead = torch.as_tensor(~live, device="cuda")
            x[dead] = float("nan")                                  # none of it is read
            values[dead], ids[dead] = float("nan"), V + 5
            lead = (B, max(T), max(U) + 1)
            x, values, ids = x.view(*lead, V), values.view(*lead, k), ids.view(*lead, k)
            rest = rest.view(lead) if with_rest else None
        x.requires_grad_()
        loss = rnnt_distill_loss(x, values, ids, i32(T), i32(U), teacher_rest=rest,
                                 temperature=tau, weight=weight, reduction=reduction)
        assert loss.dtype == torch.float32 and loss.shape == ((B,) if reduction == "none" else ())
        grad, = torch.autograd.grad(loss.sum(), x)
        assert grad.dtype == dt and grad.shape == x.shape
        check_distill(x, loss, grad, want, dt)
        with torch.no_grad():
            alone = rnnt_distill_loss(x, values, ids, i32(T), i32(U), rest, tau, weight, reduction)
        assert torch.equal(alone, loss.detach())
        again = rnnt_distill_loss(x, values, ids, i32(T), i32(U), rest, tau, weight, reduction)
        assert torch.equal(again, loss)
        assert torch.equal(torch.autograd.grad(again.sum(), x)[0], grad)


@pytest.mark.parametrize("V,k", [(29, 4), (1024, 8), (5000, 6)])
def test_distill_differences(V, k):
    """The gradient against central differences of the float64 form along random directions, and
    against differences of the call itself."""
    T, U = [3, 2], [1, 2]
    owner, live = R.rows_of(T, U, False)
    x = torch.randn(len(owner), V, device="cuda", generator=gen(7))
    values, ids, rest = make_teacher(x, k, 2.0, "plain", 3)
    leaf = x.clone().requires_grad_()
    args = (values, ids, i32(T), i32(U), rest, 2.0, 1.0, "sum")
    grad, = torch.autograd.grad(rnnt_distill_loss(leaf, *args), leaf)
    for seed in range(3):
        d = torch.randn(x.shape, device="cuda", generator=gen(seed)).double().cpu().numpy()
        h = 1e-4
        up, down = (R.distill(L.f64(x) + s * h * d, L.f64(values), ids.cpu().numpy(), L.f64(rest), 2.0)[0].sum()
                    for s in (1, -1))
        slope = (up - down) / (2 * h)
        mine = (L.f64(grad) * d).sum()
        # h^2 / 6 of a third derivative (below 10 |d|^3 a row) and the gradient's own bound
        assert abs(mine - slope) <= 1e-5 * (1 + abs(slope))


def test_distill_infinite():
    """An output that the teacher has and the student rules out: loss +inf, a finite gradient."""
    for V in (29, 1024, 5000):
        x = torch.randn(4, V, device="cuda", generator=gen(8))
        values, ids, rest = make_teacher(x, 3, 1.0, "plain", 8)
        x[1, ids[1, 0].item()] = -float("inf")
        values[2, 1] = -float("inf")                       # no weight there: nothing lost
        x[2, ids[2, 1].item()] = -float("inf")
        leaf = x.requires_grad_()
        for r in (rest, None):
            loss = rnnt_distill_loss(leaf, values, ids, i32([2, 2]), i32([0, 0]), r, reduction="none")
            grad, = torch.autograd.grad(loss.sum(), leaf)
            want = expected(leaf, values, ids, r, 1.0, *R.rows_of([2, 2], [0, 0], False), 2, 1.0, "none")
            assert torch.isinf(loss).tolist() == [True, False] and torch.isfinite(grad).all()
            check_distill(leaf, loss, grad, want, torch.float32)


@pytest.mark.parametrize("V", [29, 1024, 5000, 50000])
def test_distill_checks(V):
    x = torch.randn(6, V, device="cuda", generator=gen(9))
    values, ids, rest = make_teacher(x, 4, 1.0, "plain", 9)
    T, U = i32([2, 4]), i32([0, 0])

    def call(check=True, **kw):
        a = dict(logits=x, teacher_logits=values, teacher_ids=ids, logit_lengths=T, target_lengths=U,
                 teacher_rest=rest, reduction="none", check=check)
        a.update(kw)
        return rnnt_distill_loss(**a)

    def changed(t, at, value):
        t = t.clone()
        t[at] = value
        return t

    want = call()
    for kw in (dict(logits=changed(x, (3, 5), float("nan"))), dict(logits=changed(x, (3, 5), float("inf"))),
               dict(logits=changed(x, 3, -float("inf"))),
               dict(teacher_logits=changed(values, (3, 1), float("nan"))),
               dict(teacher_logits=changed(values, (3, 1), float("inf"))),
               dict(teacher_rest=changed(rest, 3, float("nan"))),
               dict(teacher_rest=changed(rest, 3, float("inf")))):
        with pytest.raises(ValueError, match="wanted"):
            call(**kw)
        got = call(False, **kw)
        assert got[0] == want[0] and torch.isnan(got[1])
    for bad, as_if in ((V, -1), (2 ** 31 - 1, -1)):
        with pytest.raises(ValueError, match="wanted"):
            call(teacher_ids=changed(ids, (3, 1), bad))
        assert torch.equal(call(False, teacher_ids=changed(ids, (3, 1), bad)),
                           call(teacher_ids=changed(ids, (3, 1), as_if)))
    twice = changed(ids, (3, 3), ids[3, 1])
    with pytest.raises(ValueError, match="different"):
        call(teacher_ids=twice)
    assert torch.equal(call(False, teacher_ids=twice), call(teacher_ids=changed(ids, (3, 3), -1)))
    for t, u in (([2, 3], [0, 0]), ([2, 5], [0, 0]), ([-1, 6], [0, 0]), ([2, 4], [0, -1]),
                 ([2 ** 31 - 1, 4], [2 ** 31 - 1, 0])):
        with pytest.raises(ValueError, match="T_b"):
            call(logit_lengths=i32(t), target_lengths=i32(u))
        leaf = x.clone().requires_grad_()
        got = call(False, logits=leaf, logit_lengths=i32(t), target_lengths=i32(u))
        grad, = torch.autograd.grad(got.sum(), leaf)
        counted = min(6, sum(max(a, 0) * (max(b, -1) + 1) for a, b in zip(t, u)))
        assert (grad[counted:] == 0).all() and (grad[:counted] != 0).any(1).all()


@pytest.mark.parametrize("V", [70, 1024, 5000, 50001])
def test_distill_repeated_ids(V):
    """Ids that stand many times in a row, over both halves of the places: the first counts."""
    N, k = 5, 64
    x = torch.randn(N, V, device="cuda", generator=gen(10)).requires_grad_()
    rng = np.random.default_rng(4)
    ids = rng.integers(-1, 40, size=(N, k))
    ids[0], ids[1, :32], ids[1, 32:] = 7, np.arange(32), np.arange(32)
    once = ids.copy()
    for n in range(N):
        for j in range(k):
            if ids[n, j] in ids[n, :j]:
                once[n, j] = -1
    values = torch.randn(N, k, device="cuda", generator=gen(11))
    rest = torch.randn(N, device="cuda", generator=gen(12))
    outs = []
    for which in (ids, once):
        loss = rnnt_distill_loss(x, values, i32(which), i32([N]), i32([0]), rest, check=False)
        outs += [loss, torch.autograd.grad(loss, x)[0]]
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[3])


def test_distill_upstream():
    """Factors of backward: one, another, one a sample; a second backward raises."""
    T, U, V = [3, 0, 5], [2, 1, 0], 1024
    for padded in (False, True):
        owner, live = R.rows_of(T, U, padded)
        x = torch.randn(len(owner), V, device="cuda", generator=gen(13))
        values, ids, rest = make_teacher(x, 8, 1.0, "plain", 13)
        if padded:
            lead = (3, 5, 3)
            x, values, ids, rest = (t.view(*lead, *t.shape[1:]) for t in (x, values, ids, rest))
        x.requires_grad_()
        args = (values, ids, i32(T), i32(U), rest, 1.0, 1.0)
        base, = torch.autograd.grad(rnnt_distill_loss(x, *args, "sum"), x)
        half, = torch.autograd.grad(rnnt_distill_loss(x, *args, "sum") * 0.5, x)
        assert torch.equal(half, base * 0.5)
        f = torch.tensor([2.0, 3.0, -0.25], device="cuda")
        each, = torch.autograd.grad(rnnt_distill_loss(x, *args, "none"), x, f)
        want = base.reshape(len(owner), V) * f[torch.as_tensor(owner, device="cuda")][:, None]
        assert torch.equal(each.reshape(want.shape), want)
        one, = torch.autograd.grad(rnnt_distill_loss(x, *args, "none").sum(), x)
        assert torch.equal(one, base)
        loss = rnnt_distill_loss(x, *args, "sum")
        loss.backward(retain_graph=True)
        assert torch.equal(x.grad, base)
        with pytest.raises(RuntimeError, match="only once"):
            loss.backward()
        x.grad = None


def test_distill_views():
    """Rows that begin between two vectors, strided, expanded and negative views, other types of the
    teacher's logits."""
    T, U, V, k = i32([3, 2]), i32([1, 1]), 301, 5
    big = torch.randn(12 * V + 9, device="cuda", generator=gen(14))
    x = big[:10 * V].view(10, V)
    values, ids, rest = make_teacher(x, k, 1.0, "plain", 14)

    def both(leaf, v, i, r):
        leaf = leaf.detach().requires_grad_()
        loss = rnnt_distill_loss(leaf, v, i, T, U, r)
        return loss, torch.autograd.grad(loss, leaf)[0]

    want = both(x, values, ids, rest)
    shifted = torch.cat([big[:3], x.reshape(-1)])[3:].view(10, V)
    wide = torch.stack([x, x], 2)[:, :, 1]
    for y in (shifted, wide, torch.complex(x, -x).conj().imag):
        got = both(y, values, ids, rest)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    v2 = torch.stack([values, values], 1)[:, 0]
    i2 = torch.stack([ids, ids], 2)[..., 1]
    r2 = torch.stack([rest, rest], 1)[:, 1]
    got = both(x, v2, i2, r2)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = both(x, values[:1].expand(10, k), ids[:1].expand(10, k), rest[:1].expand(10))
    copy = both(x, values[:1].repeat(10, 1), ids[:1].repeat(10, 1), rest[:1].repeat(10))
    assert torch.equal(one[0], copy[0]) and torch.equal(one[1], copy[1])
    for dt in DT.values():
        v = values.to(dt)
        a, b = both(x, v, ids, rest), both(x, v.float(), ids, rest)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_distill_many_samples():
    """More samples than a block has threads, empty ones among them, in a long compact batch."""
    rng = np.random.default_rng(5)
    T, U = rng.integers(0, 4, size=700), rng.integers(0, 3, size=700)
    owner, live = R.rows_of(T, U, False)
    x = torch.randn(len(owner), 40, device="cuda", generator=gen(15)).requires_grad_()
    values, ids, rest = make_teacher(x.detach(), 3, 1.0, "gaps", 15)
    for reduction in ("none", "mean"):
        loss = rnnt_distill_loss(x, values, ids, i32(T), i32(U), rest, reduction=reduction)
        f = torch.arange(1, 701, device="cuda") / 64 if reduction == "none" else torch.ones((), device="cuda")
        grad, = torch.autograd.grad(loss, x, f)
        want = expected(x, values, ids, rest, 1.0, owner, live, 700, 1.0, reduction)
        if reduction == "none":
            factor = f.double().cpu().numpy()[owner][:, None]
            want = (want[0], want[1] * factor, want[2], want[3] * factor)
        check_distill(x, loss, grad, want, torch.float32)


def test_student_learns_from_teacher():
    """A training step as it is used: the teacher's rows to their top logits, the transducer loss and
    the distillation loss of the student on the same lattice, one backward pass."""
    T, U, V = [12, 7], [4, 2], 1024
    owner, live = R.rows_of(T, U, False)
    targets = i32(np.random.default_rng(6).integers(1, V, size=(2, 4)))
    teacher = torch.randn(len(owner), V, device="cuda", generator=gen(16)) * 2
    student = (teacher + torch.randn(teacher.shape, device="cuda", generator=gen(17))).half().requires_grad_()
    values, ids, rest = rnnt_top_logits(teacher, 8, temperature=2.0)
    module = RNNTDistillLoss(temperature=2.0, weight=0.1)
    a = rnnt_loss(student, targets, i32(T), i32(U), blank=0)
    b = module(student, values, ids, i32(T), i32(U), rest)
    (a + b).backward()
    ga, = torch.autograd.grad(rnnt_loss(student, targets, i32(T), i32(U), blank=0), student)
    want = expected(student, values, ids, rest, 2.0, owner, live, 2, 0.1, "mean")
    check_distill(student, b, None, want, torch.float16)
    total = L.f64(ga) + want[1]
    bound = R.grad_bound(want[1], want[3], 1.0, torch.float16) + np.abs(total) * 2 ** -11 * 1.01 + 2 ** -25
    assert (np.abs(L.f64(student.grad) - total) <= bound).all()


def test_distill_captured():
    """A captured step, replayed on other inputs, and two graphs at once on streams of their own."""
    T, U, V = i32([4, 3]), i32([2, 1]), 1024
    graphs = []
    side = torch.cuda.Stream()
    for seed in (20, 21):
        x = torch.randn(18, V, device="cuda", generator=gen(seed)).requires_grad_()
        values, ids, rest = rnnt_top_logits(x.detach() + 1, 8)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            rnnt_distill_loss(x, values, ids, T, U, rest, check=False)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                top = rnnt_top_logits(x.detach() * 2, 8, check=False)
                loss = rnnt_distill_loss(x, *top[:2], T, U, top[2], check=False)
                grad, = torch.autograd.grad(loss, x)
        graphs.append((g, x, loss, grad))
    torch.cuda.synchronize()
    for turn in range(3):
        for g, x, loss, grad in graphs:
            with torch.no_grad():
                x.copy_(torch.randn(18, V, device="cuda", generator=gen(30 + turn)))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for (g, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, x, loss, grad in graphs:
            leaf = x.detach().clone().requires_grad_()
            top = rnnt_top_logits(leaf.detach() * 2, 8)
            want = rnnt_distill_loss(leaf, *top[:2], T, U, top[2])
            assert torch.equal(loss, want)
            assert torch.equal(grad, torch.autograd.grad(want, leaf)[0])


def test_distill_streams():
    """Calls on a side stream that its inputs are made on."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x = torch.randn(40, 1024, device="cuda", generator=gen(22)).requires_grad_()
        values, ids, rest = rnnt_top_logits(x.detach() + 1, 8, check=False)
        loss = rnnt_distill_loss(x, values, ids, i32([20, 20]), i32([0, 0]), rest, check=False)
        grad, = torch.autograd.grad(loss * 2, x)
    s.synchronize()
    again = rnnt_distill_loss(x, values, ids, i32([20, 20]), i32([0, 0]), rest)
    assert torch.equal(again, loss) and torch.equal(torch.autograd.grad(again * 2, x)[0], grad)


def test_distill_far_rows():
    """Row offsets beyond 2^31 elements."""
    V, N = 1024, (1 << 21) + 300                      # 2^31 elements and more, 4.3 GB of float16
    x = torch.zeros(N, V, device="cuda", dtype=torch.float16)
    x[-300:] = torch.randn(300, V, device="cuda", generator=gen(23)).half()
    top = rnnt_top_logits(x, 4)
    few = rnnt_top_logits(x[-300:].clone(), 4)
    for a, b in zip(top, few):
        assert torch.equal(a[-300:], b)
    x.requires_grad_()
    loss = rnnt_distill_loss(x, *top[:2], i32([N - 300, 300]), i32([0, 0]), reduction="none")
    grad, = torch.autograd.grad(loss.sum(), x)
    leaf = x.detach()[-300:].clone().requires_grad_()
    want = rnnt_distill_loss(leaf, *few[:2], i32([300]), i32([0]), reduction="none")
    assert loss[1] == want[0]
    assert torch.equal(grad[-300:], torch.autograd.grad(want.sum(), leaf)[0])


def test_refusals():
    x = torch.randn(6, 20, device="cuda")
    v, ids, rest = rnnt_top_logits(x, 3)
    T, U = i32([2, 4]), i32([0, 0])
    for args, kw in (((x, 0), {}), ((x, 21), {}), ((x.double(), 3), {}), ((x[None], 3), {}),
                     ((x, 3, T, U), {}), ((x.view(2, 3, 1, 20), 3, T), {}),
                     ((x.view(2, 3, 1, 20), 3, T.long(), U), {}), ((x.view(2, 3, 1, 20), 3, T[:1], U), {}),
                     ((x, 3), dict(temperature=0.0))):
        with pytest.raises(ValueError):
            rnnt_top_logits(*args, **kw)
    good = dict(logits=x, teacher_logits=v, teacher_ids=ids, logit_lengths=T, target_lengths=U,
                teacher_rest=rest)
    rnnt_distill_loss(**good)
    for kw in (dict(logits=x.double()), dict(logits=x[0]), dict(teacher_logits=v[:5]),
               dict(teacher_logits=v.double()), dict(teacher_logits=v.cpu()), dict(teacher_ids=ids.long()),
               dict(teacher_ids=ids[:, :2]), dict(teacher_rest=rest.half()), dict(teacher_rest=rest[:5]),
               dict(logit_lengths=T.long()), dict(logit_lengths=T[:1]), dict(target_lengths=U.cpu()),
               dict(logit_lengths=T[:0], target_lengths=U[:0]), dict(temperature=float("nan")),
               dict(weight=float("inf")), dict(reduction="batch"), dict(logits=x[:0], teacher_logits=v[:0],
                                                                       teacher_ids=ids[:0], teacher_rest=rest[:0]),
               dict(teacher_logits=v.clone().requires_grad_()), dict(teacher_rest=rest.clone().requires_grad_())):
        with pytest.raises(ValueError):
            rnnt_distill_loss(**{**good, **kw})
    # more than once differentiated, or forward
    leaf = x.clone().requires_grad_()
    g, = torch.autograd.grad(rnnt_distill_loss(**{**good, "logits": leaf}), leaf, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    with torch.autograd.forward_ad.dual_level(), pytest.raises(NotImplementedError):
        rnnt_distill_loss(**{**good, "logits": torch.autograd.forward_ad.make_dual(x, x)})
    assert rnnt_top_logits(x[:0], 3)[0].shape == (0, 3)
