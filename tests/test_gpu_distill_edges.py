"""GPU: the distillation loss and a teacher's top logits at the edges of what may be called."""
import numpy as np
import pytest
import torch

import distill_ref as R
import label_ref as L
import test_gpu_distill as D
from rnn_transducer_loss_gb300 import rnnt_distill_loss, rnnt_top_logits

pytestmark = pytest.mark.gpu
DT = L.DTYPES


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("V", [29, 1024, 5000])
def test_one_sample_longer_than_the_rows(V):
    """Lengths of more rows than there are, in one sample: refused, and without the check cut at the rows."""
    x = torch.randn(6, V, device="cuda", generator=gen(1))
    values, ids, rest = rnnt_top_logits(x + 1, 4)
    whole = rnnt_distill_loss(x, values, ids, i32([6]), i32([0]), rest, reduction="sum")
    for t, u in (([7], [0]), ([7, 0], [0, 0]), ([0, 7], [0, 0]), ([2], [3]), ([2 ** 31 - 1], [2 ** 31 - 2]),
                 ([0, 2 ** 31 - 1, 0], [0, 0, 5])):
        with pytest.raises(ValueError, match="T_b"):
            rnnt_distill_loss(x, values, ids, i32(t), i32(u), rest)
        got = rnnt_distill_loss(x, values, ids, i32(t), i32(u), rest, reduction="sum", check=False)
        assert torch.equal(got, whole)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [1, 2, 3, 5])
def test_top_of_rows_shorter_than_a_unit(V, dtype):
    """Unaligned rows of which several lie in one 16-byte unit: as from an aligned copy."""
    for skip in (1, 3, 7):
        for rows in (1, 2, 50):
            big = torch.randn(rows * V + 16, device="cuda", generator=gen(V)).to(DT[dtype])
            x = big[skip:skip + rows * V].view(rows, V)
            for k in {1, V}:
                for a, b in zip(rnnt_top_logits(x, k), rnnt_top_logits(x.clone(), k)):
                    assert torch.equal(a, b) or torch.allclose(a, b, rtol=4 * L.U32, atol=4 * L.U32)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [7, 29, 64])
def test_padded_short_rows_of_which_most_do_not_count(V, dtype):
    """Whole batches of rows outside their sequence beside some inside: as from the compact layout."""
    T, U, k = [2, 90, 0, 31], [3, 1, 3, 0], 4
    owner, live = R.rows_of(T, U, True)
    at = torch.as_tensor(live.nonzero()[0], device="cuda")
    x = torch.full((len(owner), V), float("nan"), device="cuda", dtype=DT[dtype])
    x[at] = torch.randn(len(at), V, device="cuda", generator=gen(V)).to(DT[dtype])
    lead = (4, 90, 4)
    x = x.view(*lead, V)
    got = rnnt_top_logits(x, k, i32(T), i32(U))
    D.check_top(torch.nan_to_num(x), k, 1.0, got, live)
    # (the order in which a thread adds its row's terms turns with its place in the batch, so sums of
    # the compact layout are held to the float64 form too, not to the padded one's bits)
    rows = [t.reshape(len(owner), *t.shape[3:]) for t in got]
    for padded in (True, False):
        leaf = (x if padded else x.view(-1, V)[at]).clone().requires_grad_()
        teacher = got if padded else [t[at].contiguous() for t in rows]
        loss = rnnt_distill_loss(leaf, *teacher[:2], i32(T), i32(U), teacher[2], reduction="none")
        grad, = torch.autograd.grad(loss.sum(), leaf)
        o, l = (owner, live) if padded else (owner[live], live[live])
        want = D.expected(torch.nan_to_num(leaf).detach().view(-1, V), *(t.reshape(len(o), -1) for t in teacher[:2]),
                          teacher[2].reshape(-1), 1.0, o, l, 4, 1.0, "none")
        D.check_distill(leaf, loss, grad, want, DT[dtype])
        assert (grad.reshape(-1, V)[torch.as_tensor(~l, device="cuda")] == 0).all()


@pytest.mark.parametrize("V", [29, 200, 1024, 5000, 70000])
def test_rest_outside_float32(V):
    """A finite rest over a small temperature is the nearer end of float32's range, not infinite."""
    most = torch.finfo(torch.float32).max
    x = torch.randn(4, V, device="cuda", generator=gen(3))
    x[0], x[1, :9], x[2] = 3e38, 1e38, -3e38
    for dtype in (torch.float32, torch.bfloat16):
        _, _, rest = rnnt_top_logits(x.to(dtype), 3, temperature=0.1)
        assert rest[:3].tolist() == [most, most, -most] and abs(rest[3]) < 100
        # and is a rest that the loss takes
        loss = rnnt_distill_loss(x * 0, torch.zeros(4, 1, device="cuda"), i32(np.zeros((4, 1))), i32([4]), i32([0]),
                                 rest, temperature=0.1)
        assert torch.isfinite(loss)


@pytest.mark.parametrize("tau", [1.0, 1.5, 0.7, 3.0])
@pytest.mark.parametrize("V", [29, 200, 1024, 5000, 70000])
def test_rest_is_rounded_once(V, tau):
    """Temperatures whose reciprocal is not a float32: the rest is off by half a step of its own and by what
    the logarithm of a sum of ``V`` terms may be off (rows far from 0, where that is a tenth of a step)."""
    x = torch.randn(300, V, device="cuda", generator=gen(V)) * 2 + torch.linspace(1e4, 2e4, 300, device="cuda")[:, None]
    values, _, rest = rnnt_top_logits(x, 3, temperature=tau)
    y = x.double() / tau
    y.scatter_(1, torch.topk(x, 3, dim=1).indices, -float("inf"))
    want = torch.logsumexp(y, 1).cpu().numpy()
    far = np.log(V) + np.abs(want - y.max(1).values.cpu().numpy())
    step = np.spacing(want.astype(np.float32)).astype(np.float64)
    assert (np.abs(L.f64(rest) - want) <= step / 2 + R.SUM + R.EXPONENT * far + 4 * L.U32 * far).all()


@pytest.mark.parametrize("V,k", [(29, 8), (1024, 64), (5000, 32)])
def test_inexact_temperatures(V, k):
    """A reciprocal of the temperature that is off shifts all rows' exponents the same way, which adds
    up over rows: the sum of many is off by half a step of its own and at most as much again."""
    N, tau = 40000, 1.5
    x = torch.randn(N, V, device="cuda", generator=gen(V)) * 2
    values, ids, rest = rnnt_top_logits(x + torch.randn(N, V, device="cuda", generator=gen(V + 1)), k, temperature=tau)
    loss = rnnt_distill_loss(x, values, ids, i32([N]), i32([0]), rest, temperature=tau, reduction="sum")
    want = 0.0
    for at in torch.arange(N, device="cuda").split(10000):
        log_q = torch.log_softmax(x[at].double() / tau, 1)
        goal = torch.cat([values[at].double() / tau, rest[at, None].double()], 1)
        mine = log_q.gather(1, ids[at].long())
        left = torch.logsumexp(log_q.scatter(1, ids[at].long(), -float("inf")), 1, keepdim=True)
        log_p = torch.log_softmax(goal, 1)
        want += (log_p.exp() * (log_p - torch.cat([mine, left], 1))).sum().item() * tau * tau
    assert abs(loss.item() - want) <= 2 * L.U32 * want


@pytest.mark.parametrize("V", [29, 200, 1024, 5000, 70000])
def test_far_teachers(V):
    """Finite logits of a teacher, however large over the temperature: what counts is how far apart they are."""
    x = torch.randn(3, V, device="cuda", generator=gen(4)).requires_grad_()
    ids = i32([[3, 1, 5]] * 3)
    far = torch.tensor([[3e38, 2.9e38, -3e38], [-3e38, -3.3e38, -float("inf")], [2e38, 2e38, 1e38]], device="cuda")
    near = torch.tensor([[0.0, -1e4, -1e4], [0.0, -1e4, -float("inf")], [0.0, 0.0, -1e4]], device="cuda")
    T, U = i32([1, 1, 1]), i32([0, 0, 0])
    for rest in (None, torch.full((3,), -float("inf"), device="cuda")):
        got, want = (rnnt_distill_loss(x, t, ids, T, U, rest, temperature=0.1, reduction="none") for t in (far, near))
        assert torch.equal(got, want)
        assert torch.equal(*(torch.autograd.grad(y.sum(), x)[0] for y in (got, want)))


@pytest.mark.parametrize("V,k,tau", [(29, 8, 4.0), (1024, 8, 2.0), (1024, 8, 8.0), (5000, 32, 3.0), (60000, 64, 3.0)])
def test_small_divergences(V, k, tau):
    """Teachers next to their students, where the divergence is small beside the logarithms it is made of.
    Off by: half a step of the sum; two roundings of each row's parts; and 3e-8 of the rest's logarithm,
    which is what ex2's mean error may leave of it and which counts |p_r - q_r| times a row."""
    N = 2000 if V > 10000 else 20000
    x = torch.randn(N, V, device="cuda", generator=gen(V)) * 2
    values, ids, rest = rnnt_top_logits(x + torch.randn(N, V, device="cuda", generator=gen(V + 1)), k, temperature=tau)
    loss = rnnt_distill_loss(x, values, ids, i32([N]), i32([0]), rest, temperature=tau, reduction="sum")
    want = apart = 0.0
    for at in torch.arange(N, device="cuda").split(1000):
        log_q = torch.log_softmax(x[at].double() / tau, 1)
        goal = torch.cat([values[at].double() / tau, rest[at, None].double()], 1)
        mine = log_q.gather(1, ids[at].long())
        left = torch.logsumexp(log_q.scatter(1, ids[at].long(), -float("inf")), 1, keepdim=True)
        log_p = torch.log_softmax(goal, 1)
        want += (log_p.exp() * (log_p - torch.cat([mine, left], 1))).sum().item()
        apart += (log_p[:, -1].exp() - left[:, 0].exp()).abs().sum().item()
    assert abs(loss.item() / tau ** 2 - want) <= 3 * L.U32 * want + 3e-8 * apart


@pytest.mark.parametrize("V", [29, 200, 1024, 5000, 70000])
def test_lowest_logits_of_a_student(V):
    """A teacher's output that the student rules out by the type's lowest value, over a temperature below 1:
    a large divergence that float32 holds, and a finite gradient."""
    tau, least = 0.7, torch.finfo(torch.float32).min
    x = torch.randn(2, V, device="cuda", generator=gen(V))
    values, ids = torch.tensor([[1.0, 0.5]] * 2, device="cuda"), i32([[2, 4]] * 2)
    x[:, 4] = least
    x.requires_grad_()
    for rest in (None, torch.zeros(2, device="cuda")):
        loss = rnnt_distill_loss(x, values, ids, i32([1, 1]), i32([0, 0]), rest, temperature=tau, weight=0.25,
                                 reduction="none")
        goal = np.array([1.0 / tau, 0.5 / tau] + ([0.0] if rest is not None else []))
        p = np.exp(goal - np.log(np.exp(goal).sum()))
        want = 0.25 * tau * p[1] * -least
        assert (np.abs(L.f64(loss) - want) <= 8 * L.U32 * want).all()
        grad, = torch.autograd.grad(loss.sum(), x)
        assert torch.isfinite(grad).all() and (grad[:, 4] < 0).all()
    # the outputs without a place ruled out, which the teacher's rest has
    y = torch.full((1, V), least, device="cuda")
    y[0, 2], y[0, 4] = 0.0, 1.0
    loss = rnnt_distill_loss(y, values[:1], ids[:1], i32([1]), i32([0]), torch.zeros(1, device="cuda"),
                             temperature=tau, weight=0.25)
    want = 0.25 * tau * p[2] * -least
    assert abs(loss.item() - want) <= 8 * L.U32 * want


@pytest.mark.parametrize("V", [29, 512, 5000])
def test_mean_of_rests(V):
    """Logarithms of sums over many rows, flat ones and peaked ones: what of their errors points one way is
    below half a step of float32 at 1.  (Sums of about 1, so that the results' own rounding is not seen.)"""
    u = torch.rand(6000, V, device="cuda", generator=gen(V), dtype=torch.float64)
    z = torch.randn(6000, V, device="cuda", generator=gen(V), dtype=torch.float64)
    for x in (-0.69 * u, -0.7 - 6 * u, u.clamp_min(1e-9).log(), 2 * z):
        x[:, :2] = x.amax(1, keepdim=True)
        x = (x - torch.logsumexp(x, 1, keepdim=True)).float()
        rest = rnnt_top_logits(x, 1)[2].double()
        y = x.double().scatter(1, x.argmax(1, keepdim=True), -float("inf"))
        err = rest - torch.logsumexp(y, 1)
        assert err.mean().abs() <= L.U32 + 5 * err.std() / 6000 ** 0.5


@pytest.mark.parametrize("V", [29, 1024, 5000])
def test_gradient_scaler(V):
    """float16 gradients that are too small for the type survive with the scaler's scale in the weight: off
    by half a step of the scaled values, where scaling behind the call finds zeros."""
    N, scale, weight = 500, 65536.0, 1e-7
    owner, live = np.zeros(N, dtype=np.int64), np.ones(N, dtype=bool)
    x = (torch.randn(N, V, device="cuda", generator=gen(V)) * 2).half()
    values, ids, rest = D.make_teacher(x, 8, 2.0, "plain", 5)
    scaler = torch.amp.GradScaler("cuda", init_scale=scale)
    leaf = x.clone().requires_grad_()
    main = torch.zeros(3, device="cuda", requires_grad=True).sum()
    T, U = i32([N]), i32([0])
    loss = scaler.scale(main) + rnnt_distill_loss(leaf, values, ids, T, U, rest, 2.0, weight * scaler.get_scale())
    loss.backward()
    want = D.expected(x, values, ids, rest, 2.0, owner, live, 1, weight * scale, "mean")
    D.check_distill(leaf, loss, leaf.grad, want, torch.float16)
    late = x.clone().requires_grad_()
    (rnnt_distill_loss(late, values, ids, T, U, rest, 2.0, weight) * scale).backward()
    assert ((late.grad == 0) & (leaf.grad != 0)).any() and (leaf.grad[late.grad != 0] != 0).all()


@pytest.mark.parametrize("padded", [False, True], ids=["compact", "padded"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("V", [1, 2, 3, 5, 7, 17, 40, 64, 100, 128])
def test_short_rows_with_many_places(V, dtype, padded):
    """Few outputs and up to 64 places, empty ones among them: rows that share 16-byte units."""
    T, U, tau = [9, 0, 14], [2, 1, 0], 2.0
    owner, live = R.rows_of(T, U, padded)
    for k in (20, 33, 64):
        x = (torch.randn(len(owner), V, device="cuda", generator=gen(k)) * 2).to(DT[dtype])
        values = torch.randn(len(owner), k, device="cuda", generator=gen(k + 1))
        order = torch.rand(len(owner), max(V, k), device="cuda", generator=gen(k + 2)).argsort(1).int()[:, :k]
        ids = torch.where(order < V, order, -1).contiguous()
        rest = torch.randn(len(owner), device="cuda", generator=gen(k + 3))
        if V <= k:
            rest = rest * 0 - float("inf")              # no output is without a place
        want = D.expected(x, values, ids, rest, tau, owner, live, 3, 1.0, "sum")
        lead = (3, max(T), max(U) + 1) if padded else (len(owner),)
        if padded:
            x[torch.as_tensor(~live, device="cuda")] = float("nan")
        leaf = x.view(*lead, V).clone().requires_grad_()
        loss = rnnt_distill_loss(leaf, values.view(*lead, k), ids.view(*lead, k), i32(T), i32(U), rest.view(lead),
                                 temperature=tau, reduction="sum")
        grad, = torch.autograd.grad(loss, leaf)
        D.check_distill(leaf, loss, grad, want, DT[dtype])
        assert (grad.reshape(-1, V)[torch.as_tensor(~live, device="cuda")] == 0).all()


@pytest.mark.parametrize("V", [29, 200, 1024, 5000, 70000])
def test_rests_far_from_the_places(V):
    """A rest and places at opposite ends of float32: one has all the weight, and the loss is that of it alone."""
    x = torch.randn(4, V, device="cuda", generator=gen(6)).requires_grad_()
    ids, T, U = i32([[3, 1]] * 4), i32([1] * 4), i32([0] * 4)
    values = torch.tensor([[3e38, 3e38], [-3e38, -3e38], [3e38, -3e38], [-3e38, -float("inf")]], device="cuda")
    rest = torch.tensor([-3e38, 3e38, -3.4e38, 3.4e38], device="cuda")
    places = torch.tensor([[0.0, 0.0], [-float("inf")] * 2, [0.0, -float("inf")], [-float("inf")] * 2], device="cuda")
    rests = torch.tensor([-float("inf"), 0.0, -float("inf"), 0.0], device="cuda")
    for tau in (1.0, 0.1, 7.0):
        got, want = (rnnt_distill_loss(x, v, ids, T, U, r, temperature=tau, reduction="none")
                     for v, r in ((values, rest), (places, rests)))
        assert torch.isfinite(got).all() and torch.equal(got, want)
        assert torch.equal(*(torch.autograd.grad(y.sum(), x)[0] for y in (got, want)))


@pytest.mark.parametrize("dtype", list(DT))
def test_largest_vocabulary(dtype):
    V, k = 1 << 20, 64
    x = torch.randn(3, V, device="cuda", generator=gen(9)).to(DT[dtype])
    top = rnnt_top_logits(x, k, temperature=2.0)
    order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(top[1], order.int()) and torch.equal(top[0], x.gather(1, order))
    y = x.double() / 2.0
    want = torch.logsumexp(y.scatter(1, order, -float("inf")), 1)
    assert (top[2].double() - want).abs().max() <= R.SUM * 20          # 1024 terms a thread instead of 256
    student = (x.float() + torch.randn(3, V, device="cuda", generator=gen(10))).to(DT[dtype]).requires_grad_()
    loss = rnnt_distill_loss(student, *top[:2], i32([2, 1]), i32([0, 0]), top[2], temperature=2.0, reduction="none")
    grad, = torch.autograd.grad(loss.sum(), student)
    log_q = torch.log_softmax(student.detach().double() / 2.0, 1)
    log_p = torch.log_softmax(torch.cat([top[0].double() / 2.0, top[2].double()[:, None]], 1), 1)
    left = torch.logsumexp(log_q.scatter(1, order, -float("inf")), 1, keepdim=True)
    rows = 4.0 * (log_p.exp() * (log_p - torch.cat([log_q.gather(1, order), left], 1))).sum(1)
    rows = torch.stack([rows[0] + rows[1], rows[2]])
    # the rest's sum may be off by SUM * 20 of itself, which counts |p_r - q_r| times
    apart = 4.0 * (log_p[:, -1].exp() - left[:, 0].exp()).abs().sum()
    assert ((loss.double() - rows).abs() <= R.SUM * 20 * apart + 1e-6 * rows).all()
    q = log_q.exp()
    g = 2.0 * (q - q * (log_p[:, -1:] - left).exp()).scatter(1, order, 0.0)
    g = g.scatter(1, order, 2.0 * (q.gather(1, order) - log_p[:, :k].exp()))
    part = 2.0 * (q + q * (log_p[:, -1:] - left).exp()).scatter(1, order, 1.0)
    limit = part * R.SUM * 20 + g.abs() * L.half_step(DT[dtype]) * 1.001 + L.smallest(DT[dtype])
    assert ((grad.double() - g).abs() <= limit).all()
