"""Cases of the operators by which a transducer learns from a teacher: the teacher's top logits, the
distillation loss with its gradient, and the sampling of labels.

``listed()`` and ``draw(rng)`` give cases, ``prepare`` a program's data for one, ``run`` one pass
(elementary torch operations, or the package's operators where ``own`` is true), ``work`` the bytes
and operations a pass cannot do without, ``exact`` the outputs in 64 bits.
"""
import math
import random
from functools import lru_cache

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_CHUNK = 1 << 26                   # elements of a piece of the 64-bit forms


# ------------------------------------------------------------------------------------ cases
def _top(B, T, U, V, k, dtype, padded=False, temperature=1.0, masked=0.0):
    return {"op": "top", "B": B, "T0": T[0], "T1": T[1], "U0": U[0], "U1": U[1], "V": V, "k": k,
            "dtype": dtype, "padded": padded, "temperature": temperature, "masked": masked}


def _distill(B, T, U, V, k, dtype, train, rest, reduction, padded=False, temperature=1.0,
             weight=1.0):
    return {"op": "distill", "B": B, "T0": T[0], "T1": T[1], "U0": U[0], "U1": U[1], "V": V, "k": k,
            "dtype": dtype, "train": train, "rest": rest, "reduction": reduction,
            "padded": padded, "temperature": temperature, "weight": weight}


def _sample(B, K, V, dtype, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, finished=0.0,
            fused=True, masked=0.0):
    return {"op": "sample", "B": B, "K": K, "V": V, "dtype": dtype, "temperature": temperature,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "finished": finished, "fused": fused,
            "masked": masked}


def listed():
    return [
        # A teacher's rows of the smallest workload: latency.
        dict(_top(2, (6, 8), (2, 3), 16, 4, "f32"), name="top tiny"),
        # A teacher over a BPE ASR batch (about 480000 lattice rows), eight outputs a row kept.
        dict(_top(16, (300, 500), (50, 100), 1024, 8, "f16", temperature=2.0), name="top bpe"),
        # Long utterances, a large vocabulary, more outputs kept.
        dict(_top(2, (500, 1000), (100, 200), 5000, 32, "f32"), name="top large vocabulary"),
        # A student's training step on the smallest workload: latency of the autograd call.
        dict(_distill(2, (6, 8), (2, 3), 16, 4, "f32", True, False, "none"), name="distill tiny"),
        # Character ASR: short rows, odd vocabulary; the teacher's rest as a class of its own.
        dict(_distill(32, (150, 200), (20, 40), 29, 8, "f32", True, True, "mean"),
             name="distill char"),
        # BPE ASR training step, softened by a temperature, a tenth of the student's loss.
        dict(_distill(16, (300, 500), (50, 100), 1024, 8, "f16", True, True, "sum",
                      temperature=2.0, weight=0.1), name="distill bpe"),
        # Validation: the loss alone, the padded layout, the teacher's top taken as the whole.
        dict(_distill(16, (300, 500), (50, 100), 1024, 16, "bf16", False, False, "mean",
                      padded=True), name="distill bpe loss"),
        # Long utterances, a large vocabulary, training step.
        dict(_distill(2, (500, 1000), (100, 200), 5000, 32, "f32", True, True, "mean"),
             name="distill large vocabulary"),
        # Serving, one utterance, four drawn hypotheses: the latency of one step.
        dict(_sample(1, 4, 1024, "f16", temperature=0.7, top_k=40), name="sample 1x4x1024"),
        # Drawn labels of a batch of character-ASR utterances, some already finished.
        dict(_sample(32, 10, 29, "f32", finished=0.25), name="sample 32x10x29"),
        # 5000 sub-words, log-probabilities from the model, the nucleus alone.
        dict(_sample(16, 8, 5000, "f32", temperature=0.8, top_p=0.95, fused=False),
             name="sample 16x8x5000"),
        # Bulk drawing for sequence-level distillation, a vocabulary of 50000.
        dict(_sample(64, 16, 50000, "bf16", top_p=0.9, min_p=0.002, finished=0.1),
             name="sample 64x16x50000"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("top", "distill", "sample"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    temperature = rng.choice((1.0, 1.0, 2.0, 4.0, 0.5))
    if op == "sample":
        while True:
            B, K, V = _log(rng, 1, 64), _log(rng, 1, 32), _log(rng, 16, 50000)
            if B * K * V * _SIZE[dtype] <= 100e6:
                break
        temperature = rng.choice((1.0, 0.6, 0.8, 1.3))
        top_k = _log(rng, 1, 200) if rng.random() < 0.4 else 0
        top_p = rng.choice((0.5, 0.8, 0.9, 0.95, 0.99)) if rng.random() < 0.5 else 1.0
        min_p = rng.choice((0.001, 0.02, 0.1)) if rng.random() < 0.3 else 0.0
        return _sample(B, K, V, dtype, temperature, top_k, top_p, min_p,
                       rng.choice((0.0, 0.0, 0.2)), rng.random() < 0.8,
                       rng.choice((0.0, 0.0, 0.5)))
    while True:
        B, T, U = _log(rng, 1, 64), _log(rng, 1, 1500), _log(rng, 1, 300) - 1
        V = _log(rng, 16, 50000)
        if rng.random() < 0.6:
            V = (V + 7) // 8 * 8
        if 1000 <= B * T * (U + 1) * V * _SIZE[dtype] <= 1.5e9:
            break
    T, U = (max(1, T // 2), T), (U // 2, U)
    k = min(_log(rng, 1, 64), V)
    padded = rng.random() < 0.3
    if op == "top":
        return _top(B, T, U, V, k, dtype, padded, temperature, rng.choice((0.0, 0.0, 0.5)))
    return _distill(B, T, U, V, k, dtype, rng.random() < 0.7, rng.random() < 0.6,
                    rng.choice(("none", "sum", "mean")), padded, temperature,
                    rng.choice((1.0, 0.5)))


# ---------------------------------------------------------------------------------- inputs
@lru_cache(maxsize=64)
def _drawn_lengths(B, T0, T1, U0, U1):
    rng = random.Random(f"{B} {T0} {T1} {U0} {U1}")
    return ([rng.randint(T0, T1) for _ in range(B)], [rng.randint(U0, U1) for _ in range(B)])


def _lengths(case):
    """(T, U) of a case's utterances: part of the case, the same for every seed."""
    return _drawn_lengths(case["B"], case["T0"], case["T1"], case["U0"], case["U1"])


def _rows(case):
    T, U = _lengths(case)
    return sum(t * (u + 1) for t, u in zip(T, U))


def _logits(shape, gen, dt, masked):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=dt) * 2.0
    x[..., 0] += 4.0                # the blank is likely, as in most rows of a transducer
    if masked:                      # outputs that a grammar rules out
        off = torch.rand(shape[-1], generator=gen, device="cuda") < masked
        off[0] = False
        x[..., off] = -math.inf
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    state = {"case": case}
    if case["op"] == "sample":
        B, K, V = case["B"], case["K"], case["V"]
        logits = _logits((B, K, V), gen, dt, case["masked"])
        if not case["fused"]:
            logits = torch.log_softmax(logits.float(), -1).to(dt)
        state["logits"] = logits
        state["scores"] = -20.0 * torch.rand(B, K, generator=gen, device="cuda")
        state["random"] = torch.rand(B, K, generator=gen, device="cuda")
        state["finished"] = (torch.rand(B, K, generator=gen, device="cuda")
                             < case["finished"]) if case["finished"] else None
        return state
    T, U = _lengths(case)
    state["T"] = torch.tensor(T, dtype=torch.int32, device="cuda")
    state["U"] = torch.tensor(U, dtype=torch.int32, device="cuda")
    V = case["V"]
    shape = (case["B"], max(T), max(U) + 1, V) if case["padded"] else (_rows(case), V)
    logits = _logits(shape, gen, dt, case.get("masked", 0.0))
    if case["op"] == "distill":
        teacher = torch.randn(shape, generator=gen, device="cuda", dtype=dt).add_(logits)
        values, ids = torch.topk(teacher, case["k"], dim=-1)
        state["values"], state["ids"], state["rest"] = values, ids.int(), None
        if case["rest"]:
            left = teacher.float().div_(case["temperature"]).scatter_(-1, ids, -math.inf)
            state["rest"] = torch.logsumexp(left, -1)
        logits.requires_grad_(case["train"])
    state["logits"] = logits
    return state


def _live(case, T, U):
    """Which rows of a padded case belong to an utterance (None: all, of a compact one)."""
    if not case["padded"]:
        return None
    t = torch.arange(max(_lengths(case)[0]), device=T.device)
    u = torch.arange(max(_lengths(case)[1]) + 1, device=T.device)
    return ((t < T[:, None])[:, :, None] & (u <= U[:, None])[:, None, :]).reshape(-1)


def _owners(case, T, U):
    """The utterance of every row."""
    b = torch.arange(case["B"], device=T.device)
    if case["padded"]:
        each = max(_lengths(case)[0]) * (max(_lengths(case)[1]) + 1)
        return b[:, None].expand(-1, each).reshape(-1)
    return torch.repeat_interleave(b, (T * (U + 1)).long(), output_size=_rows(case))


# ----------------------------------------------------------------------------------- a pass
def run(state):
    case = state["case"]
    return {"top": _run_top, "distill": _run_distill, "sample": _run_sample}[case["op"]](
        state, case)


def _order(x):
    """int64 keys in the order of the values, and of the lower place where values are equal."""
    bits = (x.float() + 0.0).view(torch.int32).long()   # + 0.0: one zero
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    V = x.shape[-1]
    return bits * (1 << 32) + torch.arange(V - 1, -1, -1, device=x.device)


def _log_sum(s):
    """log of the sum of exp(s) over the last axis, -inf where there is nothing."""
    top = s.amax(-1)
    none = torch.isneginf(top)
    total = (s - torch.where(none, 0.0, top)[..., None]).exp().sum(-1)
    return torch.where(none, top, total.log() + top)


def _run_top(state, case):
    x, V, k = state["logits"], case["V"], case["k"]
    if own:
        from rnn_transducer_loss_gb300 import rnnt_top_logits
        lengths = (state["T"], state["U"]) if case["padded"] else (None, None)
        return list(rnnt_top_logits(x, k, *lengths, temperature=case["temperature"], check=False))
    rows = x.reshape(-1, V)
    ids = (V - 1) - (torch.topk(_order(rows), k, dim=1).values & 0xFFFFFFFF)
    values = rows.gather(1, ids)
    rest = _log_sum((rows.float() / case["temperature"]).scatter_(1, ids, -math.inf))
    none = torch.isneginf(values)
    live = _live(case, state["T"], state["U"])
    if live is not None:
        none = none | ~live[:, None]
        rest = torch.where(live, rest, -math.inf)
    values = values.masked_fill(none, -math.inf)
    ids = ids.masked_fill(none, -1).int()
    lead = x.shape[:-1]
    return [values.reshape(lead + (k,)), ids.reshape(lead + (k,)), rest.reshape(lead)]


def _run_distill(state, case):
    x, tau, V, B = state["logits"], case["temperature"], case["V"], case["B"]
    if own:
        from rnn_transducer_loss_gb300 import rnnt_distill_loss
        loss = rnnt_distill_loss(x, state["values"], state["ids"], state["T"], state["U"],
                                 teacher_rest=state["rest"], temperature=tau,
                                 weight=case["weight"], reduction=case["reduction"], check=False)
        if not case["train"]:
            return [loss]
        grad, = torch.autograd.grad(loss, x, torch.ones_like(loss))
        return [loss, grad]
    s = x.detach().reshape(-1, V).float() / tau
    ids = state["ids"].reshape(-1, case["k"]).long()
    places = ids >= 0
    t = torch.where(places, state["values"].reshape(ids.shape).float() / tau, -math.inf)
    if case["rest"]:
        t = torch.cat([t, state["rest"].reshape(-1, 1)], 1)
    whole = _log_sum(t)
    log_p = t - torch.where(torch.isneginf(whole), 0.0, whole)[:, None]
    p = log_p.exp()
    top = s.amax(1, keepdim=True)
    at = s.gather(1, ids.clamp_min(0)) - top
    e = s.sub_(top).exp_()
    total = e.sum(1, keepdim=True)
    log_q = at - total.log()
    left = torch.zeros(1, device=x.device)
    if case["rest"]:
        # the terms of the outputs that are not the teacher's, behind a place for empty ids
        others = torch.cat([e, e.new_zeros(e.shape[0], 1)], 1)
        others = others.scatter_(1, torch.where(places, ids, V), 0.0)[:, :V]
        left = others.sum(1, keepdim=True)
        log_q = torch.cat([log_q, left.log() - total.log()], 1)
    row = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(1).double()
    live = _live(case, state["T"], state["U"])
    if live is not None:
        row = torch.where(live, row, 0.0)
    loss = torch.zeros(B, dtype=torch.float64, device=x.device)
    loss.index_add_(0, _owners(case, state["T"], state["U"]), row)
    loss *= tau * tau * case["weight"]
    scale = tau * case["weight"]
    if case["reduction"] == "mean":
        scale /= B
    loss = {"none": loss, "sum": loss.sum(), "mean": loss.sum() / B}[case["reduction"]].float()
    if not case["train"]:
        return [loss]
    g = e / total
    if case["rest"]:
        part = torch.where(left > 0, p[:, -1:] / left, 0.0)
        g -= others * part
    g.scatter_add_(1, ids.clamp_min(0), torch.where(places, -p[:, :case["k"]], 0.0))
    alive = p.sum(1) > 0
    if live is not None:
        alive = alive & live
    g = torch.where(alive[:, None], g.mul_(scale), 0.0)
    return [loss, g.to(x.dtype).reshape(x.shape)]


def _run_sample(state, case):
    logits, scores, finished = state["logits"], state["scores"], state["finished"]
    if own:
        from rnn_transducer_loss_gb300 import rnnt_sample
        return list(rnnt_sample(logits, scores, state["random"], temperature=case["temperature"],
                                top_k=case["top_k"] or None, top_p=case["top_p"],
                                min_p=case["min_p"], finished=finished,
                                fused_log_softmax=case["fused"], check=False))
    V, tau = case["V"], case["temperature"]
    x = logits.double().reshape(-1, V)      # 64 bits: sums that end next to a border
    x, at = torch.sort(x, dim=1, descending=True, stable=True)
    top = x[:, :1]
    e = ((x - top) / tau).exp()
    keep = ~torch.isneginf(x)
    if case["top_k"]:
        keep[:, case["top_k"]:] = False
    if case["top_p"] < 1.0:
        e = torch.where(keep, e, 0.0)
        ahead = e.cumsum(1) - e
        keep &= ahead < case["top_p"] * e.sum(1, keepdim=True)
    if case["min_p"] > 0.0:
        keep &= x - top >= tau * math.log(case["min_p"])
    e = torch.where(keep, e, 0.0)
    kept = torch.empty_like(e).scatter_(1, at, e)               # by id
    running = kept.cumsum(1)
    border = state["random"].double().reshape(-1, 1) * running[:, -1:]
    token = (running <= border).sum(1, keepdim=True)
    last = torch.where(kept > 0, torch.arange(V, device=x.device), 0).amax(1, keepdim=True)
    token = torch.minimum(token, last)
    log_p = logits.double().reshape(-1, V).gather(1, token)
    if case["fused"]:
        log_p = log_p - ((x - top).exp().sum(1, keepdim=True).log() + top)
    value = scores.double() + log_p.reshape(scores.shape)
    token = token.reshape(scores.shape).int()
    if finished is not None:
        value = torch.where(finished, scores.double(), value)
        token = torch.where(finished, -1, token)
    return [value.float(), token]


# -------------------------------------------------------------------------------- the floor
def work(case):
    s = _SIZE[case["dtype"]]
    if case["op"] == "sample":
        rows = case["B"] * case["K"]
        read = rows * (1 - case["finished"]) * case["V"]
        return {"bytes": read * s + rows * (4 + 4 + (1 if case["finished"] else 0) + 8),
                "flops": read * (4 if case["fused"] else 3)}
    rows, V, k = _rows(case), case["V"], case["k"]
    T, U = _lengths(case)
    out = case["B"] * max(T) * (max(U) + 1) if case["padded"] else rows
    if case["op"] == "top":
        return {"bytes": rows * V * s + out * (k * (s + 4) + 4), "flops": rows * V * 4}
    teacher = rows * (k * (s + 4) + (4 if case["rest"] else 0))
    read = rows * V * s + teacher + 8 * case["B"]
    if not case["train"]:
        return {"bytes": read + 4, "flops": rows * V * 4}
    return {"bytes": read + out * V * s + 4, "flops": rows * V * 6}


# ---------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(state, case)
    x = state["logits"].detach()
    V, k, tau = case["V"], case["k"], case["temperature"]
    flat = x.reshape(-1, V)
    N = flat.shape[0]
    live = _live(case, state["T"], state["U"])
    step = max(1, _CHUNK // V)
    if case["op"] == "top":
        rest = torch.empty(N, dtype=torch.float64, device="cuda")
        values = torch.empty(N, k, dtype=torch.float64, device="cuda")
        for i in range(0, N, step):
            y = flat[i:i + step].double()
            best = torch.topk(y, k, dim=1)
            values[i:i + step] = best.values
            rest[i:i + step] = torch.logsumexp((y / tau).scatter_(1, best.indices, -math.inf), 1)
        if live is not None:
            values[~live], rest[~live] = -math.inf, -math.inf
        return [values.reshape(x.shape[:-1] + (k,)), None, rest.reshape(x.shape[:-1])]
    ids = state["ids"].reshape(N, k).long()
    values = state["values"].reshape(N, k).double()
    total = torch.zeros(case["B"], dtype=torch.float64, device="cuda")
    owner = _owners(case, state["T"], state["U"])
    factor = case["weight"] / (case["B"] if case["reduction"] == "mean" else 1)
    grad = torch.zeros(N, V, dtype=torch.float64, device="cuda") if case["train"] else None
    for i in range(0, N, step):
        part = slice(i, i + step)
        log_q = torch.log_softmax(flat[part].double() / tau, 1)
        at, places = ids[part], ids[part] >= 0
        goal = (values[part] / tau).masked_fill(~places, -math.inf)
        mine = log_q.gather(1, at.clamp_min(0))
        if case["rest"]:
            goal = torch.cat([goal, state["rest"].reshape(N, 1)[part].double()], 1)
            covered = torch.zeros_like(log_q, dtype=torch.bool)
            row, col = places.nonzero(as_tuple=True)
            covered[row, at[row, col]] = True
            left = torch.logsumexp(log_q.masked_fill(covered, -math.inf), 1, keepdim=True)
            mine = torch.cat([mine, left], 1)
        some = (goal > -math.inf).any(1)
        if live is not None:
            some = some & live[part]
        log_p = torch.log_softmax(goal.masked_fill(~some[:, None], 0.0), 1)
        p = log_p.exp()
        kl = torch.where(p > 0, p * (log_p - mine), 0.0).sum(1).masked_fill(~some, 0.0)
        total.index_add_(0, owner[part], kl * tau * tau)
        if grad is None:
            continue
        q = log_q.exp()
        if case["rest"]:
            goal_of_rest = torch.where(covered, 0.0, p[:, -1:] * (log_q - left).exp())
            q -= goal_of_rest.nan_to_num_(0.0)
        q.scatter_add_(1, at.clamp_min(0), torch.where(places, -p[:, :k], 0.0))
        grad[part] = q.masked_fill_(~some[:, None], 0.0) * (tau * factor)
    loss = total * factor if case["reduction"] == "none" else total.sum() * factor
    return [loss] if grad is None else [loss, grad.reshape(x.shape)]


def _exact_sample(state, case):
    V, tau = case["V"], case["temperature"]
    x = state["logits"].double().reshape(-1, V)
    u = state["random"].double().reshape(-1)
    scores = state["scores"].double().reshape(-1)
    token = torch.empty(x.shape[0], dtype=torch.int64, device="cuda")
    value = torch.empty_like(scores)
    place = torch.arange(V, device="cuda")
    for r in range(x.shape[0]):
        row = x[r]
        some = (row > -math.inf).nonzero()[:, 0]
        some = some[torch.argsort(-row[some], stable=True)]
        if case["top_k"]:
            some = some[:case["top_k"]]
        p = torch.softmax(row[some] / tau, 0)
        if case["top_p"] < 1.0:
            reached = torch.cumsum(p, 0)
            # the first place at which the mass is reached is the last one kept
            some = some[:1 + int((reached < case["top_p"]).sum())]
        if case["min_p"] > 0.0:
            some = some[row[some] - row.amax() >= tau * math.log(case["min_p"])]
        allowed = torch.isin(place, some)
        p = torch.softmax(torch.where(allowed, row / tau, -math.inf), 0)
        by_id = torch.cumsum(p, 0) / p.sum()
        i = torch.searchsorted(by_id, u[r:r + 1], right=True).clamp_max_(int(some.max()))
        token[r] = i[0]
        lse = torch.logsumexp(row, 0) if case["fused"] else 0.0
        value[r] = scores[r] + row[i[0]] - lse
    if state["finished"] is not None:
        done = state["finished"].reshape(-1)
        token, value = torch.where(done, -1, token), torch.where(done, scores, value)
    shape = state["scores"].shape
    return [value.reshape(shape), token.int().reshape(shape)]
