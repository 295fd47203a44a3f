"""Cases of the label-side operators: label embedding, its gradient, beam selection and the
reordering of beam states.

``listed()`` and ``draw(rng)`` give cases, ``prepare`` a program's data for one, ``run`` one pass
(elementary torch operations, or the package's operators where ``own`` is true), ``work`` the bytes
and operations a pass cannot do without, ``exact`` the outputs in 64 bits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2, "i32": 4}


# ------------------------------------------------------------------------------------ cases
def _embed(B, S, low, V, D, dtype, start, zipf=False):
    return {"op": "embed", "B": B, "S": S, "low": low, "V": V, "D": D, "dtype": dtype,
            "start": start, "zipf": zipf}


def _grad(B, S, low, V, D, dtype, start, zipf=False, train=False):
    return {"op": "grad", "B": B, "S": S, "low": low, "V": V, "D": D, "dtype": dtype,
            "start": start, "zipf": zipf, "train": train}


def _select(B, K, Ko, V, dtype, finished=0.0, fused=True):
    return {"op": "select", "B": B, "K": K, "Ko": Ko, "V": V, "dtype": dtype,
            "finished": finished, "fused": fused}


def _reorder(kind, B, K, layers, width, length, capacity, dtype):
    return {"op": "reorder", "kind": kind, "B": B, "K": K, "layers": layers, "width": width,
            "length": length, "capacity": capacity, "dtype": dtype}


def listed():
    return [
        # Serving, one utterance: the four labels just selected enter the prediction network.
        dict(_embed(1, 4, 4, 1024, 512, "f16", False), name="embed 4 labels"),
        # Training, BPE ASR: 16 utterances of 50 to 100 labels behind the start symbol.
        dict(_embed(16, 100, 50, 1024, 512, "f16", True), name="embed bpe targets"),
        # Training, the longest targets the loss takes, a large vocabulary.
        dict(_embed(64, 1023, 255, 50000, 1024, "bf16", True, True), name="embed long targets"),
        # Training, character ASR: few ids, each of them many times; an odd width.
        dict(_grad(32, 40, 20, 29, 301, "f32", True), name="grad char"),
        # Training step of the lookup through autograd, BPE ASR.
        dict(_grad(16, 100, 50, 1024, 512, "f32", True, False, True), name="embed+grad bpe"),
        # The longest targets, a large vocabulary, ids as unevenly frequent as words.
        dict(_grad(64, 1023, 255, 50000, 1024, "bf16", True, True), name="grad long targets"),
        # Serving, one utterance, beam of 4: the latency of one decoding step.
        dict(_select(1, 4, 4, 1024, "f16"), name="select 1x4x1024"),
        # A batch of character-ASR utterances, some hypotheses already finished; odd vocabulary.
        dict(_select(32, 10, 10, 29, "f32", 0.25), name="select 32x10x29"),
        # A batch of utterances, 5000 sub-words, log-probabilities from the model.
        dict(_select(16, 8, 8, 5000, "f32", 0.0, False), name="select 16x8x5000"),
        # Bulk decoding, wide beams, a vocabulary of 50000.
        dict(_select(64, 16, 16, 50000, "bf16", 0.1), name="select 64x16x50000"),
        # States of a two-layer recurrent predictor and the label history of 16 x 8 hypotheses.
        dict(_reorder("lstm", 16, 8, 2, 640, 101, 101, "f32"), name="reorder lstm"),
        # Key-value caches of an attention predictor, 401 of 512 places filled.
        dict(_reorder("cache", 32, 8, 2, 8, 401, 512, "f16"), name="reorder cache"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("embed", "grad", "select", "reorder"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op in ("embed", "grad"):
        while True:
            B, S = _log(rng, 1, 64), _log(rng, 1, 1023)
            V, D = _log(rng, 29, 50000), _log(rng, 32, 2048)
            if rng.random() < 0.6:
                D = (D + 7) // 8 * 8
            if (B * (S + 1) + V) * D * _SIZE[dtype] <= 200e6:
                break
        low = rng.randint(0, S) if rng.random() < 0.7 else S
        more = (B, S, low, V, D, dtype, rng.random() < 0.7, rng.random() < 0.5)
        return _embed(*more) if op == "embed" else _grad(*more, rng.random() < 0.3)
    if op == "select":
        while True:
            B, K, V = _log(rng, 1, 64), _log(rng, 1, 32), _log(rng, 29, 50000)
            if B * K * V * _SIZE[dtype] <= 100e6:
                break
        Ko = K if rng.random() < 0.7 else _log(rng, 1, 32)
        return _select(B, K, Ko, V, dtype, rng.choice((0.0, 0.0, 0.2)), rng.random() < 0.8)
    if rng.random() < 0.5:
        return _reorder("lstm", _log(rng, 1, 64), _log(rng, 1, 32), rng.randint(1, 4),
                        _log(rng, 64, 1280), 0, 0, dtype) | _lengths(rng, 1, 400)
    while True:
        case = _reorder("cache", _log(rng, 1, 64), _log(rng, 1, 16), rng.randint(1, 4),
                        rng.choice((4, 8, 16)), 0, 0, dtype) | _lengths(rng, 1, 1000)
        if _reorder_rows(case) * case["width"] * 64 * case["length"] * _SIZE[dtype] <= 400e6:
            return case


def _lengths(rng, low, high):
    n = _log(rng, low, high)
    return {"length": n, "capacity": n + rng.choice((0, 1, 24, 111))}


def _reorder_rows(case):
    return 2 * case["layers"] * case["B"] * case["K"]


# ---------------------------------------------------------------------------------- inputs
def _tokens(case, gen):
    B, S, V = case["B"], case["S"], case["V"]
    u = torch.rand(B, S, generator=gen, device="cuda", dtype=torch.float64)
    # ids by frequency rank: id r about as often as 1 / (r + 1), or all equally often
    ids = torch.exp(u * math.log(V + 1.0)) - 1.0 if case["zipf"] else u * V
    tokens = ids.to(torch.int32).clamp_(0, V - 1)
    lengths = torch.randint(case["low"], S + 1, (B,), generator=gen, device="cuda",
                            dtype=torch.int32)
    return tokens, lengths


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    state = {"case": case}
    if case["op"] in ("embed", "grad"):
        B, S, V, D = case["B"], case["S"], case["V"], case["D"]
        state["tokens"], state["lengths"] = _tokens(case, gen)
        if case["op"] == "embed" or case["train"]:
            state["weight"] = torch.randn(V, D, generator=gen, device="cuda", dtype=dt) * D ** -0.5
            state["weight"].requires_grad_(case["op"] == "grad")
        if case["op"] == "grad":
            shape = (B, S + (1 if case["start"] else 0), D)
            state["grad_out"] = torch.randn(shape, generator=gen, device="cuda", dtype=dt) * 0.01
    elif case["op"] == "select":
        B, K, V = case["B"], case["K"], case["V"]
        logits = torch.randn(B, K, V, generator=gen, device="cuda", dtype=dt) * 2.0
        # the blank is likely, as in most steps of a transducer
        logits[:, :, 0] += 4.0
        if not case["fused"]:
            logits = torch.log_softmax(logits.float(), -1).to(dt)
        state["logits"] = logits
        steps = torch.rand(B, K, generator=gen, device="cuda") * 0.6
        state["scores"] = -20.0 - torch.cumsum(steps, 1)
        state["finished"] = (torch.rand(B, K, generator=gen, device="cuda")
                             < case["finished"]) if case["finished"] else None
    else:
        B, K, layers = case["B"], case["K"], case["layers"]
        n, cap = case["length"], case["capacity"]
        if case["kind"] == "lstm":
            shape = (layers, B, K, case["width"])
            state["states"] = [torch.randn(shape, generator=gen, device="cuda", dtype=dt)
                               for _ in range(2)]
            history = torch.randint(0, 1024, (B, K, cap), generator=gen, device="cuda",
                                    dtype=torch.int32)
            state["states"].append(history[:, :, :n])
            state["dims"] = [1, 1, 0]
        else:
            shape = (B, K, case["width"], cap, 64)
            state["states"] = [torch.randn(shape, generator=gen, device="cuda",
                                           dtype=dt)[:, :, :, :n] for _ in range(2 * layers)]
            state["dims"] = [0] * (2 * layers)
        parents = torch.randint(0, K, (B, K), generator=gen, device="cuda", dtype=torch.int32)
        state["parents"] = parents
    return state


def _start(case):
    return 0 if case["start"] else None


def _ids(case, tokens, lengths):
    """(ids, valid) of every position, the start symbol's among them."""
    S = case["S"]
    valid = torch.arange(S, device=tokens.device)[None, :] < lengths[:, None]
    ids = tokens.long()
    if case["start"]:
        first = torch.zeros_like(ids[:, :1])
        ids = torch.cat([first, ids], 1)
        valid = torch.cat([torch.ones_like(first, dtype=torch.bool), valid], 1)
    return ids, valid


def _scale(case):
    return math.sqrt(case["D"])


# ----------------------------------------------------------------------------------- a pass
def run(state):
    case = state["case"]
    return {"embed": _run_embed, "grad": _run_grad, "select": _run_select,
            "reorder": _run_reorder}[case["op"]](state, case)


def _plain_embed(weight, ids, valid, scale):
    out = weight.detach()[ids].float() * scale
    return torch.where(valid[:, :, None], out, 0.0).to(weight.dtype)


def _run_embed(state, case):
    if own:
        from rnn_transducer_loss_gb300 import rnnt_embed
        return rnnt_embed(state["weight"], state["tokens"], state["lengths"],
                          start=_start(case), scale=_scale(case), check=False)
    ids, valid = _ids(case, state["tokens"], state["lengths"])
    return _plain_embed(state["weight"], ids, valid, _scale(case))


def _run_grad(state, case):
    if own and case["train"]:
        from rnn_transducer_loss_gb300 import rnnt_embed
        out = rnnt_embed(state["weight"], state["tokens"], state["lengths"],
                         start=_start(case), scale=_scale(case), check=False)
        grad, = torch.autograd.grad(out, state["weight"], state["grad_out"])
        return [out, grad]
    if own:
        from rnn_transducer_loss_gb300 import rnnt_embed_grad
        return [rnnt_embed_grad(state["grad_out"], state["tokens"], case["V"], state["lengths"],
                                start=_start(case), scale=_scale(case), check=False)]
    ids, valid = _ids(case, state["tokens"], state["lengths"])
    out = [_plain_embed(state["weight"], ids, valid, _scale(case))] if case["train"] else []
    V, D = case["V"], case["D"]
    rows = state["grad_out"].float().reshape(-1, D) * _scale(case)
    where = torch.where(valid, ids, V).reshape(-1)      # what is padding goes to a row of its own
    total = torch.zeros(V + 1, D, device=rows.device).index_add_(0, where, rows)
    return out + [total[:V].to(state["grad_out"].dtype)]


def _order(x):
    """int64 keys in the order of the values, and of the lower place where values are equal."""
    bits = (x.float() + 0.0).view(torch.int32).long()   # + 0.0: one zero
    bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    V = x.shape[-1]
    return bits * (1 << 32) + torch.arange(V - 1, -1, -1, device=x.device)


def _run_select(state, case):
    logits, scores, finished = state["logits"], state["scores"], state["finished"]
    B, K, V, Ko = case["B"], case["K"], case["V"], case["Ko"]
    if own:
        from rnn_transducer_loss_gb300 import rnnt_beam_select
        return list(rnnt_beam_select(logits, scores, Ko, finished=finished,
                                     fused_log_softmax=case["fused"], check=False))
    n = min(Ko, V)
    token = (V - 1) - (torch.topk(_order(logits), n, dim=2).values & 0xFFFFFFFF)   # (B, K, n)
    x = logits.double()                 # 64 bits: the order of candidates next to one another
    best = x.gather(2, token)
    if case["fused"]:
        top = x.amax(2, keepdim=True)
        best = best - ((x - top).exp().sum(2, keepdim=True).log() + top)
    value = scores.double()[:, :, None] + best
    parent = torch.arange(K, device=x.device)[None, :, None].expand(B, K, n)
    if finished is not None:            # one candidate: the hypothesis as it is
        alone = torch.full_like(value, -math.inf)
        alone[:, :, 0] = scores.double()
        value = torch.where(finished[:, :, None], alone, value)
        token = torch.where(finished[:, :, None], -1, token)
    value, token, parent = value.reshape(B, -1), token.reshape(B, -1), parent.reshape(B, -1)
    if value.shape[1] < Ko:
        more = (0, Ko - value.shape[1])
        value = torch.nn.functional.pad(value, more, value=-math.inf)
        token = torch.nn.functional.pad(token, more, value=-1)
        parent = torch.nn.functional.pad(parent, more, value=-1)
    value, at = torch.sort(value, dim=1, descending=True, stable=True)
    value, at = value[:, :Ko], at[:, :Ko]
    none = torch.isneginf(value)
    token = torch.where(none, -1, token.gather(1, at)).int()
    parent = torch.where(none, -1, parent.gather(1, at)).int()
    return [value.float(), token, parent]


def _gather(x, parents, dim):
    """x with its beam axis (the one after `dim`, the batch's) taken by parents (B, K)."""
    shape = [1] * x.dim()
    shape[dim], shape[dim + 1] = parents.shape
    at = parents.long().clamp_min(0).reshape(shape)
    got = torch.take_along_dim(x, at.expand(x.shape[:dim] + parents.shape + x.shape[dim + 2:]),
                               dim + 1)
    return torch.where((parents < 0).reshape(shape), torch.zeros((), dtype=x.dtype,
                                                                 device=x.device), got)


def _run_reorder(state, case):
    if own:
        from rnn_transducer_loss_gb300 import rnnt_beam_reorder
        return rnnt_beam_reorder(state["states"], state["parents"], batch_dim=state["dims"],
                                 check=False)
    at = state["parents"].long()
    rows = torch.arange(at.shape[0], device=at.device)[:, None]
    out = []
    for x, dim in zip(state["states"], state["dims"]):
        got = x[rows, at.clamp_min(0)] if dim == 0 else x[:, rows, at.clamp_min(0)]
        none = (at < 0).reshape((1,) * dim + at.shape + (1,) * (x.dim() - dim - 2))
        out.append(got.masked_fill_(none, 0))
    return out


# -------------------------------------------------------------------------------- the floor
def work(case):
    s = _SIZE[case["dtype"]]
    if case["op"] in ("embed", "grad"):
        B, S, V, D = case["B"], case["S"], case["V"], case["D"]
        first = 1 if case["start"] else 0
        places = B * (S + first)
        filled = B * ((case["low"] + S) / 2 + first)
        if case["zipf"]:
            used = sum(1 - (1 - math.log1p(1 / (r + 1)) / math.log(V + 1)) ** filled
                       for r in range(V))
        else:
            used = V * (1 - (1 - 1 / V) ** filled)
        look = (used + places) * D * s + 4 * filled
        back = (filled + V) * D * s + 4 * filled
        if case["op"] == "embed":
            return {"bytes": look, "flops": filled * D}
        return {"bytes": back + (look if case["train"] else 0),
                "flops": filled * D * (3 if case["train"] else 2)}
    if case["op"] == "select":
        rows = case["B"] * case["K"] * (1 - case["finished"])
        per = 4 if case["fused"] else 1
        return {"bytes": rows * case["V"] * s + case["B"] * (case["K"] * 5 + case["Ko"] * 12),
                "flops": rows * case["V"] * per}
    B, K = case["B"], case["K"]
    unique = K * (1 - (1 - 1 / K) ** K)
    if case["kind"] == "lstm":
        row = 2 * case["layers"] * case["width"] * s + 4 * case["length"]
    else:
        row = 2 * case["layers"] * case["width"] * case["length"] * 64 * s
    return {"bytes": B * (K + unique) * row + 4 * B * K, "flops": 0}


# ---------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("embed", "grad"):
        B, S, V, D = case["B"], case["S"], case["V"], case["D"]
        first = 1 if case["start"] else 0
        place = torch.arange(S + first, device="cuda").expand(B, -1) - first
        ids = state["tokens"].long().gather(1, place.clamp_min(0)) if S else place
        ids = torch.where(place < 0, 0, ids)
        ids = torch.where(place < state["lengths"][:, None], ids, V)      # V: padding
        out = []
        if "weight" in state:
            table = torch.cat([state["weight"].detach().double() * math.sqrt(D),
                               torch.zeros(1, D, device="cuda", dtype=torch.float64)])
            out.append(table.index_select(0, ids.reshape(-1)).reshape(B, S + first, D))
        if case["op"] == "embed":
            return out[0]
        at = ids.reshape(-1, 1).expand(-1, D)
        rows = state["grad_out"].double().reshape(-1, D)
        total = torch.zeros(V + 1, D, device="cuda", dtype=torch.float64)
        total.scatter_add_(0, at, rows)
        return out + [total[:V] * math.sqrt(D)]
    if case["op"] == "select":
        B, K, V, Ko = case["B"], case["K"], case["V"], case["Ko"]
        value = state["logits"].double()
        if case["fused"]:
            value = value - torch.logsumexp(value, 2, keepdim=True)
        value = value + state["scores"].double()[:, :, None]
        if state["finished"] is not None:
            done = state["finished"]
            value[done] = -math.inf
            value[:, :, 0] = torch.where(done, state["scores"].double(), value[:, :, 0])
        value = value.reshape(B, K * V)
        best = torch.topk(value, min(Ko, K * V), dim=1).values
        best = torch.nn.functional.pad(best, (0, Ko - best.shape[1]), value=-math.inf)
        return [best, None, None]
    return [_gather(x, state["parents"], d) if not x.is_floating_point()
            else _gather(x.double(), state["parents"], d)
            for x, d in zip(state["states"], state["dims"])]
