"""Selection in exact arithmetic (fractions; only the logarithm of a sum is a float64), for
values of any size, and the cases of such values that the CPU and the GPU tests share."""
from fractions import Fraction

import numpy as np
import torch

import label_ref as R


def select(logits, scores, beam, fused=True):
    """(scores, tokens, parents) of one item: float64 logits (K, V); scores that round to no
    finite float32 are infinite."""
    cand = []
    for k, x in enumerate(logits):
        s = float(scores[k])
        if not -np.inf < s < np.inf:
            continue
        top = x.max()
        if np.isnan(x).any() or top == np.inf or top == -np.inf:
            continue
        lse = Fraction(float(top)) + Fraction(float(np.log(np.sum(np.exp(x - top)))))
        base = Fraction(s) - (lse if fused else 0)
        cand += [(-(base + Fraction(float(x[v]))), k, int(v)) for v in np.flatnonzero(x > -np.inf)]
    out = np.full(beam, -np.inf), np.full(beam, -1), np.full(beam, -1)
    for r, (c, k, v) in enumerate(sorted(cand)[:beam]):
        beyond = abs(c) >= 2 ** 128 - 2 ** 103          # half a step above the largest
        out[0][r] = (-np.inf if c > 0 else np.inf) if beyond else float(-c)
        out[1][r], out[2][r] = v, k
    return out


def score_error(got, want, fused):
    """Largest excess of |got - want| over the bound of a score; infinities have to be equal."""
    got, want = np.asarray(got, float), np.asarray(want, float)
    same = np.isinf(want) | np.isinf(got)
    assert (got[same] == want[same]).all()
    g, w = got[~same], want[~same]
    return float(np.max(np.abs(g - w) - R.score_bound(w, fused), initial=-1.0))


def far_cases(dtype, K, V, beam):
    """Masks of the type's lowest value that leave fewer outputs than the beam, and what else sums
    beyond float32's range: (logits (K, V), scores (K,)), to be followed for some steps."""
    g = torch.Generator().manual_seed(V + K)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max

    def logits():
        return (torch.randn(K, V, generator=g) * 2).to(dtype)

    masked = logits()
    masked[:, 2:] = low
    masked[:, 1] = -1.0
    start = np.full(K, -np.inf, np.float32)
    start[0] = 0.0
    yield masked, start                                     # one hypothesis that can go two ways
    yield masked.roll(V // 2, 1), -1.0 - np.arange(K, dtype=np.float32)
    x = logits()                                            # different sizes of what is masked
    x[:, 1::2] = low
    x[:, 2::2] = low / 2
    yield x, np.where(np.arange(K) % 2 == 0, -3.0e38, -2.5e38).astype(np.float32)
    yield torch.full_like(x, low), np.full(K, np.finfo(np.float32).min, np.float32)
    x = logits()
    x[:, V // 3] = high                                     # and upwards
    x[:, V // 2] = high / 2
    yield x, np.where(np.arange(K) % 2 == 0, 3.0e38, 2.0e38).astype(np.float32)
    yield x, np.full(K, -3.0e38, np.float32)
