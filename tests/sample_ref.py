"""Drawing in float64 (NumPy, loops; shared with no other code)."""
import numpy as np


# Sums decide as if held to 40 bits: a border that lies nearer than that to a running sum may fall on
# either side of it.  It happens: with two equal maxima, u = 1/2 and a small temperature the border is
# 1 + (sum of the others) / 2, and with as many next-best terms (e^-20 each) on one side as on the other
# it is off the running sum by e^-40, which is below 2^-57 and which float64 does not place either.
NEAR = 2.0 ** -40


def sample(logits, scores, random, tau=1.0, top_k=None, top_p=1.0, min_p=0.0, finished=None, fused=True,
           nudge=(0.0, 0.0)):
    """(scores, tokens) of float64 logits (B, K, V); the borders of top_p and of the draw are moved by
    nudge times the whole."""
    B, K, V = logits.shape
    out, tokens = np.full((B, K), -np.inf), np.full((B, K), -1, dtype=np.int64)
    for b in range(B):
        for k in range(K):
            s, x, u = scores[b, k], logits[b, k], random[b, k]
            if not s < np.inf:
                continue
            if finished is not None and finished[b, k]:
                out[b, k] = s
                continue
            if not 0 <= u < 1 or np.isnan(x).any() or (x == np.inf).any() or s == -np.inf:
                continue
            order = np.argsort(-x, kind="stable")
            order = order[x[order] > -np.inf]
            if not len(order):
                continue
            if top_k is not None:
                order = order[:top_k]
            top = x.max()
            e = np.exp((x[order] - top) / tau)
            if top_p < 1:
                ahead = np.cumsum(e) - e
                order = order[ahead < (top_p + nudge[0]) * e.sum()]
            if min_p > 0:
                order = order[x[order] - top >= tau * np.log(min_p)]
            ids = np.sort(order)
            run = np.cumsum(np.maximum(np.exp((x[ids] - top) / tau), 1e-300))
            at = min(int((run <= (u + nudge[1]) * run[-1]).sum()), len(ids) - 1)
            tokens[b, k] = ids[at]
            p = x[ids[at]]
            if fused:
                p = (p - top) - np.log(np.exp(x - top).sum())
            out[b, k] = s + p
    return out, tokens
