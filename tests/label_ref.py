"""Plain float64 forms of the label-side operators (NumPy, loops; shared with no other code), and
the rounding bounds their outputs are held to."""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24          # half a float32 step, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    """Half the spacing of the type's subnormal numbers (rounding near zero)."""
    f = torch.finfo(dtype)
    return f.smallest_normal * f.eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def place_ids(tokens, lengths, start, V):
    """(B, P) ids, -1 for padding."""
    B, S = tokens.shape
    P = S + (start is not None)
    ids = np.full((B, P), -1, dtype=np.int64)
    for b in range(B):
        row = []
        if start is not None:
            row.append(start + V if start < 0 else start)
        for s in range(S):
            inside = lengths is None or s < lengths[b]
            t = int(tokens[b, s]) if inside else -1
            row.append(t if 0 <= t < V else -1)
        ids[b] = row
    return ids


def embed(weight, ids, scale):
    """(B, P, D) float64."""
    out = np.zeros(ids.shape + (weight.shape[1],))
    for b, p in np.argwhere(ids >= 0):
        out[b, p] = weight[ids[b, p]] * scale
    return out


def embed_grad(grad_out, ids, V, scale):
    """((V, D) gradient, (V, D) sum of magnitudes, (V,) number of terms)."""
    D = grad_out.shape[2]
    total, mass, n = np.zeros((V, D)), np.zeros((V, D)), np.zeros(V, dtype=np.int64)
    for b, p in np.argwhere(ids >= 0):
        v = ids[b, p]
        total[v] += grad_out[b, p]
        mass[v] += np.abs(grad_out[b, p])
        n[v] += 1
    return total * scale, mass * abs(scale), n


def embed_bound(exact, dtype):
    """The scale and the product are each rounded to float32, then once to the type."""
    a = np.abs(exact)
    return a * (2 * U32 + half_step(dtype)) * 1.001 + smallest(dtype) + 1e-45


def grad_bound(exact, mass, n, dtype):
    """n - 1 float32 additions, each off by half a step of a partial sum that is at most the sum
    of magnitudes, the scale, the product, and the rounding to the type."""
    sums = mass * U32 * (n[:, None] + 2)
    return (sums + np.abs(exact) * half_step(dtype)) * 1.001 + smallest(dtype) + 1e-45


def select(logits, scores, beam, finished=None, fused=True):
    """(scores, tokens, parents) of float64 logits (B, K, V)."""
    B, K, V = logits.shape
    out = (np.full((B, beam), -np.inf), np.full((B, beam), -1, dtype=np.int64),
           np.full((B, beam), -1, dtype=np.int64))
    for b in range(B):
        cand = []
        for k in range(K):
            s, x = scores[b, k], logits[b, k]
            if not (-np.inf < s < np.inf):
                continue
            if finished is not None and finished[b, k]:
                cand.append((-s, k, -1))
                continue
            if np.isnan(x).any() or (x == np.inf).any() or not (x > -np.inf).any():
                continue
            top = x.max()
            # in this order: top + log(..) would lose the logarithm where top is -3.4e38
            p = (x - top) - np.log(np.sum(np.exp(x - top))) if fused else x
            cand += [(-(s + p[v]), k, v) for v in np.flatnonzero(x > -np.inf)]
        for r, (c, k, v) in enumerate(sorted(cand)[:beam]):
            out[0][b, r], out[1][b, r], out[2][b, r] = -c, v, k
    return out


def score_bound(exact, fused):
    """One float32 rounding; the log-sum-exp may be off by 4e-6 (its bound is below 2e-6 for the
    rows tested here)."""
    finite = np.where(np.isfinite(exact), np.abs(exact), 0.0)
    return finite * U32 * 1.001 + (4e-6 if fused else 0.0)
