"""Plain float64 forms of the operators that learn from a teacher (NumPy; shared with no other
code), and the rounding bounds their outputs are held to."""
import numpy as np

from label_ref import U32, half_step, smallest

# What a row's sum of exponentials may be off by, relative: 2^-22 of ex2.approx, and at most 300
# float32 additions after one another (the long-row kernel's threads add up to 1024 terms; no row
# here has more than 256 a thread).  A term's exponent is rounded three times.
SUM = 2.0 ** -22 + 300 * U32
EXPONENT = 3 * U32


def log_sum(a, axis=-1):
    top = a.max(axis=axis, keepdims=True)
    safe = np.where(np.isneginf(top), 0.0, top)
    with np.errstate(divide="ignore"):
        return (np.log(np.exp(a - safe).sum(axis=axis, keepdims=True)) + safe).squeeze(axis)


def log_softmax(a):
    a = a - a.max()                 # first: the logarithm would be lost next to -3.4e38
    return a - np.log(np.exp(a).sum())


def top(x, k, tau):
    """(values, ids, rest, bound of rest) of float64 rows (N, V)."""
    N, V = x.shape
    values, ids = np.full((N, k), -np.inf), np.full((N, k), -1, dtype=np.int64)
    rest, bound = np.full(N, -np.inf), np.zeros(N)
    for n in range(N):
        if np.isnan(x[n]).any() or (x[n] == np.inf).any():
            continue
        order = np.argsort(-x[n], kind="stable")
        order = order[x[n][order] > -np.inf]
        best, left = order[:k], order[k:]
        values[n, :len(best)], ids[n, :len(best)] = x[n][best], best
        if len(left):
            rest[n] = log_sum(x[n][left] / tau)
            first = x[n][left[0]] / tau
            # the sum is relative to the largest: the mean exponent is at most log V less its log
            far = np.log(V) + abs(rest[n] - first)
            bound[n] = SUM + EXPONENT * far + 3 * U32 * (abs(first) + abs(rest[n]) + far)
    # a finite value below float32's range comes back as its lowest
    lowest = np.finfo(np.float32).min
    far = (rest < lowest) & np.isfinite(rest)
    rest[far], bound[far] = lowest, 0
    return values, ids, rest, bound * 1.01


def distill(x, t, ids, rest, tau):
    """Per row (divergence * tau^2, gradient, bound of the divergence, relative bound of the
    gradient's parts, the parts) of a float64 student (N, V) and teacher (N, K); ids < 0 are empty,
    rest (N,) or None."""
    N, V = x.shape
    loss, grad = np.zeros(N), np.zeros((N, V))
    err, part = np.zeros(N), np.zeros((N, V))
    for n in range(N):
        use = ids[n] >= 0
        goal = [t[n][use] / tau] + ([np.array([rest[n]])] if rest is not None else [])
        goal = np.concatenate(goal)
        if not (goal > -np.inf).any():
            continue
        log_p = log_softmax(goal)
        s = x[n] / tau
        log_q = log_softmax(s)
        at = ids[n][use]
        mine = log_q[at]
        others = np.ones(V, dtype=bool)
        others[at] = False
        if rest is not None:
            left = log_sum(log_q[others]) if others.any() else -np.inf
            mine = np.append(mine, left)
        p = np.exp(log_p)
        some = p > 0
        loss[n] = tau * tau * np.sum(p[some] * (log_p[some] - mine[some]))
        grad[n] = np.exp(log_q)
        part[n] = grad[n]
        np.subtract.at(grad[n], at, p[:len(at)])
        np.add.at(part[n], at, p[:len(at)])
        if rest is not None and left > -np.inf:
            q = p[-1] * np.exp(log_q[others] - left)
            grad[n][others] -= q
            part[n][others] += q
        grad[n] *= tau
        part[n] *= tau
        # an exponent's rounding grows with its size; the logarithms are rounded once each, and p's
        # own error weighs what it multiplies
        far = np.abs(log_p[some]) + np.where(np.isfinite(mine[some]), np.abs(mine[some]), 0.0)
        gap = np.where(np.isfinite(mine[some]), np.abs(log_p[some] - mine[some]), 0.0)
        one = SUM + 10 * U32 * (1 + far + np.log(V))
        err[n] = tau * tau * np.sum(p[some] * one * (1 + gap))
        depth = s.max() - s
        part[n] *= SUM + 8 * U32 * (4 + np.where(np.isfinite(depth), depth, 0.0) + np.log(V)
                                    + np.abs(log_p[some]).max())
    return loss, grad, err * 1.01, part * 1.01


def grad_bound(exact, part, scale, dtype):
    return part * abs(scale) + np.abs(exact) * (half_step(dtype) + 3 * U32) * 1.001 + \
        smallest(dtype) + 1e-44


def rows_of(T, U, padded):
    """(sample of each row, whether it counts) in the layout."""
    owner, live = [], []
    for b, (t, u) in enumerate(zip(T, U)):
        if padded:
            inside = np.zeros((max(max(T), 1), max(U) + 1), dtype=bool)
            inside[:t, :u + 1] = True
            owner += [b] * inside.size
            live += list(inside.reshape(-1))
        else:
            owner += [b] * (t * (u + 1))
            live += [True] * (t * (u + 1))
    return np.array(owner, dtype=np.int64), np.array(live, dtype=bool)
