"""Plain fp64 restatement of the sampling distributions (temperature, top-k, top-p, min-p) and of the
draw from them: one row at a time, tokens let in one after another, no shortcuts."""
import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def clean(row):
    """A row as fp64: NaN counts as -inf, +inf as the largest finite fp32 number."""
    z = np.array(row, np.float64)
    z[np.isnan(z)] = -np.inf
    return np.minimum(z, F32_MAX)


def places(z):
    """Indices of the tokens above -inf, the largest first, the lower index first on ties."""
    order = np.lexsort((np.arange(len(z)), -z))
    return order[z[order] > -np.inf]


def kept(row, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(indices in their order, weights, how far each cut's nearest border is away, relative)."""
    z = clean(row)
    order = places(z)
    if len(order) == 0:
        return order, np.zeros(0), np.inf
    if not temperature > 0:
        return order[:1], np.ones(1), np.inf
    if 0 < top_k < len(z):
        order = order[:top_k]
    with np.errstate(over="ignore"):
        w = np.exp((z[order] - z[order[0]]) / temperature)
    total, n, near = w.sum(), len(order), np.inf
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        n = min(n, int((before < top_p * total).sum()))
        if top_p > 0:
            near = min(near, np.abs(before[1:] / (top_p * total) - 1).min(initial=np.inf))
    if min_p > 0:
        floor = min(float(min_p), 1.0)
        n = min(n, int((w >= floor).sum()))
        near = min(near, np.abs(w[1:] / floor - 1).min(initial=np.inf))
    n = max(n, 1)
    return order[:n], w[:n], near


def probs(row, **setting):
    at, w, _ = kept(row, **setting)
    out = np.zeros(len(row))
    if len(at):
        out[at] = w / w.sum()
    return out


def token(row, u, **setting):
    """(token, probability, distance of u from the nearest step of the cumulative sum)."""
    at, w, _ = kept(row, **setting)
    if len(at) == 0:
        return -1, 0.0, np.inf
    by_index = np.argsort(at)
    at, w = at[by_index], w[by_index]
    c = np.cumsum(w) / w.sum()
    u = min(max(float(u), 0.0), 1 - 2.0 ** -24) if u == u else 0.0
    i = min(int(np.searchsorted(c, u, side="right")), len(at) - 1)
    return int(at[i]), float(w[i] / w.sum()), float(np.abs(c[:-1] - u).min(initial=np.inf))
