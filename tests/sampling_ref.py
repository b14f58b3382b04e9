"""What sample_tokens computes, from the definition, in 64 bits on the CPU: for one row the kept tokens, their sums in index
order, and which token a number u draws."""
import numpy as np

NO_TOKEN = -1


def kept(l, t=1.0, k=0, p=1.0, mp=0.0):
    """Indices (ascending) that the settings leave of logits l (float64), and their weights."""
    top = l.max()
    order = np.lexsort((np.arange(l.size), -l))
    order = order[l[order] > -np.inf]
    if t == 0:
        return order[:1], np.ones(1)
    w = np.exp((l[order] - top) / t)
    if k > 0:
        order, w = order[:k], w[:k]
    if mp > 0:
        ok = (l[order] - top >= t * np.log(mp)) if mp < 1 else (l[order] == top)
        order, w = order[ok], w[ok]
    if p < 1:
        # sums from the largest down: exact enough for a border between two tokens that are not within 1e-15 of it
        n = 1 + int((np.cumsum(w) < p * w.sum()).sum())
        order, w = order[:n], w[:n]
    by = np.argsort(order)
    return order[by], w[by]


def draw(l, u, **settings):
    """(token, logprob, distance of u to the nearest border of that token)."""
    i, w = kept(l, **settings)
    cum = np.cumsum(w)
    cum /= cum[-1]
    at = int(np.searchsorted(cum, u, side="right"))
    at = min(at, i.size - 1)
    low = cum[at - 1] if at else -1.0
    high = cum[at] if at + 1 < i.size else 2.0
    return int(i[at]), float(np.log(w[at] / w.sum())), min(u - low, high - u)
