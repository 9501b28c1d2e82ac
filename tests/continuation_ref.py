"""Plain implementations, in 64 bits, of the operators that decoding several
continuations adds to a step. Nothing here is shared with the library."""
import numpy as np


# ------------------------------------------------------------------ norms around a block
def block_norm(y, h, gate, w_post, w_pre, post, h_scale, y_scale, eps, offset):
    """float64 arrays (or None); gate already one row for each token. Returns
    h', x, the magnitude |a h| + |s g z| that rounding errors of h' scale with,
    and the same for x: (|terms| and, through the mean, their share of h') times
    the row's factor and weight."""
    def normed(x, w):
        f = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        return f * np.ones_like(x) if w is None else f * (w + (1.0 if offset else 0.0))

    size = np.abs(h_scale * h)
    out = h_scale * h
    if y is not None:
        z = y * normed(y, w_post) if post else y
        if gate is not None:
            z = z * gate
        out = out + y_scale * z
        size = size + np.abs(y_scale * z)
    f = normed(out, w_pre)
    rms = lambda a: np.sqrt((a * a).mean(-1, keepdims=True))  # noqa: E731
    spread = rms(size) / np.maximum(rms(out), 1e-300)
    return out, out * f, size, np.abs(f) * (size + np.abs(out) * spread)


# ------------------------------------------------------------------ sampling
def kept_weights(l, T, k, p, m):
    """One row of logits (float64) -> weights e_i of what is kept, 0 elsewhere."""
    V = len(l)
    out = np.zeros(V)
    l = np.where(np.isnan(l), -np.inf, l)
    if not (l > -np.inf).any():
        return out
    order = np.lexsort((np.arange(V), -(l + 0.0)))
    order = order[l[order] > -np.inf]
    first = not T > 0
    if first:
        T = 1.0
    with np.errstate(over="ignore", invalid="ignore"):
        x = l[order] / T
        e = (x == np.inf).astype(float) if x[0] == np.inf else np.exp(x - x[0])
    n = len(order)
    if 0 < k < V:
        n = min(n, k)
    if p < 1:
        total = e[:n].sum()
        before = np.concatenate([[0.0], np.cumsum(e[:n])[:-1]])
        n = max(1, int((before < p * total).sum()))
    if m > 0:
        n = max(1, int((e[:n] >= m).sum()))
    if first:
        n = 1
    out[order[:n]] = e[:n]
    return out


def draw(e, u):
    """The token that u (a number in [0, 1]) names, -1 if nothing is kept."""
    if not (e > 0).any():
        return -1
    run = np.cumsum(e)
    hit = np.nonzero((run > u * run[-1]) & (e > 0))[0]
    return int(hit[0]) if len(hit) else int(np.nonzero(e)[0][-1])
