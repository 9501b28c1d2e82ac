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
