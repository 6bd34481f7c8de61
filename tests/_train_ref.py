"""Plain 64-bit statements (numpy) of the operators around the layer: layer
norm forward and backward, Newton-Schulz and the Muon step."""
import numpy as np


def layer_norm(h, w, b, eps):
    mu = h.mean(axis=1, keepdims=True)
    var = ((h - mu) ** 2).mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt(var + eps)
    y = (h - mu) * r * w
    return (y if b is None else y + b), mu[:, 0], r[:, 0]


def layer_norm_grad(dy, x, w, mu, r, d_stream=None):
    n = (x - mu[:, None]) * r[:, None]
    p = dy * w
    dx = r[:, None] * (p - p.mean(axis=1, keepdims=True) - n * (p * n).mean(axis=1, keepdims=True))
    if d_stream is not None:
        dx = dx + d_stream
    return dx, (dy * n).sum(axis=0), dy.sum(axis=0)


def newton_schulz(g, coefficients, eps):
    """One matrix; coefficients: a list of (a, b, c), one for each step."""
    x = g / (np.sqrt((g ** 2).sum()) + eps)
    flip = x.shape[0] > x.shape[1]
    if flip:
        x = x.T
    for a, b, c in coefficients:
        q = x @ x.T
        x = a * x + (b * q + c * (q @ q)) @ x
    return x.T if flip else x


def muon_step(w, g, m, lr, momentum, nesterov, weight_decay, scale, coefficients, eps):
    """Stacks [B, rows, cols]; returns (w, m) after the step."""
    m = momentum * m + g
    u = g + momentum * m if nesterov else m
    o = np.stack([newton_schulz(v, coefficients, eps) for v in u])
    return w * (1 - lr * weight_decay) - lr * scale * o, m
