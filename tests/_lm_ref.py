"""Plain 64-bit statements (numpy) of the ends of a language model: embedding,
cross entropy and distillation over a vocabulary, with their gradients."""
import numpy as np


def embedding(ids, table, scale):
    known = (ids >= 0) & (ids < len(table))
    return np.where(known[:, None], scale * table[np.where(known, ids, 0)], 0.0)


def embedding_grad(d_out, ids, V, scale, add=None):
    out = np.zeros((V, d_out.shape[1])) if add is None else add.copy()
    for t, i in enumerate(ids):
        if 0 <= i < V:
            out[i] += scale * d_out[t]
    return out


def log_sum_exp(z):
    m = z.max(axis=1, keepdims=True)
    return (m + np.log(np.exp(z - m).sum(axis=1, keepdims=True)))[:, 0]


def cross_entropy(x, W, labels):
    z = x @ W.T
    lse = log_sum_exp(z)
    known = (labels >= 0) & (labels < len(W))
    at = z[np.arange(len(z)), np.where(known, labels, 0)]
    return np.where(known, lse - at, 0.0), lse


def cross_entropy_dz(x, W, labels, d_loss, d_lse=None):
    z = x @ W.T
    q = np.exp(z - log_sum_exp(z)[:, None])
    known = (labels >= 0) & (labels < len(W))
    d = np.where(known, d_loss, 0.0)
    dz = q * (d if d_lse is None else d + d_lse)[:, None]
    dz[np.arange(len(z))[known], labels[known]] -= d[known]
    return dz


def teacher(ids, logits, tau, V):
    """(probabilities [T, K] among a token's entries, entries there are)."""
    known = (ids >= 0) & (ids < V) & (logits > -np.inf)
    p = np.zeros(ids.shape)
    for t in range(len(ids)):
        k = known[t]
        if k.any():
            e = np.exp((logits[t, k] - logits[t, k].max()) / tau)
            p[t, k] = e / e.sum()
    return p, known


def distill(x, W, ids, logits, tau):
    V = len(W)
    z = x @ W.T
    lse = log_sum_exp(z / tau)
    p, _ = teacher(ids, logits, tau, V)
    inside = (ids >= 0) & (ids < V)
    at = np.where(inside, np.take_along_axis(z, np.where(inside, ids, 0), axis=1), 0.0)
    log_p = np.log(np.where(p > 0, p, 1.0))
    return np.where(p > 0, p * (log_p - at / tau + lse[:, None]), 0.0).sum(axis=1), lse, at


def distill_dz(x, W, ids, logits, tau, d_loss):
    V = len(W)
    z = x @ W.T / tau
    p, _ = teacher(ids, logits, tau, V)
    dz = np.exp(z - log_sum_exp(z)[:, None]) * p.sum(axis=1, keepdims=True)
    for t in range(len(ids)):
        for j in range(ids.shape[1]):
            if p[t, j] > 0:
                dz[t, ids[t, j]] -= p[t, j]
    return dz * (d_loss / tau)[:, None]
