"""fp64 oracle of what a step has around the expert layer: the RMS norm and its
backward, the balance loss of sequences with the z loss, and gradient clipping.
NumPy, written from the formulas; test infrastructure only."""
from __future__ import annotations

import numpy as np


def rms_norm(h, w, eps):
    """y and r = (mean h^2 + eps)^-1/2 of the rows of h."""
    r = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return h * r * w, r


def rms_norm_bwd(dy, h, w, eps, d_residual=None):
    """dh (with the residual's gradient) and dw."""
    _, r = rms_norm(h, w, eps)
    g = dy * w
    dh = r * g - r ** 3 * (g * h).mean(1, keepdims=True) * h
    if d_residual is not None:
        dh = dh + d_residual
    return dh, (dy * h * r).sum(0)


def live_tokens(T, offsets, mask=None):
    """Index arrays of the live tokens of each sequence."""
    off = np.clip(np.asarray(offsets, np.int64), 0, T)
    mask = np.ones(T, bool) if mask is None else np.asarray(mask, bool)
    return [a + np.nonzero(mask[a:b])[0] if b > a else np.zeros(0, np.int64)
            for a, b in zip(off[:-1], off[1:])]


def probabilities(x, sigmoid):
    """p, dL/dlogit's factor J, softmax and lse of rows of logits x; a row of -inf alone: zeros."""
    x = np.where(np.isnan(x), -np.inf, x)
    some = (x > -np.inf).any(1, keepdims=True)
    m = np.where(some, np.max(x, 1, keepdims=True, initial=-np.inf), 0.0)
    e = np.exp(x - m)
    total = np.where(some, e.sum(1, keepdims=True), 1.0)
    soft = e / total
    lse = np.where(some, m + np.log(total), 0.0)
    if not sigmoid:
        return soft, soft, soft, lse
    # by logarithms, so that scores that vanish keep their proportions
    log_s = -np.logaddexp(0.0, -x)
    top = np.where(some, np.max(log_s, 1, keepdims=True, initial=-np.inf), 0.0)
    p = np.exp(log_s - top)
    p = p / np.where(some, p.sum(1, keepdims=True), 1.0)
    return p, p * np.exp(-np.logaddexp(0.0, x)), soft, lse


def seq_aux(logits, idx, offsets, mask, sigmoid, coeff, z_coeff):
    """loss [2], counts, tokens, probs [B, E], d_logits, and the sizes that bound its rounding."""
    T, E = logits.shape
    k = idx.shape[1]
    seqs = live_tokens(T, offsets, mask)
    B = len(seqs)
    S, N = max(1, sum(len(t) > 0 for t in seqs)), max(1, sum(len(t) for t in seqs))
    counts, tokens = np.zeros((B, E), np.int64), np.zeros(B, np.int64)
    probs, d, size = np.zeros((B, E)), np.zeros((T, E)), np.zeros((T, E))
    loss = np.zeros(2)
    for b, t in enumerate(seqs):
        n = tokens[b] = len(t)
        if n == 0:
            continue
        p, jac, soft, lse = probabilities(logits[t].astype(np.float64), sigmoid)
        c = idx[t].ravel()
        counts[b] = np.bincount(c[(c >= 0) & (c < E)], minlength=E)
        probs[b] = p.mean(0)
        f = E * counts[b] / (k * n)
        loss += coeff / S * (f @ probs[b]), z_coeff / N * (lse ** 2).sum()
        g0, gz = coeff / (S * n), 2.0 * z_coeff / N
        mean = p @ f
        d[t] = g0 * jac * (f - mean[:, None]) + gz * lse * soft
        size[t] = abs(g0) * jac * (f + mean[:, None]) + abs(gz * lse) * soft
    return dict(loss=loss, counts=counts, tokens=tokens, probs=probs, d_logits=d, size=size)


def clip(grads, max_norm, scale):
    """(norm, factor) of fp64 gradients."""
    norm = scale * np.sqrt(sum(float((g * g).sum()) for g in grads))
    if not np.isfinite(norm):
        return norm, scale
    return norm, scale * min(1.0, max_norm / (norm + 1e-6))
