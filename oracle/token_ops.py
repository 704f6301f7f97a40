"""Token operators in float64 (NumPy): embedding lookup and gradient, residual RMS norm with its gradient and 8-bit
output scales, policy loss with its gradient. Written from the formulas, row by row; test infrastructure only."""

import numpy as np


def embedding(table, ids, scale):
    return np.stack([scale * table[i] for i in ids]) if len(ids) else np.zeros((0, table.shape[1]))


def embedding_grad(grad_out, ids, rows, scale, padding_idx=-1, start=None):
    """(gradient, sum of the absolute terms, number of terms per row)."""
    got = np.zeros((rows, grad_out.shape[1])) if start is None else start.astype(np.float64).copy()
    size = np.abs(got)
    count = np.zeros(rows, dtype=np.int64)
    for i, v in enumerate(ids):
        if 0 <= v < rows and v != padding_idx:
            got[v] += scale * grad_out[i]
            size[v] += np.abs(scale * grad_out[i])
            count[v] += 1
    return got, size, count


def add_rmsnorm(x, residual, gain, eps):
    """(y, h)"""
    h = x if residual is None else x + residual
    rho = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return h * rho * (1.0 if gain is None else gain), h


def group_scales(y, group):
    """max |y| / 448 over each group of columns (0: the row); 1 for a group of zeros."""
    group = group or y.shape[1]
    tops = np.stack([np.abs(y[:, k:k + group]).max(axis=1) for k in range(0, y.shape[1], group)], axis=1)
    return np.where(tops == 0, 1.0, np.maximum(tops / 448.0, 2.0 ** -126))


def add_rmsnorm_grad(dy, h, gain, dh, eps):
    """(dx, dgain, size of the terms of dx, size of the terms of dgain)"""
    dim = h.shape[1]
    rho = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    d = dy * (1.0 if gain is None else gain)
    back = h * rho ** 3 / dim
    dx = rho * d - back * (d * h).sum(axis=1, keepdims=True)
    size = rho * np.abs(d) + np.abs(back) * np.abs(d * h).sum(axis=1, keepdims=True)
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    terms = dy * h * rho
    return dx, terms.sum(axis=0), size, np.abs(terms).sum(axis=0)


def log_softmax(logits, temperature):
    z = logits / temperature
    m = z.max(axis=1, keepdims=True)
    return z - m - np.log(np.exp(z - m).sum(axis=1, keepdims=True))


def policy_loss(logits, targets, old_logp, advantages, weights, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
                temperature=1.0):
    """(loss, logp, dlogits, the rows' terms, the rows' d loss / d logp)"""
    n, vocab = logits.shape
    logp, terms, coef = np.zeros(n), np.zeros(n), np.zeros(n)
    dlogits = np.zeros((n, vocab))
    for t in range(n):
        a = int(targets[t])
        if weights[t] == 0 or not 0 <= a < vocab:
            continue
        ls = log_softmax(logits[t:t + 1], temperature)[0]
        logp[t] = ls[a]
        r = np.exp(logp[t] - old_logp[t])
        whole = r * advantages[t]
        cut = min(max(r, 1.0 - clip_low), 1.0 + clip_high) * advantages[t]
        each, c = -min(whole, cut), -whole if whole <= cut else 0.0
        if ref_logp is not None and kl_coef:
            d = ref_logp[t] - logp[t]
            each += kl_coef * (np.exp(d) - d - 1.0)
            c += kl_coef * (1.0 - np.exp(d))
        terms[t], coef[t] = weights[t] * each, weights[t] * c
        dlogits[t] = -np.exp(ls) * coef[t] / temperature
        dlogits[t, a] += coef[t] / temperature
    return terms.sum(), logp, dlogits, terms, coef
