"""Token operators in float64 (NumPy): embedding lookup and gradient, residual RMS norm with its gradient and 8-bit
output scales, policy loss with its gradient, per-head norm with rotation, attention and token statistics with theirs.
Written from the formulas, row by row; test infrastructure only."""

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


# ---------------------------------------------------------------------------- per-head norm and rotation


def turns(positions, rotary_dim, base=10000.0, freqs=None, sections=None):
    """Angles, n x rotary_dim / 2; positions (n,), or (axes, n) with sections."""
    half = rotary_dim // 2
    f = np.array([base ** (-2.0 * j / rotary_dim) for j in range(half)]) if freqs is None else np.asarray(freqs, float)
    if sections is None:
        return positions[:, None].astype(np.float64) * f
    axis = np.repeat(np.arange(len(sections)), sections)
    return positions.astype(np.float64)[axis].T * f


def turn(z, angles, rotary_dim, interleaved):
    """z (n, heads, dim) with its pairs turned by the angles."""
    out = z.copy()
    half = rotary_dim // 2
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + (1 if interleaved else half)
    c, s = np.cos(angles)[:, None], np.sin(angles)[:, None]
    out[..., first] = z[..., first] * c - z[..., second] * s
    out[..., second] = z[..., second] * c + z[..., first] * s
    return out


def qk_norm_rotary(x, gain, angles, rotary_dim, interleaved=False, norm=True, eps=1e-6):
    """One of the two tensors: (n, heads, dim)."""
    z = x
    if norm:
        z = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * (1.0 if gain is None else gain)
    return turn(z, angles, rotary_dim, interleaved)


def qk_norm_rotary_grad(dy, x, gain, angles, rotary_dim, interleaved=False, norm=True, eps=1e-6):
    """(dx, dgain, size of the terms of dx, size of the terms of dgain)"""
    d = turn(dy, -angles, rotary_dim, interleaved)
    # |d| as the sum of the absolute values of its two terms
    half = rotary_dim // 2
    size = np.abs(dy).copy()
    first = np.arange(half) * 2 if interleaved else np.arange(half)
    second = first + (1 if interleaved else half)
    both = np.abs(dy[..., first]) + np.abs(dy[..., second])
    size[..., first] = size[..., second] = both
    if not norm:
        return d, None, size, None
    dim = x.shape[-1]
    g = np.ones(dim) if gain is None else gain
    rho = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    back = x * rho ** 3 / dim
    dx = rho * d * g - back * (d * g * x).sum(axis=-1, keepdims=True)
    dx_size = rho * size * np.abs(g) + np.abs(back) * (size * np.abs(g * x)).sum(axis=-1, keepdims=True)
    return dx, (d * x * rho).sum(axis=(0, 1)), dx_size, (size * np.abs(x) * rho).sum(axis=(0, 1))


# ---------------------------------------------------------------------------- attention


def _scores(q, k, ends, s, head, kv, causal, scale):
    b, e = ends[s], ends[s + 1]
    x = q[b:e, head] @ k[b:e, kv].T * scale
    if causal:
        x = np.where(np.arange(e - b)[None] > np.arange(e - b)[:, None], -np.inf, x)
    return b, e, x


def attention(q, k, v, ends, causal=True, scale=None):
    """(out, lse, sum of p |v|, largest sum of |q_c k_c| scale of each row); rows of no sequence are zeros."""
    n, heads, dim = q.shape
    scale = dim ** -0.5 if scale is None else scale
    group = heads // k.shape[1]
    out, size = np.zeros((n, heads, dim)), np.zeros((n, heads, dim))
    lse, reach = np.zeros((heads, n)), np.zeros((heads, n))
    for s in range(len(ends) - 1):
        for h in range(heads):
            b, e, x = _scores(q, k, ends, s, h, h // group, causal, scale)
            if e == b:
                continue
            m = x.max(axis=1)
            p = np.exp(x - m[:, None])
            total = p.sum(axis=1)
            lse[h, b:e] = m + np.log(total)
            out[b:e, h] = p @ v[b:e, h // group] / total[:, None]
            size[b:e, h] = p @ np.abs(v[b:e, h // group]) / total[:, None]
            reach[h, b:e] = (np.abs(q[b:e, h]) @ np.abs(k[b:e, h // group]).T).max(axis=1) * abs(scale)
    return out, lse, size, reach


def attention_grad(dout, q, k, v, out, lse, ends, causal=True, scale=None, p_off=0.0, dot_off=0.0):
    """(dq, dk, dv) at the stored out and lse, and the bounds of what they are off by where every p is off by p_off of
    itself and dout . v and D by dot_off of the sum of their absolute terms. The sum of a row's ds, 0 but for what out
    lost in its rounding, may be added to D, in whole or in part: it counts to the bounds."""
    n, heads, dim = q.shape
    scale = dim ** -0.5 if scale is None else scale
    group = heads // k.shape[1]
    got = [np.zeros(t.shape) for t in (q, k, v)]
    off = [np.zeros(t.shape) for t in (q, k, v)]
    for s in range(len(ends) - 1):
        for h in range(heads):
            kv = h // group
            b, e, x = _scores(q, k, ends, s, h, kv, causal, scale)
            if e == b:
                continue
            p = np.exp(x - lse[h, b:e, None])
            do = dout[b:e, h]
            along = do @ v[b:e, kv].T
            delta = (do * out[b:e, h]).sum(axis=1, keepdims=True)
            ds = p * (along - delta)
            ds_off = p * (dot_off * (np.abs(do) @ np.abs(v[b:e, kv]).T + np.abs(do * out[b:e, h]).sum(axis=1, keepdims=True)))
            ds_off += p_off * np.abs(ds) + p * np.abs(ds.sum(axis=1, keepdims=True))
            got[0][b:e, h] = scale * ds @ k[b:e, kv]
            off[0][b:e, h] = abs(scale) * ds_off @ np.abs(k[b:e, kv])
            got[1][b:e, kv] += scale * ds.T @ q[b:e, h]
            off[1][b:e, kv] += abs(scale) * ds_off.T @ np.abs(q[b:e, h])
            got[2][b:e, kv] += p.T @ do
            off[2][b:e, kv] += p_off * p.T @ np.abs(do)
    return got, off


# ---------------------------------------------------------------------------- token statistics


def token_stats(logits, targets, top, temperature=1.0):
    """(logp, entropy, top_logp, top_ids, norm); a row without a target is zeros and -1."""
    n, vocab = logits.shape
    logp, entropy, norm = np.zeros(n), np.zeros(n), np.zeros((n, 2))
    top_logp, top_ids = np.zeros((n, top)), np.full((n, top), -1, dtype=np.int64)
    for t in range(n):
        if targets is not None and not 0 <= targets[t] < vocab:
            continue
        x = logits[t]
        ls = log_softmax(x[None], temperature)[0]
        p = np.exp(ls)
        if targets is not None:
            logp[t] = ls[targets[t]]
        entropy[t] = -(p[p > 0] * ls[p > 0]).sum()
        norm[t] = x.max(), np.exp((x - x.max()) / temperature).sum()
        ids = sorted(range(vocab), key=lambda j: (-x[j], j))[:top]
        top_ids[t], top_logp[t] = ids, ls[ids]
    return logp, entropy, top_logp, top_ids, norm


def token_stats_grad(logits, targets, dlogp, dentropy, temperature=1.0):
    """(dlogits, size of its terms)"""
    n, vocab = logits.shape
    got, size = np.zeros((n, vocab)), np.zeros((n, vocab))
    for t in range(n):
        if targets is not None and not 0 <= targets[t] < vocab:
            continue
        ls = log_softmax(logits[t:t + 1], temperature)[0]
        p = np.exp(ls)
        lp = np.where(p > 0, ls, 0.0)
        entropy = -(p * lp).sum()
        g, h = (0.0 if dlogp is None else dlogp[t]), (0.0 if dentropy is None else dentropy[t])
        got[t] = -p * (g + h * (lp + entropy))
        size[t] = p * (abs(g) + abs(h) * (np.abs(lp) + entropy))
        if targets is not None:
            got[t, targets[t]] += g
            size[t, targets[t]] += abs(g)
    return got / temperature, size / temperature
