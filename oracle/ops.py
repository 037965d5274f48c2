"""Float64 reference of the operators beside the optimizer step (test
infrastructure only): embedding, distillation loss, query/key norm with
rotation.  float64 NumPy in and out, written from the definitions."""
from __future__ import annotations

import numpy as np


def embedding(table, tokens, scale=1.0):
    """scale * table[tokens]; zero rows for tokens outside the table."""
    table, tokens = np.asarray(table, np.float64), np.asarray(tokens).reshape(-1)
    out = np.zeros((tokens.size, table.shape[1]))
    known = (tokens >= 0) & (tokens < table.shape[0])
    out[known] = scale * table[tokens[known]]
    return out


def embedding_plan(tokens, vocab):
    """(order, slot, rows, row_index, count) of dmuon_embedding_plan."""
    tokens = np.asarray(tokens).reshape(-1)
    n = tokens.size
    key = np.where((tokens >= 0) & (tokens < vocab), tokens, vocab)
    order = np.argsort(key, kind="stable")
    distinct = np.unique(key[key < vocab])
    rows = np.full(min(n, vocab), -1)
    rows[:distinct.size] = distinct
    row_index = np.full(vocab, -1)
    row_index[distinct] = np.arange(distinct.size)
    slot = np.where(key[order] < vocab, row_index[np.minimum(key[order], vocab - 1)], -1)
    return order, slot, rows, row_index, distinct.size


def embedding_grad(dout, tokens, vocab, scale=1.0):
    """(gradient, sum of the terms' magnitudes, number of terms) per table row."""
    dout, tokens = np.asarray(dout, np.float64), np.asarray(tokens).reshape(-1)
    grad, size = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1]))
    count = np.zeros(vocab, dtype=np.int64)
    for t in np.nonzero((tokens >= 0) & (tokens < vocab))[0]:
        grad[tokens[t]] += scale * dout[t]
        size[tokens[t]] += np.abs(scale * dout[t])
        count[tokens[t]] += 1
    return grad, size, count


def _log_softmax(z):
    top = z.max()
    with np.errstate(invalid="ignore"):
        return z - top - np.log(np.exp(z - top).sum())


def distill_loss(logits, index, teacher, labels=None, temperature=1.0, kd=1.0, ce=0.0, weight=None, grad_scale=1.0):
    """(losses, dlogits) of dmuon_distill_loss, row by row."""
    logits = np.asarray(logits, np.float64)
    n, vocab = logits.shape
    losses, dz = np.zeros(n), np.zeros((n, vocab))
    for r in range(n):
        w = 1.0 if weight is None else float(weight[r])
        if w == 0.0:
            continue
        z, loss, g = logits[r], 0.0, np.zeros(vocab)
        if kd != 0.0:
            ok = (index[r] >= 0) & (index[r] < vocab)
            idx, y = index[r][ok], np.asarray(teacher[r], np.float64)[ok] / temperature
            if idx.size and not np.all(y == -np.inf):
                logq = _log_softmax(y)
                q, logp = np.exp(logq), _log_softmax(z / temperature)
                use = q > 0
                loss += kd * temperature ** 2 * np.sum(q[use] * (logq[use] - logp[idx[use]]))
                t = np.exp(logp)
                np.subtract.at(t, idx, q)
                g += kd * temperature * t
        if ce != 0.0 and labels is not None and 0 <= labels[r] < vocab:
            logp = _log_softmax(z)
            loss -= ce * logp[labels[r]]
            t = np.exp(logp)
            t[labels[r]] -= 1.0
            g += ce * t
        losses[r] = w * loss
        dz[r] = grad_scale * w * g
    return losses, dz


def _pairs(dim, rot, interleaved):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _turn(x, cos, sin, interleaved):
    """x (tokens, heads, dim) with its pairs turned by cos, sin (tokens, rot / 2)."""
    out = x.copy()
    i, j = _pairs(x.shape[-1], 2 * cos.shape[1], interleaved)
    c, s = cos[:, None], sin[:, None]
    out[..., i] = x[..., i] * c - x[..., j] * s
    out[..., j] = x[..., i] * s + x[..., j] * c
    return out


def _angles(positions, rope, n):
    if rope is None:
        return np.zeros((n, 0)), np.zeros((n, 0)), np.zeros(n, bool)
    rope, positions = np.asarray(rope, np.float64), np.asarray(positions)
    at = rope[np.clip(positions, 0, rope.shape[0] - 1)]
    at[positions >= rope.shape[0]] = np.nan
    half = rope.shape[1] // 2
    return at[:, :half], at[:, half:], positions < 0


def qk_norm_rope(x, gain, positions, rope, eps=1e-6, interleaved=False, offset=0.0):
    """One of q, k: RMS norm per head, gain, rotation; zeros where the position
    is negative."""
    x = np.asarray(x, np.float64)
    cos, sin, pad = _angles(positions, rope, x.shape[0])
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    if gain is not None:
        y = y * (offset + np.asarray(gain, np.float64))
    y = _turn(y, cos, sin, interleaved)
    y[pad] = 0.0
    return y


def qk_norm_rope_grad(dy, x, gain, positions, rope, eps=1e-6, interleaved=False, offset=0.0):
    """(dx, dgain) of qk_norm_rope."""
    dy, x = np.asarray(dy, np.float64).copy(), np.asarray(x, np.float64)
    cos, sin, pad = _angles(positions, rope, x.shape[0])
    dy[pad] = 0.0
    dn = _turn(dy, cos, -sin, interleaved)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh = x * r
    xh[pad] = 0.0
    w = 1.0 if gain is None else offset + np.asarray(gain, np.float64)
    g = dn * w
    dx = r * (g - xh * np.mean(g * xh, -1, keepdims=True))
    dx[pad] = 0.0
    return dx, (dn * xh).sum((0, 1))
