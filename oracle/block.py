"""Float64 reference of the operators between a decoder block's projections
(test infrastructure only): norms around a block, attention over packed
sequences, gated feed-forward.  float64 NumPy in and out, written from the
definitions, one sequence, head and row at a time where that is plainest."""
from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------- norms around a block
def _rms(x, eps):
    return np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)


def block_norm_stream(x, h, post, gate, eps, scale, offset, post_norm):
    """The residual stream behind the block."""
    b = h / _rms(h, eps) if post_norm else h
    if post is not None:
        b = b * (offset + post)
    return x + scale * (1.0 if gate is None else gate) * b


def block_norm_out(x_out, pre, eps, offset):
    """The normed stream."""
    return x_out / _rms(x_out, eps) * (1.0 if pre is None else offset + pre)


def block_norm_grad(dx_out, dy, x_out, h, pre, post, gate, eps, scale, offset, post_norm):
    """(dx, dh, dpre, dpost, dgate), every one whether its weight is there or not."""
    gpre = 1.0 if pre is None else offset + pre
    gpost = 1.0 if post is None else offset + post
    gt = 1.0 if gate is None else gate
    lx = _rms(x_out, eps)
    xh = x_out / lx
    u = dy * gpre
    t = (u - xh * np.mean(u * xh, -1, keepdims=True)) / lx + (0.0 if dx_out is None else dx_out)
    lh = _rms(h, eps) if post_norm else 1.0
    hh = h / lh
    d = scale * gt * gpost * t
    dh = (d - hh * np.mean(d * hh, -1, keepdims=True)) / lh if post_norm else d
    return t, dh, (dy * xh).sum(0), (scale * gt * t * hh).sum(0), (scale * gpost * t * hh).sum(0)


# ---------------------------------------------------------------- attention
def visible(lq, lk, causal, window):
    """Truth values (lq, lk): the keys that each query sees."""
    i, j = np.arange(lq)[:, None] + (lk - lq), np.arange(lk)[None, :]
    see = np.ones((lq, lk), bool)
    if causal:
        see = j <= i
        if window:
            see &= j > i - window
    return see


def _each(q_offsets, k_offsets, q_heads, k_heads):
    for b in range(len(q_offsets) - 1):
        for h in range(q_heads):
            yield (slice(q_offsets[b], q_offsets[b + 1]), slice(k_offsets[b], k_offsets[b + 1]), h,
                   h // (q_heads // k_heads))


def attention(q, k, v, q_offsets, k_offsets, causal=True, window=0, scale=None):
    """(out (tokens, heads, dim), lse (heads, tokens)); rows of no sequence are NaN."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    out, lse = np.full(q.shape, np.nan), np.full((q.shape[1], q.shape[0]), np.nan)
    for rq, rk, h, kv in _each(q_offsets, k_offsets, q.shape[1], k.shape[1]):
        see = visible(rq.stop - rq.start, rk.stop - rk.start, causal, window)
        for i in range(rq.stop - rq.start):
            on = see[i]
            if not on.any():
                out[rq.start + i, h], lse[h, rq.start + i] = 0.0, -math.inf
                continue
            z = scale * (k[rk, kv][on] @ q[rq.start + i, h])
            e = np.exp(z - z.max())
            out[rq.start + i, h] = e @ v[rk, kv][on] / e.sum()
            lse[h, rq.start + i] = z.max() + math.log(e.sum())
    return out, lse


def attention_grad(dout, q, k, v, q_offsets, k_offsets, causal=True, window=0, scale=None, out=None, lse=None):
    """(dq, dk, dv); rows of no sequence are NaN.  out, lse: the forward's, if not exact ones."""
    scale = q.shape[2] ** -0.5 if scale is None else scale
    exact = attention(q, k, v, q_offsets, k_offsets, causal, window, scale)
    out, lse = exact[0] if out is None else out, exact[1] if lse is None else lse
    dq, dk, dv = np.full(q.shape, np.nan), np.full(k.shape, np.nan), np.full(v.shape, np.nan)
    for rq, rk, h, kv in _each(q_offsets, k_offsets, q.shape[1], k.shape[1]):
        if h % (q.shape[1] // k.shape[1]) == 0:
            dk[rk, kv] = dv[rk, kv] = 0.0
        see = visible(rq.stop - rq.start, rk.stop - rk.start, causal, window)
        z = scale * (q[rq, h] @ k[rk, kv].T)
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.where(see, np.exp(z - lse[h, rq][:, None]), 0.0)
        dp = dout[rq, h] @ v[rk, kv].T
        ds = p * (dp - (dout[rq, h] * out[rq, h]).sum(-1, keepdims=True)) * scale
        dq[rq, h] = ds @ k[rk, kv]
        dk[rk, kv] += ds.T @ q[rq, h]
        dv[rk, kv] += p.T @ dout[rq, h]
    return dq, dk, dv


# ---------------------------------------------------------------- gated feed-forward
def activation(g, kind):
    """(act(g), act'(g)) of "silu" or "gelu" (its tanh form)."""
    if kind == "silu":
        sig = 0.5 * (1.0 + np.tanh(0.5 * g))
        return g * sig, sig + g * sig * (1.0 - sig)
    c, a = math.sqrt(2.0 / math.pi), 0.044715
    t = np.tanh(c * (g + a * g ** 3))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * a * g * g)


def gated_ffn(x, w_gate, w_up, kind="silu"):
    return activation(x @ w_gate.T, kind)[0] * (x @ w_up.T)


def gated_ffn_grad(dh, x, w_gate, w_up, kind="silu"):
    """(dx, dw_gate, dw_up)."""
    a, da = activation(x @ w_gate.T, kind)
    dg, du = dh * (x @ w_up.T) * da, dh * a
    return dg @ w_gate + du @ w_up, dg.T @ x, du.T @ x
