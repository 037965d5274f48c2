"""Attention in float64 on the device, with bounds for what the kernels may be off."""
import numpy as np
import torch

from ops_util import U32, half_step

# What lies below the least normal float32 may become 0, so a probability is also
# off by this, and so is whatever is formed of it: scores that lie 88 below their
# row's maximum have probabilities under it, which float64 still holds.
TINY = 2.0 ** -126


def visible(lq, lk, causal, window, device):
    i, j = torch.arange(lq, device=device)[:, None] + (lk - lq), torch.arange(lk, device=device)[None]
    if not causal:
        return torch.ones(lq, lk, dtype=torch.bool, device=device)
    return (j <= i) & (j > i - window) if window else j <= i


def spans(q_offsets, k_offsets):
    return [(slice(a, b), slice(c, d)) for a, b, c, d in zip(q_offsets, q_offsets[1:], k_offsets, k_offsets[1:])]


def forward(q, k, v, q_offsets, k_offsets, causal, window, scale, dtype):
    """(out, its bound, lse, its bound); NaN on rows of no sequence.

    A score sums D products: off by (D + 16) units of their magnitudes.  In base
    2 it is scaled and the maximum taken off (4 units of the largest score),
    and exp2 rounds (2 units).  So a probability is off by `rel`, relative, and
    bf16 rounds it once more in front of its product.  Sums over n keys add
    n + 64 units."""
    q, k, v = q.double(), k.double(), v.double()
    (n, qh, d), kh = q.shape, k.shape[1]
    nan = lambda *s: torch.full(s, float("nan"), dtype=torch.float64, device=q.device)  # noqa: E731
    out, ob, lse, lb = nan(n, qh, d), nan(n, qh, d), nan(qh, n), nan(qh, n)
    half = half_step(dtype)
    p_half = half if dtype == torch.bfloat16 else 0.0
    for rq, rk in spans(q_offsets, k_offsets):
        lq, lk = rq.stop - rq.start, rk.stop - rk.start
        if lq == 0:
            continue
        see = visible(lq, lk, causal, window, q.device)
        none = ~see.any(1)
        for h in range(qh):
            kk, vv, qq = k[rk, h // (qh // kh)], v[rk, h // (qh // kh)], q[rq, h]
            z = (qq @ kk.T * scale).masked_fill(~see, -float("inf"))
            size = (qq.abs() @ kk.T.abs() * scale).masked_fill(~see, 0.0)
            if lk == 0:
                out[rq, h], ob[rq, h], lse[h, rq], lb[h, rq] = 0.0, 0.0, -float("inf"), 0.0
                continue
            s = torch.logsumexp(z, 1)
            p = torch.exp(z - s[:, None]).masked_fill(none[:, None], 0.0)
            rel = U32 * ((d + 16) * size.amax(1) + 8 * size.amax(1) + 8)
            o = p @ vv
            b = (p_half + 2 * rel + (lk + 64) * U32)[:, None] * (p @ vv.abs()) + TINY * (1 + vv.abs().sum(0))
            out[rq, h], ob[rq, h] = o, b + half * (o.abs() + b)
            lse[h, rq] = s
            lb[h, rq] = torch.where(none, 0.0, rel + (lk + 64) * U32 + 4 * U32 * s.abs().masked_fill(none, 0.0))
    return out, ob, lse, lb


def backward(dout, q, k, v, o, lse, q_offsets, k_offsets, causal, window, scale, dtype):
    """((dq, bound), (dk, bound), (dv, bound)) for the stored o and lse."""
    dout, q, k, v, o, lse = (t.double() for t in (dout, q, k, v, o, lse))
    (n, qh, d), (nk, kh) = q.shape, k.shape[:2]
    nan = lambda t: torch.full_like(t, float("nan"))  # noqa: E731
    dq, bq, dk, bk, dv, bv = nan(q), nan(q), nan(k), nan(k), nan(v), nan(v)
    half = half_step(dtype)
    p_half = half if dtype == torch.bfloat16 else 0.0
    for rq, rk in spans(q_offsets, k_offsets):
        lq, lk = rq.stop - rq.start, rk.stop - rk.start
        for t in (dk, bk, dv, bv):
            t[rk] = 0.0
        for t in (dq, bq):
            t[rq] = 0.0
        if lq == 0 or lk == 0:
            continue
        see = visible(lq, lk, causal, window, q.device)
        terms = lq * (qh // kh)
        for h in range(qh):
            kv = h // (qh // kh)
            qq, kk, vv, dd, oo = q[rq, h], k[rk, kv], v[rk, kv], dout[rq, h], o[rq, h]
            z = qq @ kk.T * scale
            size = qq.abs() @ kk.T.abs() * scale
            s = lse[h, rq][:, None]
            p = torch.exp(z - s).masked_fill(~see, 0.0)
            rel = U32 * ((d + 24) * size + 4 * s.abs().masked_fill(torch.isinf(s), 0.0) + 8)
            dp, delta = dd @ vv.T, (dd * oo).sum(1, keepdim=True)
            near = U32 * (d + 24) * (dd.abs() @ vv.abs().T + (dd * oo).abs().sum(1, keepdim=True))
            ds = p * (dp - delta)
            e_p = p * (rel + p_half) + TINY
            e_ds = p * (rel * (dp - delta).abs() * 2 + near * 2) + (p_half + 4 * U32) * (ds.abs() + 2 * p * near) + TINY * (1 + dp.abs() + delta.abs())
            add = (lk + 64) * U32
            dq[rq, h] = ds @ kk * scale
            bq[rq, h] = (e_ds + add * ds.abs()) @ kk.abs() * scale * (1 + 4 * U32)
            add = (terms + 64) * U32
            dk[rk, kv] += ds.T @ qq * scale
            bk[rk, kv] += (e_ds + add * ds.abs()).T @ qq.abs() * scale * (1 + 4 * U32)
            dv[rk, kv] += p.T @ dd
            bv[rk, kv] += (e_p + add * p).T @ dd.abs()
    return tuple((w, b + TINY + half * (w.abs() + b)) for w, b in ((dq, bq), (dk, bk), (dv, bv)))


def offsets(lengths, device="cuda"):
    ends = np.concatenate([[0], np.cumsum(lengths)]).astype(int).tolist()
    return ends, torch.tensor(ends, dtype=torch.int32, device=device)
