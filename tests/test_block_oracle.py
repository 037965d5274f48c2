"""The float64 reference of the block operators against something other than
itself: differences of the forward for every gradient, closed forms, and
autograd of plain torch."""
import numpy as np
import pytest
import torch

from oracle import block


def rng(seed):
    return np.random.default_rng(seed)


def by_differences(f, x, at, step=1e-6):
    """df/dx[at] by a central difference."""
    hi, lo = x.copy(), x.copy()
    hi[at] += step
    lo[at] -= step
    return (f(hi) - f(lo)) / (2 * step)


def some(x, r, n=6):
    return [tuple(int(r.integers(0, s)) for s in x.shape) for _ in range(n)]


@pytest.mark.parametrize("post_norm", [False, True])
def test_block_norm_gradient_is_the_forwards(post_norm):
    r = rng(1)
    x, h, cx, cy = (r.standard_normal((5, 7)) for _ in range(4))
    pre, post, gate = (r.standard_normal(7) for _ in range(3))
    post = post if post_norm else None
    kw = dict(eps=1e-3, scale=0.7, offset=0.5)

    def value(x=x, h=h, pre=pre, post=post, gate=gate):
        s = block.block_norm_stream(x, h, post, gate, 1e-3, 0.7, 0.5, post_norm)
        return float((cx * s).sum() + (cy * block.block_norm_out(s, pre, 1e-3, 0.5)).sum())

    s = block.block_norm_stream(x, h, post, gate, post_norm=post_norm, **kw)
    got = block.block_norm_grad(cx, cy, s, h, pre, post, gate, post_norm=post_norm, **kw)
    for name, arr, g in (("x", x, got[0]), ("h", h, got[1]), ("pre", pre, got[2]), ("post", post, got[3]), ("gate", gate, got[4])):
        if arr is None:
            continue
        for at in some(arr, r):
            assert g[at] == pytest.approx(by_differences(lambda t: value(**{name: t}), arr, at), rel=1e-5, abs=1e-7), name


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 3)])
def test_attention_and_its_gradient(causal, window):
    r = rng(2)
    qo, ko = [0, 4, 4, 9], [0, 6, 9, 12]      # more keys than queries, no queries, more queries than keys
    q, c = r.standard_normal((9, 4, 5)), r.standard_normal((9, 4, 5))
    k, v = r.standard_normal((12, 2, 5)), r.standard_normal((12, 2, 5))
    out, lse = block.attention(q, k, v, qo, ko, causal, window)
    if causal:   # the last sequence's first two queries see no key
        assert not out[4:6].any() and np.isneginf(lse[:, 4:6]).all()
    # the same by a dense softmax with a mask
    for b in range(3):
        rq, rk = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b + 1])
        see = torch.from_numpy(block.visible(qo[b + 1] - qo[b], ko[b + 1] - ko[b], causal, window))
        for h in range(4):
            z = torch.from_numpy(q[rq, h] @ k[rk, h // 2].T) * 5 ** -0.5
            p = z.masked_fill(~see, -1e30).softmax(-1) * see
            np.testing.assert_allclose(out[rq, h], (p @ torch.from_numpy(v[rk, h // 2])).numpy(), rtol=1e-12, atol=1e-14)

    def value(q=q, k=k, v=v):
        return float((c * block.attention(q, k, v, qo, ko, causal, window)[0]).sum())

    got = block.attention_grad(c, q, k, v, qo, ko, causal, window)
    for name, arr, g in (("q", q, got[0]), ("k", k, got[1]), ("v", v, got[2])):
        for at in some(arr, r, 10):
            assert g[at] == pytest.approx(by_differences(lambda t: value(**{name: t}), arr, at), rel=1e-5, abs=1e-8), name


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gated_ffn_and_its_gradient(kind):
    r = rng(3)
    x, wg, wu, c = r.standard_normal((4, 3)), r.standard_normal((6, 3)), r.standard_normal((6, 3)), r.standard_normal((4, 6))
    f = torch.nn.functional.silu if kind == "silu" else lambda t: torch.nn.functional.gelu(t, approximate="tanh")
    tx, tg, tu = (torch.from_numpy(t).requires_grad_() for t in (x, wg, wu))
    want = f(tx @ tg.T) * (tx @ tu.T)
    np.testing.assert_allclose(block.gated_ffn(x, wg, wu, kind), want.detach().numpy(), rtol=1e-12)
    (want * torch.from_numpy(c)).sum().backward()
    for got, t in zip(block.gated_ffn_grad(c, x, wg, wu, kind), (tx, tg, tu)):
        np.testing.assert_allclose(got, t.grad.numpy(), rtol=1e-10, atol=1e-13)
