"""Norm of queries and keys with the rotation, forward and backward, against the
float64 reference."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa
from oracle import ops

from ops_util import DT, U32, dev, half_step, host, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


def make(n, qh, kh, d, rot, dtype, wdt, seed, shift=0, pitch=0, pads=True, idx=torch.int64):
    """A packed projection (queries, keys, values), gains, positions, table."""
    rng = np.random.default_rng(seed)
    width = (qh + 2 * kh) * d + pitch
    packed = dev(rng.standard_normal((n, width)) * 1.5, dtype, shift)
    q, k = (packed[:, a * d:b * d].unflatten(1, (b - a, d)) for a, b in ((0, qh), (qh, qh + kh)))
    qw, kw = (dev(rng.standard_normal(d) * 0.2, wdt) for _ in range(2))
    rope = nsa.rope_table(50, rot, 10000.0) if rot else None
    pos = rng.integers(0, 50, n)
    if pads and n > 2:
        pos[::5] = -1
    return packed, q, k, qw, kw, dev(pos, idx), pos, rope


def turned(x, pos, rope, inter):
    """|a cos| + |b sin| per element: the size of what a rotation adds."""
    if rope is None:
        return np.abs(x)
    t = np.abs(np.asarray(rope, np.float64))[np.clip(pos, 0, len(rope) - 1)]
    half = t.shape[1] // 2
    i, j = (np.arange(half) * 2, np.arange(half) * 2 + 1) if inter else (np.arange(half), np.arange(half) + half)
    c, s, ax = t[:, None, :half], t[:, None, half:], np.abs(x)
    out = ax.copy()
    out[..., i] = ax[..., i] * c + ax[..., j] * s
    out[..., j] = ax[..., i] * s + ax[..., j] * c
    return out


def check_forward(x, w, got, pos, rope, eps, inter, offset, dtype):
    """The sum of squares takes 8 + 6 additions and a product per element, the
    mean, eps, root and reciprocal four more roundings (half of what precedes
    the root counts): r is within 14 units, the normed value times its gain
    within 18, the rotation adds 3: 24 fp32 units of the rotated magnitudes."""
    xh, wh = host(x), None if w is None else host(w)
    want = ops.qk_norm_rope(xh, wh, pos, None if rope is None else host(rope), eps, inter, offset)
    r = 1 / np.sqrt(np.mean(xh * xh, -1, keepdims=True) + eps)
    mag = turned(np.abs(xh * r) * (1.0 if wh is None else abs(offset) + np.abs(wh)), pos, None if rope is None else host(rope), inter)
    b = 24 * U32 * mag
    within(host(got), want, b + half_step(dtype) * (np.abs(want) + b), "forward")


def check_backward(dy, x, w, dx, dw, pos, rope, eps, inter, offset, dtype, wdt):
    """dn within 3 units of its magnitude; xh within 16; g = dn w within 21;
    the mean of D products of 37 units, summed in 14 steps: 52; dx = r (g - xh
    mean): 80 covers both terms.  dw adds tokens x heads products, each lane in
    sequence and the lanes and blocks after that: fewer additions than tokens x
    heads + 300."""
    rp = None if rope is None else host(rope)
    dyh, xh, wh = host(dy), host(x), None if w is None else host(w)
    want, wantw = ops.qk_norm_rope_grad(dyh, xh, wh, pos, rp, eps, inter, offset)
    r = 1 / np.sqrt(np.mean(xh * xh, -1, keepdims=True) + eps)
    dyh[pos < 0] = 0.0
    dn, n = turned(dyh, pos, rp, inter), np.abs(xh * r)
    g = dn * (1.0 if wh is None else abs(offset) + np.abs(wh))
    b = 80 * U32 * r * (g + n * np.mean(g * n, -1, keepdims=True))
    within(host(dx), want, b + half_step(dtype) * (np.abs(want) + b), "dx")
    if dw is not None:
        size = (dn * n).sum((0, 1))
        b = (min(dn.shape[0] * dn.shape[1], 4000) + 340) * U32 * size
        within(host(dw), wantw, b + half_step(wdt) * (np.abs(wantw) + b), "dw")


CASES = [  # n, q heads, k heads, D, rot
    (1, 1, 1, 1, 0), (1, 32, 8, 128, 128), (3, 3, 1, 2, 2), (7, 5, 2, 8, 8), (16, 4, 2, 64, 32), (5, 6, 3, 80, 80),
    (33, 2, 1, 96, 64), (9, 3, 3, 7, 4), (4, 7, 1, 30, 10), (130, 4, 4, 256, 256), (6, 2, 1, 512, 512), (5, 1, 1, 511, 256),
    (4100, 3, 2, 16, 16), (5000, 5, 3, 40, 24)]


@pytest.mark.parametrize("dt,wdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(case, inter, dt, wdt):
    n, qh, kh, d, rot = case
    offset = 1.0 if n % 2 else 0.0
    packed, q, k, qw, kw, pos_d, pos, rope = make(n, qh, kh, d, rot, DT[dt], DT[wdt], n + d)
    p = None if rope is None else pos_d
    kwargs = dict(eps=1e-6, interleaved=inter, weight_offset=offset)
    eps = float(np.float32(1e-6))
    if rope is None:
        pos = np.zeros(n, np.int64)
    out = nsa.qk_norm_rope(q, k, qw, kw, p, rope, **kwargs)
    for x, w, got in zip((q, k), (qw, kw), out):
        check_forward(x, w, got, pos, rope, eps, inter, offset, DT[dt])
    rng = np.random.default_rng(d)
    dq, dk = (dev(rng.standard_normal(t.shape), DT[dt]) for t in (q, k))
    grads = nsa.qk_norm_rope_grad(dq, dk, q, k, qw, kw, p, rope, **kwargs)
    for dy, x, w, dx, dw in zip((dq, dk), (q, k), (qw, kw), grads[:2], grads[2:]):
        check_backward(dy, x, w, dx, dw, pos, rope, eps, inter, offset, DT[dt], DT[wdt])


@pytest.mark.parametrize("shift,pitch", [(1, 0), (0, 3), (8, 8)])
def test_strides_in_place_and_packed_gradients(shift, pitch):
    for dt in (torch.float32, torch.bfloat16):
        packed, q, k, qw, kw, pos_d, pos, rope = make(21, 4, 2, 64, 64, dt, dt, 3, shift, pitch, idx=torch.int32)
        want = nsa.qk_norm_rope(q.contiguous(), k.contiguous(), qw, kw, pos_d, rope)
        dy = [torch.randn_like(t) for t in want]
        wantg = nsa.qk_norm_rope_grad(*dy, q.contiguous(), k.contiguous(), qw, kw, pos_d, rope)
        dpacked = torch.full_like(packed, 5.0)
        dq, dk = (dpacked[:, a * 64:b * 64].unflatten(1, (b - a, 64)) for a, b in ((0, 4), (4, 6)))
        got = nsa.qk_norm_rope_grad(*dy, q, k, qw, kw, pos_d, rope, dq=dq, dk=dk)
        for a, b in zip(got, wantg):
            assert torch.equal(a, b)
        assert dpacked[:, 6 * 64:].eq(5.0).all()
        values = packed[:, 6 * 64:].clone()
        out = nsa.qk_norm_rope(q, k, qw, kw, pos_d, rope, q_out=q, k_out=k)
        assert out[0] is q and all(torch.equal(a, b) for a, b in zip(out, want))
        assert torch.equal(packed[:, 6 * 64:], values)
        again = nsa.qk_norm_rope_grad(*(t.clone() for t in dy), *(t.contiguous() for t in out), qw, kw, pos_d, rope)
        own = [t.clone() for t in dy]
        nsa.qk_norm_rope_grad(*own, out[0], out[1], qw, kw, pos_d, rope, dq=own[0], dk=own[1])
        assert torch.equal(own[0], again[0]) and torch.equal(own[1], again[1])


def test_no_gain_one_tensor_and_one_gain():
    _, q, k, qw, kw, pos_d, pos, rope = make(40, 3, 2, 32, 32, torch.float32, torch.float32, 4)
    eps = float(np.float32(1e-6))
    out = nsa.qk_norm_rope(q, k, None, None, pos_d, rope)
    check_forward(q, None, out[0], pos, rope, eps, False, 0.0, torch.float32)
    dq, dk = torch.randn_like(out[0]), torch.randn_like(out[1])
    g = nsa.qk_norm_rope_grad(dq, dk, q, k, None, kw, pos_d, rope)
    assert g[2] is None
    check_backward(dq, q, None, g[0], None, pos, rope, eps, False, 0.0, torch.float32, torch.float32)
    check_backward(dk, k, kw, g[1], g[3], pos, rope, eps, False, 0.0, torch.float32, torch.float32)
    only = nsa.qk_norm_rope(q, k[:, :0], qw, None, pos_d, rope)
    assert torch.equal(only[0], nsa.qk_norm_rope(q, k, qw, kw, pos_d, rope)[0]) and only[1].numel() == 0


def test_padding_is_not_read_and_far_positions_are_nan():
    _, q, k, qw, kw, pos_d, pos, rope = make(10, 2, 1, 16, 8, torch.float32, torch.float32, 5, pads=False)
    q, k = q.clone(), k.clone()
    pos_d[3], pos_d[7] = -1, -2 ** 40
    q[3], k[7] = float("nan"), float("inf")
    dq, dk = torch.randn_like(q), torch.randn_like(k)
    dq[3] = float("nan")
    for eps in (1e-6, 0.0):
        out = nsa.qk_norm_rope(q, k, qw, kw, pos_d, rope, eps=eps)
        grads = nsa.qk_norm_rope_grad(dq, dk, q, k, qw, kw, pos_d, rope, eps=eps)
        for t in (*out, *grads[:2]):
            assert not t[3].any() and not t[7].any() and torch.isfinite(t).all()
        assert torch.isfinite(grads[2]).all() and torch.isfinite(grads[3]).all()
    pos_d[5] = 50
    out = nsa.qk_norm_rope(q, k, qw, kw, pos_d, rope)
    assert torch.isnan(out[0][5]).all() and torch.isnan(out[1][5]).all() and torch.isfinite(out[0][6]).all()
    grads = nsa.qk_norm_rope_grad(dq, dk, q, k, qw, kw, pos_d, rope)
    assert torch.isnan(grads[0][5]).all() and torch.isnan(grads[2]).all()


def test_no_tokens():
    z = torch.zeros(0, 2, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    pos = torch.zeros(0, dtype=torch.int64, device="cuda")
    rope = nsa.rope_table(4, 8)
    assert nsa.qk_norm_rope(z, z, w, w, pos, rope)[0].shape == z.shape
    g = nsa.qk_norm_rope_grad(z, z, z, z, w, w, pos, rope)
    assert not g[2].any() and not g[3].any()


def test_gradient_against_a_difference():
    rng = np.random.default_rng(6)
    _, q, k, qw, kw, pos_d, pos, rope = make(30, 3, 2, 24, 16, torch.float32, torch.float32, 7)
    dq, dk = torch.randn(q.shape, device="cuda"), torch.randn(k.shape, device="cuda")
    g = nsa.qk_norm_rope_grad(dq, dk, q, k, qw, kw, pos_d, rope, eps=1e-3, weight_offset=1.0)
    kw_ = dict(positions=pos, rope=host(rope), eps=float(np.float32(1e-3)), offset=1.0)
    x, w, dy, h = host(q), host(qw), host(dq), 1e-6
    v, u = rng.standard_normal(x.shape), rng.standard_normal(w.shape)
    fx = lambda a: float((dy * ops.qk_norm_rope(a, w, **kw_)).sum())  # noqa: E731
    fw = lambda a: float((dy * ops.qk_norm_rope(x, a, **kw_)).sum())  # noqa: E731
    # fp32 gradients: 100 units of the summed magnitudes; the difference: 1e-7 of the function's size
    size = np.abs(dy).sum() * 3
    assert abs(float((host(g[0]) * v).sum()) - (fx(x + h * v) - fx(x - h * v)) / (2 * h)) <= 100 * U32 * size + 1e-7 * size
    assert abs(float((host(g[2]) * u).sum()) - (fw(w + h * u) - fw(w - h * u)) / (2 * h)) <= 100 * U32 * size + 1e-7 * size


def test_reproducible_on_streams_and_in_a_graph():
    packed, q, k, qw, kw, pos_d, pos, rope = make(300, 8, 2, 64, 64, torch.bfloat16, torch.bfloat16, 8)
    dq, dk = torch.randn_like(q), torch.randn_like(k)

    def step(stream=None):
        return (*nsa.qk_norm_rope(q, k, qw, kw, pos_d, rope, stream=stream),
                *nsa.qk_norm_rope_grad(dq, dk, q, k, qw, kw, pos_d, rope, stream=stream))

    first = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = step(side), step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, t) for x, t in zip(a, first)) and all(torch.equal(x, t) for x, t in zip(b, first))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(4):
        packed.normal_()
        pos_d.random_(-1, 50)
        g.replay()
        torch.cuda.synchronize()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, t) for x, t in zip(outs, want))
