"""Norms around a block with gate and residual scale, forward and backward,
against the float64 reference."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa
from oracle import block

from ops_util import U32, dev, half_step, host, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


def rows_of(rng, n, dim, std, dtype, shift=0, pitch=0):
    """(n, dim) with `pitch` more elements between rows, `shift` elements behind an aligned address."""
    return dev(rng.standard_normal((n, dim + pitch)) * std, dtype, shift)[:, :dim]


def make(n, dim, dtype, branch, wdt, seed, shift=0, pitch=0):
    rng = np.random.default_rng(seed)
    x, h = rows_of(rng, n, dim, 2.0, dtype, shift, pitch), rows_of(rng, n, dim, 0.5, branch, shift, 2 * pitch)
    dx, dy = rows_of(rng, n, dim, 0.1, dtype, shift, pitch), rows_of(rng, n, dim, 0.1, branch, shift, pitch)
    pre, post, gate = (dev(rng.standard_normal(dim) * 0.2 + m, wdt, shift) for m in (1.0, 0.9, 0.5))
    return x, h, dx, dy, pre, post, gate


def opt(t):
    return None if t is None else host(t)


def check(n, dim, dtype, branch, wdt, seed=0, shift=0, pitch=0, post_norm=True, gains=True, gated=True, stream=True,
          eps=1e-6, scale=0.8, offset=0.0):
    """A sum over a row takes at most 64 additions in a lane, 6 across it and 15
    across the waves, and a product or two per element: relative to its terms'
    magnitudes it is within 88 units; a reciprocal length (half of that, and
    root, reciprocal and mean) within 50, what is scaled by both within 120."""
    x, h, dx, dy, pre, post, gate = make(n, dim, dtype, branch, wdt, seed, shift, pitch)
    if not gains:
        pre = post = None
    if not post_norm:
        post = None
    if not gated:
        gate = None
    kw = dict(eps=eps, residual_scale=scale, weight_offset=offset, post_norm=post_norm)
    eps, scale = float(np.float32(eps)), float(np.float32(scale))
    x_out, y = nsa.block_norm(x, h, pre, post, gate, **kw)
    assert x_out.dtype == dtype and y.dtype == branch and x_out.is_contiguous() and y.is_contiguous()
    xh, hh, gp, gq, gt = host(x), host(h), opt(pre), opt(post), opt(gate)
    want = block.block_norm_stream(xh, hh, gq, gt, eps, scale, offset, post_norm)
    b = 120 * U32 * np.abs(want - xh) + 2 * U32 * (np.abs(xh) + np.abs(want))
    within(host(x_out), want, b + half_step(dtype) * (np.abs(want) + b), "x_out")
    xo = host(x_out)                        # y reads the stored stream
    want = block.block_norm_out(xo, gp, eps, offset)
    b = 120 * U32 * np.abs(xo / np.sqrt(np.mean(xo * xo, -1, keepdims=True) + eps)) * (
        1.0 if gp is None else abs(offset) + np.abs(gp))
    within(host(y), want, b + half_step(branch) * (np.abs(want) + b), "y")

    got = nsa.block_norm_grad(dx if stream else None, dy, x_out, h, pre, post, gate, **kw)
    dxh, dyh = host(dx) if stream else None, host(dy)
    want = block.block_norm_grad(dxh, dyh, xo, hh, gp, gq, gt, eps, scale, offset, post_norm)
    one = np.ones(dim)
    gpre, gpost = (one if g is None else abs(offset) + np.abs(g) for g in (gp, gq))
    ga = one if gt is None else np.abs(gt)
    rx = 1 / np.sqrt(np.mean(xo * xo, -1, keepdims=True) + eps)
    rh = 1 / np.sqrt(np.mean(hh * hh, -1, keepdims=True) + eps) if post_norm else np.ones((n, 1))
    ux, uh = np.abs(xo * rx), np.abs(hh * rh)
    u = np.abs(dyh) * gpre
    # t: both terms within 88 + 2 * 50 + 12
    t = rx * (u + ux * np.mean(u * ux, -1, keepdims=True)) + (0.0 if dxh is None else np.abs(dxh))
    b = 200 * U32 * t
    within(host(got[0]), want[0], b + half_step(dtype) * (np.abs(want[0]) + b), "dx")
    # d = s gate g_post t, then the same once more around h
    mag = abs(scale)   # bounds are magnitudes: a negative scale must not turn them around
    d = mag * ga * gpost * t
    size = rh * (d + uh * np.mean(d * uh, -1, keepdims=True)) if post_norm else d
    b = 420 * U32 * size
    within(host(got[1]), want[1], b + half_step(branch) * (np.abs(want[1]) + b), "dh")
    # sums over rows: 200 + 60 units a term, and fewer than rows + 120 additions
    sums = ((pre, np.abs(dyh) * ux), (post, mag * ga * t * uh), (gate, mag * gpost * t * uh))
    for k, (w, size) in enumerate(sums):
        if w is None:
            assert got[2 + k] is None
            continue
        assert got[2 + k].dtype == wdt
        b = (380 + n) * U32 * size.sum(0)
        within(host(got[2 + k]), want[2 + k], b + half_step(wdt) * (np.abs(want[2 + k]) + b), f"weight {k}")


# every width's layout: one wave a row, four, sixteen, the wide rows; ragged ends of each
@pytest.mark.parametrize("dim", [1, 7, 8, 64, 511, 512, 513, 1024, 1025, 2048, 2051, 4096, 4099, 8192, 8193, 16384, 20001, 40007,
                                 65536])
@pytest.mark.parametrize("dtype,branch,wdt", [(F32, F32, F32), (BF16, BF16, BF16), (F32, BF16, F32)])
def test_widths(dim, dtype, branch, wdt):
    check(5, dim, dtype, branch, wdt, seed=dim)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 63, 777, 3000])
@pytest.mark.parametrize("dim", [40, 1000, 2056])
def test_rows(n, dim):
    check(n, dim, F32, F32, F32, seed=n)
    check(n, dim, BF16, BF16, F32, seed=n + 1)


def test_many_wide_rows():
    check(300, 8200, BF16, F32, BF16, seed=1)


@pytest.mark.parametrize("shift,pitch", [(1, 0), (0, 3), (3, 5), (0, 8)])
@pytest.mark.parametrize("dim", [64, 1001, 4096, 9000])
def test_strides_and_alignment(dim, shift, pitch):
    check(6, dim, F32, BF16, BF16, seed=3, shift=shift, pitch=pitch)
    check(6, dim, BF16, BF16, F32, seed=4, shift=shift, pitch=pitch)


@pytest.mark.parametrize("post_norm", [False, True])
@pytest.mark.parametrize("gains", [False, True])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("stream", [False, True])
def test_parts(post_norm, gains, gated, stream):
    for dim in (100, 1500, 8300):
        check(9, dim, F32, F32, F32, 5, 0, 0, post_norm, gains, gated, stream, scale=-1.5, offset=1.0, eps=1e-2)


def test_strides_do_not_change_a_bit():
    x, h, dx, dy, pre, post, gate = make(50, 1000, BF16, BF16, BF16, 6)
    x2, h2, dx2, dy2, *_ = make(50, 1000, BF16, BF16, BF16, 6, shift=1, pitch=3)
    for a, b in ((x2, x), (h2, h), (dx2, dx), (dy2, dy)):
        a.copy_(b)
    kw = dict(post_norm=True)
    one, two = nsa.block_norm(x, h, pre, post, gate, **kw), nsa.block_norm(x2, h2, pre, post, gate, **kw)
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    back = [nsa.block_norm_grad(a, b, c, d, pre, post, gate, **kw) for a, b, c, d in
            ((dx, dy, x, h), (dx2, dy2, x2, h2), (dx, dy, x, h))]
    for other in back[1:]:
        assert all(torch.equal(a, b) for a, b in zip(back[0], other))


# 513, 1030, 4099, 16390: the last run begins in one wave and is loaded together with another's last elements
@pytest.mark.parametrize("dim", [5, 100, 513, 1030, 4099, 5000, 9000, 16390])
@pytest.mark.parametrize("post_norm", [False, True])
def test_in_place(dim, post_norm):
    x, h, dx, dy, pre, post, gate = make(20, dim, F32, BF16, F32, 7)
    post = post if post_norm else None
    kw = dict(post_norm=post_norm, residual_scale=0.5)
    want = nsa.block_norm(x, h, pre, post, gate, **kw)
    back = nsa.block_norm_grad(dx, dy, want[0], h, pre, post, gate, **kw)
    got = nsa.block_norm_grad(dx, dy, want[0], h, pre, post, gate, dx=dx, **kw)
    assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(back, got) if a is not None)
    got = nsa.block_norm(x, h, pre, post, gate, x_out=x, y=h, **kw)
    assert got[0] is x and got[1] is h and torch.equal(x, want[0]) and torch.equal(h, want[1])


def test_no_rows():
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    a, b = nsa.block_norm(x, x, w, None, w)
    assert a.shape == b.shape == (0, 64)
    got = nsa.block_norm_grad(None, x, x, x, w, w, w, post_norm=True)
    assert got[0].shape == (0, 64) and not any(t.any() for t in got[2:])


def test_nan_and_infinity_stay_in_their_rows():
    x, h, dx, dy, pre, post, gate = make(12, 700, F32, F32, F32, 8)
    x[3, 5], h[7, 1] = float("nan"), float("inf")
    a, b = nsa.block_norm(x, h, pre, post, gate, post_norm=True)
    bad = torch.zeros(12, dtype=torch.bool, device="cuda")
    bad[3] = bad[7] = True
    assert torch.isfinite(a[~bad]).all() and torch.isfinite(b[~bad]).all()
    assert not torch.isfinite(b[bad]).all(1).any()
