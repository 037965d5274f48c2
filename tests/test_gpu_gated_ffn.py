"""The gated feed-forward product, forward and backward, against float64."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa
from oracle import block

from ops_util import U32, half_step, host, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


def make(n, dim, hidden, dtype, seed, shift=0, pitch=0, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)

    def rows(r, width, std, extra=0):
        t = torch.randn(r * (width + extra) + shift, generator=g, device="cuda").mul_(std).to(dtype)
        return t[shift:].view(r, width + extra)[:, :width]

    return (rows(n, dim, std, pitch), rows(hidden, dim, 1.2 * dim ** -0.5), rows(hidden, dim, dim ** -0.5),
            rows(n, hidden, 0.1, pitch))


def activation(g, kind):
    """act, act' and the largest |act''| near g, by autograd of the definition."""
    g = g.detach().requires_grad_()
    if kind == "silu":
        a = g * torch.sigmoid(g)
    else:
        a = 0.5 * g * (1 + torch.tanh((2 / np.pi) ** 0.5 * (g + 0.044715 * g ** 3)))
    da, = torch.autograd.grad(a.sum(), g)
    return a.detach(), da


def check(n, dim, hidden, dtype, kind="silu", seed=0, shift=0, pitch=0, back=True, std=1.0):
    """A projection sums dim products: off by (dim + 16) units of their
    magnitudes, G and U.  |act'| <= 1.13 and |act''| <= 0.8 for both, and the
    activation itself is within 24 units of |g|, its slope within 60 (exponential,
    reciprocal, and cubes of g up to where the slope still differs from 0 or 1:
    2 |y| < 32 turns 4 units of y into 64)."""
    x, wg, wu, dh = make(n, dim, hidden, dtype, seed, shift, pitch, std)
    got = nsa.gated_ffn(x, wg, wu, kind)
    assert got.shape == (n, hidden) and got.dtype == dtype and got.is_contiguous()
    xd, gd, ud, hd = (t.double() for t in (x, wg, wu, dh))
    g, u = xd @ gd.T, xd @ ud.T
    eg, eu = ((dim + 16) * U32 * (xd.abs() @ w.abs().T) for w in (gd, ud))
    a, da = activation(g, kind)
    want = a * u
    ea = 1.13 * eg + 100 * U32 * g.abs()
    b = ea * u.abs() + (a.abs() + ea) * eu + 4 * U32 * want.abs()
    half = half_step(dtype)
    within(host(got), want.cpu().numpy(), (b + half * (want.abs() + b)).cpu().numpy(), "h")
    if not back:
        return
    got = nsa.gated_ffn_grad(dh, x, wg, wu, kind)
    assert [t.shape for t in got] == [x.shape, wg.shape, wu.shape] and all(t.dtype == dtype for t in got)
    eda = 0.8 * eg + 200 * U32
    dg, du = hd * u * da, hd * a
    store = half if dtype == BF16 else 0.0   # rounded once, as operands of the next products
    edg = hd.abs() * (u.abs() * eda + eu * (da.abs() + eda)) + (store + 4 * U32) * dg.abs() * 1.01
    edu = hd.abs() * ea + (store + 4 * U32) * du.abs() * 1.01
    dx = dg @ gd + du @ ud
    add = (2 * hidden + 64) * U32
    b = (edg + add * dg.abs()) @ gd.abs() + (edu + add * du.abs()) @ ud.abs()
    within(host(got[0]), dx.cpu().numpy(), (b * 1.01 + half * (dx.abs() + b)).cpu().numpy(), "dx")
    add = (n + 64) * U32
    for what, t, d, e in (("dw_gate", got[1], dg, edg), ("dw_up", got[2], du, edu)):
        want, b = d.T @ xd, (e + add * d.abs()).T @ xd.abs()
        within(host(t), want.cpu().numpy(), (b * 1.01 + half * (want.abs() + b)).cpu().numpy(), what)


def test_reference_is_the_oracles():
    x, wg, wu, dh = make(7, 9, 11, F32, 1)
    for kind in ("silu", "gelu"):
        a, da = activation(x.double() @ wg.double().T, kind)
        wa, wda = block.activation(host(x) @ host(wg).T, kind)
        np.testing.assert_allclose(a.cpu().numpy(), wa, rtol=1e-12, atol=1e-15)
        np.testing.assert_allclose(da.cpu().numpy(), wda, rtol=1e-10, atol=1e-13)


# one token to the last that goes without tiles, and around the tiles' sizes
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 32, 33, 63, 64, 65, 127, 128, 200, 256, 257, 513])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tokens(n, dtype):
    check(n, 128, 192, dtype, seed=n)
    check(n, 192, 130, dtype, "gelu", seed=n + 1)


@pytest.mark.parametrize("dim", [1, 3, 8, 31, 32, 64, 72, 100, 256, 264, 500, 1024, 1100])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_dims(dim, dtype):
    check(5, dim, 96, dtype, seed=dim)
    check(150, dim, 96, dtype, seed=dim)


@pytest.mark.parametrize("hidden", [1, 5, 8, 15, 16, 17, 63, 64, 127, 128, 129, 300, 1000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_hidden_widths(hidden, dtype):
    check(3, 64, hidden, dtype, "gelu", seed=hidden)
    check(130, 64, hidden, dtype, "gelu", seed=hidden)
    check(130, 320, hidden, dtype, seed=hidden)


@pytest.mark.parametrize("shift,pitch", [(1, 0), (0, 3), (8, 8), (2, 5)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_alignment(shift, pitch, dtype):
    for n in (4, 40, 140):
        check(n, 128, 200, dtype, seed=1, shift=shift, pitch=pitch)
        check(n, 130, 72, dtype, "gelu", seed=1, shift=shift, pitch=pitch)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_far_from_zero(kind, dtype):
    """Projections of some hundreds: the activation is 0 or its argument."""
    for n in (9, 100):
        check(n, 64, 80, dtype, kind, seed=3, std=200.0)


def test_wide_contractions():
    check(700, 2048, 1400, BF16, seed=4)
    check(300, 1024, 700, F32, "gelu", seed=5)


def test_the_same_bits_again_and_for_other_strides():
    x, wg, wu, dh = make(100, 128, 192, BF16, 6)
    x2, wg2, wu2, dh2 = make(100, 128, 192, BF16, 7, shift=1, pitch=3)
    for a, b in ((x2, x), (wg2, wg), (wu2, wu), (dh2, dh)):
        a.copy_(b)
    assert torch.equal(nsa.gated_ffn(x, wg, wu), nsa.gated_ffn(x2, wg2, wu2))
    assert torch.equal(nsa.gated_ffn(x[:20], wg, wu), nsa.gated_ffn(x2[:20], wg2, wu2))
    one, two = nsa.gated_ffn_grad(dh, x, wg, wu), nsa.gated_ffn_grad(dh2, x2, wg2, wu2)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_given_results_and_packed_weights():
    x, wg, wu, dh = make(90, 128, 192, BF16, 8)
    packed = torch.cat([wg, wu])                 # one buffer of both, as a fused projection keeps them
    grads = torch.full_like(packed, 7.0)
    wide = torch.full((90, 300), 7.0, dtype=BF16, device="cuda")
    want, back = nsa.gated_ffn(x, wg, wu), nsa.gated_ffn_grad(dh, x, wg, wu)
    out = nsa.gated_ffn(x, packed[:192], packed[192:], out=wide[:, 5:197])
    assert torch.equal(out, want) and (wide[:, :5] == 7).all() and (wide[:, 197:] == 7).all()
    dx = torch.full_like(x, 7.0)
    got = nsa.gated_ffn_grad(dh, x, packed[:192], packed[192:], dx=dx, dw_gate=grads[:192], dw_up=grads[192:])
    assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(got, back))


def test_no_tokens():
    x, wg, wu, dh = make(0, 64, 80, BF16, 9)
    assert nsa.gated_ffn(x, wg, wu).shape == (0, 80)
    dx, dg, du = nsa.gated_ffn_grad(dh, x, wg, wu)
    assert dx.shape == (0, 64) and not dg.any() and not du.any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [10, 100])
def test_nan_and_infinity_stay_in_their_rows(n, dtype):
    x, wg, wu, dh = make(n, 128, 150, dtype, 10)
    want = nsa.gated_ffn(x, wg, wu)
    x = x.clone()
    x[n - 1, 3], x[4, 7] = float("nan"), float("inf")
    got = nsa.gated_ffn(x, wg, wu)
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[4] = keep[n - 1] = False
    assert torch.equal(got[keep], want[keep]) and got[n - 1].isnan().all()
    back = nsa.gated_ffn_grad(dh, x, wg, wu)[0]
    assert torch.isfinite(back[keep]).all() and back[n - 1].isnan().all()


def test_gradient_by_differences():
    x, wg, wu, dh = make(70, 64, 96, F32, 11)
    grads = nsa.gated_ffn_grad(dh, x, wg, wu, "gelu")
    step = 2.0 ** -7
    for which, g in enumerate(grads):
        d = torch.randn(g.shape, generator=torch.Generator("cuda").manual_seed(which), device="cuda")
        d *= [x, wg, wu][which].std()
        values = []
        for sign in (1, -1):
            t = [x, wg, wu]
            t[which] = t[which] + sign * step * d
            values.append(float((nsa.gated_ffn(*t, "gelu").double() * dh.double()).sum()))
        got, want = float((g.double() * d.double()).sum()), (values[0] - values[1]) / (2 * step)
        # the third derivative's share (step^2 / 6 of a value of this size) and the results' roundings over the step
        assert abs(got - want) <= 2e-3 * (abs(want) + float((g.double() * d.double()).norm())), which


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 70])
def test_activation_is_zero_or_its_argument_far_out(n, dtype, kind):
    """One input column of 1s: the projections are the weights, and beyond +-200 act is 0 or g and
    its derivative 0 or 1, to less than half a step of any type.  The gradients of 1 or 64 tokens,
    a power of two each, add up to 1 without rounding."""
    tokens = 64 if n == 70 else n
    g = torch.tensor([s * 2.0 ** e for e in (8, 20, 43, 60, 83, 100) for s in (1, -1)], device="cuda").to(dtype)
    x, one = torch.ones(n, 1, dtype=dtype, device="cuda"), torch.ones_like(g)[:, None]
    want = torch.where(g > 0, g, torch.zeros_like(g))
    out = nsa.gated_ffn(x, g[:, None], one, kind)
    assert torch.equal(out, want.expand(n, -1))
    dh = torch.zeros(n, len(g), dtype=dtype, device="cuda")
    dh[:tokens] = 1 / tokens
    dx, dg, du = nsa.gated_ffn_grad(dh, x, g[:, None], one, kind)
    assert torch.equal(dg[:, 0], (g > 0).to(dtype)) and torch.equal(du[:, 0], want)
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("stride", [(1 << 22) - 4, 1 << 22, (1 << 22) + 4])
def test_strides_around_the_limit_of_short_offsets(stride):
    """Aligned fp32 rows up to and beyond 16 MiB apart: the same bits as rows side by side."""
    n, dim, hidden = 70, 12, 40
    near, wg, wu, dh = make(n, dim, hidden, F32, 5)
    x = torch.empty((n - 1) * stride + dim, device="cuda").as_strided((n, dim), (stride, 1))
    x.copy_(near)
    assert torch.equal(nsa.gated_ffn(x, wg, wu), nsa.gated_ffn(near, wg, wu))
    for a, b in zip(nsa.gated_ffn_grad(dh, x, wg, wu), nsa.gated_ffn_grad(dh, near, wg, wu)):
        assert torch.equal(a, b)
