"""The block operators where elements lie more than 2^31 behind a tensor's first:
long caches, wide strides, large intermediate results."""
import pytest
import torch

import newton_schulz_08_amd as nsa

import attention_util as ref
import test_gpu_gated_ffn as ffn
from ops_util import U32, half_step, host, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()
    yield
    torch.cuda.empty_cache()


def far(n, width, stride, dtype, seed):
    """(n, width), `stride` elements between rows, over 2^31 from first to last."""
    assert (n - 1) * stride > 1 << 31
    big = torch.empty((n - 1) * stride + width, dtype=dtype, device="cuda")
    t = big.as_strided((n, width), (stride, 1))
    t.normal_(generator=torch.Generator("cuda").manual_seed(seed))
    return t


@pytest.mark.parametrize("pitch", [0, 1])
def test_attention_over_a_long_cache(pitch):
    lens, d, kh = [40000, 3, 35000], 64, 2
    n = sum(lens)
    kv = far(n, 2 * kh * d, 40000 + pitch, BF16, 1).unflatten(1, (2 * kh, d))   # pitch 1: no aligned runs
    ke, ko = ref.offsets(lens)
    for lq in ([1, 1, 2], [100, 3, 40]):
        qe, qo = ref.offsets(lq)
        q = torch.randn(qe[-1], 4, d, device="cuda").to(BF16)
        k, v = kv[:, :kh], kv[:, kh:]
        out, lse = nsa.attention(q, k, v, qo, ko)
        w, b, wl, lb = ref.forward(q, k, v, qe, ke, True, 0, d ** -0.5, BF16)
        within(host(out), w.cpu().numpy(), b.cpu().numpy(), "out")
        within(host(lse), wl.cpu().numpy(), lb.cpu().numpy(), "lse")


def test_attention_gradient_with_wide_strides():
    lens, d = [300, 212], 64
    n = sum(lens)
    e, off = ref.offsets(lens)
    stride = (1 << 31) // 400
    q, k, v, dout = (far(n, h * d, stride + 8 * i, BF16, i).unflatten(1, (h, d)) for i, h in enumerate((4, 2, 2, 4)))
    out, lse = nsa.attention(q, k, v, off, off)
    dq = far(n, 4 * d, stride, BF16, 9).unflatten(1, (4, d))
    got = nsa.attention_grad(dout, q, k, v, out, lse, off, off, dq=dq)
    for g, (w, b) in zip(got, ref.backward(dout, q, k, v, out, lse, e, e, True, 0, d ** -0.5, BF16)):
        within(host(g), w.cpu().numpy(), b.cpu().numpy(), "gradient")


def test_block_norm_with_wide_strides():
    n, dim = 300, 200
    stride = (1 << 31) // 250
    x, h, dx = (far(n, dim, stride + i, dt, i) for i, dt in enumerate((F32, BF16, F32)))
    w = torch.randn(dim, device="cuda")
    near = [t.contiguous() for t in (x, h, dx)]
    kw = dict(post_norm=True)
    assert all(torch.equal(a, b) for a, b in zip(nsa.block_norm(x, h, w, w, w, **kw), nsa.block_norm(*near[:2], w, w, w, **kw)))
    got = nsa.block_norm_grad(dx, h, x, h, w, w, w, dx=dx, **kw)
    want = nsa.block_norm_grad(near[2], near[1], near[0], near[1], w, w, w, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [30, 200])
def test_feed_forward_with_wide_strides(n, dtype):
    stride = (1 << 31) // (n - 5)
    x, dh = far(n, 72, stride, dtype, 1), far(n, 96, stride, dtype, 2)
    wg, wu = (torch.randn(96, 72, device="cuda").to(dtype) for _ in range(2))
    out, dx = far(n, 96, stride, dtype, 3), far(n, 72, stride, dtype, 4)
    nsa.gated_ffn(x, wg, wu, out=out)
    assert torch.equal(out, nsa.gated_ffn(x.contiguous(), wg, wu))
    got = nsa.gated_ffn_grad(dh, x, wg, wu, dx=dx)
    want = nsa.gated_ffn_grad(dh.contiguous(), x.contiguous(), wg, wu)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_feed_forward_gradient_of_many_tokens(dtype):
    n, dim, hidden = 36000, 64, 32768            # 2 n hidden > 2^31 intermediate numbers
    x, wg, wu, dh = ffn.make(n, dim, hidden, dtype, 1)
    dx, dg, du = nsa.gated_ffn_grad(dh, x, wg, wu)
    half = half_step(dtype)
    store = half if dtype == BF16 else 0.0

    def parts(rows, cols):
        """d_gate, d_up with bounds, for some rows and hidden columns (bounds as in the operator's own test)."""
        xr, g_, u_, d_ = x[rows].double(), wg[cols].double(), wu[cols].double(), dh[rows][:, cols].double()
        g, u = xr @ g_.T, xr @ u_.T
        eg, eu = ((dim + 16) * U32 * (xr.abs() @ w.abs().T) for w in (g_, u_))
        a, da = ffn.activation(g, "silu")
        ea, eda = 1.13 * eg + 100 * U32 * g.abs(), 0.8 * eg + 200 * U32
        a_, b_ = d_ * u * da, d_ * a
        return (a_, d_.abs() * (u.abs() * eda + eu * (da.abs() + eda)) + (store + 4 * U32) * a_.abs() * 1.01,
                b_, d_.abs() * ea + (store + 4 * U32) * b_.abs() * 1.01)

    rows = torch.tensor([0, 1, n // 2, n - 2, n - 1], device="cuda")
    every = slice(None)
    a, ea, b, eb = parts(rows, every)
    w = a @ wg.double() + b @ wu.double()
    add = (2 * hidden + 64) * U32
    e = (ea + add * a.abs()) @ wg.double().abs() + (eb + add * b.abs()) @ wu.double().abs()
    within(host(dx[rows]), w.cpu().numpy(), (e * 1.01 + half * (w.abs() + e)).cpu().numpy(), "dx")
    cols = torch.tensor([0, 1, hidden // 2, hidden - 1], device="cuda")
    a, ea, b, eb = parts(every, cols)
    add = (n + 64) * U32
    for what, t, d_, e in (("dw_gate", dg, a, ea), ("dw_up", du, b, eb)):
        w, e = d_.T @ x.double(), (e + add * d_.abs()).T @ x.double().abs()
        within(host(t[cols]), w.cpu().numpy(), (e * 1.01 + half * (w.abs() + e)).cpu().numpy(), what)


def test_attention_gradient_of_one_query_behind_many_keys():
    """1024 heads share four million keys, and a window leaves the query the last three of them."""
    n, heads, window = 1 << 22, 1024, 3
    q, dout = (torch.randn(1, heads, 1, device="cuda") for _ in range(2))
    k, v = (torch.randn(n, 1, 1, device="cuda") for _ in range(2))
    out, lse = nsa.attention(q, k, v, window=window)
    dq, dk, dv = nsa.attention_grad(dout, q, k, v, out, lse, window=window)
    assert not dk[:-window].any() and not dv[:-window].any()
    for g, (w, b) in zip((dq, dk[-window:], dv[-window:]),
                         ref.backward(dout, q, k[-window:], v[-window:], out, lse, [0, 1], [0, window], True, window, 1.0, F32)):
        within(host(g), w.cpu().numpy(), b.cpu().numpy(), "gradient")
