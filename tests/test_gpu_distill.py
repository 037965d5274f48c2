"""Distillation loss and gradient against the float64 reference."""
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


def spread(x):
    """max - x over the finite entries of each row."""
    x = np.where(np.isfinite(x), x, np.nan)
    top = np.fmax.reduce(x, axis=1, initial=-np.inf)
    low = np.fmin.reduce(x, axis=1, initial=np.inf)
    return np.where(np.isfinite(top) & np.isfinite(low), top - low, 0.0)


def bounds(z, y, losses, dz, dtype, temperature, kd, ce, weight, scale):
    """How far the losses and gradients may be off.

    An exponential of (z - max) / T: the difference, the scaled argument (two
    products) and the function itself are each rounded, which makes the value
    4 |z - max| / T + 2 fp32 units off, relatively.  A row's sum adds at most
    vocab / 256 + 24 rounded additions and as many rescalings, each rescaling
    again an exponential whose arguments add up to the row's spread: delta.
    The loss moves by delta through the logarithm; through q by at most twice
    q's relative error times the largest |log q - log p|.  A gradient element is
    p (the exponential over the sum) less q, each with its own error, scaled
    and rounded once more."""
    n, vocab = z.shape
    steps = vocab / 256 + 24
    d1, dt_, dy = spread(z), spread(z) / temperature, spread(y) / temperature
    delta_t, delta_1 = ((8 * d + 5 * steps) * U32 for d in (dt_, d1))
    dq = (8 * dy + 16) * U32
    far = dt_ + np.log(vocab) + dy + np.log(max(y.shape[1], 2))
    w = np.ones(n) if weight is None else np.abs(weight)
    loss_b = w * (abs(kd) * temperature ** 2 * (delta_t + 2 * dq * far) + abs(ce) * delta_1) + 4 * U32 * np.abs(losses)
    rel_t, rel_1 = delta_t + (4 * dt_ + 6) * U32, delta_1 + (4 * d1 + 6) * U32
    zf = np.where(np.isfinite(z), z, -1e30)
    top = zf.max(1, keepdims=True)
    soft = lambda t: np.exp((zf - top) / t) / np.exp((zf - top) / t).sum(1, keepdims=True)  # noqa: E731
    part = abs(kd) * temperature * (soft(temperature) * rel_t[:, None] + (dq + 4 * U32)[:, None])
    part += abs(ce) * (soft(1.0) * rel_1[:, None] + 4 * U32)
    fp32 = abs(scale) * w[:, None] * part
    return loss_b, fp32 + half_step(dtype) * (np.abs(dz) + fp32) + 1e-40


def make(n, vocab, k, dtype, seed, holes=True, idx_dtype=torch.int64):
    rng = np.random.default_rng(seed)
    z = dev(rng.standard_normal((n, vocab)) * 3, dtype)
    idx = np.stack([rng.choice(vocab, k, replace=k > vocab) for _ in range(n)]) if k else np.zeros((n, 0), np.int64)
    y = (rng.standard_normal((n, k)) * 2).astype(np.float32)
    lab = rng.integers(0, vocab, n)
    w = rng.random(n).astype(np.float32) + 0.5
    if holes:
        lab[::3] = -100
        w[1::4] = 0.0
        idx[2::5] = -1                        # no teacher entry
        if k > 2:
            idx[:, 1] = idx[:, 0]             # the same element twice
            idx[3::7, 2] = vocab              # one entry less
            y[4::6, 0] = -np.inf
            lab[4::6] = idx[4::6, 0] if k else 0
    return z, idx, y, lab, w


def check(z, idx, y, lab, w, temperature, kd, ce, scale, idx_dtype=torch.int64, **kw):
    index, teacher = dev(idx, idx_dtype), dev(y, torch.float32)
    labels = None if lab is None else dev(lab, idx_dtype)
    weight = None if w is None else dev(w, torch.float32)
    zh = host(z)
    want, wantg = ops.distill_loss(zh, idx, y, lab, temperature, kd, ce, w, scale)
    if not idx.shape[1]:
        index = teacher = None
    args = dict(temperature=temperature, kd_weight=kd, ce_weight=ce, row_weight=weight, grad_scale=scale)
    alone, none = nsa.distill_loss(z, index, teacher, labels, grad=False, **args)
    losses, dz = nsa.distill_loss(z, index, teacher, labels, **args, **kw)
    assert none is None and torch.equal(alone, losses)
    lb, gb = bounds(zh, np.where(idx >= 0, y, np.nan) if idx.shape[1] else np.zeros((len(zh), 1)), want, wantg, z.dtype,
                    temperature, kd, ce, w, scale)
    within(host(losses), want, lb, "losses")
    within(host(dz), wantg, gb, "dlogits")
    return losses, dz


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("temperature,kd,ce", [(1.0, 1.0, 0.0), (2.0, 0.7, 0.4), (1.0, 0.5, 0.5), (0.7, 0.0, 1.0)])
@pytest.mark.parametrize("n,vocab,k", [(1, 1, 1), (2, 3, 3), (9, 1000, 8), (31, 4099, 33), (3, 32003, 20), (5, 50000, 200)])
def test_loss_and_gradient(dtype, temperature, kd, ce, n, vocab, k):
    temperature, kd, ce = (float(np.float32(x)) for x in (temperature, kd, ce))
    z, idx, y, lab, w = make(n, vocab, k, DT[dtype], n * 7 + k)
    check(z, idx, y, lab, w, temperature, kd, ce, 0.125)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_vocabulary_many_entries(dtype):
    z, idx, y, lab, w = make(6, 128256, 1024, DT[dtype], 3)
    check(z, idx, y, lab, w, 2.0, 1.0, 0.25, 1.0)


def test_many_rows():
    z, idx, y, lab, w = make(1500, 600, 5, torch.bfloat16, 4, idx_dtype=torch.int32)
    check(z, idx, y, lab, w, 2.0, 1.0, 0.25, 1.0, idx_dtype=torch.int32)


def test_labels_alone():
    z, idx, y, lab, w = make(7, 777, 0, torch.float32, 5)
    check(z, idx, y, lab, w, 1.0, 0.0, 1.0, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,pitch,shift", [(1000, 1008, 0), (1003, 1005, 0), (999, 1000, 1)])
def test_strided_rows_in_place_and_gaps(dtype, vocab, pitch, shift):
    z, idx, y, lab, w = make(5, vocab, 12, DT[dtype], 6)
    want = check(z, idx, y, lab, w, 2.0, 1.0, 0.5, 1.0)
    buf = torch.full((5 * pitch + shift,), 9.0, dtype=DT[dtype], device="cuda")
    rows = buf[shift:].view(5, pitch)[:, :vocab]
    rows.copy_(z)
    got = nsa.distill_loss(rows, dev(idx, torch.int64), dev(y, torch.float32), dev(lab, torch.int64), temperature=2.0,
                           ce_weight=0.5, row_weight=dev(w, torch.float32), dlogits=rows)
    within(host(got[0]), host(want[0]), 1e-5 * (1 + np.abs(host(want[0]))), "losses")   # another order of the same sum
    _, gb = bounds(host(z), np.where(idx >= 0, y, np.nan), host(want[0]), host(want[1]), DT[dtype], 2.0, 1.0, 0.5, w, 1.0)
    within(host(rows), host(want[1]), 2 * gb, "in place")
    assert buf[shift:].view(5, pitch)[:, vocab:].eq(9.0).all()


def test_masked_and_extreme_logits():
    rng = np.random.default_rng(8)
    for dtype in (torch.float32, torch.bfloat16):
        z = torch.from_numpy(rng.standard_normal((6, 9000)) * 2).to("cuda", dtype)
        z[0, 100:] = -float("inf")            # slices that hold nothing
        z[1, :8500] = torch.finfo(dtype).min  # the type's lowest value
        z[2] = 0.0
        z[2, 7] = 30000.0
        z[3] = -float("inf")                  # no distribution
        z[4, 17] = float("nan")
        z[5, 3] = float("inf")
        idx = np.tile(np.array([3, 50, 7]), (6, 1))
        y = rng.standard_normal((6, 3)).astype(np.float32)
        lab = np.full(6, 20)
        losses, dz = nsa.distill_loss(z, dev(idx, torch.int64), dev(y, torch.float32), dev(lab, torch.int64),
                                      temperature=2.0, ce_weight=0.5)
        zh = host(z)
        with np.errstate(invalid="ignore", over="ignore"):
            want, wantg = ops.distill_loss(zh[:3], idx[:3], y[:3], lab[:3], 2.0, 1.0, 0.5)
        lb, gb = bounds(np.where(zh[:3] < -1e30, -np.inf, zh[:3]), y[:3], want, wantg, dtype, 2.0, 1.0, 0.5, None, 1.0)
        # row 1: named elements of probability 0 cost the lowest value's size
        within(host(losses)[[0, 2]], want[[0, 2]], lb[[0, 2]], "losses")
        assert abs(host(losses)[1] - want[1]) <= 1e-6 * abs(want[1]) or np.isinf(host(losses)[1])
        within(host(dz)[:3], wantg, gb, "dlogits")
        assert torch.isnan(losses[3:]).all() and torch.isnan(dz[3:]).any(1).all()


@pytest.mark.parametrize("temperature", [0.01, 4.0, 100.0])
def test_far_temperatures(temperature):
    z, idx, y, lab, w = make(9, 3001, 8, torch.float32, 13)
    check(z, idx, y, lab, w, float(np.float32(temperature)), 1.0, 0.5, 1.0)


@pytest.mark.parametrize("temperature", [1e-6, 1e6])
@pytest.mark.parametrize("vocab", [500, 9000, 70000])
def test_limits_of_the_temperature_with_masked_logits(temperature, vocab):
    """At the smallest temperature all of the weight is on the largest logit, at
    the largest it is spread evenly over the elements that are not masked."""
    rng = np.random.default_rng(14)
    z = torch.from_numpy(rng.standard_normal((3, vocab)).astype(np.float32)).cuda()
    z[:, 5:vocab // 2] = -float("inf")
    z[:, 3] = 40.0
    idx = torch.tensor([[3, 4], [3, vocab - 1], [3, 0]], device="cuda")
    y = torch.tensor([[0.0, -float("inf")]] * 3, device="cuda")     # the teacher names element 3 alone
    losses, dz = nsa.distill_loss(z, idx, y, temperature=temperature, kd_weight=1.0 / temperature)
    assert torch.isfinite(losses).all() and torch.isfinite(dz).all() and not dz[:, 5:vocab // 2].any()
    kept = vocab - (vocab // 2 - 5)
    p = torch.zeros_like(z) if temperature < 1 else torch.where(torch.isinf(z), 0.0, 1.0 / kept)
    q = torch.zeros_like(z)
    q[:, 3] = 1.0
    if temperature < 1:
        p = q
    # the spread 45 / 1e6 moves a probability by that share of it
    torch.testing.assert_close(dz, p - q, rtol=2e-4, atol=1e-6)


def test_every_named_element_of_a_large_batch():
    """Beyond the memory-side cache: each named element is rewritten behind the
    sweep that wrote its neighbours."""
    n, vocab, k = 2600, 70000, 40
    torch.manual_seed(15)
    z = torch.randn(n, vocab, device="cuda", dtype=torch.bfloat16)
    idx = torch.stack([torch.randperm(vocab, device="cuda")[:k] for _ in range(n)])
    y, lab = torch.randn(n, k, device="cuda"), torch.randint(0, vocab, (n,), device="cuda")
    _, dz = nsa.distill_loss(z, idx, y, lab, temperature=1.0, ce_weight=0.5)
    p = torch.stack([z[r].double().log_softmax(0).exp() for r in range(n)])
    want = 1.5 * p
    named = torch.zeros(n, vocab, dtype=torch.bool, device="cuda")
    want.scatter_add_(1, idx, -y.double().softmax(1))
    want.scatter_add_(1, lab[:, None], torch.full((n, 1), -0.5, dtype=torch.float64, device="cuda"))
    named.scatter_(1, idx, True).scatter_(1, lab[:, None], True)
    # sums of 70000 positive terms, 140 additions to a thread: 5e-5 covers 800 fp32 units
    err, bound = (dz.double() - want).abs(), (half_step(torch.bfloat16) + 5e-5) * want.abs() + 5e-5 * 1.5 * p + 1e-7
    assert bool((err[named] <= bound[named]).all()) and bool((err <= bound).all())


def test_skipped_rows_are_not_read():
    z = torch.full((4, 5000), float("nan"), device="cuda")
    z[3] = 1.0
    idx = torch.tensor([[1, 2], [-1, -1], [-1, 7000], [1, 2]], device="cuda")
    y = torch.zeros(4, 2, device="cuda")
    lab = torch.tensor([3, -1, 5000, 2], device="cuda")
    w = torch.tensor([0.0, 1.0, 1.0, 1.0], device="cuda")
    losses, dz = nsa.distill_loss(z, idx, y, lab, ce_weight=1.0, row_weight=w)
    assert not losses[:3].any() and not dz[:3].any() and torch.isfinite(dz[3]).all() and losses[3] > 0
    assert nsa.distill_loss(z[:0], idx[:0], y[:0])[1].shape == (0, 5000)


def test_gradient_against_a_difference():
    rng = np.random.default_rng(9)
    z, idx, y, lab, w = make(8, 500, 6, torch.float32, 10)
    _, dz = nsa.distill_loss(z, dev(idx, torch.int64), dev(y, torch.float32), dev(lab, torch.int64), temperature=2.0,
                             ce_weight=0.5, row_weight=dev(w, torch.float32))
    v, h, zh = rng.standard_normal((8, 500)), 1e-5, host(z)
    f = lambda x: ops.distill_loss(x, idx, y, lab, 2.0, 1.0, 0.5, w)[0].sum()  # noqa: E731
    want = (f(zh + h * v) - f(zh - h * v)) / (2 * h)
    _, gb = bounds(zh, np.where(idx >= 0, y, np.nan), np.zeros(8), host(dz), torch.float32, 2.0, 1.0, 0.5, w, 1.0)
    assert abs(float((host(dz) * v).sum()) - want) <= float((gb * np.abs(v)).sum()) + 1e-8


def test_reproducible_on_streams_and_in_a_graph():
    z, idx, y, lab, w = make(12, 20000, 16, torch.bfloat16, 11)
    index, teacher, labels, weight = dev(idx, torch.int64), dev(y, torch.float32), dev(lab, torch.int64), dev(w, torch.float32)
    run = lambda **kw: nsa.distill_loss(z, index, teacher, labels, temperature=2.0, ce_weight=0.5, row_weight=weight, **kw)  # noqa: E731
    first = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a, b = run(stream=side), run()
    torch.cuda.synchronize()
    assert all(torch.equal(x, t) for x, t in zip(a, first)) and all(torch.equal(x, t) for x, t in zip(b, first))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for k in range(4):
        z.copy_(make(12, 20000, 16, torch.bfloat16, 20 + k)[0])
        g.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(x, t) for x, t in zip(outs, want))
