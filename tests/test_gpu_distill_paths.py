"""Distillation loss of batches, on every kernel variant that the size of a row,
the type and the temperature choose, against the float64 reference."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa

from ops_util import DT, U32, dev, half_step, host
from test_gpu_distill import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()
    yield
    torch.cuda.empty_cache()


# bytes of a row, on both sides of where another variant begins
ROWS = [3200, 4096, 4104, 12288, 12296, 35984, 36016, 65536, 65544, 200008]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("temperature,ce", [(0.7, 0.5), (2.0, 0.5), (4.0, 0.25), (1.0, 0.5), (3.0, 0.0)])
@pytest.mark.parametrize("row_bytes", ROWS)
def test_batches(row_bytes, temperature, ce, dtype):
    vocab = row_bytes // (4 if dtype == "f32" else 2)
    n = 129 if row_bytes > 40000 else 200
    z, idx, y, lab, w = make(n, vocab, 7, DT[dtype], row_bytes)
    t = float(np.float32(temperature))
    losses, dz = check(z, idx, y, lab, w, t, 1.0, ce, 0.25)
    # over the logits: the same bits
    args = dict(temperature=t, ce_weight=ce, row_weight=dev(w, torch.float32), grad_scale=0.25)
    got = nsa.distill_loss(z, dev(idx, torch.int64), dev(y, torch.float32), dev(lab, torch.int64), dlogits=z, **args)
    assert got[1] is z and torch.equal(got[0], losses) and torch.equal(z, dz)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("row_bytes", [2000, 12288, 65544])
def test_batches_with_many_teacher_entries(row_bytes, dtype):
    """From 256 entries on, a short row takes 256 threads."""
    for k in (255, 256, 400):
        z, idx, y, lab, w = make(140, row_bytes // (4 if dtype == "f32" else 2), k, DT[dtype], k)
        check(z, idx, y, lab, w, 2.0, 1.0, 0.5, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", [(5, 1003), (5, 30001), (5, 70003), (150, 1003), (150, 9001), (150, 40003)])
@pytest.mark.parametrize("pitch,shift", [(5, 0), (0, 1), (8, 3)])
def test_bits_do_not_depend_on_strides_and_addresses(n, vocab, pitch, shift, dtype):
    """The order of a sum follows the shape of the call, never where its rows lie."""
    z, idx, y, lab, w = make(n, vocab, 9, DT[dtype], vocab)
    args = dev(idx, torch.int64), dev(y, torch.float32), dev(lab, torch.int64)
    kw = dict(temperature=2.0, ce_weight=0.5, row_weight=dev(w, torch.float32))
    want = nsa.distill_loss(z, *args, **kw)
    pitch += vocab
    buf = torch.full((n * pitch + shift,), 9.0, dtype=DT[dtype], device="cuda")
    rows = buf[shift:].view(n, pitch)[:, :vocab]
    rows.copy_(z)
    apart = nsa.distill_loss(rows, *args, **kw)
    got = nsa.distill_loss(rows, *args, dlogits=rows, **kw)
    assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(apart, want, got))
    assert buf[:shift].eq(9.0).all() and buf[shift:].view(n, pitch)[:, vocab:].eq(9.0).all()


@pytest.mark.parametrize("dtype,n,vocab", [("bf16", 1300, 70000), ("f32", 700, 70000), ("bf16", 6000, 16000), ("f32", 6000, 8000),
                                           ("bf16", 30000, 3000), ("f32", 9000, 4001)])
@pytest.mark.parametrize("temperature", [2.0, 0.7])
def test_batches_beyond_the_memory_side_cache(dtype, n, vocab, temperature):
    """The streaming variants, in place, with labels and masked rows; the
    reference in float64 on the device."""
    g = torch.Generator("cuda").manual_seed(n)
    z = (torch.randn(n, vocab, generator=g, device="cuda") * 2).to(DT[dtype])
    assert z.nbytes * 2 > 256e6 and not z.isinf().any()
    idx = torch.randint(0, vocab, (n, 12), generator=g, device="cuda")      # the same element twice now and then
    idx[::7] = -1
    idx[1::5, 3:] = vocab
    y = torch.randn(n, 12, generator=g, device="cuda") * 2
    lab = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    lab[::3] = -1
    w = (torch.rand(n, generator=g, device="cuda") > 0.2).float() * 1.25
    t = float(np.float32(temperature))
    kept = z.clone()
    losses, dz = nsa.distill_loss(z, idx, y, lab, temperature=t, ce_weight=0.5, row_weight=w, grad_scale=0.5, dlogits=z)
    step = max(1, (1 << 26) // vocab)
    for r in range(0, n, step):
        s = slice(r, r + step)
        zz, yy = kept[s].double(), torch.where((idx[s] >= 0) & (idx[s] < vocab), y[s].double(), -torch.inf) / t
        has_kd, has_ce = torch.isfinite(yy).any(1), lab[s] >= 0
        yy[~has_kd] = 0.0
        q, logq = yy.softmax(1), yy.log_softmax(1)
        logp, log1 = (zz / t).log_softmax(1), zz.log_softmax(1)
        at, label = idx[s].clamp(0, vocab - 1), lab[s].clamp(min=0)[:, None]
        kd = t * t * torch.where(q > 0, q * (logq - logp.gather(1, at)), 0.0).sum(1)
        kd, ce = torch.where(has_kd, kd, 0.0), torch.where(has_ce, -log1.gather(1, label)[:, 0], 0.0)
        ws = w[s].double()
        want = ws * (kd + 0.5 * ce)
        # a sum of positive terms: vocab / 64 + 24 additions to a thread at most, five
        # units each (a rescaling among them); an exponential is 8 spread + 8 units off
        delta = (8.0 * 22.0 / min(t, 1.0) + 5.0 * (vocab / 64 + 24)) * U32
        dq = (8.0 * 16.0 / t + 16.0) * U32
        far = 22.0 / t + np.log(vocab) + 16.0 / t + np.log(12)
        bound = ws * (t * t * (delta + 2 * dq * far) + 0.5 * delta) + 4 * U32 * want.abs()
        assert bool(((losses[s].double() - want).abs() <= bound).all())
        p, p1 = logp.exp_(), log1.exp_()
        grad = t * p * has_kd[:, None] + 0.5 * p1 * has_ce[:, None]
        size = grad.clone()
        grad.scatter_add_(1, at, -t * q * has_kd[:, None])
        grad.scatter_add_(1, label, -0.5 * has_ce[:, None].double())
        scale = (0.5 * ws)[:, None]
        fp32 = scale * (size * (2 * delta + 16 * U32) + torch.zeros_like(size).scatter_add_(
            1, at, t * q * has_kd[:, None] * (dq + 4 * U32)).scatter_add_(1, label, 4 * U32 * 0.5 * has_ce[:, None].double()))
        grad *= scale
        err = (dz[s].double() - grad).abs()
        assert bool((err <= fp32 + half_step(DT[dtype]) * (grad.abs() + fp32) + 1e-40).all())
