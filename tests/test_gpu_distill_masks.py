"""Distillation loss of rows that hold finite masks or lie far from zero,
against the float64 reference: on every path that a row can take (one wave, 256,
512 and 1024 threads, slices over several blocks)."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa
from oracle import ops

from ops_util import DT, U32, dev, host, within
from test_gpu_distill import bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


MASKS = [-1e5, -1e9, -1e10, -1e12, -1e20, -1e25, -1e30, "lowest"]
PATTERNS = ["first vector", "leading third", "every other 512", "all but the named", "all"]
# (rows, vocabulary): which path, fp32 / bf16
SHAPES = [(40, 3001), (40, 20011), (40, 70001), (160, 900), (160, 2900), (160, 12001), (160, 40009)]


def near(z, temperature):
    """z less its rows' largest, with the elements that have probability 0 in any
    precision at -inf: e^-800 is below every float64."""
    d = z - z.max(1, keepdims=True)
    return np.where(d < -800.0 * max(temperature, 1.0), -np.inf, d)


def check(z, idx, y, lab, w, temperature, kd, ce, in_place=False, extra=0.0):
    """`extra`: a relative share of the loss, for rows that name masked elements."""
    zh = host(z)
    want, wantg = ops.distill_loss(zh, idx, y, lab, temperature, kd, ce, w, 0.5)
    args = dict(temperature=temperature, kd_weight=kd, ce_weight=ce, grad_scale=0.5,
                row_weight=None if w is None else dev(w, torch.float32))
    tensors = dev(idx, torch.int64), dev(y, torch.float32), dev(lab, torch.int64)
    alone, _ = nsa.distill_loss(z, *tensors, grad=False, **args)
    kept = z.clone()
    losses, dz = nsa.distill_loss(z, *tensors, dlogits=z if in_place else None, **args)
    assert torch.equal(alone, losses)
    assert in_place or torch.equal(z, kept)
    lb, gb = bounds(near(zh, temperature), y, want, wantg, z.dtype, temperature, kd, ce, w, 0.5)
    within(host(losses), want, lb + extra * np.abs(want), "losses")
    within(host(dz), wantg, gb, "dlogits")


def masked(n, vocab, dtype, seed):
    """Row r: mask r % 8 in pattern r // 8 % 5."""
    rng = np.random.default_rng(seed)
    z = rng.standard_normal((n, vocab)) * 3
    idx = np.stack([rng.choice(vocab, 6, replace=False) for _ in range(n)])
    y = (rng.standard_normal((n, 6)) * 2).astype(np.float32)
    lab = rng.integers(0, vocab, n)
    for r in range(n):
        mask = MASKS[r % len(MASKS)]
        mask = torch.finfo(dtype).min if mask == "lowest" else mask
        pattern = PATTERNS[r // len(MASKS) % len(PATTERNS)]
        open_ = np.append(idx[r], lab[r])
        kept = z[r, open_].copy()
        if pattern == "first vector":
            z[r, :8] = mask
        elif pattern == "leading third":
            z[r, :vocab // 3] = mask
        elif pattern == "every other 512":
            z[r, (np.arange(vocab) // 512) % 2 == 0] = mask
        else:
            z[r] = mask
        if pattern != "all":
            z[r, open_] = kept
    return dev(z, dtype), idx, y, lab


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("temperature,ce", [(1.0, 0.5), (2.0, 0.5), (4.0, 0.5), (0.7, 0.5), (3.0, 0.0)])
@pytest.mark.parametrize("n,vocab", SHAPES)
def test_finite_masks(dtype, temperature, ce, n, vocab):
    z, idx, y, lab = masked(n, vocab, DT[dtype], vocab)
    check(z, idx, y, lab, None, float(np.float32(temperature)), 1.0, ce)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", SHAPES)
def test_finite_masks_labels_alone_in_place(dtype, n, vocab):
    z, idx, y, lab = masked(n, vocab, DT[dtype], vocab + 1)
    check(z, idx, y, lab, None, 1.0, 0.0, 1.0, in_place=True)
    z, idx, y, lab = masked(n, vocab, DT[dtype], vocab + 2)
    check(z, idx, y, lab, None, 2.0, 1.0, 0.25, in_place=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", SHAPES)
def test_named_elements_that_are_masked(dtype, n, vocab):
    """The loss is then of the mask's size; q's relative error (16 + 8 spread
    units, counted twice) goes into it as a whole."""
    rng = np.random.default_rng(vocab)
    z = rng.standard_normal((n, vocab)) * 3
    idx = np.tile(np.array([5, vocab // 2, vocab - 1]), (n, 1))
    y = rng.standard_normal((n, 3)).astype(np.float32)
    lab = np.full(n, 5)
    for r in range(n):
        z[r, :vocab // 3] = [-1e5, -1e10, -1e20, -1e30][r % 4]
        z[r, vocab // 3] = 4.0
    check(dev(z, DT[dtype]), idx, y, lab, None, 2.0, 1.0, 0.5, extra=2 * (16 + 8 * 8) * U32)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("top", [1e7, -1e7, 1e10, -1e10, 1e20, 1e30, -1e30, 3e38])
def test_far_tops(dtype, top):
    """A few equal elements far above all others share the row."""
    for n, vocab in SHAPES:
        rng = np.random.default_rng(vocab)
        z = rng.standard_normal((n, vocab)) * 3 + min(top, 0.0) * 1.125
        at = np.array([1, vocab // 2, vocab - 2])
        z[:, at] = top
        idx = np.tile(at[:2], (n, 1))
        y = rng.standard_normal((n, 2)).astype(np.float32)
        w = np.where(np.arange(n) % 5 == 3, 0.0, 1.5).astype(np.float32)
        for temperature in (1.0, 2.0, 0.7):
            check(dev(z, DT[dtype]), idx, y, np.full(n, vocab - 2), w, float(np.float32(temperature)), 1.0, 0.5)


@pytest.mark.parametrize("temperature", [1.0, 2.0, 4.0, 0.7])
@pytest.mark.parametrize("n,vocab", SHAPES)
def test_rows_on_both_sides_of_the_exponent_limit(temperature, n, vocab):
    """fp32 logits around +- 2^22 T / log2(e) that differ by little: parts of a
    row lie on either side of what the fused exponent takes, and all count."""
    temperature = float(np.float32(temperature))
    rng = np.random.default_rng(vocab)
    for base in (1.0, -1.0):
        for wide in {temperature, 1.0}:
            z = np.round((rng.standard_normal((n, vocab)) * 2) * 4) / 4 + np.round(base * 2 ** 22 / 1.4426950408889634 * wide)
            z[:, vocab // 2:] -= 3.0                   # the second half: other slices, mostly other threads
            z[::2, :vocab // 2] -= 6.0
            idx = np.stack([rng.choice(vocab, 6, replace=False) for _ in range(n)])
            y = (rng.standard_normal((n, 6)) * 2).astype(np.float32)
            check(dev(z, torch.float32), idx, y, rng.integers(0, vocab, n), None, temperature, 1.0, 0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab", SHAPES)
def test_smallest_temperature_with_large_logits(dtype, n, vocab):
    rng = np.random.default_rng(vocab)
    z = rng.standard_normal((n, vocab)) * 40
    z[:, 7] = 2000.0
    z[::3, 7] = 30000.0
    z[1::3] -= 5000.0
    idx = np.tile(np.array([7, vocab - 3]), (n, 1))
    y = np.tile(np.array([0.0, -np.inf], np.float32), (n, 1))
    check(dev(z, DT[dtype]), idx, y, np.full(n, 3), None, float(np.float32(1e-6)), 1e6, 0.0)
