"""Helpers of the operator tests: host copies, misaligned tensors, bounds."""
import numpy as np
import torch

from gpu_util import to_host_f64

U32 = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    """A rounding to `dtype` is off by at most this, relative to the value."""
    return torch.finfo(dtype).eps / 2


def dev(a, dtype, shift: int = 0) -> torch.Tensor:
    """`a` on the GPU; with `shift`, that many elements behind an aligned address."""
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)
    if shift:
        big = torch.empty(t.numel() + shift, dtype=dtype, device="cuda")
        big[shift:] = t.reshape(-1)
        t = big[shift:].view(t.shape)
    return t


def empty(shape, dtype, shift: int = 0) -> torch.Tensor:
    n = int(np.prod(shape))
    big = torch.full((n + shift,), float("nan"), dtype=dtype, device="cuda")
    return big[shift:].view(shape)


def host(t: torch.Tensor) -> np.ndarray:
    if t.dtype in (torch.int32, torch.int64):
        return t.cpu().numpy()
    return to_host_f64(t)


def within(got, want, bound, what=""):
    """|got - want| <= bound element by element (NaN only where wanted)."""
    got, want, bound = np.broadcast_arrays(got, want, bound)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what}: infinities differ"
    err = np.abs(got[fine] - want[fine])
    bad = err > bound[fine] * 1.0000001
    if bad.any():
        worst = np.argmax(err / np.maximum(bound[fine], 1e-300))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of bound; worst {err[worst]:.3e} against "
                             f"{bound[fine][worst]:.3e}")
