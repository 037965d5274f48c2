"""The gated feed-forward product where only its results lie off multiples of 16
bytes: an odd hidden width, a result or a gradient that is a shifted slice.  The
operands are read as fast as ever, and no bit changes."""
import pytest
import torch

import newton_schulz_08_amd as nsa
from test_gpu_gated_ffn import check, make

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()
    yield
    torch.cuda.empty_cache()


def fastest(calls, repeats=5, n=20):
    """The least time of each call, taken in turn."""
    best = [float("inf")] * len(calls)
    for call in calls:
        call()
    for _ in range(repeats):
        for i, call in enumerate(calls):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(n):
                call()
            b.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], a.elapsed_time(b))
    return best


# two weights of 14336 x 4096 are read once, whatever becomes of the result: reading
# them element by element takes 2 to 7 times as long
@pytest.mark.parametrize("dtype,n", [(BF16, 4), (BF16, 32), (F32, 32)])
def test_results_anywhere_do_not_slow_the_reads(dtype, n):
    dim, hidden = 4096, 14336
    x, wg, wu, _ = make(n, dim, hidden + 1, dtype, 1)
    even = [w[:hidden] for w in (wg, wu)]
    wide = torch.empty(n, hidden + 9, dtype=dtype, device="cuda")
    base, odd, shifted = fastest([lambda: nsa.gated_ffn(x, *even), lambda: nsa.gated_ffn(x, wg, wu),
                                  lambda: nsa.gated_ffn(x, *even, out=wide[:, 1:hidden + 1])])
    assert odd < 1.5 * base and shifted < 1.5 * base, (base, odd, shifted)


@pytest.mark.parametrize("shift", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("n", [3, 20, 50, 130])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_shifted_results_and_gradients(dtype, n, shift):
    x, wg, wu, dh = make(n, 128, 193, dtype, n)
    want, back = nsa.gated_ffn(x, wg, wu), nsa.gated_ffn_grad(dh, x, wg, wu)

    def inside(rows, width):
        t = torch.full((rows, width + 9), 7.0, dtype=dtype, device="cuda")
        return t, t[:, shift:shift + width]

    whole, out = inside(n, 193)
    assert torch.equal(nsa.gated_ffn(x, wg, wu, out=out), want)
    assert (whole[:, :shift] == 7).all() and (whole[:, shift + 193:] == 7).all()
    (whole, dx), (_, dh2) = inside(n, 128), inside(n, 193)
    dh2.copy_(dh)
    flat = torch.full((2 * 193 * 128 + 8 + shift,), 7.0, dtype=dtype, device="cuda")
    dwg, dwu = (flat[shift + k * 193 * 128:][:193 * 128].view(193, 128) for k in range(2))
    got = nsa.gated_ffn_grad(dh2, x, wg, wu, dx=dx, dw_gate=dwg, dw_up=dwu)
    assert all(torch.equal(a, b) for a, b in zip(got, back))
    assert (whole[:, :shift] == 7).all() and (whole[:, shift + 128:] == 7).all()
    assert (flat[:shift] == 7).all() and (flat[shift + 2 * 193 * 128:] == 7).all()


@pytest.mark.parametrize("hidden", [65, 66, 67, 1001])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_odd_hidden_widths(dtype, hidden):
    for n in (2, 40, 150):
        check(n, 256, hidden, dtype, seed=hidden + n)
