"""Embedding lookup, plan and gradient at their largest and beyond the
memory-side cache."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa
from oracle import ops

from ops_util import DT, U32, dev, half_step, host
from test_gpu_embedding import draw_tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind,n,vocab", [("zipf", 524288, 128256), ("mixed", 524289, 50000), ("zipf", 1000003, 1 << 24),
                                          ("one", 700001, 9), ("zipf", 4194304, 200000), ("mixed", 5000, 1 << 24),
                                          ("mixed", 300, 1 << 24)])
def test_plan_up_to_the_limits(kind, n, vocab):
    tok = draw_tokens(kind, n, vocab, n)
    plan = nsa.embedding_plan(dev(tok, torch.int64), vocab)
    for name, want in zip(("order", "slot", "rows", "row_index", "count"), ops.embedding_plan(tok, vocab)):
        assert np.array_equal(host(getattr(plan, name)), np.reshape(want, -1)), name


@pytest.mark.parametrize("tdt", ["f32", "bf16"])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [4096, 4099])
def test_lookup_of_a_large_batch(tdt, odt, dim):
    n = 34000 if odt == "bf16" else 17000
    g = torch.Generator("cuda").manual_seed(dim)
    table = torch.randn(5000, dim, generator=g, device="cuda").to(DT[tdt])
    tok = torch.randint(-200, 5200, (n,), generator=g, device="cuda")
    out = nsa.embedding(table, tok, scale=0.5, out_dtype=DT[odt])
    assert out.nbytes > 256e6
    known = (tok >= 0) & (tok < 5000)
    want = torch.where(known[:, None], table[tok.clamp(0, 4999)].float() * 0.5, 0.0).to(DT[odt])   # a half is exact
    assert torch.equal(out, want)


@pytest.mark.parametrize("ddt,gdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("form", ["dense", "add", "rows"])
@pytest.mark.parametrize("dim", [4096, 4090])
def test_gradient_of_a_large_batch(ddt, gdt, form, dim):
    n, vocab = (33000 if ddt == "bf16" else 17000), 6000
    tok = draw_tokens("zipf", n, vocab, dim)
    tok[::9] = -1
    t = dev(tok, torch.int64)
    g = torch.Generator("cuda").manual_seed(dim)
    dout = torch.randn(n, dim, generator=g, device="cuda").to(DT[ddt])
    assert dout.nbytes > 256e6
    plan = nsa.embedding_plan(t, vocab)
    old = torch.randn(vocab, dim, generator=g, device="cuda").to(DT[gdt])
    got = nsa.embedding_grad(plan, dout, scale=0.5, form=form, dtype=DT[gdt], out=old.clone() if form == "add" else None)
    # float64 sums on the device; a bound of (occurrences + 2) fp32 roundings of the summed magnitudes
    known = t >= 0
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, t[known], dout[known].double() * 0.5)
    size = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, t[known], dout[known].double().abs() * 0.5)
    count = torch.bincount(t[known], minlength=vocab)
    fp32 = (count[:, None] + 2) * (U32 * 1.001) * size
    if form == "add":
        want += old.double()
        fp32 += U32 * (want.abs() + fp32)
    bound = fp32 + half_step(DT[gdt]) * (want.abs() + fp32)
    if form == "add":
        bound[count == 0] = 0.0
    if form == "rows":
        used = int(plan.count)
        rows = plan.rows[:used].long()
        assert not got[used:].any() and torch.equal(rows, torch.nonzero(count)[:, 0])
        got, want, bound = got[:used], want[rows], bound[rows]
    assert bool(((got.double() - want).abs() <= bound).all())
