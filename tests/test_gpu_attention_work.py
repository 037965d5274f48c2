"""What the timing record says of attention's work: the pairs that the masks leave."""
import pytest
import torch

import newton_schulz_08_amd as nsa
from attention_util import offsets, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 16), (True, 1000)])
@pytest.mark.parametrize("sequences,lq,lk", [(1, 200, 200), (3, 70, 70), (2, 1, 900), (2, 30, 500), (1, 90, 40)])
def test_work_is_that_of_the_visible_pairs(sequences, lq, lk, causal, window):
    d, qh, kh = 24, 4, 2
    q, k, v = (torch.randn(sequences * n, h, d, device="cuda") for n, h in ((lq, qh), (lk, kh), (lk, kh)))
    (_, qo), (_, ko) = offsets([lq] * sequences), offsets([lk] * sequences)
    kw = dict(causal=causal, window=window)
    out, lse = nsa.attention(q, k, v, qo, ko, **kw)
    torch.cuda.synchronize()
    nsa.profile_read()
    nsa.profile_enable(True)
    try:
        nsa.attention(q, k, v, qo, ko, **kw)
        nsa.attention_grad(q, q, k, v, out, lse, qo, ko, **kw)
        stats = nsa.profile_read()
    finally:
        nsa.profile_enable(False)
    see = visible(lq, lk, causal, window, "cpu")
    pairs, keys = int(see.sum()) * sequences * qh, int(see.any(0).sum()) * sequences
    assert stats["attention"]["flops"] == 4 * d * pairs
    assert stats["attention_grad"]["flops"] == 10 * d * pairs
    rows, cols, seen = q.numel(), k.numel(), keys * kh * d
    assert stats["attention"]["bytes"] == 4 * 2 * (rows + seen)                  # q, out; the keys and values that are seen
    assert stats["attention_grad"]["bytes"] == 4 * (4 * rows + 2 * seen + 2 * cols)   # q, out, dout, dq; k, v; dk, dv
