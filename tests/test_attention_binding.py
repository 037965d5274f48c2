"""Numbers that a C int cannot hold are refused by attention's binding, not wrapped."""
import pytest
import torch

import newton_schulz_08_amd as nsa
from newton_schulz_08_amd import _lib

from test_block_abi import AT, ATG, at_shape
from test_ops_abi import BAD, accepted, refused

WRAPS = 1 << 32   # 0 in an int: no window at all


def test_workspace_queries():
    assert nsa.attention_workspace_bytes(8, 65536, 32, 8, 128, 8) > 0
    for args in ((8, 65536, WRAPS + 32, 8, 128, 8), (8, 65536, 32, WRAPS + 8, 128, 8), (8, 65536, 32, 8, WRAPS + 128, 8)):
        with pytest.raises(ValueError, match="too large"):
            nsa.attention_workspace_bytes(*args)
    with pytest.raises(ValueError, match="too large"):
        nsa.attention_grad_workspace_bytes(8, WRAPS + 32)
    for args in ((8, WRAPS + 4, 2, 64), (8, 4, WRAPS + 2, 64), (8, 4, 2, 64 - WRAPS)):
        with pytest.raises(ValueError, match="too large"):
            nsa.qk_norm_rope_grad_workspace_bytes(*args)


@pytest.mark.gpu
def test_windows():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    q, k, v = (torch.randn(300, 4, 64, device="cuda") for _ in range(3))
    out, lse = nsa.attention(q, k, v)
    assert torch.equal(nsa.attention(q, k, v, window=1 << 30)[0], out)
    for window in (WRAPS, WRAPS + 5, 5 - WRAPS):
        with pytest.raises(ValueError, match="window"):
            nsa.attention(q, k, v, window=window)
        with pytest.raises(ValueError, match="window"):
            nsa.attention_grad(q, q, k, v, out, lse, window=window)
    with pytest.raises(nsa.DmuonError, match="window"):
        nsa.attention(q, k, v, window=(1 << 30) + 1)


def test_scales_that_overflow_in_base_2():
    """Exponentials are base 2: a scale that is infinite times log2(e) would make a score of 0 a NaN."""
    lib, largest = _lib.load(), 3.4028234e38 / 1.4426952
    for f, good in ((lib.dmuon_attention_forward, AT), (lib.dmuon_attention_backward, ATG)):
        good = dict(good, shape=at_shape(k_tokens=6))
        refused(f, good, [(dict(shape=at_shape(k_tokens=6, scale=s)), BAD) for s in (largest * 1.0001, 3.4e38)])
        accepted(f, dict(good, shape=at_shape(k_tokens=6, scale=largest * 0.9999)))


@pytest.mark.gpu
def test_heads_of_no_elements_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    two, one, lse = torch.empty(5, 2, 0, device="cuda"), torch.empty(5, 1, 0, device="cuda"), torch.zeros(1, 5, device="cuda")
    with pytest.raises(ValueError, match="next to each other"):   # torch takes a step of 1 between heads of nothing
        nsa.attention(two, two, two)
    with pytest.raises(nsa.DmuonError, match="head_dim"):
        nsa.attention(one, one, one)
    with pytest.raises(nsa.DmuonError, match="head_dim"):
        nsa.attention_grad(one, one, one, one, one, lse)
