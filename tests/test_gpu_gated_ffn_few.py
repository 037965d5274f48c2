"""The gated feed-forward product of few tokens on both sides of the rule that
leaves the streaming kernel for tiles: wide weights, more than a few tokens."""
import pytest
import torch

import newton_schulz_08_amd as nsa
from test_gpu_gated_ffn import check
from test_gpu_gated_ffn_odd import fastest

F32, BF16 = torch.float32, torch.bfloat16


def test_tiles_take_copies_and_the_streaming_kernel_none():
    need = lambda n, dim, hidden: nsa.gated_ffn_workspace_bytes(n, dim, hidden, BF16, aligned=False)  # noqa: E731
    for n, dim, hidden in ((1, 4096, 14336), (32, 4096, 14336), (64, 4096, 8192), (64, 512, 28672)):
        assert need(n, dim, hidden) == 0
    for n, dim, hidden in ((64, 4096, 14336), (32, 4096, 28672), (64, 1024, 14336)):
        assert need(n, dim, hidden) > 0 and nsa.gated_ffn_workspace_bytes(n, dim, hidden, BF16) == 0
    assert nsa.gated_ffn_workspace_bytes(64, 4096, 14336, F32) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,dim,hidden,tokens", [(BF16, 1024, 16384, (33, 48, 49, 63, 64)), (BF16, 1032, 28672, (27, 28, 64)),
                                                     (F32, 320, 8191, (32, 33, 64)), (F32, 320, 8192, (32, 33, 64))])
def test_both_sides(dtype, dim, hidden, tokens):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    for n in tokens:
        check(n, dim, hidden, dtype, "gelu", seed=n, back=False)
        check(n, dim, hidden, dtype, seed=n, shift=1, pitch=3, back=False)


@pytest.mark.gpu
def test_one_token_more_costs_no_less():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    wg, wu = (torch.randn(28672, 4096, device="cuda").mul_(0.02).to(BF16) for _ in range(2))
    x = torch.randn(65, 4096, device="cuda").to(BF16)
    some, more = fastest([lambda: nsa.gated_ffn(x[:64], wg, wu), lambda: nsa.gated_ffn(x, wg, wu)])
    assert some < 1.2 * more, (some, more)
