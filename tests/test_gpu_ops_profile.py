"""Kernel timing of the operators: every family is recorded while timing is on,
and a call that a graph records is not (its events would carry no times)."""
import pytest
import torch

import newton_schulz_08_amd as nsa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


def test_families_and_capture():
    tok = torch.arange(50, device="cuda") % 7
    table, m, v = torch.randn(9, 64, device="cuda"), torch.zeros(9, 64, device="cuda"), torch.zeros(9, 64, device="cuda")
    dout, z = torch.randn(50, 64, device="cuda"), torch.randn(50, 200, device="cuda")
    idx, y = torch.randint(0, 200, (50, 4), device="cuda"), torch.randn(50, 4, device="cuda")
    q, k, w = torch.randn(50, 4, 64, device="cuda"), torch.randn(50, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    rope, pos = nsa.rope_table(60, 64), torch.arange(50, device="cuda")

    def calls():
        nsa.embedding(table, tok)
        plan = nsa.embedding_plan(tok, 9)
        nsa.adamw_rows_step_(table, nsa.embedding_grad(plan, dout, form="rows"), plan.row_index, m, v, 1)
        nsa.distill_loss(z, idx, y)
        nsa.qk_norm_rope(q, k, w, w, pos, rope)
        nsa.qk_norm_rope_grad(q, k, q, k, w, w, pos, rope)

    calls()
    torch.cuda.synchronize()
    nsa.profile_read()
    nsa.profile_enable(True)
    try:
        calls()
        stats = nsa.profile_read()
        assert set(stats) == {"embedding", "embedding_plan", "embedding_grad", "adamw_rows", "distill_loss", "qk_norm_rope",
                              "qk_norm_rope_grad"}
        assert all(s["launches"] == 1 and s["total_ms"] > 0 and s["bytes"] > 0 for s in stats.values())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        assert nsa.profile_read() == {}
        g.replay()
        torch.cuda.synchronize()
    finally:
        nsa.profile_enable(False)
