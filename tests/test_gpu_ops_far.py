"""The operators where an element's offset passes 2^31 (and its bytes 2^32)."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa
from oracle import ops

from ops_util import U32, half_step, host, within

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()
    yield
    torch.cuda.empty_cache()


def test_embedding_and_adamw_of_a_large_table():
    vocab, dim = 530000, 4100
    assert vocab * dim > 2 ** 31
    torch.manual_seed(1)
    table = torch.randn(vocab, dim, device="cuda", dtype=BF16)
    tok = torch.tensor([0, vocab - 1, 523777, 262144, vocab - 1, vocab], device="cuda")
    out = nsa.embedding(table, tok)
    assert torch.equal(out[:5], table[tok[:5]]) and not out[5].any()
    dout = torch.randn(6, dim, device="cuda", dtype=BF16)
    plan = nsa.embedding_plan(tok, vocab)
    dense = nsa.embedding_grad(plan, dout)
    rows = nsa.embedding_grad(plan, dout, form="rows")
    assert torch.equal(dense[plan.rows[:4].long()], rows[:4]) and int((dense != 0).any(1).sum()) == 4
    want = host(dout[1]) + host(dout[4])
    within(host(rows[3]), want, (U32 + half_step(BF16)) * 1.01 * np.abs(want) + U32 * (np.abs(host(dout[1])) + np.abs(host(dout[4]))),
           "last row")
    a, b = [table, torch.zeros(vocab, dim, device="cuda"), torch.zeros(vocab, dim, device="cuda")], None
    b = [t.clone() for t in a]
    nsa.adamw_rows_step_(a[0], rows, plan.row_index, a[1], a[2], 1)
    nsa.adamw_step_([b[0]], [dense], [b[1]], [b[2]], 1)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_embedding_gradient_of_a_large_batch():
    n, dim, vocab = 530000, 4100, 7
    assert n * dim > 2 ** 31
    dout = torch.zeros(n, dim, device="cuda", dtype=BF16)
    tok = torch.randint(0, vocab - 1, (n,), device="cuda")
    tok[-3:] = vocab - 1
    dout[-3:] = torch.randn(3, dim, device="cuda")
    got = nsa.embedding_grad(nsa.embedding_plan(tok, vocab), dout, dtype=torch.float32)
    want, size = host(dout[-3:]).sum(0), np.abs(host(dout[-3:])).sum(0)
    assert not got[:-1].any()
    within(host(got[-1]), want, 4 * U32 * size, "last token")


def test_distill_of_many_logits():
    n, vocab = 17000, 128256
    assert n * vocab > 2 ** 31
    torch.manual_seed(2)
    z = torch.randn(n, vocab, device="cuda", dtype=BF16)
    idx = torch.randint(0, vocab, (n, 4), device="cuda")
    y = torch.randn(n, 4, device="cuda")
    losses, dz = nsa.distill_loss(z, idx, y)
    tail = slice(n - 2, n)
    alone, dz2 = nsa.distill_loss(z[tail].clone(), idx[tail].contiguous(), y[tail].contiguous())
    want, wantg = ops.distill_loss(host(z[tail]), host(idx[tail]), host(y[tail]))
    # 128256 exponentials summed in fp32, 500 additions to a thread: 1e-4 is
    # 3 times 550 fp32 units of a sum of positive terms
    for got, grad in ((losses[tail], dz[tail]), (alone, dz2)):
        within(host(got), want, 1e-4 * np.abs(want), "losses")
        within(host(grad), wantg, (half_step(BF16) + 1e-4) * np.abs(wantg) + 1e-7, "dlogits")


def test_qk_of_many_tokens():
    n, qh, kh, d = 220000, 48, 16, 128
    packed = torch.empty(n, (qh + 2 * kh) * d, device="cuda", dtype=BF16).normal_()
    assert packed.numel() > 2 ** 31
    q, k = packed[:, :qh * d].unflatten(1, (qh, d)), packed[:, qh * d:(qh + kh) * d].unflatten(1, (kh, d))
    w = torch.ones(d, device="cuda")
    rope = nsa.rope_table(64, d)
    pos = torch.arange(n, device="cuda") % 64
    tail = slice(n - 3, n)
    small = [t[tail].contiguous() for t in (q, k)]
    want = nsa.qk_norm_rope(*small, w, w, pos[tail].contiguous(), rope)
    wantg = nsa.qk_norm_rope_grad(*small, *small, w, w, pos[tail].contiguous(), rope)
    g = nsa.qk_norm_rope_grad(q, k, q, k, w, w, pos, rope)
    assert torch.equal(g[0][tail], wantg[0]) and torch.equal(g[1][tail], wantg[1])
    del g
    nsa.qk_norm_rope(q, k, w, w, pos, rope, q_out=q, k_out=k)
    assert torch.equal(q[tail], want[0]) and torch.equal(k[tail], want[1])
