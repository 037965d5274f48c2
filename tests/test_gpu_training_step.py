"""The operators together, as one training step of a small model uses them:
embedding, query/key projections with norm and rotation, causal attention,
output projection, tied-width head, distillation loss; then the gradients back
through the same operators, clipping, Muon on the projections, AdamW on gains
and head, AdamW on the embedding's row gradient.

The gradients are checked against float64 autograd of the same model, the
updates against the same optimizer calls on the dense gradient."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa

pytestmark = pytest.mark.gpu

VOCAB, DIM, HEADS, KV, HD, N = 997, 320, 4, 2, 80, 160


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


def make():
    g = torch.Generator().manual_seed(3)
    r = lambda *s, std=1.0: torch.randn(*s, generator=g, dtype=torch.float64) * std  # noqa: E731
    p = dict(table=r(VOCAB, DIM, std=0.5), qkv=r((HEADS + 2 * KV) * HD, DIM, std=DIM ** -0.5), o=r(DIM, HEADS * HD, std=0.06),
             qw=r(HD, std=0.1), kw=r(HD, std=0.1), head=r(VOCAB, DIM, std=0.1))
    data = dict(tok=torch.randint(0, VOCAB // 4, (N,), generator=g), pos=torch.arange(N) % 80,
                idx=torch.stack([torch.randperm(VOCAB, generator=g)[:8] for _ in range(N)]),
                teacher=r(N, 8, std=2.0).float(), lab=torch.randint(0, VOCAB, (N,), generator=g),
                w=(torch.rand(N, generator=g) > 0.2).float())
    data["tok"][-5:] = -1
    data["w"][-5:] = 0
    return {k: v.float() for k, v in p.items()}, data


def attention(q, k, v):
    """Causal attention over (tokens, heads, dim), keys shared by heads."""
    k, v = (t.repeat_interleave(HEADS // KV, 1) for t in (k, v))
    s = torch.stack([q[:, h] @ k[:, h].T for h in range(HEADS)]) * HD ** -0.5
    s = s.masked_fill(torch.ones(N, N, dtype=torch.bool, device=q.device).triu(1), float("-inf")).softmax(-1)
    return torch.stack([s[h] @ v[:, h] for h in range(HEADS)], 1).flatten(1)


def reference(params, d, rope):
    """float64 losses and gradients by autograd, on the host."""
    p = {k: v.double().requires_grad_() for k, v in params.items()}
    x = torch.where((d["tok"] >= 0)[:, None], p["table"][d["tok"].clamp(min=0)] * DIM ** 0.5, 0.0)
    qkv = (x @ p["qkv"].T).view(N, HEADS + 2 * KV, HD)
    cos, sin = rope.double()[d["pos"]][:, None].chunk(2, -1)

    def norm(t, w):
        t = t / (t.square().mean(-1, keepdim=True) + float(np.float32(1e-6))).sqrt() * (1.0 + w)
        a, b = t.chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

    q, k = norm(qkv[:, :HEADS], p["qw"]), norm(qkv[:, HEADS:HEADS + KV], p["kw"])
    h = x + attention(q, k, qkv[:, HEADS + KV:]) @ p["o"].T
    z = h @ p["head"].T
    y = d["teacher"].double() / 2.0
    kd = 4.0 * (y.softmax(1) * (y.log_softmax(1) - (z / 2.0).log_softmax(1).gather(1, d["idx"]))).sum(1)
    ce = -z.log_softmax(1).gather(1, d["lab"][:, None])[:, 0]
    losses = d["w"].double() * (kd + 0.5 * ce)
    (losses.sum() / N).backward()
    return losses.detach(), {k: v.grad for k, v in p.items()}


def gradients(p, d, rope):
    """The same through the operators; plain torch for the products between."""
    x = nsa.embedding(p["table"], d["tok"], scale=DIM ** 0.5)
    qkv = (x @ p["qkv"].T).view(N, HEADS + 2 * KV, HD)
    q0, k0, v0 = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], qkv[:, HEADS + KV:]
    q, k = nsa.qk_norm_rope(q0, k0, p["qw"], p["kw"], d["pos"], rope, weight_offset=1.0)
    leaves = [t.detach().requires_grad_() for t in (q, k, v0)]
    att = attention(*leaves)
    h = x + att.detach() @ p["o"].T
    z = h @ p["head"].T
    losses, dz = nsa.distill_loss(z, d["idx"], d["teacher"], d["lab"], temperature=2.0, ce_weight=0.5, row_weight=d["w"],
                                  grad_scale=1.0 / N, dlogits=z)   # over the logits
    g = {"head": dz.T @ h}
    dh = dz @ p["head"]
    g["o"] = dh.T @ att.detach()
    dq, dk, dv = torch.autograd.grad(att, leaves, dh @ p["o"])
    dqkv = torch.empty_like(qkv)
    dqkv[:, HEADS + KV:] = dv
    _, _, g["qw"], g["kw"] = nsa.qk_norm_rope_grad(dq, dk, q0, k0, p["qw"], p["kw"], d["pos"], rope, weight_offset=1.0,
                                                   dq=dqkv[:, :HEADS], dk=dqkv[:, HEADS:HEADS + KV])
    dqkv = dqkv.flatten(1)
    g["qkv"] = dqkv.T @ x
    dx = dh + dqkv @ p["qkv"]
    plan = nsa.embedding_plan(d["tok"], VOCAB)
    rows = nsa.embedding_grad(plan, dx, scale=DIM ** 0.5, form="rows")
    g["table"] = nsa.embedding_grad(plan, dx, scale=DIM ** 0.5)
    return losses, g, plan, rows


def test_training_step():
    params, data = make()
    rope = nsa.rope_table(80, HD, 10000.0, device="cpu")
    want_losses, want = reference(params, data, rope)
    p = {k: v.cuda() for k, v in params.items()}
    d = {k: v.cuda() for k, v in data.items()}
    losses, g, plan, rows = gradients(p, d, rope.cuda())
    # fp32 products over 320 .. 997 terms, a dozen operations deep: each is off
    # by at most sqrt(997) 2^-24 of its norm for roundings of random sign, and
    # softmax and norm pass a relative error on at most a few times
    tol = 12 * 4 * 997 ** 0.5 * 2.0 ** -24
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(losses, want_losses) <= tol
    for k in want:
        assert rel(g[k], want[k]) <= tol, k
    used = plan.rows >= 0
    assert torch.equal(rows[used], g["table"][plan.rows[used].long()]) and not rows[~used].any()

    # the norm that clipping sees does not depend on the gradient's form
    dense = {k: v.clone() for k, v in g.items()}
    names = [k for k in g if k != "table"]
    total = nsa.clip_grad_norm_([g[k] for k in names] + [rows], 0.05)
    total_dense = nsa.clip_grad_norm_([dense[k] for k in names] + [dense["table"]], 0.05)
    assert abs(float(total / total_dense) - 1) <= 1e-5 and float(total) > 0.05
    assert abs(float(total) / float(torch.cat([w.flatten() for w in want.values()]).norm()) - 1) <= 1e-4

    # the updates: row gradient against dense gradient, scaled alike
    coef = 0.05 / (float(total) + 1e-6)
    torch.testing.assert_close(rows[used], coef * want["table"].cuda()[plan.rows[used].long()].float(), rtol=1e-3, atol=1e-7)
    scattered = torch.zeros_like(p["table"])
    scattered[plan.rows[used].long()] = rows[used]
    state = [torch.zeros_like(p["table"]) for _ in range(4)]
    table_dense, before_table = p["table"].clone(), p["table"].clone()
    nsa.adamw_rows_step_(p["table"], rows, plan.row_index, state[0], state[1], 1)
    nsa.adamw_step_([table_dense], [scattered], [state[2]], [state[3]], 1)
    assert torch.equal(p["table"], table_dense) and torch.equal(state[0], state[2]) and torch.equal(state[1], state[3])
    before = {k: p[k].clone() for k in names}
    mats = ["qkv", "o"]
    nsa.muon_step([p[k] for k in mats], [g[k] for k in mats], [torch.zeros_like(p[k]) for k in mats], lr=0.02)
    rest = [k for k in names if k not in mats]
    table = before_table.clone()
    nsa.AdamWStep([p[k] for k in rest] + [table], [g[k] for k in rest] + [(rows, plan.row_index)])()
    assert torch.equal(table, p["table"])   # the optimizer's own way to the row step
    for k in names:
        assert torch.isfinite(p[k]).all() and not torch.equal(p[k], before[k])
