"""The operators together, as one training step of a two-block decoder uses them:
embedding, norms around every block, query/key norm with rotation, attention
over packed sequences, gated feed-forward, distillation loss, the gradients
back through the same operators, and the optimizer's steps on them.

The gradients are checked against float64 autograd of the same model; plain
products (projections) are torch's."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa

pytestmark = pytest.mark.gpu

VOCAB, DIM, HEADS, KV, HD, HIDDEN, LAYERS = 499, 192, 6, 2, 40, 300, 2
LENGTHS, WINDOW, SCALE = [50, 1, 77], 33, 0.75
N = sum(LENGTHS)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


def make():
    g = torch.Generator().manual_seed(5)
    r = lambda *s, std=1.0, at=0.0: torch.randn(*s, generator=g) * std + at  # noqa: E731
    p = dict(table=r(VOCAB, DIM, std=0.7), first=r(DIM, std=0.1, at=1.0), head=r(VOCAB, DIM, std=0.1))
    for i in range(LAYERS):
        p.update({f"{i}.qkv": r((HEADS + 2 * KV) * HD, DIM, std=DIM ** -0.5), f"{i}.o": r(DIM, HEADS * HD, std=(HEADS * HD) ** -0.5),
                  f"{i}.qw": r(HD, std=0.1), f"{i}.kw": r(HD, std=0.1), f"{i}.wg": r(HIDDEN, DIM, std=DIM ** -0.5),
                  f"{i}.wu": r(HIDDEN, DIM, std=DIM ** -0.5), f"{i}.wd": r(DIM, HIDDEN, std=HIDDEN ** -0.5)})
        for part in ("attn", "ffn"):
            p.update({f"{i}.{part}.post": r(DIM, std=0.1, at=1.0), f"{i}.{part}.gate": r(DIM, std=0.1, at=0.6),
                      f"{i}.{part}.pre": r(DIM, std=0.1, at=1.0)})
    data = dict(tok=torch.randint(0, VOCAB, (N,), generator=g), pos=torch.cat([torch.arange(n) for n in LENGTHS]),
                idx=torch.stack([torch.randperm(VOCAB, generator=g)[:6] for _ in range(N)]), teacher=r(N, 6, std=2.0))
    return p, data


def reference(params, d, rope):
    """float64 losses and gradients by autograd, on the host."""
    p = {k: v.double().requires_grad_() for k, v in params.items()}
    eps, s = float(np.float32(1e-6)), float(np.float32(SCALE))
    cos, sin = rope.double()[d["pos"]][:, None].chunk(2, -1)
    rms = lambda t: t / (t.square().mean(-1, keepdim=True) + eps).sqrt()  # noqa: E731

    def turned(t, w):
        a, b = (rms(t) * (1.0 + w)).chunk(2, -1)
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

    def attention(q, k, v):
        ends = np.concatenate([[0], np.cumsum(LENGTHS)])
        rows = []
        for a, b in zip(ends, ends[1:]):
            i, j = torch.arange(b - a)[:, None], torch.arange(b - a)[None]
            see = (j <= i) & (j > i - WINDOW)
            heads = []
            for h in range(HEADS):
                z = (q[a:b, h] @ k[a:b, h // (HEADS // KV)].T) * HD ** -0.5
                heads.append(z.masked_fill(~see, float("-inf")).softmax(-1) @ v[a:b, h // (HEADS // KV)])
            rows.append(torch.stack(heads, 1))
        return torch.cat(rows)

    x = p["table"][d["tok"]]
    y = rms(x) * p["first"]
    for i in range(LAYERS):
        qkv = (y @ p[f"{i}.qkv"].T).view(N, HEADS + 2 * KV, HD)
        q, k = turned(qkv[:, :HEADS], p[f"{i}.qw"]), turned(qkv[:, HEADS:HEADS + KV], p[f"{i}.kw"])
        for part in ("attn", "ffn"):
            if part == "attn":
                h = attention(q, k, qkv[:, HEADS + KV:]).flatten(1) @ p[f"{i}.o"].T
            else:
                h = (torch.nn.functional.silu(y @ p[f"{i}.wg"].T) * (y @ p[f"{i}.wu"].T)) @ p[f"{i}.wd"].T
            x = x + s * p[f"{i}.{part}.gate"] * rms(h) * p[f"{i}.{part}.post"]
            y = rms(x) * p[f"{i}.{part}.pre"]
    z = y @ p["head"].T
    t = d["teacher"].double()
    losses = (t.softmax(1) * (t.log_softmax(1) - z.log_softmax(1).gather(1, d["idx"]))).sum(1)
    (losses.sum() / N).backward()
    return losses.detach(), {k: v.grad for k, v in p.items()}


def step(p, d, rope, off):
    """The same through the operators: losses and gradients."""
    kw = dict(post_norm=True, residual_scale=SCALE)
    zero = torch.zeros(N, DIM, device="cuda")
    x, y = nsa.block_norm(nsa.embedding(p["table"], d["tok"]), zero, p["first"])
    x0, tape = x, []
    for i in range(LAYERS):
        w = lambda k: p[f"{i}.{k}"]  # noqa: B023,E731
        y_in = y
        qkv = (y @ w("qkv").T).view(N, HEADS + 2 * KV, HD)
        q, k = nsa.qk_norm_rope(qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], w("qw"), w("kw"), d["pos"], rope, weight_offset=1.0)
        att, lse = nsa.attention(q, k, qkv[:, HEADS + KV:], off, off, window=WINDOW)
        h1 = att.flatten(1) @ w("o").T
        x1, y1 = nsa.block_norm(x, h1, w("attn.pre"), w("attn.post"), w("attn.gate"), **kw)
        f = nsa.gated_ffn(y1, w("wg"), w("wu"))
        h2 = f @ w("wd").T
        x, y = nsa.block_norm(x1, h2, w("ffn.pre"), w("ffn.post"), w("ffn.gate"), **kw)
        tape.append((y_in, qkv, q, k, att, lse, h1, x1, y1, f, h2, x))
    z = y @ p["head"].T
    losses, dz = nsa.distill_loss(z, d["idx"], d["teacher"], grad_scale=1.0 / N)
    g = {"head": dz.T @ y}
    dy, dx = dz @ p["head"], None
    for i in reversed(range(LAYERS)):
        w = lambda k: p[f"{i}.{k}"]  # noqa: B023,E731
        y_in, qkv, q, k, att, lse, h1, x1, y1, f, h2, x2 = tape[i]
        dx, dh, g[f"{i}.ffn.pre"], g[f"{i}.ffn.post"], g[f"{i}.ffn.gate"] = nsa.block_norm_grad(
            dx, dy, x2, h2, w("ffn.pre"), w("ffn.post"), w("ffn.gate"), **kw)
        g[f"{i}.wd"] = dh.T @ f
        dy, g[f"{i}.wg"], g[f"{i}.wu"] = nsa.gated_ffn_grad(dh @ w("wd"), y1, w("wg"), w("wu"))
        dx, dh, g[f"{i}.attn.pre"], g[f"{i}.attn.post"], g[f"{i}.attn.gate"] = nsa.block_norm_grad(
            dx, dy, x1, h1, w("attn.pre"), w("attn.post"), w("attn.gate"), dx=dx, **kw)
        g[f"{i}.o"] = dh.T @ att.flatten(1)
        dqkv = torch.empty_like(qkv)
        v = qkv[:, HEADS + KV:]
        dq, dk, _ = nsa.attention_grad((dh @ w("o")).view(N, HEADS, HD), q, k, v, att, lse, off, off, window=WINDOW,
                                       dv=dqkv[:, HEADS + KV:])
        _, _, g[f"{i}.qw"], g[f"{i}.kw"] = nsa.qk_norm_rope_grad(
            dq, dk, qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV], w("qw"), w("kw"), d["pos"], rope, weight_offset=1.0,
            dq=dqkv[:, :HEADS], dk=dqkv[:, HEADS:HEADS + KV])
        dqkv = dqkv.flatten(1)
        g[f"{i}.qkv"] = dqkv.T @ y_in
        dy = dqkv @ w("qkv")
    dx, _, g["first"], _, _ = nsa.block_norm_grad(dx, dy, x0, zero, p["first"])
    g["table"] = nsa.embedding_grad(nsa.embedding_plan(d["tok"], VOCAB), dx)
    return losses, g


def on_device():
    params, data = make()
    off = torch.tensor([0, *np.cumsum(LENGTHS)], dtype=torch.int32, device="cuda")
    return params, data, {k: v.cuda() for k, v in params.items()}, {k: v.cuda() for k, v in data.items()}, off


def test_training_step():
    rope = nsa.rope_table(100, HD, device="cpu")
    params, data, p, d, off = on_device()
    want_losses, want = reference(params, data, rope)
    losses, g = step(p, d, rope.cuda(), off)
    # fp32 products over up to 499 terms, some thirty operations deep: each is off
    # by at most sqrt(499) 2^-24 of its norm for roundings of random sign, and
    # softmaxes and norms pass a relative error on at most a few times
    tol = 30 * 4 * 499 ** 0.5 * 2.0 ** -24
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(losses, want_losses) <= tol
    assert set(g) == set(want)
    for k in want:
        assert rel(g[k], want[k]) <= tol, k

    # the optimizer takes them: Muon the projections, AdamW the rest
    mats = [k for k, v in p.items() if v.dim() == 2 and k not in ("table", "head")]
    rest = [k for k in p if k not in mats]
    before = {k: v.clone() for k, v in p.items()}
    nsa.muon_step([p[k] for k in mats], [g[k] for k in mats], [torch.zeros_like(p[k]) for k in mats], lr=0.02)
    nsa.AdamWStep([p[k] for k in rest], [g[k] for k in rest])()
    for k in p:
        assert torch.isfinite(p[k]).all() and not torch.equal(p[k], before[k]), k


def test_the_step_recorded_and_replayed():
    """Forward and backward as one graph; every replay is the eager step's bits."""
    rope = nsa.rope_table(100, HD)
    _, _, p, d, off = on_device()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):      # the library products' own first calls
        step(p, d, rope, off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        losses, g = step(p, d, rope, off)
    for _ in range(3):
        for k in p:
            p[k].add_(0.01 * torch.randn_like(p[k]))
        graph.replay()
        torch.cuda.synchronize()
        want_losses, want = step(p, d, rope, off)
        torch.cuda.synchronize()
        rel = lambda a, b: float((a.double() - b.double()).norm() / b.double().norm())  # noqa: E731
        # the library's products may take another kernel in a graph; within that, the same step
        tol = 30 * 4 * 499 ** 0.5 * 2.0 ** -24
        assert rel(losses, want_losses) <= tol
        for k in want:
            assert rel(g[k], want[k]) <= tol, k
