"""Embedding lookup, plan, gradient and the row-gradient AdamW step against the
float64 references; the plan exactly, the AdamW step bitwise against the dense
one."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa
from oracle import ops

from ops_util import DT, U32, dev, empty, half_step, host, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


def draw_tokens(kind, n, vocab, seed):
    rng = np.random.default_rng(seed)
    if kind == "zipf":
        t = np.minimum(vocab ** rng.random(n), vocab).astype(np.int64) - 1
        return rng.permutation(vocab)[np.maximum(t, 0)]
    if kind == "one":
        return np.full(n, vocab - 1)
    if kind == "none":
        return rng.choice([-1, vocab, -100, vocab + 7], n)
    if kind == "distinct":
        return rng.permutation(max(n, vocab))[:n] % vocab
    t = rng.integers(0, vocab, n)                # "mixed": a padded batch
    t[rng.random(n) < 0.2] = -1
    t[rng.random(n) < 0.05] = vocab
    return t


# ---------------------------------------------------------------- lookup
@pytest.mark.parametrize("tdt", ["f32", "bf16"])
@pytest.mark.parametrize("odt", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim,shift", [(1, 1, 1, 0), (3, 7, 8, 0), (5, 100, 24, 1), (17, 33, 100, 0),
                                               (64, 50, 2056, 0), (9, 300, 4096, 0), (2, 5, 65536, 0), (300, 11, 72, 3)])
def test_lookup(tdt, odt, n, vocab, dim, shift):
    rng = np.random.default_rng(n * 1000 + dim)
    table = dev(rng.standard_normal((vocab, dim)) * 0.02, DT[tdt], shift)
    tok = draw_tokens("mixed", n, vocab, 7)
    out = empty((n, dim), DT[odt], shift)
    for dt in (torch.int32, torch.int64):
        got = nsa.embedding(table, dev(tok, dt), scale=22.5, out=out)
        want = ops.embedding(host(table), tok, 22.5)
        # the product is rounded to fp32, then to the output's type
        within(host(got), want, ((1 + U32) * (1 + half_step(DT[odt])) - 1) * np.abs(want), "lookup")


def test_lookup_shapes_and_no_tokens():
    table = torch.randn(10, 16, device="cuda")
    tok = torch.tensor([[1, 2, -1], [9, 0, 3]], device="cuda")
    out = nsa.embedding(table, tok)
    assert out.shape == (2, 3, 16) and torch.equal(out[1, 0], table[9]) and not out[0, 2].any()
    assert nsa.embedding(table, tok[:0]).shape == (0, 3, 16)


def test_lookup_reads_no_row_of_unknown_tokens():
    table = torch.full((4, 64), float("nan"), device="cuda")
    tok = torch.tensor([-1, 4, -2 ** 40, 2 ** 40], device="cuda")
    assert not nsa.embedding(table, tok).any()


# ---------------------------------------------------------------- plan
PLANS = [("zipf", 1, 5), ("mixed", 64, 1), ("mixed", 65, 2), ("one", 1000, 7), ("none", 1000, 7), ("zipf", 4095, 511),
         ("zipf", 4096, 512), ("mixed", 4096, 130000), ("mixed", 4097, 513), ("one", 5000, 40000), ("none", 6000, 3),
         ("zipf", 70001, 128256), ("distinct", 20000, 300000), ("mixed", 140000, 31), ("zipf", 300007, 1 << 20)]


@pytest.mark.parametrize("kind,n,vocab", PLANS)
def test_plan(kind, n, vocab):
    tok = draw_tokens(kind, n, vocab, n)
    for dt in (torch.int32, torch.int64):
        plan = nsa.embedding_plan(dev(tok, dt), vocab)
        for name, want in zip(("order", "slot", "rows", "row_index", "count"), ops.embedding_plan(tok, vocab)):
            assert np.array_equal(host(getattr(plan, name)), np.reshape(want, -1)), name


def test_plan_of_nothing_and_refill():
    plan = nsa.embedding_plan(torch.zeros(0, dtype=torch.int32, device="cuda"), 9)
    assert plan.count.item() == 0 and plan.row_index.eq(-1).all() and plan.rows.numel() == 0
    tok = torch.tensor([3, 3, 8], device="cuda")
    plan = nsa.embedding_plan(tok, 9)
    again = nsa.embedding_plan(torch.tensor([0, 8, 0], device="cuda"), 9, plan=plan)
    assert again is plan and plan.rows.tolist() == [0, 8, -1] and plan.row_index.tolist() == [0] + [-1] * 7 + [1]


# ---------------------------------------------------------------- gradient
def check_grad(kind, n, vocab, dim, ddt, gdt, form, shift=0, scale=1.5):
    rng = np.random.default_rng(n + dim)
    tok = draw_tokens(kind, n, vocab, n + 1)
    dout = rng.standard_normal((n, dim)) * 1e-2
    dout[(tok < 0) | (tok >= vocab)] = np.nan    # never read
    dout = dev(dout, DT[ddt], shift)
    plan = nsa.embedding_plan(dev(tok, torch.int64), vocab)
    exact, size, count = ops.embedding_grad(host(dout), tok, vocab, scale)
    cap = min(n, vocab)
    out = empty((cap if form == "rows" else vocab, dim), DT[gdt], shift)
    if form == "add":
        old = dev(rng.standard_normal((vocab, dim)) * 1e-2, DT[gdt])
        out.copy_(old)
    got = host(nsa.embedding_grad(plan, dout, scale=scale, form=form, out=out))
    # count - 1 additions, the scale, and one addition more with "add"
    sums = (count[:, None] + 2) * U32 * 1.001 * size
    if form == "add":
        want = exact + host(old)
        bound = sums + (U32 + half_step(DT[gdt])) * (np.abs(want) + sums)
        bound[count == 0] = 0.0
    else:
        want = exact
        bound = sums + half_step(DT[gdt]) * (np.abs(exact) + sums)
    if form == "rows":
        rows = host(plan.rows)
        used = rows >= 0
        assert not got[~used].any()
        got, want, bound = got[used], want[rows[used]], bound[rows[used]]
    within(got, want, bound, f"{form} gradient")


@pytest.mark.parametrize("form", ["dense", "add", "rows"])
@pytest.mark.parametrize("ddt,gdt", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("kind,n,vocab,dim", [("zipf", 1, 3, 1), ("mixed", 50, 20, 8), ("one", 700, 3, 40),
                                              ("mixed", 333, 4, 100), ("zipf", 2000, 300, 256), ("none", 100, 5, 16)])
def test_gradient(form, ddt, gdt, kind, n, vocab, dim):
    check_grad(kind, n, vocab, dim, ddt, gdt, form)


@pytest.mark.parametrize("form", ["dense", "rows"])
@pytest.mark.parametrize("kind,n,vocab,dim,ddt,shift", [("zipf", 5000, 1000, 2056, "bf16", 0), ("one", 9000, 2, 24, "bf16", 0),
                                                        ("mixed", 4500, 7, 520, "f32", 0), ("zipf", 600, 90, 72, "bf16", 1),
                                                        ("mixed", 300, 40, 1030, "f32", 1), ("zipf", 200, 40, 65536, "bf16", 0)])
def test_gradient_long(form, kind, n, vocab, dim, ddt, shift):
    check_grad(kind, n, vocab, dim, ddt, ddt, form, shift)


def test_gradient_of_nothing():
    plan = nsa.embedding_plan(torch.zeros(0, dtype=torch.int64, device="cuda"), 5)
    none = torch.zeros(0, 8, device="cuda")
    assert not nsa.embedding_grad(plan, none, out=torch.ones(5, 8, device="cuda")).any()
    assert nsa.embedding_grad(plan, none, form="add", out=torch.ones(5, 8, device="cuda")).eq(1).all()
    assert nsa.embedding_grad(plan, none, form="rows").shape == (0, 8)


def test_gradient_is_reproducible_and_against_a_difference():
    rng = np.random.default_rng(11)
    tok = draw_tokens("zipf", 3000, 200, 12)
    dout = dev(rng.standard_normal((3000, 64)), torch.float32)
    t = dev(tok, torch.int64)
    plan = nsa.embedding_plan(t, 200)
    grad = nsa.embedding_grad(plan, dout, scale=2.0)
    assert torch.equal(grad, nsa.embedding_grad(nsa.embedding_plan(t, 200), dout, scale=2.0))
    # the lookup is linear: <dout, lookup(v)> = <grad, v> up to the sums' roundings
    v = dev(rng.standard_normal((200, 64)), torch.float32)
    lhs = float((dout.double() * nsa.embedding(v, t, scale=2.0).double()).sum())
    rhs = float((grad.double() * v.double()).sum())
    _, size, count = ops.embedding_grad(host(dout), tok, 200, 2.0)
    slack = float(((count[:, None] + 3) * U32 * size * np.abs(host(v))).sum())
    assert abs(lhs - rhs) <= slack


# ---------------------------------------------------------------- AdamW, gradient as rows
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,n", [(1, 1, 1), (7, 5, 3), (100, 40, 64), (33, 4096, 20), (3000, 12, 500), (65, 1032, 300),
                                        (40, 4100, 9), (9, 65536, 4)])
def test_adamw_rows_is_the_dense_step(dtype, rows, dim, n):
    rng = np.random.default_rng(rows)
    tok = dev(rng.integers(0, rows, n), torch.int64)
    plan = nsa.embedding_plan(tok, rows)
    dout = dev(rng.standard_normal((n, dim)), dtype)
    state = [dev(rng.standard_normal((rows, dim)), dtype), dev(rng.standard_normal((rows, dim)) * 1e-2, torch.float32),
             dev(rng.random((rows, dim)) * 1e-3, torch.float32)]
    a, b = [t.clone() for t in state], [t.clone() for t in state]
    for step in (1, 2, 9):
        nsa.adamw_rows_step_(a[0], nsa.embedding_grad(plan, dout, form="rows"), plan.row_index, a[1], a[2], step, lr=1e-2)
        nsa.adamw_step_([b[0]], [nsa.embedding_grad(plan, dout)], [b[1]], [b[2]], step, lr=1e-2)
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_adamw_rows_unaligned_and_indices_outside():
    rng = np.random.default_rng(5)
    for dim in (8, 6):
        p, m, v = (dev(rng.random((50, dim)), torch.float32, 1) for _ in range(3))
        q, k, w = p.clone(), m.clone(), v.clone()
        g = dev(rng.standard_normal((3, dim)), torch.float32, 1)
        index = torch.full((50,), -1, dtype=torch.int32, device="cuda")
        index[4], index[10], index[11], index[49], index[0] = 0, 2, 2, 3, 2 ** 31 - 1   # 3 and 2^31 - 1 name no row
        dense = torch.zeros(50, dim, device="cuda")
        dense[4], dense[10], dense[11] = g[0], g[2], g[2]
        nsa.adamw_rows_step_(p, g, index, m, v, 3)
        nsa.adamw_step_([q], [dense], [k], [w], 3)
        assert torch.equal(p, q) and torch.equal(m, k) and torch.equal(v, w)
    # no gradient row at all
    nsa.adamw_rows_step_(p, g[:0], index, m, v, 4)
    nsa.adamw_step_([q], [torch.zeros_like(q)], [k], [w], 4)
    assert torch.equal(p, q) and torch.equal(m, k) and torch.equal(v, w)


def test_optimizer_takes_row_gradients_beside_dense_ones():
    rng = np.random.default_rng(9)
    tok = dev(rng.integers(0, 60, 90), torch.int64)
    dout = dev(rng.standard_normal((90, 32)), torch.float32)
    plan = nsa.embedding_plan(tok, 60)
    rows, dense = nsa.embedding_grad(plan, dout, form="rows"), nsa.embedding_grad(plan, dout)
    table, gain, g = (dev(rng.standard_normal(s), torch.float32) for s in ((60, 32), 32, 32))
    a, b = [table.clone(), gain.clone()], [table.clone(), gain.clone()]
    one = nsa.AdamWStep(a, [(rows, plan.row_index), g], lr=1e-2)
    two = nsa.AdamWStep(b, [dense, g], lr=1e-2)
    for _ in range(3):
        one()
        two()
    assert one.step == 3 and all(torch.equal(x, y) for x, y in zip(a + one.exp_avg + one.exp_avg_sq, b + two.exp_avg + two.exp_avg_sq))
    alone = nsa.AdamWStep([table], [(rows, plan.row_index)], lr=1e-2)
    for _ in range(3):
        alone()
    assert torch.equal(table, a[0])
    with pytest.raises(ValueError):
        nsa.AdamWStep([table], [(rows,)])
    with pytest.raises(ValueError):
        nsa.AdamWStep([table], [])


# ---------------------------------------------------------------- streams and graphs
def test_graph_replays_see_new_tokens():
    rng = np.random.default_rng(6)
    for n, vocab, dim in ((512, 300, 64), (9000, 2000, 32)):
        tok = dev(draw_tokens("zipf", n, vocab, 1), torch.int64)
        dout = dev(rng.standard_normal((n, dim)), torch.bfloat16)
        table, m, v = (torch.rand(vocab, dim, device="cuda") for _ in range(3))
        table = table.bfloat16()
        static = [table.clone(), m.clone(), v.clone()]

        def step(state):
            out = nsa.embedding(state[0], tok)
            plan = nsa.embedding_plan(tok, vocab)
            rows = nsa.embedding_grad(plan, dout, form="rows")
            nsa.adamw_rows_step_(state[0], rows, plan.row_index, state[1], state[2], 3)
            return out, nsa.embedding_grad(plan, dout), plan.rows

        step([t.clone() for t in static])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step(static)
        for t, s in zip((table, m, v), static):
            s.copy_(t)
        for k in range(4):
            tok.copy_(dev(draw_tokens("mixed" if k == 2 else "zipf", n, vocab, 20 + k), torch.int64))
            dout.copy_(dev(rng.standard_normal((n, dim)), torch.bfloat16))
            g.replay()
            torch.cuda.synchronize()
            want = step([table, m, v])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
            assert all(torch.equal(a, b) for a, b in zip(static, (table, m, v)))


def test_other_stream_with_own_workspaces():
    rng = np.random.default_rng(8)
    side = torch.cuda.Stream()
    results = []
    inputs = [(dev(draw_tokens("zipf", 6000, 700, s), torch.int64), dev(rng.standard_normal((6000, 128)), torch.float32))
              for s in (1, 2)]
    torch.cuda.synchronize()
    for (tok, dout), stream in zip(inputs, (None, side)):
        plan = nsa.embedding_plan(tok, 700, stream=stream)
        results.append(nsa.embedding_grad(plan, dout, stream=stream))
    torch.cuda.synchronize()
    for (tok, dout), got in zip(inputs, results):
        assert torch.equal(got, nsa.embedding_grad(nsa.embedding_plan(tok, 700), dout))
