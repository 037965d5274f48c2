"""Calls on another stream than the current one: what they allocate is not memory
that the current stream still works on, whatever its last owner left there."""
import pytest
import torch

import newton_schulz_08_amd as nsa

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()
    yield
    torch.cuda.empty_cache()


def calls():
    """{name: (call on a stream, what to free before it: shapes and types of its results and workspace)}"""
    g = torch.Generator("cuda").manual_seed(1)
    r = lambda *s, dtype=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    n, vocab, dim = 6000, 9000, 512
    table, dout = r(vocab, dim), r(n, dim)
    tok = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    plan = nsa.embedding_plan(tok, vocab)
    z = r(5, 90000, dtype=BF16)
    idx, y = torch.randint(0, 90000, (5, 6), generator=g, device="cuda"), r(5, 6)
    q, k, dq, dk = (r(n, h, 64) for h in (4, 2, 4, 2))
    w, rope, pos = r(64), nsa.rope_table(n, 64), torch.arange(n, device="cuda")
    xs = [r(512, 1024, dtype=BF16), r(1024, 512, dtype=BF16)]
    grads = [r(300000), r(1000)]
    u8, f32 = torch.uint8, torch.float32

    def muon(stream):
        p, m, u = [x.clone() for x in xs], [torch.zeros_like(x, dtype=f32) for x in xs], [torch.empty_like(x, dtype=f32) for x in xs]
        torch.cuda.synchronize()
        return lambda: nsa.muon_step(p, xs, m, update_out=u, stream=stream) or u

    def clip(stream):
        own = [t.clone() for t in grads]
        torch.cuda.synchronize()
        return lambda: [nsa.clip_grad_norm_(own, 0.5, stream=stream), *own]

    arrays = lambda p: [p.order, p.slot, p.rows, p.row_index, p.count]  # noqa: E731
    at_once = lambda f: lambda stream: lambda: f(stream)  # noqa: E731
    return {
        "embedding": (at_once(lambda s: nsa.embedding(table, tok, stream=s)), [((n, dim), f32)]),
        "plan": (at_once(lambda s: arrays(nsa.embedding_plan(tok, vocab, stream=s))),
                 [(tuple(plan._buf.shape), torch.int32), ((nsa.embedding_plan_workspace_bytes(n, vocab),), u8)]),
        "gradient": (at_once(lambda s: nsa.embedding_grad(plan, dout, stream=s)),
                     [((vocab, dim), f32), ((nsa.embedding_grad_workspace_bytes(n, dim, f32),), u8)]),
        "loss": (at_once(lambda s: nsa.distill_loss(z, idx, y, stream=s)),
                 [((5, 90000), BF16), ((5,), f32), ((nsa.distill_loss_workspace_bytes(5, 90000),), u8)]),
        "q/k": (at_once(lambda s: nsa.qk_norm_rope(q, k, w, w, pos, rope, stream=s)), [((n, 4, 64), f32), ((n, 2, 64), f32)]),
        "q/k gradient": (at_once(lambda s: nsa.qk_norm_rope_grad(dq, dk, q, k, w, w, pos, rope, stream=s)),
                         [((n, 4, 64), f32), ((n, 2, 64), f32), ((64,), f32), ((64,), f32),
                          ((nsa.qk_norm_rope_grad_workspace_bytes(n, 4, 2, 64),), u8)]),
        "Newton-Schulz": (at_once(lambda s: nsa.ns_batched(xs, stream=s)),
                          [(x.shape, BF16) for x in xs] + [((nsa.ns_workspace_bytes([x.shape for x in xs], BF16),), u8)]),
        "Muon": (muon, [((nsa.muon_step_workspace_bytes([x.shape for x in xs], BF16),), u8)]),
        "clipping": (clip, [((1,), f32), ((nsa.clip_grad_norm_workspace_bytes([t.numel() for t in grads]),), u8)]),
    }


def tensors(out):
    return [out] if isinstance(out, torch.Tensor) else list(out)


def test_freed_memory_is_not_written_while_the_current_stream_reads_it():
    side = torch.cuda.Stream()
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    for name, (prepare, blocks) in calls().items():
        want = [t.clone() for t in tensors(prepare(None)())]
        call = prepare(side)
        victims = [torch.empty(shape, dtype=dtype, device="cuda").fill_(3) for shape, dtype in blocks for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(60):
            big.fill_(1)                       # some 10 ms of work on the current stream, before ...
        kept = [v.clone() for v in victims]    # ... it reads the victims
        victims.clear()                        # freed, while those reads are still to come
        got = call()                           # the side stream does not wait
        torch.cuda.synchronize()
        for t in kept:
            assert bool((t == 3).all()), f"{name}: written while it was read"
        for a, b in zip(tensors(got), want):
            assert torch.equal(a, b), name


def test_results_are_kept_until_the_current_stream_has_read_them():
    side = torch.cuda.Stream()
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    for name, (prepare, _) in calls().items():
        want = [t.clone() for t in tensors(prepare(None)())]
        call = prepare(side)
        torch.cuda.synchronize()
        got = call()
        torch.cuda.current_stream().wait_stream(side)
        for _ in range(60):
            big.fill_(1)
        read = [t.clone() for t in tensors(got)]
        sizes = [(t.shape, t.dtype) for t in tensors(got)]
        del got
        with torch.cuda.stream(side):          # the side stream's next blocks of these sizes
            junk = [torch.zeros(s, dtype=d, device="cuda") for s, d in sizes]
        torch.cuda.synchronize()
        for a, b in zip(read, want):
            assert torch.equal(a, b), name
        del junk


def test_a_plan_outlives_the_call_that_reads_it():
    side = torch.cuda.Stream()
    g = torch.Generator("cuda").manual_seed(2)
    tok = torch.randint(0, 700, (50000,), generator=g, device="cuda")
    dout = torch.randn(50000, 1024, generator=g, device="cuda")
    want = nsa.embedding_grad(nsa.embedding_plan(tok, 700), dout)
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    plan = nsa.embedding_plan(tok, 700)
    size = plan._buf.shape
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):
            big.fill_(1)
    got = nsa.embedding_grad(plan, dout, stream=side)
    del plan
    junk = torch.zeros(size, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not junk.any()


def test_calls_on_a_forked_stream_are_recorded():
    """A graph whose capture forks to a second stream: what is allocated there
    belongs to the graph, and replays follow their inputs."""
    g = torch.Generator("cuda").manual_seed(3)
    table = torch.randn(500, 256, generator=g, device="cuda")
    tok = torch.randint(0, 500, (9000,), generator=g, device="cuda")
    z = torch.randn(4, 70000, generator=g, device="cuda")
    idx, y = torch.randint(0, 70000, (4, 5), generator=g, device="cuda"), torch.randn(4, 5, generator=g, device="cuda")

    def both(stream):
        x = nsa.embedding(table, tok, stream=stream)
        grad = nsa.embedding_grad(nsa.embedding_plan(tok, 500, stream=stream), x, stream=stream)
        return (x, grad, *nsa.distill_loss(z, idx, y, stream=stream))

    both(None)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        outs = both(side)
        torch.cuda.current_stream().wait_stream(side)
        total = outs[2] + 1.0
    for _ in range(4):
        table.normal_()
        z.normal_()
        tok.random_(-3, 520)
        graph.replay()
        torch.cuda.synchronize()
        want = both(None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and torch.equal(total, want[2] + 1.0)
        del want
        junk = [torch.full_like(o, 5.0) for o in outs]   # eager work between the replays
        torch.cuda.synchronize()
        del junk
