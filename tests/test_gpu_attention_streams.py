"""Attention, whole and over caches, and its gradient on other streams than the
current one: recorded on a forked stream, several at once, with a workspace that
two graphs share, and beside memory that the current stream still reads."""
import pytest
import torch

import newton_schulz_08_amd as nsa

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
QH, KH = 6, 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()
    yield
    torch.cuda.empty_cache()


class Inputs:
    """Sequences that take every token, so that every row of a result is written; `refill` draws new ones in place."""

    def __init__(self, seed, dtype=BF16, d=64):
        self.g = torch.Generator("cuda").manual_seed(seed)
        e = lambda *s: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.q, self.kv, self.dout = e(480, QH, d), e(480, 2 * KH, d), e(480, QH, d)
        self.token, self.cache = e(3, QH, d), e(6000, 2 * KH, d)
        i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.off, self.tok_off, self.cache_off = i(0, 130, 131, 480), i(0, 1, 2, 3), i(0, 2500, 2600, 6000)
        self.refill()

    def refill(self):
        for t in (self.q, self.kv, self.dout, self.token, self.cache):
            t.normal_(generator=self.g)

    def forward(self, **kw):
        return nsa.attention(self.q, self.kv[:, :KH], self.kv[:, KH:], self.off, self.off, **kw)

    def tokens(self, **kw):
        return nsa.attention(self.token, self.cache[:, :KH], self.cache[:, KH:], self.tok_off, self.cache_off, **kw)

    def backward(self, out, lse, **kw):
        return nsa.attention_grad(self.dout, self.q, self.kv[:, :KH], self.kv[:, KH:], out, lse, self.off, self.off, **kw)

    def all(self, **kw):
        out, lse = self.forward(**{k: v for k, v in kw.items() if k != "workspace"})
        return (out, lse, *self.backward(out, lse, **kw), *self.tokens(**kw))


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 80)])
def test_recorded_on_a_forked_stream(dtype, d):
    s = Inputs(1, dtype, d)
    s.all()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = s.all(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(4):
        s.refill()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, s.all())
        torch.cuda.synchronize()


def test_side_streams_at_once():
    s = Inputs(2)
    want = [t.clone() for t in s.all()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        got = [s.all(stream=streams[i % 3]) for i in range(9)]
        torch.cuda.synchronize()
        assert all(same(g, want) for g in got)


def test_two_graphs_with_one_workspace():
    """Row statistics and slices' sums of one call are nothing to the next."""
    s, t = Inputs(3), Inputs(4)
    need = max(nsa.attention_grad_workspace_bytes(480, QH), nsa.attention_workspace_bytes(3, 6000, QH, KH, 64, 3))
    assert nsa.attention_workspace_bytes(3, 6000, QH, KH, 64, 3) > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    s.all(workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for inputs in (s, t):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = inputs.all(workspace=ws)
        graphs.append((graph, outs, inputs))
    for _ in range(3):
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        ws.fill_(255)    # NaN, where a number is read that was not written
        for graph, outs, inputs in graphs:
            graph.replay()
            torch.cuda.synchronize()
            kept = [o.clone() for o in outs]
            assert same(kept, inputs.all(workspace=ws))


def test_freed_memory_is_not_written_while_the_current_stream_reads_it():
    s, side = Inputs(5), torch.cuda.Stream()
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    out, lse = (t.clone() for t in s.forward())
    calls = {
        "forward": (lambda **kw: s.forward(**kw), [((480, QH, 64), BF16), ((QH, 480), F32)]),
        "tokens": (lambda **kw: s.tokens(**kw), [((3, QH, 64), BF16), ((QH, 3), F32),
                                                 ((nsa.attention_workspace_bytes(3, 6000, QH, KH, 64, 3),), torch.uint8)]),
        "backward": (lambda **kw: s.backward(out, lse, **kw), [((480, QH, 64), BF16), ((480, KH, 64), BF16),
                                                              ((nsa.attention_grad_workspace_bytes(480, QH),), torch.uint8)]),
    }
    for name, (call, shapes) in calls.items():
        want = [t.clone() for t in call()]
        victims = [torch.empty(shape, dtype=dtype, device="cuda").fill_(3) for shape, dtype in shapes for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(60):
            big.fill_(1)                       # some 10 ms of work on the current stream, before ...
        kept = [v.clone() for v in victims]    # ... it reads the victims
        victims.clear()                        # freed, while those reads are still to come
        got = call(stream=side)                # the side stream does not wait
        torch.cuda.synchronize()
        for t in kept:
            assert bool((t == 3).all()), f"{name}: written while it was read"
        assert same(got, want), name


def test_given_results_on_a_side_stream():
    """Rows behind the last sequence, filled on the same stream, stay as they were."""
    s, side = Inputs(6), torch.cuda.Stream()
    want = [t.clone() for t in s.forward()]
    want += [t.clone() for t in s.backward(*want)]
    torch.cuda.synchronize()
    last = torch.tensor([0, 130, 131, 300], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        out, lse = torch.full_like(s.q, 7.0), torch.full((QH, 480), 7.0, device="cuda")
        grads = [torch.full((480, h, 64), 7.0, dtype=BF16, device="cuda") for h in (QH, KH, KH)]
    k, v = s.kv[:, :KH], s.kv[:, KH:]
    nsa.attention(s.q, k, v, last, last, out=out, lse=lse, stream=side)
    nsa.attention_grad(s.dout, s.q, k, v, out, lse, last, last, dq=grads[0], dk=grads[1], dv=grads[2], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out[:300], want[0][:300]) and torch.equal(lse[:, :300], want[1][:, :300])
    assert torch.equal(grads[0][:300], want[2][:300])
    assert all(torch.equal(g[:131], w[:131]) for g, w in zip(grads[1:], want[3:]))
    assert all((t[300:] == 7).all() for t in (out, *grads)) and (lse[:, 300:] == 7).all()
