"""The block operators as a program calls them: recorded into graphs and replayed,
on other streams than the current one, several at once, with given results and
workspaces, timed."""
import pytest
import torch

import newton_schulz_08_amd as nsa

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()
    yield
    torch.cuda.empty_cache()


class Inputs:
    """Inputs of one call of each operator; `refill` draws new ones in place."""

    def __init__(self, seed=0):
        self.g = torch.Generator("cuda").manual_seed(seed)
        e = lambda *s, dtype=BF16: torch.empty(*s, device="cuda", dtype=dtype)  # noqa: E731
        self.x, self.h, self.dx, self.dy = e(300, 1030, dtype=F32), e(300, 1030), e(300, 1030, dtype=F32), e(300, 1030)
        self.pre, self.post, self.gate = e(1030), e(1030), e(1030)
        self.wide, self.wh, self.wpre = e(40, 9000), e(40, 9000), e(9000)
        self.q, self.kv, self.dout = e(500, 6, 64), e(500, 4, 64), e(500, 6, 64)
        self.token, self.cache = e(3, 4, 80, dtype=F32), e(6000, 2, 80, dtype=F32)
        self.f, self.wg, self.wu, self.df = e(200, 100), e(150, 100), e(150, 100), e(200, 150)
        self.few = e(7, 100)
        self.floats = [t for t in vars(self).values() if isinstance(t, torch.Tensor)]
        self.off = torch.tensor([0, 130, 131, 480], dtype=torch.int32, device="cuda")
        self.tok_off = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
        self.cache_off = torch.tensor([0, 2500, 2600, 6000], dtype=torch.int32, device="cuda")
        self.refill()

    def refill(self):
        for t in self.floats:
            t.normal_(generator=self.g)

    def calls(self, stream=None):
        """{name: call}, the backward ones behind their forward's results."""
        kw = dict(stream=stream)
        bn = dict(kw, post_norm=True, residual_scale=0.7)
        k, v = self.kv[:, :2], self.kv[:, 2:]

        def attend():
            # rows behind the last sequence are the caller's
            out, lse = torch.zeros_like(self.q), torch.zeros(6, 500, device="cuda")
            nsa.attention(self.q, k, v, self.off, self.off, out=out, lse=lse, **kw)
            grads = [torch.zeros(t.shape, dtype=BF16, device="cuda") for t in (self.q, k, v)]
            nsa.attention_grad(self.dout, self.q, k, v, out, lse, self.off, self.off, dq=grads[0], dk=grads[1], dv=grads[2], **kw)
            return (out, lse, *grads)

        return {
            "norm": lambda: nsa.block_norm(self.x, self.h, self.pre, self.post, self.gate, **bn),
            "norm gradient": lambda: nsa.block_norm_grad(self.dx, self.dy, self.x, self.h, self.pre, self.post, self.gate, **bn),
            "wide norm gradient": lambda: nsa.block_norm_grad(None, self.wh, self.wide, self.wh, self.wpre, **kw)[:3],
            "attention": attend,
            "tokens": lambda: nsa.attention(self.token, self.cache[:, :1], self.cache[:, 1:], self.tok_off, self.cache_off, **kw),
            "ffn": lambda: (nsa.gated_ffn(self.f, self.wg, self.wu, **kw), nsa.gated_ffn(self.few, self.wg, self.wu, "gelu", **kw)),
            "ffn gradient": lambda: nsa.gated_ffn_grad(self.df, self.f, self.wg, self.wu, **kw),
        }


def test_recorded_and_replayed():
    s = Inputs()
    for call in s.calls().values():
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = {name: call() for name, call in s.calls().items()}
    for _ in range(4):
        s.refill()
        graph.replay()
        torch.cuda.synchronize()
        for name, call in s.calls().items():
            assert all(torch.equal(a, b) for a, b in zip(got[name], call())), name
        torch.cuda.synchronize()
        junk = [torch.full_like(t, 5.0) for outs in got.values() for t in outs]   # eager work between the replays
        torch.cuda.synchronize()
        del junk


def test_recorded_on_a_forked_stream():
    s = Inputs(1)
    want = {name: [t.clone() for t in call()] for name, call in s.calls().items() if name != "attention"}
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = {name: call() for name, call in s.calls(side).items() if name in want}
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for name, outs in want.items():
            assert all(torch.equal(a, b) for a, b in zip(got[name], outs)), name


def test_two_graphs_with_one_workspace():
    """A call leaves nothing behind in its workspace for the next."""
    s, t = Inputs(2), Inputs(3)
    need = max(nsa.block_norm_grad_workspace_bytes(300, 1030), nsa.gated_ffn_grad_workspace_bytes(200, 100, 150, BF16, aligned=False))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def both(s):
        a = nsa.gated_ffn_grad(s.df, s.f, s.wg, s.wu, workspace=ws)
        b = nsa.block_norm_grad(s.dx, s.dy, s.x, s.h, s.pre, s.post, s.gate, post_norm=True, workspace=ws)
        return (*a, *b)

    both(s)
    torch.cuda.synchronize()
    graphs = []
    for inputs in (s, t):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = both(inputs)
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
            assert all(torch.equal(a, b) for a, b in zip(kept, both(inputs)))


def test_side_streams_at_once():
    s = Inputs(4)
    want = {name: [t.clone() for t in call()] for name, call in s.calls().items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        got = []
        for i in range(6):
            for name, call in s.calls(streams[i % 3]).items():
                if name != "attention":   # its given results are filled on the current stream
                    got.append((name, call()))
        torch.cuda.synchronize()
        for name, outs in got:
            assert all(torch.equal(a, b) for a, b in zip(outs, want[name])), name


def test_freed_memory_is_not_written_while_the_current_stream_reads_it():
    s, side = Inputs(5), torch.cuda.Stream()
    big = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    blocks = {
        "norm": [((300, 1030), F32), ((300, 1030), BF16)],
        "norm gradient": [((300, 1030), F32), ((300, 1030), BF16), ((1030,), BF16), ((nsa.block_norm_grad_workspace_bytes(300, 1030),), torch.uint8)],
        "tokens": [((3, 4, 80), F32), ((4, 3), F32), ((nsa.attention_workspace_bytes(3, 6000, 4, 1, 80, 3),), torch.uint8)],
        "ffn": [((200, 150), BF16), ((7, 150), BF16)],
        "ffn gradient": [((200, 100), BF16), ((150, 100), BF16),
                         ((nsa.gated_ffn_grad_workspace_bytes(200, 100, 150, BF16, aligned=False),), torch.uint8)],
    }
    for name, shapes in blocks.items():
        want = [t.clone() for t in s.calls()[name]()]
        call = s.calls(side)[name]
        victims = [torch.empty(shape, dtype=dtype, device="cuda").fill_(3) for shape, dtype in shapes for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(60):
            big.fill_(1)                       # some 10 ms of work on the current stream, before ...
        kept = [v.clone() for v in victims]    # ... it reads the victims
        victims.clear()                        # freed, while those reads are still to come
        got = call()                           # the side stream does not wait
        torch.cuda.synchronize()
        for t in kept:
            assert bool((t == 3).all()), f"{name}: written while it was read"
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_families_are_timed_and_recorded_calls_are_not():
    s = Inputs(6)
    for call in s.calls().values():
        call()
    torch.cuda.synchronize()
    nsa.profile_read()
    nsa.profile_enable(True)
    try:
        for call in s.calls().values():
            call()
        stats = nsa.profile_read()
        assert set(stats) == {"block_norm", "block_norm_grad", "attention", "attention_grad", "gated_ffn", "gated_ffn_grad"}
        assert all(v["launches"] >= 1 and v["total_ms"] > 0 and v["bytes"] > 0 and v["flops"] > 0 for v in stats.values())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.calls()["ffn"]()
        assert nsa.profile_read() == {}
    finally:
        nsa.profile_enable(False)


def test_refusals_leave_results_alone():
    s = Inputs(7)
    out = torch.full((500, 6, 64), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((6, 500), 7.0, device="cuda")
    k, v = s.kv[:, :2], s.kv[:, 2:]
    with pytest.raises(nsa.DmuonError, match="window"):
        nsa.attention(s.q, k, v, s.off, s.off, causal=False, window=3, out=out, lse=lse)
    with pytest.raises(nsa.DmuonError, match="overlap"):
        nsa.attention(s.q, k, v, s.off, s.off, out=s.q, lse=lse)
    with pytest.raises(nsa.DmuonError, match="multiple"):
        nsa.attention(s.q[:, :5], k, v, s.off, s.off)
    with pytest.raises(ValueError, match="together"):
        nsa.attention(s.q, k, v, s.off)
    with pytest.raises(TypeError, match="int32"):
        nsa.attention(s.q, k, v, s.off.long(), s.off.long())
    with pytest.raises(ValueError, match="expected"):
        nsa.attention(s.q, k, s.kv[:400, 2:], s.off, s.off)
    with pytest.raises(ValueError, match="next to each other"):
        nsa.attention(s.q.transpose(0, 1).contiguous().transpose(0, 1), k, v, s.off, s.off)
    with pytest.raises(ValueError, match="h is"):
        nsa.block_norm(s.x, s.h[:, :1000])
    with pytest.raises(nsa.DmuonError, match="post"):
        nsa.block_norm(s.x, s.h, s.pre, s.post)
    with pytest.raises(ValueError, match="contiguous rows"):
        nsa.block_norm(s.x.t(), s.h.t())
    with pytest.raises(TypeError, match="dtype"):
        nsa.gated_ffn(s.f, s.wg.float(), s.wu.float())
    with pytest.raises(ValueError, match="hidden"):
        nsa.gated_ffn(s.f, s.wg[:, :50].contiguous(), s.wu)
    with pytest.raises(ValueError, match="dh is"):
        nsa.gated_ffn_grad(s.df[:, :100], s.f, s.wg, s.wu)
    with pytest.raises(nsa.DmuonError, match="overlap"):
        nsa.gated_ffn_grad(s.df, s.f, s.wg, s.wu, dw_gate=s.wg)
    torch.cuda.synchronize()
    assert (out == 7).all() and (lse == 7).all()
