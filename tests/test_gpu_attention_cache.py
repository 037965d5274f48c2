"""Decoding several sequences over caches that grow in place: the room behind each
is a sequence without queries, and only the offsets change from token to token."""
import pytest
import torch

import newton_schulz_08_amd as nsa
import attention_util as ref
from ops_util import host, within

F32, BF16 = torch.float32, torch.bfloat16


def test_room_does_not_take_the_slices():
    """16 tokens over 16 caches of 4096 of 8192 keys are few tiles with long caches, as without room."""
    assert nsa.attention_workspace_bytes(16, 16 * 4096, 32, 8, 128, 16) > 0
    assert nsa.attention_workspace_bytes(16, 16 * 8192, 32, 8, 128, 32) > 0
    # one query among a million sequences: the workspace stays small
    assert nsa.attention_workspace_bytes(1, 1 << 22, 8, 1, 256, 1 << 20) == 0


class Caches:
    """`room` keys for each of len(used) sequences; keys that are not in use hold NaN."""

    def __init__(self, used, room, kh, d, dtype, seed=0):
        self.g, self.used, self.room = torch.Generator("cuda").manual_seed(seed), list(used), room
        self.kv = torch.full((len(used) * room, 2 * kh, d), float("nan"), dtype=dtype, device="cuda")
        self.k, self.v = self.kv[:, :kh], self.kv[:, kh:]
        for b, n in enumerate(used):
            self.kv[b * room:b * room + n].normal_(generator=self.g)
        self.q_offsets, self.k_offsets = (torch.zeros(2 * len(used) + 1, dtype=torch.int32, device="cuda") for _ in range(2))

    def take(self, new):
        """new[b] more tokens of sequence b: their keys, and the offsets in place."""
        q, k = [0], [0]
        for b, n in enumerate(new):
            at = b * self.room + self.used[b]
            self.kv[at:at + n].normal_(generator=self.g)
            self.used[b] += n
            q += [q[-1] + n] * 2
            k += [b * self.room + self.used[b], (b + 1) * self.room]
        self.q_offsets.copy_(torch.tensor(q, dtype=torch.int32))
        self.k_offsets.copy_(torch.tensor(k, dtype=torch.int32))
        return q, k

    def packed(self):
        rows = torch.cat([torch.arange(b * self.room, b * self.room + n, device="cuda") for b, n in enumerate(self.used)])
        return self.k[rows], self.v[rows], ref.offsets(self.used)

    def check(self, q, new, out, lse, causal=True, window=0):
        k, v, (ke, _) = self.packed()
        qe, _ = ref.offsets(new)
        w, b, wl, lb = ref.forward(q, k, v, qe, ke, causal, window, q.shape[2] ** -0.5, q.dtype)
        within(host(out), w.cpu().numpy(), b.cpu().numpy(), "out")
        within(host(lse), wl.cpu().numpy(), lb.cpu().numpy(), "lse")


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,window", [(BF16, 128, 0), (BF16, 64, 300), (F32, 80, 0)])
def test_prompts_then_tokens(gpu, dtype, d, window):
    c = Caches([0, 0, 0, 0], 2500, 2, d, dtype)
    for new in ([40, 1, 300, 7], [1000, 1000, 0, 2000], [1, 1, 1, 1], [1, 1, 1, 1], [0, 2, 1, 0]):
        c.take(new)
        q = torch.randn(sum(new), 6, d, generator=c.g, device="cuda").to(dtype)
        out, lse = nsa.attention(q, c.k, c.v, c.q_offsets, c.k_offsets, window=window)
        c.check(q, new, out, lse, window=window)


@pytest.mark.gpu
def test_gradients_leave_the_room_zero(gpu):
    c, new = Caches([0, 0, 0], 200, 2, 64, BF16), [130, 1, 77]
    c.take(new)
    q = torch.randn(sum(new), 4, 64, generator=c.g, device="cuda").to(BF16)
    out, lse = nsa.attention(q, c.k, c.v, c.q_offsets, c.k_offsets)
    got = nsa.attention_grad(q, q, c.k, c.v, out, lse, c.q_offsets, c.k_offsets)
    k, v, (ke, ko) = c.packed()
    want = nsa.attention_grad(q, q, k, v, out, lse, ko, ko)
    rows = torch.zeros(600, dtype=torch.bool, device="cuda")
    for b, n in enumerate(new):
        rows[b * 200:b * 200 + n] = True
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[rows], b) and not a[~rows].any()


@pytest.mark.gpu
def test_a_recorded_step_over_growing_caches(gpu):
    """One graph serves every token: the offsets, queries and new keys change in place."""
    c = Caches([1500, 10, 2047, 900], 2400, 2, 128, BF16)
    c.take([1] * 4)
    q = torch.randn(4, 8, 128, generator=c.g, device="cuda").to(BF16)
    nsa.attention(q, c.k, c.v, c.q_offsets, c.k_offsets)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = nsa.attention(q, c.k, c.v, c.q_offsets, c.k_offsets)
    for _ in range(4):
        c.take([1] * 4)
        q.normal_(generator=c.g)
        graph.replay()
        torch.cuda.synchronize()
        c.check(q, [1] * 4, out, lse)
        again = nsa.attention(q, c.k, c.v, c.q_offsets, c.k_offsets)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
