"""Attention over packed sequences, forward and backward, against float64."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa
from oracle import block

import attention_util as ref
from ops_util import DT, host, within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    nsa.load()


def make(nq, nk, qh, kh, d, dtype, seed, shift=0, pitch=0, std=1.0):
    """Queries, keys, values and an output gradient: slices of packed tensors, `shift` elements behind an aligned address."""
    g = torch.Generator("cuda").manual_seed(seed)

    def packed(n, heads):
        width = heads * d + pitch
        t = torch.randn(n * width + shift, generator=g, device="cuda").mul_(std).to(dtype)
        return t[shift:].view(n, width)[:, :heads * d].unflatten(1, (heads, d))

    q, dout = packed(nq, qh), packed(nq, qh)
    kv = packed(nk, 2 * kh)
    return q, kv[:, :kh], kv[:, kh:], dout


def close(got, want, bound, what):
    within(host(got), host_f64(want), host_f64(bound), what)


def host_f64(t):
    return t.cpu().numpy()


def check(lq, lk, qh, kh, d, dtype, causal=True, window=0, scale=None, seed=0, shift=0, pitch=0, tail=0, back=True,
          single=False, std=1.0):
    """tail: tokens behind the last sequence, left as they were."""
    qe, qo = ref.offsets(lq)
    ke, ko = ref.offsets(lk)
    q, k, v, dout = make(qe[-1] + tail, ke[-1] + 2 * tail, qh, kh, d, dtype, seed, shift, pitch, std)
    kw = dict(causal=causal, window=window, scale=scale)
    c = float(np.float32(d ** -0.5 if scale is None else scale))
    offs = (None, None) if single else (qo, ko)
    out, lse = torch.full(q.shape, 7.0, dtype=dtype, device="cuda"), torch.full((qh, q.shape[0]), 7.0, device="cuda")
    got = nsa.attention(q, k, v, *offs, out=out, lse=lse, **kw)
    assert got[0] is out and got[1] is lse
    want, ob, wl, lb = ref.forward(q, k, v, qe, ke, causal, window, c, dtype)
    if tail:
        assert (out[qe[-1]:] == 7).all() and (lse[:, qe[-1]:] == 7).all()
    n = qe[-1]
    close(out[:n], want[:n], ob[:n], "out")
    close(lse[:, :n], wl[:, :n], lb[:, :n], "lse")
    if back:
        grads = [torch.full(t.shape, 7.0, dtype=dtype, device="cuda") for t in (q, k, v)]
        nsa.attention_grad(dout, q, k, v, out, lse, *offs, dq=grads[0], dk=grads[1], dv=grads[2], **kw)
        for g, end, name, (w, b) in zip(grads, (n, ke[-1], ke[-1]), ("dq", "dk", "dv"),
                                        ref.backward(dout, q, k, v, out, lse, qe, ke, causal, window, c, dtype)):
            assert not tail or (g[end:] == 7).all(), name
            close(g[:end], w[:end], b[:end], name)
    return q, k, v, dout, out, lse, qo, ko


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 5)])
def test_reference_is_the_oracles(dtype, causal, window):
    q, k, v, dout = make(20, 26, 4, 2, 12, dtype, 1)
    qe, ke = [0, 7, 7, 20], [0, 11, 20, 26]
    want = block.attention(*(host(t) for t in (q, k, v)), qe, ke, causal, window)
    out, _, lse, _ = ref.forward(q, k, v, qe, ke, causal, window, 12 ** -0.5, dtype)
    np.testing.assert_allclose(host_f64(out), want[0], rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(host_f64(lse), want[1], rtol=1e-10, atol=1e-12)
    got = ref.backward(dout, q, k, v, out, lse, qe, ke, causal, window, 12 ** -0.5, dtype)
    for a, b in zip(got, block.attention_grad(*(host(t) for t in (dout, q, k, v)), qe, ke, causal, window)):
        np.testing.assert_allclose(host_f64(a[0]), b, rtol=1e-9, atol=1e-12)


# lengths around the tiles of 32, 64 and 128, one token, none
@pytest.mark.parametrize("lengths", [[1], [2], [31], [32, 33], [63, 64, 65], [127, 128, 129], [0, 5, 0, 1, 0], [300], [257, 1, 40]])
@pytest.mark.parametrize("qh,kh", [(1, 1), (4, 1), (6, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_lengths(lengths, qh, kh, dtype):
    check(lengths, lengths, qh, kh, 64, dtype, seed=len(lengths))
    check(lengths, lengths, qh, kh, 128, dtype, causal=False, seed=1)


@pytest.mark.parametrize("d", [1, 5, 8, 16, 40, 64, 66, 72, 80, 96, 100, 104, 128, 136, 160, 192, 200, 250, 256])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_head_sizes(d, dtype):
    check([70, 131], [70, 131], 4, 2, d, dtype, seed=d)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 64, 100, 1000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_windows(window, dtype):
    check([200, 3, 333], [200, 3, 333], 3, 1, 64, dtype, window=window, seed=window)
    check([50, 3, 90], [200, 3, 333], 4, 2, 80, dtype, window=window, seed=window)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_more_keys_than_queries_and_fewer(causal, dtype):
    check([5, 1, 130], [300, 40, 200], 4, 2, 64, dtype, causal, seed=1)
    # rows that see nothing: out 0, lse -infinity, no part in any gradient
    check([200, 90, 3], [70, 1, 0], 4, 2, 96, dtype, causal, seed=2)
    check([0, 90], [33, 60], 2, 2, 128, dtype, causal, seed=3)
    if causal:
        check([200, 90], [70, 1], 4, 2, 64, dtype, causal, window=3, seed=4)


@pytest.mark.parametrize("lq,lk,qh,kh", [([1], [3000], 8, 2), ([1, 1, 2], [2000, 10, 5000], 4, 1), ([3, 0, 1], [1100, 1024, 1500], 5, 1),
                                         ([40], [4097], 2, 2), ([1, 1], [0, 9000], 16, 4)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_few_queries_over_long_keys(lq, lk, qh, kh, dtype):
    for d in (64, 80, 128, 256):
        assert nsa.attention_workspace_bytes(sum(lq), sum(lk), qh, kh, d, len(lq)) > 0    # in slices
        check(lq, lk, qh, kh, d, dtype, seed=d, back=d == 64)
        check(lq, lk, qh, kh, d, dtype, window=700, seed=d, back=False)


@pytest.mark.parametrize("qh,kh", [(7, 7), (5, 1), (12, 4), (32, 8), (33, 3), (64, 1)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_heads(qh, kh, dtype):
    check([45, 77], [45, 77], qh, kh, 32, dtype, seed=qh)


@pytest.mark.parametrize("shift,pitch", [(1, 0), (0, 3), (8, 8), (3, 5)])
@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_alignment(shift, pitch, d, dtype):
    check([70, 150], [70, 150], 4, 2, d, dtype, seed=1, shift=shift, pitch=pitch)
    check([1, 2], [2000, 1500], 4, 2, d, dtype, seed=1, shift=shift, pitch=pitch, back=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_behind_the_last_sequence(dtype):
    check([40, 100], [90, 100], 4, 2, 64, dtype, tail=50)
    check([1, 1], [2000, 3000], 4, 2, 128, dtype, tail=9)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_sequence_without_offsets(dtype):
    check([133], [133], 4, 2, 64, dtype, single=True)
    check([2], [5000], 4, 2, 64, dtype, single=True, back=False)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores(dtype):
    """Maxima far from zero and softmaxes of one key."""
    check([150], [150], 2, 1, 64, dtype, scale=4.0, std=1.5, seed=5)
    check([150], [150], 2, 1, 64, dtype, scale=1e-6, seed=6)


def test_long_sequences():
    check([2500, 1700], [2500, 1700], 4, 1, 128, BF16, seed=7)
    check([1500], [1500], 2, 2, 64, F32, seed=8, window=300)


def test_many_short_sequences():
    lengths = np.random.default_rng(0).integers(0, 40, 500).tolist()
    check(lengths, lengths, 2, 1, 64, BF16, seed=9)


def test_the_same_bits_again_and_for_other_strides():
    q, k, v, dout, out, lse, qo, ko = check([150, 260], [150, 260], 4, 2, 80, BF16, seed=10)
    q2, k2, v2, dout2 = make(410, 410, 4, 2, 80, BF16, 11, shift=1, pitch=3)
    for a, b in ((q2, q), (k2, k), (v2, v), (dout2, dout)):
        a.copy_(b)
    again = nsa.attention(q2, k2, v2, qo, ko)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    one, two = nsa.attention_grad(dout, q, k, v, out, lse, qo, ko), nsa.attention_grad(dout2, q2, k2, v2, out, lse, qo, ko)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_results_into_a_packed_gradient():
    q, k, v, dout, out, lse, qo, ko = check([70, 60], [70, 60], 4, 2, 64, BF16, seed=12)
    packed = torch.full((130, 8, 64), 7.0, dtype=BF16, device="cuda")
    want = nsa.attention_grad(dout, q, k, v, out, lse, qo, ko)
    nsa.attention_grad(dout, q, k, v, out, lse, qo, ko, dq=packed[:, :4], dk=packed[:, 4:6], dv=packed[:, 6:])
    assert all(torch.equal(a, b) for a, b in zip(want, (packed[:, :4], packed[:, 4:6], packed[:, 6:])))


def test_other_sequences_do_not_see_a_nan():
    qe, qo = ref.offsets([100, 60, 90])
    q, k, v, dout = (t.clone() for t in make(250, 250, 4, 2, 64, BF16, 13))
    clean = nsa.attention(q, k, v, qo, qo)
    back = nsa.attention_grad(dout, q, k, v, *clean, qo, qo)
    bad = slice(100, 160)
    for t in (q, k, v, dout):
        t[bad] = float("nan")
    k[120], v[130] = float("inf"), -float("inf")
    got = nsa.attention(q, k, v, qo, qo)
    dgot = nsa.attention_grad(dout, q, k, v, *got, qo, qo)
    for keep in (slice(0, 100), slice(160, 250)):
        assert torch.equal(got[0][keep], clean[0][keep]) and torch.equal(got[1][:, keep], clean[1][:, keep])
        assert all(torch.equal(a[keep], b[keep]) for a, b in zip(dgot, back))


def test_offsets_outside_the_tokens_stay_inside():
    """Offsets that promise more tokens than there are: every access stays within the tensors."""
    q, k, v, dout = make(64, 64, 2, 1, 64, BF16, 14)
    want = nsa.attention(q, k, v)
    off = torch.tensor([-5, 1000], dtype=torch.int32, device="cuda")
    got = nsa.attention(q, k, v, off, off)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    grads = nsa.attention_grad(dout, q, k, v, *want), nsa.attention_grad(dout, q, k, v, *want, off, off)
    assert all(torch.equal(a, b) for a, b in zip(*grads))


def test_gradient_by_differences():
    q, k, v, dout = make(40, 40, 4, 2, 32, F32, 15)
    _, qo = ref.offsets([25, 15])
    out, lse = nsa.attention(q, k, v, qo, qo)
    grads = nsa.attention_grad(dout, q, k, v, out, lse, qo, qo)
    step = 2.0 ** -7
    for which, g in enumerate(grads):
        d = torch.randn(g.shape, generator=torch.Generator("cuda").manual_seed(which), device="cuda")
        values = []
        for sign in (1, -1):
            t = [q, k, v]
            t[which] = t[which] + sign * step * d
            values.append(float((nsa.attention(*t, qo, qo)[0].double() * dout.double()).sum()))
        got, want = float((g.double() * d.double()).sum()), (values[0] - values[1]) / (2 * step)
        # the third derivative's share (step^2 / 6 of a value of this size) and the results' roundings over the step
        assert abs(got - want) <= 2e-3 * (abs(want) + float((g.double() * d.double()).norm())), which
