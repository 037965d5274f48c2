"""dq of keys that have much in common.

A row of dS adds up to 0, so the keys' common part cancels in dq = dS K, but not
in the errors of dS: rounded to bf16 once, it alone would be further off than
all of dq's rounding.  The bound here leaves no room for that; it takes dS as
two bf16 numbers, which hold it to 2^-16."""
import pytest
import torch

import newton_schulz_08_amd as nsa
import attention_util as ref
from ops_util import U32, half_step, host, within

F32, BF16 = torch.float32, torch.bfloat16


def make(lq, lk, qh, kh, d, seed, device):
    """Keys of a head share a vector four times as long as any other operand, eight times what sets them apart."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, dout = r(sum(lq), qh, d), r(sum(lq), qh, d)
    k, v = 4 * r(1, kh, d) + 0.5 * r(sum(lk), kh, d), r(sum(lk), kh, d)
    return [t.to(BF16).to(device) for t in (q, k, v, dout)]


def dq(dout, q, k, v, o, lse, qe, ke, causal, window, dtype, form=lambda ds: ds):
    """(dq, bound) as attention_util.backward forms them, but with dS held to 2^-16 where it holds it to a half step.
    form: what becomes of dS in front of its product."""
    dout, q, k, v, o, lse = (t.double() for t in (dout, q, k, v, o, lse))
    (n, qh, d), kh = q.shape, k.shape[1]
    scale, half, want, bound = d ** -0.5, half_step(dtype), torch.zeros_like(q), torch.zeros_like(q)
    held = 2.0 ** -16 if dtype == BF16 else 0.0
    for rq, rk in ref.spans(qe, ke):
        lq, lk = rq.stop - rq.start, rk.stop - rk.start
        if lq == 0 or lk == 0:
            continue
        see = ref.visible(lq, lk, causal, window, q.device)
        for h in range(qh):
            kv = h // (qh // kh)
            qq, kk, vv, dd, oo, s = q[rq, h], k[rk, kv], v[rk, kv], dout[rq, h], o[rq, h], lse[h, rq][:, None]
            p = torch.exp(qq @ kk.T * scale - s).masked_fill(~see, 0.0)
            rel = U32 * ((d + 24) * (qq.abs() @ kk.T.abs() * scale) + 4 * s.abs().masked_fill(torch.isinf(s), 0.0) + 8)
            dp, delta = dd @ vv.T, (dd * oo).sum(1, keepdim=True)
            near = U32 * (d + 24) * (dd.abs() @ vv.abs().T + (dd * oo).abs().sum(1, keepdim=True))
            ds = p * (dp - delta)
            e = p * (rel * (dp - delta).abs() * 2 + near * 2) + (held + 4 * U32) * (ds.abs() + 2 * p * near) + ref.TINY * (
                1 + dp.abs() + delta.abs())
            want[rq, h] = form(ds) @ kk * scale
            bound[rq, h] = (e + (lk + 64) * U32 * ds.abs()) @ kk.abs() * scale * (1 + 4 * U32)
    return want, bound + ref.TINY + half * (want.abs() + bound)


def once(ds):
    return ds.to(BF16).double()


def twice(ds):
    return once(ds) + once(ds - once(ds))


CASES = [([16, 9], [16, 9], 4, 2, 16, True, 0), ([24], [40], 3, 1, 16, False, 0), ([40], [40], 2, 2, 32, True, 12)]


@pytest.mark.parametrize("lq,lk,qh,kh,d,causal,window", CASES)
def test_the_bound_tells_one_rounding_from_two(lq, lk, qh, kh, d, causal, window):
    q, k, v, dout = make(lq, lk, qh, kh, d, 1, "cpu")
    (qe, _), (ke, _) = ref.offsets(lq, "cpu"), ref.offsets(lk, "cpu")
    o, _, lse, _ = ref.forward(q, k, v, qe, ke, causal, window, d ** -0.5, BF16)
    args = dout, q, k, v, o.to(BF16), lse.float(), qe, ke, causal, window, BF16
    want, bound = dq(*args)
    two, one = dq(*args, form=twice)[0].to(BF16).double(), dq(*args, form=once)[0].to(BF16).double()
    assert ((two - want).abs() <= bound).all()
    assert ((one - want).abs() > bound).double().mean() > 0.05
    # and by the whole: dq's own rounding is at most a half step of it, and of its error
    half = half_step(BF16)
    assert (two - want).norm() <= 1.1 * half * want.norm() < (one - want).norm()


@pytest.mark.gpu
@pytest.mark.parametrize("lq,lk,qh,kh,d,causal,window", CASES + [([70, 131], [70, 131], 4, 2, 64, True, 0), ([50], [200], 4, 1, 96, True, 0),
                                                                ([150], [150], 2, 2, 128, True, 60), ([90], [90], 2, 1, 256, False, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_common_keys_cancel(lq, lk, qh, kh, d, causal, window, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    for shift in (0, 1):      # whole runs of 16 bytes, and none
        q, k, v, dout = (t.to(dtype) for t in make(lq, lk, qh, kh, d, 1, "cuda"))
        if shift:
            q, k, v, dout = (torch.cat([t.flatten()[:1], t.flatten()])[1:].view(t.shape) for t in (q, k, v, dout))
        (qe, qo), (ke, ko) = ref.offsets(lq), ref.offsets(lk)
        out, lse = nsa.attention(q, k, v, qo, ko, causal=causal, window=window)
        got = nsa.attention_grad(dout, q, k, v, out, lse, qo, ko, causal=causal, window=window)[0]
        want, bound = dq(dout, q, k, v, out, lse, qe, ke, causal, window, dtype)
        within(host(got), want.cpu().numpy(), bound.cpu().numpy(), "dq")
