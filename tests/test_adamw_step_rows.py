"""AdamWStep with a table's gradient as rows beside dense ones: all of its
parameters take a step, or none does.  The checks alone need no GPU."""
import pytest
import torch

import newton_schulz_08_amd as nsa
from newton_schulz_08_amd import _lib

from test_ops_abi import ADAM, BAD, INF, NAN, TYPE, addr, refused

CHECK = {k: v for k, v in ADAM.items() if k != "stream"}


def test_checks_without_a_device():
    lib = _lib.load()
    assert lib.dmuon_adamw_rows_check(*CHECK.values()) == _lib.DMUON_OK
    assert lib.dmuon_adamw_rows_check(*dict(CHECK, grad=0, n=0).values()) == _lib.DMUON_OK
    refused(lib.dmuon_adamw_rows_check, CHECK, [
        (dict(dt=2), TYPE), (dict(rows=0), BAD), (dict(dim=0), BAD), (dict(dim=_lib.DMUON_MAX_DIM + 1), BAD), (dict(n=-1), BAD),
        (dict(n=_lib.DMUON_MAX_TOKENS + 1), BAD), (dict(step=0), BAD), (dict(lr=NAN), BAD), (dict(wd=INF), BAD),
        (dict(eps=-1.0), BAD), (dict(b1=1.0), BAD), (dict(b2=NAN), BAD), (dict(param=0), BAD), (dict(grad=0), BAD),
        (dict(index=0), BAD), (dict(m=addr(4)), BAD), (dict(grad=addr(0) + 4), BAD), (dict(param=addr(0) + 1), BAD)])


def make():
    g = torch.Generator("cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    params = [r(300), r(20, 16), r(50, 16)]
    index = torch.full((50,), -1, dtype=torch.int32, device="cuda")
    index[torch.tensor([3, 7, 49], device="cuda")] = torch.arange(3, dtype=torch.int32, device="cuda")
    return params, [r(300), (r(3, 16), torch.full((20,), -1, dtype=torch.int32, device="cuda")), (r(3, 16), index)]


@pytest.mark.gpu
def test_a_refused_call_changes_nothing():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    params, grads = make()
    step = nsa.AdamWStep(params, grads, lr=0.1)
    step()
    state = lambda: [*step.params, *step.exp_avg, *step.exp_avg_sq]  # noqa: E731
    before = [t.clone() for t in state()]
    rows, index = grads[2]
    bad = [(rows.double(), index), (rows[:, :8].contiguous(), index), (rows, index.long()), (rows, index[:49]),
           (rows.cpu(), index), (rows.T.contiguous().T, index), (rows, None), (step.params[2][:3], index)]
    for pair in bad:
        step.grads[2] = pair
        with pytest.raises((TypeError, ValueError, _lib.DmuonError)):
            step()
        torch.cuda.synchronize()
        assert step.step == 1 and all(torch.equal(a, b) for a, b in zip(state(), before)), pair
    step.grads[2] = grads[2]
    step.lr = float("nan")
    with pytest.raises(_lib.DmuonError):
        step()
    step.lr, step.grads[0] = 0.1, grads[0].bfloat16()
    with pytest.raises(ValueError):
        step()
    torch.cuda.synchronize()
    assert step.step == 1 and all(torch.equal(a, b) for a, b in zip(state(), before))
    # the retry is the step that was refused
    step.grads[0] = grads[0]
    step()
    fresh = make()[0]
    again = nsa.AdamWStep(fresh, grads, lr=0.1)
    again()
    again()
    assert step.step == again.step == 2
    assert all(torch.equal(a, b) for a, b in zip(state(), [*again.params, *again.exp_avg, *again.exp_avg_sq]))
    assert not torch.equal(step.params[2], before[2])


@pytest.mark.gpu
def test_gradients_may_change_their_form():
    """The lists are read at each call: a table's gradient as rows now, dense later."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    params, grads = make()
    dense = torch.zeros(50, 16, device="cuda")
    dense[torch.tensor([3, 7, 49], device="cuda")] = grads[2][0]
    other = [p.clone() for p in params]
    a = nsa.AdamWStep(params, [grads[0], grads[1], dense])
    b = nsa.AdamWStep(other, [grads[0], grads[1], dense])
    for pair in ((grads[2], dense), (dense, grads[2])):
        a.grads[2], b.grads[2] = pair
        a()
        b()
    assert all(torch.equal(x, y) for x, y in zip(params, other))


def test_a_row_gradient_is_a_pair():
    with pytest.raises(ValueError, match="pair"):
        nsa.AdamWStep([torch.zeros(2, 2)], [(torch.zeros(2, 2),)])
    with pytest.raises(ValueError, match="length"):
        nsa.AdamWStep([torch.zeros(2, 2)], [])
