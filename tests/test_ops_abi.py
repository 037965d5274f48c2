"""Refusals of the operators' C entry points and their binding: nothing here
reaches a device (every call is turned down before it would)."""
import ctypes

import pytest
import torch

import newton_schulz_08_amd as nsa
from newton_schulz_08_amd import _lib

E = _lib
A = 0x100000   # made-up, well separated addresses
BAD, TYPE, WS = E.DMUON_ERR_INVALID_ARG, E.DMUON_ERR_UNSUPPORTED_DTYPE, E.DMUON_ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def addr(k):
    return A * 0x1000 * (k + 1)


def refused(fn, good, changes):
    """Each change to the good arguments is refused with its status."""
    names = list(good)
    for change, status in changes:
        args = dict(good, **change)
        assert set(args) == set(names), change
        got = fn(*(args[n] for n in names))
        assert got == status, (change, got, _lib.last_error())
        assert _lib.last_error()


def accepted(fn, args):
    """The arguments pass every check (without a GPU the device check follows;
    with one this must not be called: the addresses are made up)."""
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only without a GPU")
    assert fn(*args.values()) == E.DMUON_ERR_NO_DEVICE


EMBED = dict(table=addr(0), vocab=10, dim=8, tdt=0, tokens=addr(1), n=4, kdt=2, scale=1.0, out=addr(2), odt=1, stream=None)


def test_embedding_forward(lib):
    accepted(lib.dmuon_embedding_forward, EMBED)
    accepted(lib.dmuon_embedding_forward, dict(EMBED, n=0, table=0, tokens=0, out=0))
    refused(lib.dmuon_embedding_forward, EMBED, [
        (dict(tdt=2), TYPE), (dict(odt=7), TYPE), (dict(kdt=0), TYPE), (dict(vocab=0), BAD), (dict(dim=0), BAD),
        (dict(dim=65537), BAD), (dict(n=-1), BAD), (dict(n=E.DMUON_MAX_TOKENS + 1), BAD),
        (dict(vocab=E.DMUON_MAX_VOCAB + 1), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD), (dict(table=0), BAD),
        (dict(tokens=0), BAD), (dict(out=0), BAD), (dict(out=addr(0)), BAD), (dict(out=addr(0) + 300), BAD),
        (dict(out=addr(1)), BAD), (dict(table=addr(0) + 2), BAD), (dict(tokens=addr(1) + 2), BAD), (dict(out=addr(2) + 1), BAD)])


PLAN = dict(tokens=addr(0), n=5000, kdt=3, vocab=100, order=addr(1), slot=addr(2), rows=addr(3), index=addr(4),
            count=addr(5), ws=addr(6), bytes=1 << 30, stream=None)


def test_embedding_plan(lib):
    accepted(lib.dmuon_embedding_plan, PLAN)
    accepted(lib.dmuon_embedding_plan, dict(PLAN, n=100, ws=0, bytes=0))   # small batches need none
    need = nsa.embedding_plan_workspace_bytes(5000, 100)
    refused(lib.dmuon_embedding_plan, PLAN, [
        (dict(kdt=1), TYPE), (dict(n=-1), BAD), (dict(vocab=0), BAD), (dict(tokens=0), BAD), (dict(order=0), BAD),
        (dict(slot=0), BAD), (dict(rows=0), BAD), (dict(index=0), BAD), (dict(count=0), BAD), (dict(ws=0), WS),
        (dict(bytes=need - 1), WS), (dict(ws=addr(6) + 64), WS), (dict(slot=addr(1)), BAD), (dict(order=addr(0)), BAD),
        (dict(count=addr(4) + 396), BAD), (dict(rows=addr(3) + 2), BAD), (dict(index=addr(6)), BAD)])
    out = ctypes.c_size_t()
    assert lib.dmuon_embedding_plan_workspace_bytes(1, 1, None) == BAD
    assert lib.dmuon_embedding_plan_workspace_bytes(-1, 1, ctypes.byref(out)) == BAD
    assert nsa.embedding_plan_workspace_bytes(4096, 1000) == 0 and nsa.embedding_plan_workspace_bytes(0, 1) == 0


GRAD = dict(dout=addr(0), n=5000, dim=64, ddt=1, scale=1.0, order=addr(1), slot=addr(2), rows=addr(3), index=addr(4),
            count=addr(5), vocab=100, form=0, grad=addr(7), gdt=0, ws=addr(6), bytes=1 << 30, stream=None)


def test_embedding_backward(lib):
    for form in (0, 1, 2):
        accepted(lib.dmuon_embedding_backward, dict(GRAD, form=form))
    need = nsa.embedding_grad_workspace_bytes(5000, 64, torch.bfloat16)
    assert need > 0 and nsa.embedding_grad_workspace_bytes(1, 64, torch.float32) == 0
    refused(lib.dmuon_embedding_backward, GRAD, [
        (dict(ddt=2), TYPE), (dict(gdt=3), TYPE), (dict(form=3), BAD), (dict(form=-1), BAD), (dict(scale=INF), BAD),
        (dict(n=-3), BAD), (dict(dim=0), BAD), (dict(vocab=0), BAD), (dict(dout=0), BAD), (dict(order=0), BAD),
        (dict(slot=0), BAD), (dict(rows=0), BAD), (dict(index=0), BAD), (dict(count=0), BAD), (dict(grad=0), BAD),
        (dict(ws=0), WS), (dict(bytes=need - 1), WS), (dict(ws=addr(6) + 4), WS), (dict(grad=addr(0)), BAD),
        (dict(grad=addr(4)), BAD), (dict(grad=addr(6)), BAD), (dict(dout=addr(0) + 1), BAD)])


ADAM = dict(param=addr(0), grad=addr(1), n=3, index=addr(2), m=addr(3), v=addr(4), rows=10, dim=8, dt=1, step=1, lr=1e-3,
            b1=0.9, b2=0.999, eps=1e-8, wd=0.0, stream=None)


def test_adamw_rows(lib):
    accepted(lib.dmuon_adamw_rows_step, ADAM)
    accepted(lib.dmuon_adamw_rows_step, dict(ADAM, grad=0, n=0))
    refused(lib.dmuon_adamw_rows_step, ADAM, [
        (dict(dt=2), TYPE), (dict(rows=0), BAD), (dict(dim=0), BAD), (dict(n=-1), BAD), (dict(step=0), BAD),
        (dict(lr=NAN), BAD), (dict(wd=INF), BAD), (dict(eps=-1.0), BAD), (dict(b1=1.0), BAD), (dict(b2=-0.1), BAD),
        (dict(b1=NAN), BAD), (dict(param=0), BAD), (dict(grad=0), BAD), (dict(index=0), BAD), (dict(m=0), BAD),
        (dict(v=0), BAD), (dict(m=addr(4)), BAD), (dict(grad=addr(0)), BAD), (dict(param=addr(0) + 1), BAD),
        (dict(m=addr(3) + 2), BAD), (dict(index=addr(3)), BAD)])


LOSS = dict(logits=addr(0), n=4, vocab=80000, stride=80008, dt=1, index=addr(1), idt=3, teacher=addr(2), k=5, labels=addr(3),
            t=2.0, kd=1.0, ce=0.5, w=addr(4), scale=1.0, losses=addr(5), dz=addr(6), dstride=80000, ws=addr(7), bytes=1 << 20,
            stream=None)


def test_distill_loss(lib):
    accepted(lib.dmuon_distill_loss, LOSS)
    accepted(lib.dmuon_distill_loss, dict(LOSS, dz=addr(0), dstride=80008))              # in place
    accepted(lib.dmuon_distill_loss, dict(LOSS, dz=0, dstride=0, labels=0, ce=0.0, w=0))
    accepted(lib.dmuon_distill_loss, dict(LOSS, k=0, kd=0.0, index=0, teacher=0))
    accepted(lib.dmuon_distill_loss, dict(LOSS, n=1, stride=0, dstride=0))
    accepted(lib.dmuon_distill_loss, dict(LOSS, vocab=4096, ws=0, bytes=0))   # a block takes the whole row
    need = nsa.distill_loss_workspace_bytes(4, 80000)
    assert need > 0
    refused(lib.dmuon_distill_loss, LOSS, [
        (dict(dt=2), TYPE), (dict(idt=0), TYPE), (dict(n=-1), BAD), (dict(vocab=0), BAD), (dict(k=-1), BAD),
        (dict(k=1025), BAD), (dict(t=0.0), BAD), (dict(t=-1.0), BAD), (dict(t=NAN), BAD), (dict(t=INF), BAD), (dict(t=9e-7), BAD), (dict(t=1.1e6), BAD),
        (dict(kd=NAN), BAD), (dict(ce=INF), BAD), (dict(scale=NAN), BAD), (dict(k=0), BAD), (dict(labels=0), BAD),
        (dict(stride=79999), BAD), (dict(dstride=79999), BAD), (dict(logits=0), BAD), (dict(index=0), BAD),
        (dict(teacher=0), BAD), (dict(losses=0), BAD), (dict(ws=0), WS), (dict(bytes=need - 1), WS),
        (dict(dz=addr(0)), BAD), (dict(dz=addr(0) + 2, dstride=80008), BAD), (dict(losses=addr(4)), BAD),
        (dict(logits=addr(0) + 1), BAD), (dict(labels=addr(3) + 4), BAD), (dict(ws=addr(7) + 8), WS)])


def qk_shape(**kw):
    s = dict(tokens=6, q_heads=4, k_heads=2, head_dim=16, rot_dim=8, interleaved=0, max_pos=100, eps=1e-6,
             weight_offset=0.0, dtype=1, weight_dtype=0, pos_dtype=3)
    s.update(kw)
    return _lib.QkShape(**s)


QK = dict(shape=qk_shape(), q=addr(0), qs=128, k=addr(0) + 128, ks=128, qw=addr(1), kw=addr(2), pos=addr(3),
          rope=addr(4), qo=addr(5), qos=64, ko=addr(6), kos=32, stream=None)
QKG = dict(shape=qk_shape(), dqo=addr(7), dqos=64, dko=addr(8), dkos=32, q=addr(0), qs=128, k=addr(0) + 128, ks=128,
           qw=addr(1), kw=addr(2), pos=addr(3), rope=addr(4), dq=addr(5), dqs=96, dk=addr(5) + 128, dks=96,
           dqw=addr(6), dkw=addr(9), ws=addr(10), bytes=1 << 20, stream=None)

SHAPES = [(dict(dtype=3), TYPE), (dict(weight_dtype=2), TYPE), (dict(pos_dtype=1), TYPE), (dict(tokens=-1), BAD),
          (dict(q_heads=-1), BAD), (dict(k_heads=1025), BAD), (dict(q_heads=0, k_heads=0), BAD), (dict(head_dim=0), BAD),
          (dict(head_dim=513), BAD), (dict(rot_dim=18), BAD), (dict(rot_dim=7), BAD), (dict(rot_dim=-2), BAD),
          (dict(eps=-1e-6), BAD), (dict(eps=NAN), BAD), (dict(weight_offset=INF), BAD), (dict(max_pos=0), BAD)]


def test_qk_forward(lib):
    f = lib.dmuon_qk_norm_rope_forward
    accepted(f, QK)
    accepted(f, dict(QK, qo=QK["q"], qos=128, ko=QK["k"], kos=128))          # in place, one packed buffer
    accepted(f, dict(QK, shape=qk_shape(tokens=1), qo=QK["q"], qos=64, ko=QK["k"], kos=32))   # one token has no stride
    accepted(f, dict(QK, qw=0, kw=0))
    accepted(f, dict(QK, shape=qk_shape(rot_dim=0), pos=0, rope=0))
    accepted(f, dict(QK, shape=qk_shape(k_heads=0), k=0, ks=0, ko=0, kos=0))
    refused(f, QK, [(dict(shape=qk_shape(**s)), st) for s, st in SHAPES])
    refused(f, QK, [
        (dict(shape=None), BAD), (dict(q=0), BAD), (dict(k=0), BAD), (dict(qo=0), BAD), (dict(ko=0), BAD), (dict(pos=0), BAD),
        (dict(rope=0), BAD), (dict(qs=63), BAD), (dict(kos=31), BAD), (dict(qo=QK["q"]), BAD), (dict(ko=addr(5)), BAD),
        (dict(ko=QK["k"], kos=64), BAD), (dict(qo=QK["q"] + 2, qos=128), BAD), (dict(qo=QK["k"], qos=128), BAD),
        (dict(q=addr(0) + 1), BAD), (dict(qw=addr(1) + 2), BAD), (dict(pos=addr(3) + 4), BAD), (dict(qo=addr(4)), BAD)])


def test_qk_backward(lib):
    f = lib.dmuon_qk_norm_rope_backward
    accepted(f, QKG)
    accepted(f, dict(QKG, dq=addr(7), dqs=64, dk=addr(8), dks=32))           # over the incoming gradients
    accepted(f, dict(QKG, dqw=0, dkw=0, ws=0, bytes=0))                      # no sums, no workspace
    accepted(f, dict(QKG, dqw=0))
    refused(f, QKG, [(dict(shape=qk_shape(**s)), st) for s, st in SHAPES])
    need = nsa.qk_norm_rope_grad_workspace_bytes(6, 4, 2, 16)
    refused(f, QKG, [
        (dict(dqo=0), BAD), (dict(dko=0), BAD), (dict(q=0), BAD), (dict(dq=0), BAD), (dict(dk=0), BAD), (dict(ws=0), WS),
        (dict(bytes=need - 1), WS), (dict(ws=addr(10) + 128), WS), (dict(dqw=addr(9)), BAD), (dict(dqw=addr(1)), BAD),
        (dict(dk=addr(5) + 64), BAD), (dict(dqs=32), BAD), (dict(dkos=2), BAD), (dict(dq=addr(4)), BAD),
        (dict(dqw=addr(6) + 1), BAD)])


def test_binding_refuses_host_tensors_and_wrong_types():
    t = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device"):
        nsa.embedding(t, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="device"):
        nsa.embedding_plan(torch.zeros(3, dtype=torch.int64), 4)
    with pytest.raises(ValueError, match="form"):
        nsa.embedding_grad(None, t, form="sparse")
    with pytest.raises(ValueError, match="device"):
        nsa.adamw_rows_step_(t, t, t, t, t, 1)
    with pytest.raises(ValueError, match="device"):
        nsa.distill_loss(t, None, None)
    with pytest.raises(ValueError, match="device"):
        nsa.qk_norm_rope(t[None], t[None], None, None, None, None)
    with pytest.raises(TypeError):
        nsa.embedding("table", t)
