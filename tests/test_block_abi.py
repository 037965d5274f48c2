"""Refusals of the block operators' C entry points and their binding: nothing here
reaches a device (every call is turned down before it would)."""
import ctypes

import pytest
import torch

import newton_schulz_08_amd as nsa
from newton_schulz_08_amd import _lib

from test_ops_abi import BAD, INF, NAN, TYPE, WS, accepted, addr, refused

E = _lib


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


# ---------------------------------------------------------------- norms around a block
def bn_shape(**kw):
    s = dict(rows=6, dim=16, post_norm=1, eps=1e-6, residual_scale=1.0, weight_offset=0.0, dtype=0, branch_dtype=1, weight_dtype=1)
    s.update(kw)
    return _lib.BlockNormShape(**s)


BN_SHAPES = [(dict(dtype=2), TYPE), (dict(branch_dtype=3), TYPE), (dict(weight_dtype=7), TYPE), (dict(rows=-1), BAD),
             (dict(rows=E.DMUON_MAX_TOKENS + 1), BAD), (dict(dim=0), BAD), (dict(dim=65537), BAD), (dict(eps=-1.0), BAD),
             (dict(eps=NAN), BAD), (dict(residual_scale=INF), BAD), (dict(weight_offset=NAN), BAD)]
BN = dict(shape=bn_shape(), x=addr(0), xs=16, h=addr(1), hs=20, pre=addr(2), post=addr(3), gate=addr(4), xo=addr(5), xos=16,
          y=addr(6), ys=16, stream=None)
BNG = dict(shape=bn_shape(), dxo=addr(0), dxos=16, dy=addr(1), dys=16, x=addr(2), xs=16, h=addr(3), hs=16, pre=addr(4),
           post=addr(5), gate=addr(6), dx=addr(7), dxs=16, dh=addr(8), dhs=16, dpre=addr(9), dpost=addr(10), dgate=addr(11),
           ws=addr(12), bytes=1 << 20, stream=None)


def test_block_norm_forward(lib):
    f = lib.dmuon_block_norm_forward
    accepted(f, BN)
    accepted(f, dict(BN, xo=addr(0), y=addr(1), ys=20))                                 # in place
    accepted(f, dict(BN, pre=0, post=0, gate=0))
    accepted(f, dict(BN, shape=bn_shape(post_norm=0), post=0))
    accepted(f, dict(BN, shape=bn_shape(rows=0), x=0, h=0, xo=0, y=0))
    accepted(f, dict(BN, shape=bn_shape(rows=1), xs=0, hs=-5))                          # one row has no stride
    refused(f, BN, [(dict(shape=bn_shape(**s)), st) for s, st in BN_SHAPES])
    refused(f, BN, [
        (dict(shape=None), BAD), (dict(x=0), BAD), (dict(h=0), BAD), (dict(xo=0), BAD), (dict(y=0), BAD), (dict(xs=15), BAD),
        (dict(hs=(1 << 31) + 1), BAD), (dict(shape=bn_shape(post_norm=0)), BAD), (dict(xo=addr(0), xos=20), BAD),
        (dict(xo=addr(0) + 4), BAD), (dict(y=addr(1)), BAD), (dict(y=addr(5)), BAD), (dict(xo=addr(1)), BAD), (dict(y=addr(4)), BAD),
        (dict(x=addr(0) + 2), BAD), (dict(h=addr(1) + 1), BAD), (dict(pre=addr(2) + 1), BAD)])


def test_block_norm_backward(lib):
    f = lib.dmuon_block_norm_backward
    need = nsa.block_norm_grad_workspace_bytes(6, 16)
    accepted(f, BNG)
    accepted(f, dict(BNG, dxo=0, dxos=0))
    accepted(f, dict(BNG, dx=addr(0)))                                                  # over the incoming gradient
    accepted(f, dict(BNG, dpre=0, dpost=0, dgate=0, ws=0, bytes=0))
    accepted(f, dict(BNG, shape=bn_shape(post_norm=0), post=0, dpost=0))
    refused(f, BNG, [(dict(shape=bn_shape(**s)), st) for s, st in BN_SHAPES])
    refused(f, BNG, [
        (dict(dy=0), BAD), (dict(x=0), BAD), (dict(h=0), BAD), (dict(dx=0), BAD), (dict(dh=0), BAD), (dict(ws=0), WS),
        (dict(bytes=need - 1), WS), (dict(ws=addr(12) + 64), WS), (dict(dx=addr(2)), BAD), (dict(dh=addr(1)), BAD), (dict(dh=addr(3)), BAD),
        (dict(dpre=addr(4)), BAD), (dict(dgate=addr(10)), BAD), (dict(dxs=8), BAD), (dict(dx=addr(0), dxs=20), BAD),
        (dict(shape=bn_shape(post_norm=0), post=0), BAD), (dict(shape=bn_shape(post_norm=0), dpost=0), BAD), (dict(dpost=addr(10) + 1), BAD)])
    out = ctypes.c_size_t()
    assert lib.dmuon_block_norm_backward_workspace_bytes(bn_shape(), None) == BAD
    assert lib.dmuon_block_norm_backward_workspace_bytes(None, ctypes.byref(out)) == BAD


# ---------------------------------------------------------------- attention
def at_shape(**kw):
    s = dict(q_tokens=6, k_tokens=9, sequences=2, q_heads=4, k_heads=2, head_dim=16, causal=1, window=0, scale=0.25, dtype=1)
    s.update(kw)
    return _lib.AttentionShape(**s)


AT_SHAPES = [(dict(dtype=2), TYPE), (dict(q_tokens=-1), BAD), (dict(k_tokens=-1), BAD), (dict(q_tokens=E.DMUON_MAX_TOKENS + 1), BAD),
             (dict(sequences=0), BAD), (dict(q_heads=0), BAD), (dict(k_heads=0), BAD), (dict(q_heads=1025), BAD), (dict(q_heads=5), BAD),
             (dict(head_dim=0), BAD), (dict(head_dim=257), BAD), (dict(window=-1), BAD), (dict(window=4, causal=0), BAD),
             (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=NAN), BAD), (dict(scale=INF), BAD),
             (dict(q_tokens=1 << 22, q_heads=1024, k_heads=1), BAD), (dict(sequences=1 << 22, k_heads=8, q_heads=8), BAD)]
AT = dict(shape=at_shape(), q=addr(0), qs=128, k=addr(0) + 128, ks=128, v=addr(0) + 192, vs=128, qo=addr(1), ko=addr(2), out=addr(3),
          os=64, lse=addr(4), ws=0, bytes=0, stream=None)
ATG = dict(shape=at_shape(), dout=addr(0), dos=64, q=addr(1), qs=64, k=addr(2), ks=64, v=addr(2) + 64, vs=64, out=addr(3), os=64,
           lse=addr(4), qo=addr(5), ko=addr(6), dq=addr(7), dqs=128, dk=addr(7) + 128, dks=128, dv=addr(7) + 192, dvs=128, ws=addr(8),
           bytes=1 << 20, stream=None)


def test_attention_forward(lib):
    f = lib.dmuon_attention_forward
    packed = dict(AT, shape=at_shape(k_tokens=6))
    accepted(f, packed)
    accepted(f, dict(AT, k=addr(5), v=addr(6), ks=32, vs=40))
    accepted(f, dict(packed, shape=at_shape(k_tokens=6, sequences=1), qo=0, ko=0))
    accepted(f, dict(packed, shape=at_shape(q_tokens=0, k_tokens=0), q=0, k=0, v=0, out=0, lse=0))
    accepted(f, dict(packed, shape=at_shape(q_tokens=1, k_tokens=1), qs=0, ks=0, vs=0, os=0))
    refused(f, packed, [(dict(shape=at_shape(**s)), st) for s, st in AT_SHAPES])
    refused(f, packed, [
        (dict(shape=None), BAD), (dict(q=0), BAD), (dict(k=0), BAD), (dict(v=0), BAD), (dict(out=0), BAD), (dict(lse=0), BAD),
        (dict(qo=0), BAD), (dict(ko=0), BAD), (dict(qo=0, ko=0), BAD), (dict(qs=63), BAD), (dict(os=32), BAD), (dict(out=addr(0)), BAD),
        (dict(out=addr(0) + 128, os=128), BAD), (dict(lse=addr(1)), BAD), (dict(lse=addr(3)), BAD), (dict(q=addr(0) + 1), BAD),
        (dict(qo=addr(1) + 2), BAD), (dict(lse=addr(4) + 2), BAD)])
    few = dict(AT, shape=at_shape(q_tokens=2, k_tokens=8000), k=addr(5), v=addr(6), ks=32, vs=32)   # in slices
    need = nsa.attention_workspace_bytes(2, 8000, 4, 2, 16, 2)
    assert need > 0
    accepted(f, dict(few, ws=addr(9), bytes=need))
    refused(f, few, [(dict(ws=0), WS), (dict(ws=addr(9), bytes=need - 1), WS), (dict(ws=addr(9) + 16, bytes=need), WS),
                     (dict(ws=addr(3), bytes=need), BAD)])
    assert lib.dmuon_attention_workspace_bytes(at_shape(), None) == BAD


def test_attention_backward(lib):
    f = lib.dmuon_attention_backward
    packed = dict(ATG, shape=at_shape(k_tokens=6))
    need = nsa.attention_grad_workspace_bytes(6, 4)
    accepted(f, packed)
    accepted(f, dict(ATG, dk=addr(9), dks=32, dv=addr(10), dvs=32))
    refused(f, packed, [(dict(shape=at_shape(**s)), st) for s, st in AT_SHAPES])
    refused(f, packed, [
        (dict(dout=0), BAD), (dict(q=0), BAD), (dict(k=0), BAD), (dict(v=0), BAD), (dict(out=0), BAD), (dict(lse=0), BAD), (dict(dq=0), BAD),
        (dict(dk=0), BAD), (dict(dv=0), BAD), (dict(ws=0), WS), (dict(bytes=need - 1), WS), (dict(ws=addr(8) + 8), WS),
        (dict(dq=addr(0), dqs=64), BAD), (dict(dk=addr(2), dks=64), BAD), (dict(dv=addr(7) + 128), BAD), (dict(dks=31), BAD),
        (dict(dq=addr(8)), BAD), (dict(qo=0), BAD), (dict(ko=addr(7)), BAD), (dict(dv=addr(7) + 193), BAD)])


# ---------------------------------------------------------------- gated feed-forward
def ff_shape(**kw):
    s = dict(tokens=100, dim=64, hidden=80, activation=0, dtype=1)
    s.update(kw)
    return _lib.GatedFfnShape(**s)


FF_SHAPES = [(dict(dtype=2), TYPE), (dict(tokens=-1), BAD), (dict(tokens=E.DMUON_MAX_TOKENS + 1), BAD), (dict(dim=0), BAD),
             (dict(dim=65537), BAD), (dict(hidden=0), BAD), (dict(hidden=65537), BAD), (dict(activation=2), BAD), (dict(activation=-1), BAD)]
FF = dict(shape=ff_shape(), x=addr(0), xs=64, wg=addr(1), wu=addr(2), h=addr(3), hs=80, ws=0, bytes=0, stream=None)
FFG = dict(shape=ff_shape(), dh=addr(0), dhs=80, x=addr(1), xs=64, wg=addr(2), wu=addr(3), dx=addr(4), dxs=64, dwg=addr(5), dwu=addr(6),
           ws=addr(7), bytes=1 << 26, stream=None)


def test_gated_ffn_forward(lib):
    f = lib.dmuon_gated_ffn_forward
    accepted(f, FF)
    accepted(f, dict(FF, shape=ff_shape(tokens=0), x=0, wg=0, wu=0, h=0))
    accepted(f, dict(FF, shape=ff_shape(tokens=5), xs=65))                 # few tokens take no copies
    accepted(f, dict(FF, shape=ff_shape(dtype=0, dim=63)))
    refused(f, FF, [(dict(shape=ff_shape(**s)), st) for s, st in FF_SHAPES])
    refused(f, FF, [
        (dict(shape=None), BAD), (dict(x=0), BAD), (dict(wg=0), BAD), (dict(wu=0), BAD), (dict(h=0), BAD), (dict(xs=63), BAD), (dict(hs=79), BAD),
        (dict(h=addr(0)), BAD), (dict(h=addr(2)), BAD)])
    need = nsa.gated_ffn_workspace_bytes(100, 64, 80, torch.bfloat16, aligned=False)
    assert need > 0 and nsa.gated_ffn_workspace_bytes(100, 64, 80, torch.bfloat16) == 0
    assert nsa.gated_ffn_workspace_bytes(100, 72, 80, torch.bfloat16) > 0
    for change in (dict(xs=65), dict(x=addr(0) + 2), dict(wu=addr(2) + 2), dict(xs=(1 << 22) + 8)):
        refused(f, FF, [(change, WS), (dict(change, ws=addr(9), bytes=need - 1), WS)])
        accepted(f, dict(FF, **change, ws=addr(9), bytes=need))
    refused(f, dict(FF, xs=65, ws=addr(9), bytes=need), [(dict(ws=addr(9) + 64), WS), (dict(ws=addr(3)), BAD), (dict(x=addr(0) + 1), BAD),
                                                         (dict(wg=addr(1) + 1), BAD)])
    assert lib.dmuon_gated_ffn_workspace_bytes(ff_shape(), 1, None) == BAD


def test_gated_ffn_backward(lib):
    f = lib.dmuon_gated_ffn_backward
    accepted(f, FFG)
    accepted(f, dict(FFG, shape=ff_shape(tokens=0), dh=0, x=0, wg=0, wu=0, dx=0))
    refused(f, FFG, [(dict(shape=ff_shape(**s)), st) for s, st in FF_SHAPES])
    need = nsa.gated_ffn_grad_workspace_bytes(100, 64, 80, torch.bfloat16)
    refused(f, FFG, [
        (dict(dh=0), BAD), (dict(x=0), BAD), (dict(wg=0), BAD), (dict(wu=0), BAD), (dict(dx=0), BAD), (dict(dwg=0), BAD), (dict(dwu=0), BAD),
        (dict(ws=0), WS), (dict(bytes=need - 1), WS), (dict(ws=addr(7) + 32), WS), (dict(dx=addr(1)), BAD), (dict(dwg=addr(2)), BAD),
        (dict(dwu=addr(5)), BAD), (dict(dx=addr(7)), BAD), (dict(dxs=60), BAD), (dict(dhs=79), BAD), (dict(dwu=addr(6) + 1), BAD),
        (dict(shape=ff_shape(tokens=0), dwg=0), BAD)])


# ---------------------------------------------------------------- the binding
def test_binding_refuses_host_tensors_and_wrong_types():
    t, h = torch.zeros(4, 8), torch.zeros(4, 2, 8)
    with pytest.raises(ValueError, match="device"):
        nsa.block_norm(t, t)
    with pytest.raises(ValueError, match="device"):
        nsa.block_norm_grad(None, t, t, t)
    with pytest.raises(ValueError, match="device"):
        nsa.attention(h, h, h)
    with pytest.raises(ValueError, match="device"):
        nsa.attention_grad(h, h, h, h, h, t)
    with pytest.raises(ValueError, match="device"):
        nsa.gated_ffn(t, t, t)
    with pytest.raises(ValueError, match="activation"):
        nsa.gated_ffn_grad(t, t, t, t, "relu")
    for f in (nsa.block_norm, lambda a, b: nsa.attention(a, b, b), lambda a, b: nsa.gated_ffn(a, b, b)):
        with pytest.raises(TypeError):
            f("x", t)


def test_launches_beyond_a_grid(lib):
    """As many tiles as a launch cannot hold; one sequence, or one token, fewer is taken as far as the operands."""
    wide = dict(AT, shape=at_shape(q_tokens=0, k_tokens=0, sequences=1 << 22, q_heads=4, k_heads=4), q=0, k=0, v=0, out=0, lse=0)
    refused(lib.dmuon_attention_forward, dict(AT, shape=at_shape(k_tokens=6)), [(wide, BAD)])
    accepted(lib.dmuon_attention_forward, dict(wide, shape=at_shape(q_tokens=0, k_tokens=0, sequences=(1 << 22) - 1, q_heads=4, k_heads=4),
                                               qo=addr(1), ko=addr(1) + (1 << 25), stream=None))
    many = E.DMUON_MAX_TOKENS
    refused(lib.dmuon_gated_ffn_forward, FF, [(dict(shape=ff_shape(tokens=many, hidden=65536), hs=65536), BAD),
                                              (dict(shape=ff_shape(tokens=many, hidden=8192, dtype=0), hs=8192), BAD)])
    refused(lib.dmuon_gated_ffn_backward, FFG, [(dict(shape=ff_shape(tokens=many, dim=65536, hidden=16, dtype=0), xs=65536, dxs=65536), BAD)])
