"""Norm of queries and keys without a rotation, in a batch with padding."""
import numpy as np
import pytest
import torch

import newton_schulz_08_amd as nsa

from ops_util import DT, dev
from test_gpu_qknorm import check_backward, check_forward
from test_ops_abi import QK, QKG, TYPE, BAD, accepted, addr, qk_shape, refused
from newton_schulz_08_amd import _lib


def test_positions_without_a_rotation_are_checked():
    lib = _lib.load()
    for f, good in ((lib.dmuon_qk_norm_rope_forward, QK), (lib.dmuon_qk_norm_rope_backward, QKG)):
        good = dict(good, shape=qk_shape(rot_dim=0, max_pos=0), rope=0)
        if not torch.cuda.is_available():
            accepted(f, good)
            accepted(f, dict(good, pos=0))
            accepted(f, dict(good, pos=0, shape=qk_shape(rot_dim=0, max_pos=0, pos_dtype=0)))
        refused(f, good, [(dict(shape=qk_shape(rot_dim=0, max_pos=0, pos_dtype=1)), TYPE), (dict(pos=addr(3) + 4), BAD)])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,qh,kh,d", [(1, 4, 2, 64), (7, 3, 1, 30), (300, 8, 2, 128), (5000, 2, 2, 16)])
@pytest.mark.parametrize("table", [False, True])   # no table, or one without columns
def test_padding_without_a_rotation(n, qh, kh, d, dt, table):
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    rng = np.random.default_rng(n)
    q, k, dq, dk = (dev(rng.standard_normal((n, h, d)), DT[dt]) for h in (qh, kh, qh, kh))
    qw, kw = (dev(rng.standard_normal(d) * 0.2 + 1.0, DT[dt]) for _ in range(2))
    pos = np.full(n, 10 ** 6)
    pos[::3] = -1 - np.arange(len(pos[::3]))
    pads = torch.from_numpy(pos < 0).cuda()
    rope = torch.empty(4, 0, device="cuda") if table else None
    eps, bare = float(np.float32(1e-6)), torch.empty(4, 0)   # the reference's table: nothing turns, signs count
    kept = [t.clone() for t in (q, k)]
    for t in (q, k, dq, dk):
        t[pads] = float("nan")
    for t in kept:
        t[pads] = 1.0                          # what the reference puts in a padding token's place is not looked at
    for kind in (torch.int64, torch.int32):
        p = dev(pos, kind)
        out = nsa.qk_norm_rope(q, k, qw, kw, p, rope)
        grads = nsa.qk_norm_rope_grad(dq, dk, q, k, qw, kw, p, rope)
        for x, w, y, g, dx, dw in zip(kept, (qw, kw), out, (dq, dk), grads[:2], grads[2:]):
            check_forward(x, w, y, pos, bare, eps, False, 0.0, DT[dt])
            check_backward(g, x, w, dx, dw, pos, bare, eps, False, 0.0, DT[dt], DT[dt])
            assert not y[pads].any() and not dx[pads].any()
    none = nsa.qk_norm_rope(*kept, qw, kw, None, None)
    assert all(torch.equal(a[~pads], b[~pads]) and b.isfinite().all() for a, b in zip(out, none))
