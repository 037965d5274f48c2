"""Python binding of the operators between a decoder block's projections: norms
around the block, attention over packed sequences, gated feed-forward.

Everything that ops.py says of its calls (allocation, devices, streams, graphs,
autograd) holds here too.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .api import _alloc, dtype_code
from .ops import _c_int, _heads, _query, _rows, _run, _tensor, _workspace

_ACTIVATIONS = {"silu": _lib.DMUON_ACT_SILU, "gelu": _lib.DMUON_ACT_GELU}


def _row(t, name: str, like: Optional[torch.Tensor] = None) -> Tuple[int, int]:
    """(address, row stride) of a 2-D device tensor with contiguous rows."""
    stride = _rows(t, name, like)
    return t.data_ptr(), stride


def _out(out, name: str, like: torch.Tensor, stream) -> Tuple[torch.Tensor, int, int]:
    """(tensor, address, row stride) of a result like the 2-D `like`, given or allocated here."""
    if out is None:
        new = like.new_empty
        out = new(like.shape) if stream is None else _alloc(stream, new, like.shape)
        return out, out.data_ptr(), like.shape[1]
    return out, *_row(out, name, like)


# ---------------------------------------------------------------- norms around a block
def _bn_args(x, h, pre_weight, post_weight, gate, eps, residual_scale, weight_offset, post_norm):
    """(device index, dmuon_block_norm_shape, [x, stride, h, stride], [gains and gate])."""
    head = [*_row(x, "x"), *_row(h, "h")]
    dev, (n, dim) = x.get_device(), x.shape
    if h.shape != x.shape or h.get_device() != dev:
        raise ValueError(f"h is {tuple(h.shape)} on {h.device}, x {tuple(x.shape)} on {x.device}")
    weights, wdt = [], None
    for w, name in ((pre_weight, "pre_weight"), (post_weight, "post_weight"), (gate, "gate")):
        if w is None:
            weights.append(0)
        else:
            weights.append(_tensor(w, name, dev, wdt, (dim,)))
            wdt = w.dtype
    s = _lib.BlockNormShape(n, dim, 1 if post_norm else 0, eps, residual_scale, weight_offset, dtype_code(x.dtype),
                            dtype_code(h.dtype), dtype_code(wdt or h.dtype))
    return dev, s, head, weights


def block_norm(x: torch.Tensor, h: torch.Tensor, pre_weight: Optional[torch.Tensor] = None,
               post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, *, eps: float = 1e-6,
               residual_scale: float = 1.0, weight_offset: float = 0.0, post_norm: bool = False,
               x_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """dmuon_block_norm_forward: (x_out, y), the residual stream behind a block
    and its norm in front of the next one.

    x (rows, dim): the stream; h (rows, dim): the block's output, normed first
    with `post_norm`, times its gain, `gate` (dim) and residual_scale, then
    added.  y has h's type.  Gains count as weight_offset + weight; None is a
    factor of 1.  x_out may be x, y may be h.  Outside autograd: the gradients
    are block_norm_grad's."""
    dev, s, head, weights = _bn_args(x, h, pre_weight, post_weight, gate, eps, residual_scale, weight_offset, post_norm)
    x_out, *xo = _out(x_out, "x_out", x, stream)
    y, *yo = _out(y, "y", h, stream)
    _run("dmuon_block_norm_forward", dev, stream, s, *head, *weights, *xo, *yo)
    return x_out, y


def block_norm_grad_workspace_bytes(rows: int, dim: int) -> int:
    return _query("dmuon_block_norm_backward_workspace_bytes", _lib.BlockNormShape(rows=rows, dim=dim))


def block_norm_grad(dx_out: Optional[torch.Tensor], dy: torch.Tensor, x_out: torch.Tensor, h: torch.Tensor,
                    pre_weight: Optional[torch.Tensor] = None, post_weight: Optional[torch.Tensor] = None,
                    gate: Optional[torch.Tensor] = None, *, eps: float = 1e-6, residual_scale: float = 1.0,
                    weight_offset: float = 0.0, post_norm: bool = False, dx: Optional[torch.Tensor] = None,
                    dh: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """dmuon_block_norm_backward: (dx, dh, dpre_weight, dpost_weight, dgate)
    from the gradients of block_norm's results (dx_out None: the stream has no
    other reader) and its x_out and h; a weight's gradient is None where the
    weight is.  dx may be dx_out."""
    dev, s, head, weights = _bn_args(x_out, h, pre_weight, post_weight, gate, eps, residual_scale, weight_offset,
                                     post_norm)
    grads = [*((0, 0) if dx_out is None else _row(dx_out, "dx_out", x_out)), *_row(dy, "dy", h)]
    dx, *dxo = _out(dx, "dx", x_out, stream)
    dh, *dho = _out(dh, "dh", h, stream)
    dws = [None if w is None else torch.empty_like(w) if stream is None else _alloc(stream, torch.empty_like, w)
           for w in (pre_weight, post_weight, gate)]
    need = _query("dmuon_block_norm_backward_workspace_bytes", s) if any(weights) else 0
    _ws, ptr, nbytes = _workspace(workspace, need, dev, stream)
    _run("dmuon_block_norm_backward", dev, stream, s, *grads, *head, *weights, *dxo, *dho,
         *[0 if w is None else w.data_ptr() for w in dws], ptr, nbytes)
    return (dx, dh, *dws)


# ---------------------------------------------------------------- attention
def _packed(out, name: str, like: torch.Tensor, stream) -> Tuple[torch.Tensor, int, int]:
    """(tensor, address, token stride) of a result like `like` (tokens, heads, dim), given or allocated here."""
    if out is None:
        new = like.new_empty
        out = new(like.shape) if stream is None else _alloc(stream, new, like.shape)
        return out, out.data_ptr(), like.shape[1] * like.shape[2]
    return out, *_heads(out, name, like)


def _attn_args(q, k, v, q_offsets, k_offsets, causal, window, scale):
    """(device index, dmuon_attention_shape, [q, stride, k, stride, v, stride], [offsets])."""
    head = [*_heads(q, "q"), *_heads(k, "k"), *_heads(v, "v", k)]
    dev, (n, qh, d), (nk, kh, dk) = q.get_device(), q.shape, k.shape
    if dk != d or k.dtype != q.dtype or k.get_device() != dev:
        raise ValueError(f"q is {q.dtype} {tuple(q.shape)} on {q.device}, k {k.dtype} {tuple(k.shape)} on {k.device}")
    if (q_offsets is None) != (k_offsets is None):
        raise ValueError("q_offsets and k_offsets come together")
    sequences, offs = 1, [0, 0]
    if q_offsets is not None:
        offs = [_tensor(q_offsets, "q_offsets", dev, torch.int32),
                _tensor(k_offsets, "k_offsets", dev, torch.int32, q_offsets.shape)]
        if q_offsets.dim() != 1 or q_offsets.shape[0] < 2:
            raise ValueError(f"q_offsets must hold one entry more than there are sequences, got shape {tuple(q_offsets.shape)}")
        sequences = q_offsets.shape[0] - 1
    s = _lib.AttentionShape(n, nk, sequences, _c_int(qh, "q_heads"), _c_int(kh, "k_heads"), _c_int(d, "head_dim"),
                            1 if causal else 0, _c_int(window, "window"), max(d, 1) ** -0.5 if scale is None else scale,
                            dtype_code(q.dtype))
    return dev, s, head, offs


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, q_offsets: Optional[torch.Tensor] = None,
              k_offsets: Optional[torch.Tensor] = None, *, causal: bool = True, window: int = 0,
              scale: Optional[float] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """dmuon_attention_forward: (out, lse) of packed sequences.

    q (tokens, q_heads, head_dim); k, v (keys, k_heads, head_dim), k_heads a
    divisor of q_heads; all may be slices of a packed projection: only a token's
    heads have to be contiguous.  q_offsets, k_offsets: int32 (sequences + 1),
    where each sequence begins and the last ends; None for one sequence.  A
    sequence's last query stands at its last key: with more keys than queries
    the first ones are a cache.  The room behind a cache that grows in place is
    a sequence of its own, without queries: q_offsets [0, 1, 1, 2, 2], k_offsets
    [0, n0, C, C + n1, 2 C] for two caches of C keys with n0, n1 in use.
    causal, window: which keys a query sees.
    scale: head_dim ** -0.5 by default.  lse: float32 (q_heads, tokens).
    Rows behind the last sequence are left as they were (unset, where the
    results are allocated here).  Outside autograd: the gradients are
    attention_grad's."""
    dev, s, head, offs = _attn_args(q, k, v, q_offsets, k_offsets, causal, window, scale)
    out, *o = _packed(out, "out", q, stream)
    if lse is None:
        new, shape = q.new_empty, (q.shape[1], q.shape[0])
        lse = new(shape, dtype=torch.float32) if stream is None else _alloc(stream, new, shape, dtype=torch.float32)
        at = lse.data_ptr()
    else:
        at = _tensor(lse, "lse", dev, torch.float32, (q.shape[1], q.shape[0]))
    _ws, ptr, nbytes = _workspace(workspace, _query("dmuon_attention_workspace_bytes", s), dev, stream)
    _run("dmuon_attention_forward", dev, stream, s, *head, *offs, *o, at, ptr, nbytes)
    return out, lse


def attention_workspace_bytes(q_tokens: int, k_tokens: int, q_heads: int, k_heads: int, head_dim: int,
                              sequences: int = 1) -> int:
    return _query("dmuon_attention_workspace_bytes",
                  _lib.AttentionShape(q_tokens, k_tokens, sequences, _c_int(q_heads, "q_heads"), _c_int(k_heads, "k_heads"),
                                      _c_int(head_dim, "head_dim"), scale=1.0))


def attention_grad(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                   lse: torch.Tensor, q_offsets: Optional[torch.Tensor] = None,
                   k_offsets: Optional[torch.Tensor] = None, *, causal: bool = True, window: int = 0,
                   scale: Optional[float] = None, dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                   dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """dmuon_attention_backward: (dq, dk, dv) from the gradient of attention's
    out, its inputs, and its out and lse.  dq, dk, dv may be given, as slices of
    a packed gradient.  Rows behind the last sequence are left as they were."""
    dev, s, head, offs = _attn_args(q, k, v, q_offsets, k_offsets, causal, window, scale)
    first, back = _heads(dout, "dout", q), _heads(out, "out", q)
    at = _tensor(lse, "lse", dev, torch.float32, (q.shape[1], q.shape[0]))
    dq, *dqo = _packed(dq, "dq", q, stream)
    dk, *dko = _packed(dk, "dk", k, stream)
    dv, *dvo = _packed(dv, "dv", v, stream)
    _ws, ptr, nbytes = _workspace(workspace, _query("dmuon_attention_backward_workspace_bytes", s), dev, stream)
    _run("dmuon_attention_backward", dev, stream, s, *first, *head, *back, at, *offs, *dqo, *dko, *dvo, ptr, nbytes)
    return dq, dk, dv


def attention_grad_workspace_bytes(q_tokens: int, q_heads: int) -> int:
    return _query("dmuon_attention_backward_workspace_bytes",
                  _lib.AttentionShape(q_tokens, 0, 1, _c_int(q_heads, "q_heads"), q_heads, 1, scale=1.0))


# ---------------------------------------------------------------- gated feed-forward
def _ffn_args(x, w_gate, w_up, activation):
    """(device index, dmuon_gated_ffn_shape, [x, stride, w_gate, w_up], whether they are aligned)."""
    if activation not in _ACTIVATIONS:
        raise ValueError(f"activation must be 'silu' or 'gelu', got {activation!r}")
    head = [*_row(x, "x")]
    dev, (n, dim) = x.get_device(), x.shape
    head.append(_tensor(w_gate, "w_gate", dev, x.dtype))
    if w_gate.dim() != 2 or w_gate.shape[1] != dim:
        raise ValueError(f"w_gate has shape {tuple(w_gate.shape)}, expected (hidden, {dim})")
    head.append(_tensor(w_up, "w_up", dev, x.dtype, w_gate.shape))
    pitch = head[1] * x.element_size() if n > 1 else 0
    fits = not (head[0] | head[2] | head[3] | pitch) % 16 and pitch <= 1 << 23
    return dev, _lib.GatedFfnShape(n, dim, w_gate.shape[0], _ACTIVATIONS[activation], dtype_code(x.dtype)), head, fits


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, activation: str = "silu", *,
              out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """dmuon_gated_ffn_forward: act(x w_gate^T) * (x w_up^T), (tokens, hidden).

    x (tokens, dim), rows contiguous; w_gate, w_up (hidden, dim), all of one
    type; activation "silu" or "gelu" (its tanh form).  Outside autograd: the
    gradients are gated_ffn_grad's."""
    dev, s, head, fits = _ffn_args(x, w_gate, w_up, activation)
    if out is None:
        new, shape = x.new_empty, (x.shape[0], w_gate.shape[0])
        out = new(shape) if stream is None else _alloc(stream, new, shape)
        at = out.data_ptr(), shape[1]
    else:
        at = _row(out, "out")
        if out.dtype != x.dtype or out.get_device() != dev or out.shape != (x.shape[0], w_gate.shape[0]):
            raise ValueError(f"out is {out.dtype} {tuple(out.shape)} on {out.device}, expected {x.dtype} "
                             f"{(x.shape[0], w_gate.shape[0])} on {x.device}")
    _ws, ptr, nbytes = _workspace(workspace, _query("dmuon_gated_ffn_workspace_bytes", s, fits), dev, stream)
    _run("dmuon_gated_ffn_forward", dev, stream, s, *head, *at, ptr, nbytes)
    return out


def gated_ffn_workspace_bytes(tokens: int, dim: int, hidden: int, dtype: torch.dtype, aligned: bool = True) -> int:
    """aligned: x and the weights begin at multiples of 16 bytes, and x's rows
    are a multiple of 16 bytes, at most 8 MiB, apart."""
    return _query("dmuon_gated_ffn_workspace_bytes", _lib.GatedFfnShape(tokens, dim, hidden, 0, dtype_code(dtype)), aligned)


def gated_ffn_grad(dh: torch.Tensor, x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor,
                   activation: str = "silu", *, dx: Optional[torch.Tensor] = None,
                   dw_gate: Optional[torch.Tensor] = None, dw_up: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """dmuon_gated_ffn_backward: (dx, dw_gate, dw_up) from the gradient of
    gated_ffn's result and its inputs; the weights' gradients have the weights'
    type and shape, as muon_step takes them."""
    dev, s, head, fits = _ffn_args(x, w_gate, w_up, activation)
    first = _row(dh, "dh")
    if dh.dtype != x.dtype or dh.get_device() != dev or dh.shape != (x.shape[0], w_gate.shape[0]):
        raise ValueError(f"dh is {dh.dtype} {tuple(dh.shape)} on {dh.device}, expected {x.dtype} "
                         f"{(x.shape[0], w_gate.shape[0])} on {x.device}")
    dx, *dxo = _out(dx, "dx", x, stream)
    grads = []
    for dw, w, name in ((dw_gate, w_gate, "dw_gate"), (dw_up, w_up, "dw_up")):
        if dw is None:
            dw = torch.empty_like(w) if stream is None else _alloc(stream, torch.empty_like, w)
        else:
            _tensor(dw, name, dev, w.dtype, w.shape)
        grads.append(dw)
    _ws, ptr, nbytes = _workspace(workspace, _query("dmuon_gated_ffn_backward_workspace_bytes", s, fits), dev, stream)
    _run("dmuon_gated_ffn_backward", dev, stream, s, *first, *head, *dxo, *[t.data_ptr() for t in grads], ptr, nbytes)
    return dx, grads[0], grads[1]


def gated_ffn_grad_workspace_bytes(tokens: int, dim: int, hidden: int, dtype: torch.dtype, aligned: bool = True) -> int:
    """aligned: as in gated_ffn_workspace_bytes."""
    return _query("dmuon_gated_ffn_backward_workspace_bytes",
                  _lib.GatedFfnShape(tokens, dim, hidden, 0, dtype_code(dtype)), aligned)
