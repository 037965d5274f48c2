"""Python binding of the operators that feed the non-matrix parameters of a
training step: embedding lookup and gradient, AdamW on row gradients, the
distillation loss, and the norm of queries and keys with their rotation.

Like api.py this only marshals arguments; the work runs in libdmuon.so
(include/dmuon.h, from dmuon_embedding_forward on).  Results are allocated
unless given.  All tensors of a call lie on one device, which need not be the
current one; `stream` is a stream of that device (default: its current one).
Calls can be recorded into a graph; give a call on another stream than the
current one its own workspace and outputs if they outlive it.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import check
from .api import _used_on, alloc_workspace, dtype_code

_INDEX = {torch.int32: _lib.DMUON_I32, torch.int64: _lib.DMUON_I64}
_FORMS = {"dense": _lib.DMUON_EMBED_DENSE, "add": _lib.DMUON_EMBED_ADD, "rows": _lib.DMUON_EMBED_ROWS}


def _index_code(t: torch.Tensor, name: str) -> int:
    try:
        return _INDEX[t.dtype]
    except KeyError:
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}") from None


def _tensor(t, name: str, device: Optional[torch.device] = None, dtype: Optional[torch.dtype] = None,
            shape=None) -> torch.Tensor:
    """A contiguous device tensor, of that device, dtype and shape where given."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _run(name: str, device: torch.device, stream, *args) -> None:
    """One C call on `device`: the library works on the current device."""
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif stream.device != device:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to {device}")
    fn = getattr(_lib.load(), name)
    if device.index == torch.cuda.current_device():
        st = fn(*args, stream.cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, stream.cuda_stream)
    check(st, name)


def _query(name: str, *args) -> int:
    out = ctypes.c_size_t(0)
    check(getattr(_lib.load(), name)(*args, ctypes.byref(out)), name)
    return int(out.value)


def _workspace(given: Optional[torch.Tensor], need: int, device) -> Tuple[Optional[torch.Tensor], int, int]:
    """(workspace allocated here or None, address, bytes)."""
    if given is not None:
        if not given.is_cuda or given.device != device or given.dtype != torch.uint8 or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
        return None, given.data_ptr(), given.numel()
    if need == 0:
        return None, 0, 0
    ws = alloc_workspace(need, device)
    return ws, ws.data_ptr(), ws.numel()


# ---------------------------------------------------------------- embedding
def embedding(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0,
              out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """dmuon_embedding_forward: scale * table[tokens], of shape tokens.shape +
    (dim,) and dtype `out_dtype` (default: the table's).  A token outside
    [0, vocab) gives a zero row."""
    _tensor(table, "table")
    if table.dim() != 2:
        raise ValueError(f"table must be 2-D, got shape {tuple(table.shape)}")
    dev = table.device
    _tensor(tokens, "tokens", dev)
    vocab, dim = table.shape
    shape = tokens.shape + (dim,)
    own = out is None
    if own:
        out = torch.empty(shape, dtype=out_dtype or table.dtype, device=dev)
    else:
        _tensor(out, "out", dev, out_dtype, shape)
    _run("dmuon_embedding_forward", dev, stream, table.data_ptr(), vocab, dim, dtype_code(table.dtype),
         tokens.data_ptr(), tokens.numel(), _index_code(tokens, "tokens"), scale, out.data_ptr(), dtype_code(out.dtype))
    if own:
        _used_on(stream, out)
    return out


class EmbeddingPlan:
    """Sorted order of one batch's tokens (dmuon_embedding_plan), in device
    int32 tensors: `order`, `slot` (n), `rows` (min(n, vocab)), `row_index`
    (vocab) and `count` (1)."""

    def __init__(self, n: int, vocab: int, device: torch.device):
        self.n, self.vocab, self.cap, self.device = n, vocab, min(n, vocab), device
        at, self._at = 0, []
        for size in (n, n, self.cap, vocab, 1):
            self._at.append((at, size))
            at += (size + 63) // 64 * 64   # each on its own 256 bytes
        self._buf = torch.empty(max(at, 64), dtype=torch.int32, device=device)
        base = self._buf.data_ptr()
        self._ptrs = [base + 4 * a for a, _ in self._at]

    def _view(self, k: int) -> torch.Tensor:
        at, size = self._at[k]
        return self._buf[at:at + size]

    order = property(lambda self: self._view(0))
    slot = property(lambda self: self._view(1))
    rows = property(lambda self: self._view(2))
    row_index = property(lambda self: self._view(3))
    count = property(lambda self: self._view(4))


def embedding_plan_workspace_bytes(n: int, vocab: int) -> int:
    return _query("dmuon_embedding_plan_workspace_bytes", n, vocab)


def embedding_plan(tokens: torch.Tensor, vocab: int, plan: Optional[EmbeddingPlan] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> EmbeddingPlan:
    """dmuon_embedding_plan of `tokens` (any shape); with `plan`, into an
    existing plan of the same size."""
    _tensor(tokens, "tokens")
    code, n, dev, vocab = _index_code(tokens, "tokens"), tokens.numel(), tokens.device, int(vocab)
    need = embedding_plan_workspace_bytes(n, vocab)   # also the check of n and vocab
    own = plan is None
    if own:
        plan = EmbeddingPlan(n, vocab, dev)
    elif (plan.n, plan.vocab, plan.device) != (n, vocab, dev):
        raise ValueError(f"plan is for {plan.n} tokens of {plan.vocab} on {plan.device}, not {n} of {vocab} on {dev}")
    ws, ptr, nbytes = _workspace(workspace, need, dev)
    _run("dmuon_embedding_plan", dev, stream, tokens.data_ptr(), n, code, vocab, *plan._ptrs, ptr, nbytes)
    _used_on(stream, ws, plan._buf if own else None)
    return plan


def embedding_grad_workspace_bytes(n: int, dim: int, dtype: torch.dtype) -> int:
    return _query("dmuon_embedding_backward_workspace_bytes", n, dim, dtype_code(dtype))


def embedding_grad(plan: EmbeddingPlan, dout: torch.Tensor, scale: float = 1.0, form: str = "dense",
                   dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dmuon_embedding_backward: the gradient of `embedding` with respect to
    its table, for the tokens of `plan` and the output's gradient `dout`
    (tokens.shape + (dim,)).

    form: "dense" (vocab, dim), zero rows for tokens not in the batch; "add",
    the same added to `out`; "rows" (plan.cap, dim), row i for token
    plan.rows[i] and zero rows from plan.count on, as adamw_rows_step_ takes
    it.  dtype: of the gradient (default: dout's)."""
    if form not in _FORMS:
        raise ValueError(f"form must be 'dense', 'add' or 'rows', got {form!r}")
    dev = plan.device
    _tensor(dout, "dout", dev)
    if dout.dim() < 2:
        raise ValueError(f"dout must have the tokens' shape and a last dimension, got {tuple(dout.shape)}")
    dim = dout.shape[-1]
    if dim == 0 or dout.numel() // dim != plan.n:
        raise ValueError(f"dout has shape {tuple(dout.shape)}, the plan {plan.n} tokens")
    shape = (plan.cap if form == "rows" else plan.vocab, dim)
    own = out is None
    if own:
        if form == "add":
            raise ValueError("form 'add' needs out")
        out = torch.empty(shape, dtype=dtype or dout.dtype, device=dev)
    else:
        _tensor(out, "out", dev, dtype, shape)
    code = dtype_code(dout.dtype)
    need = _query("dmuon_embedding_backward_workspace_bytes", plan.n, dim, code)
    ws, ptr, nbytes = _workspace(workspace, need, dev)
    _run("dmuon_embedding_backward", dev, stream, dout.data_ptr(), plan.n, dim, code, scale, *plan._ptrs, plan.vocab,
         _FORMS[form], out.data_ptr(), dtype_code(out.dtype), ptr, nbytes)
    _used_on(stream, ws, out if own else None)
    return out


# ---------------------------------------------------------------- AdamW, gradient as rows
def adamw_rows_step_(param: torch.Tensor, grad_rows: torch.Tensor, row_index: torch.Tensor, exp_avg: torch.Tensor,
                     exp_avg_sq: torch.Tensor, step: int, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                     weight_decay: float = 0.01, stream=None) -> None:
    """dmuon_adamw_rows_step: one AdamW step of a (rows, dim) table in place.
    Row r has the gradient grad_rows[row_index[r]], or zero where row_index[r]
    names none: embedding_grad(plan, ..., form="rows") with plan.row_index.
    Defaults as in adamw_step_."""
    _tensor(param, "param")
    if param.dim() != 2:
        raise ValueError(f"param must be 2-D, got shape {tuple(param.shape)}")
    dev, (rows, dim) = param.device, param.shape
    _tensor(grad_rows, "grad_rows", dev, param.dtype)
    if grad_rows.dim() != 2 or grad_rows.shape[1] != dim:
        raise ValueError(f"grad_rows has shape {tuple(grad_rows.shape)}, expected (n, {dim})")
    _tensor(row_index, "row_index", dev, torch.int32, (rows,))
    _tensor(exp_avg, "exp_avg", dev, torch.float32, param.shape)
    _tensor(exp_avg_sq, "exp_avg_sq", dev, torch.float32, param.shape)
    b1, b2 = betas
    _run("dmuon_adamw_rows_step", dev, stream, param.data_ptr(), grad_rows.data_ptr(), grad_rows.shape[0],
         row_index.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), rows, dim, dtype_code(param.dtype),
         int(step), lr, b1, b2, eps, weight_decay)


# ---------------------------------------------------------------- distillation loss
def distill_loss_workspace_bytes(n: int, vocab: int) -> int:
    return _query("dmuon_distill_loss_workspace_bytes", n, vocab)


def _rows(t, name: str, device=None, dtype=None, shape=None) -> int:
    """Stride between the rows of a 2-D device tensor with contiguous rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2 or not t.is_cuda or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D device tensor with contiguous rows")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.stride(0)


def distill_loss(logits: torch.Tensor, teacher_index: Optional[torch.Tensor],
                 teacher_logits: Optional[torch.Tensor], labels: Optional[torch.Tensor] = None, *,
                 temperature: float = 1.0, kd_weight: float = 1.0, ce_weight: float = 0.0,
                 row_weight: Optional[torch.Tensor] = None, grad: bool = True, grad_scale: float = 1.0,
                 dlogits: Optional[torch.Tensor] = None, losses: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """dmuon_distill_loss: per-row losses (float32) and, with `grad`, their
    gradient with respect to the logits times `grad_scale` (1 / rows for the
    gradient of a mean); (losses, None) without.

    logits (n, vocab), rows contiguous; teacher_index, teacher_logits (n, k),
    entries outside the vocabulary left out, or both None for the label's term
    alone (kd_weight 0); labels (n), those outside the vocabulary ignored;
    row_weight (n) float32, rows of weight 0 skipped.  dlogits may be logits
    itself: the gradient then takes its place."""
    stride = _rows(logits, "logits")
    dev, (n, vocab) = logits.device, logits.shape
    if (teacher_index is None) != (teacher_logits is None):
        raise ValueError("teacher_index and teacher_logits come together")
    k, iptr, tptr, code = 0, 0, 0, _lib.DMUON_I64
    if teacher_index is not None:
        if teacher_index.dim() != 2 or teacher_index.shape[0] != n:
            raise ValueError(f"teacher_index has shape {tuple(teacher_index.shape)}, expected ({n}, k)")
        k, code = teacher_index.shape[1], _index_code(teacher_index, "teacher_index")
        iptr = _tensor(teacher_index, "teacher_index", dev).data_ptr()
        tptr = _tensor(teacher_logits, "teacher_logits", dev, torch.float32, teacher_index.shape).data_ptr()
    lptr = 0
    if labels is not None:
        want = labels.dtype if teacher_index is None else teacher_index.dtype
        lptr = _tensor(labels, "labels", dev, want, (n,)).data_ptr()
        code = _index_code(labels, "labels")
    wptr = 0 if row_weight is None else _tensor(row_weight, "row_weight", dev, torch.float32, (n,)).data_ptr()
    own_losses, own_grad, dstride = losses is None, grad and dlogits is None, 0
    if own_losses:
        losses = torch.empty(n, dtype=torch.float32, device=dev)
    else:
        _tensor(losses, "losses", dev, torch.float32, (n,))
    if not grad:
        dlogits = None
    else:
        if own_grad:
            dlogits = torch.empty((n, vocab), dtype=logits.dtype, device=dev)
        dstride = _rows(dlogits, "dlogits", dev, logits.dtype, logits.shape)
    ws, ptr, nbytes = _workspace(workspace, distill_loss_workspace_bytes(n, vocab), dev)
    _run("dmuon_distill_loss", dev, stream, logits.data_ptr(), n, vocab, stride, dtype_code(logits.dtype), iptr, code,
         tptr, k, lptr, temperature, kd_weight, ce_weight, wptr, grad_scale, losses.data_ptr(),
         dlogits.data_ptr() if grad else 0, dstride, ptr, nbytes)
    _used_on(stream, ws, losses if own_losses else None, dlogits if own_grad else None)
    return losses, dlogits


# ---------------------------------------------------------------- query / key norm
def rope_table(max_pos: int, rot_dim: int, theta: float = 10000.0, device=None) -> torch.Tensor:
    """Rotation table for qk_norm_rope: float32 (max_pos, rot_dim), the cosines
    of position * theta^(-2 i / rot_dim), then the sines; angles in float64."""
    freq = theta ** (-torch.arange(rot_dim // 2, dtype=torch.float64) * 2 / rot_dim)
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device or "cuda")


def _heads(t, name: str, like: Optional[torch.Tensor] = None) -> int:
    """Stride between the tokens of (tokens, heads, dim), heads contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3 or not t.is_cuda:
        raise ValueError(f"{name} must be a (tokens, heads, head_dim) device tensor")
    if like is not None and (t.device != like.device or t.dtype != like.dtype):
        raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")
    n, h, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}'s heads must lie next to each other (strides {t.stride()})")
    return t.stride(0)


def _qk_args(q, k, q_weight, k_weight, positions, rope, eps, interleaved, weight_offset):
    """(dmuon_qk_shape, strides, gains, positions, rope) of a call."""
    strides = _heads(q, "q"), _heads(k, "k", q)
    n, qh, d = q.shape
    if k.shape[0] != n or k.shape[2] != d:
        raise ValueError(f"q and k have shapes {tuple(q.shape)} and {tuple(k.shape)}")
    dev = q.device
    gain = q_weight if q_weight is not None else k_weight
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _tensor(w, name, dev, gain.dtype, (d,))
    s = _lib.QkShape(tokens=n, q_heads=qh, k_heads=k.shape[1], head_dim=d, interleaved=1 if interleaved else 0, eps=eps,
                     weight_offset=weight_offset, dtype=dtype_code(q.dtype),
                     weight_dtype=dtype_code(q.dtype if gain is None else gain.dtype))
    pos = table = 0
    if rope is not None:
        _tensor(rope, "rope", dev, torch.float32)
        if rope.dim() != 2:
            raise ValueError(f"rope must be (max_pos, rot_dim), got shape {tuple(rope.shape)}")
        _tensor(positions, "positions", dev, None, (n,))
        s.max_pos, s.rot_dim = rope.shape
        s.pos_dtype = _index_code(positions, "positions")
        pos, table = positions.data_ptr(), rope.data_ptr()
    gains = [0 if w is None else w.data_ptr() for w in (q_weight, k_weight)]
    return s, strides, gains, pos, table


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: Optional[torch.Tensor],
                 k_weight: Optional[torch.Tensor], positions: Optional[torch.Tensor], rope: Optional[torch.Tensor],
                 *, eps: float = 1e-6, interleaved: bool = False, weight_offset: float = 0.0,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """dmuon_qk_norm_rope_forward: every head of q (tokens, q_heads, head_dim)
    and k (tokens, k_heads, head_dim) divided by its root mean square, times
    weight_offset + gain, rotated by its token's position.

    q and k may be slices of a packed projection: only a token's heads have to
    be contiguous.  positions (tokens); negative ones mark padding (zeros out).
    rope: rope_table(...), float32 (max_pos, rot_dim); None leaves the rotation
    out.  q_out, k_out may be q and k themselves."""
    s, strides, gains, pos, table = _qk_args(q, k, q_weight, k_weight, positions, rope, eps, interleaved,
                                             weight_offset)
    outs, own, ostr = [], [], []
    for out, x, name in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        own.append(out is None)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        elif out.shape != x.shape:
            raise ValueError(f"{name} has shape {tuple(out.shape)}, expected {tuple(x.shape)}")
        ostr.append(_heads(out, name, q))
        outs.append(out)
    _run("dmuon_qk_norm_rope_forward", q.device, stream, s, q.data_ptr(), strides[0], k.data_ptr(), strides[1], *gains,
         pos, table, outs[0].data_ptr(), ostr[0], outs[1].data_ptr(), ostr[1])
    _used_on(stream, *(o for o, mine in zip(outs, own) if mine))
    return outs[0], outs[1]


def qk_norm_rope_grad_workspace_bytes(tokens: int, q_heads: int, k_heads: int, head_dim: int) -> int:
    s = _lib.QkShape(tokens=tokens, q_heads=q_heads, k_heads=k_heads, head_dim=head_dim)
    return _query("dmuon_qk_norm_rope_backward_workspace_bytes", s)


def qk_norm_rope_grad(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                      q_weight: Optional[torch.Tensor], k_weight: Optional[torch.Tensor],
                      positions: Optional[torch.Tensor], rope: Optional[torch.Tensor], *, eps: float = 1e-6,
                      interleaved: bool = False, weight_offset: float = 0.0, dq: Optional[torch.Tensor] = None,
                      dk: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """dmuon_qk_norm_rope_backward: (dq, dk, dq_weight, dk_weight) from the
    gradients of qk_norm_rope's outputs and its inputs; a gain's gradient is
    None where the gain is.  dq, dk may be given, as slices of a packed
    gradient, dq_out, dk_out, or q, k themselves."""
    s, strides, gains, pos, table = _qk_args(q, k, q_weight, k_weight, positions, rope, eps, interleaved,
                                             weight_offset)
    args, outs, own = [], [], []
    for dy, x, name in ((dq_out, q, "dq_out"), (dk_out, k, "dk_out")):
        st = _heads(dy, name, q)
        if dy.shape != x.shape:
            raise ValueError(f"{name} has shape {tuple(dy.shape)}, expected {tuple(x.shape)}")
        args += [dy.data_ptr(), st]
    args += [q.data_ptr(), strides[0], k.data_ptr(), strides[1], *gains, pos, table]
    for out, x, name in ((dq, q, "dq"), (dk, k, "dk")):
        own.append(out is None)
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        elif out.shape != x.shape:
            raise ValueError(f"{name} has shape {tuple(out.shape)}, expected {tuple(x.shape)}")
        args += [out.data_ptr(), _heads(out, name, q)]
        outs.append(out)
    dw = [None if w is None else torch.empty_like(w) for w in (q_weight, k_weight)]
    need = 0
    if q_weight is not None or k_weight is not None:
        need = _query("dmuon_qk_norm_rope_backward_workspace_bytes", s)
    ws, ptr, nbytes = _workspace(workspace, need, q.device)
    _run("dmuon_qk_norm_rope_backward", q.device, stream, s, *args, *(0 if w is None else w.data_ptr() for w in dw),
         ptr, nbytes)
    _used_on(stream, ws, *(o for o, mine in zip(outs, own) if mine), *dw)
    return outs[0], outs[1], dw[0], dw[1]
