"""Python binding of the operators that feed the non-matrix parameters of a
training step: embedding lookup and gradient, AdamW on row gradients, the
distillation loss, and the norm of queries and keys with their rotation.

Like api.py this only marshals arguments; the work runs in libdmuon.so
(include/dmuon.h, from dmuon_embedding_forward on).  Results are allocated
unless given.  All tensors of a call lie on one device, which need not be the
current one; `stream` is a stream of that device (default: its current one).
A call on another stream than the current one does not wait for it: the caller
orders the two around the call's inputs and results, as for any kernel.  What
the call allocates comes from that stream's own pool and may be dropped at any
time.  Calls can be recorded into a graph.

The results do not take part in autograd, whatever the inputs require: a
gradient goes through the call that this module has for it.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import check
from .api import _alloc, _alloc_workspace, _used_on, alloc_workspace, dtype_code

_INDEX = {torch.int32: _lib.DMUON_I32, torch.int64: _lib.DMUON_I64}
_FORMS = {"dense": _lib.DMUON_EMBED_DENSE, "add": _lib.DMUON_EMBED_ADD, "rows": _lib.DMUON_EMBED_ROWS}

# The handle of a device's current stream, without a Stream object (about 2 us)
# where this build of torch offers it: small calls cost little more than that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _index_code(t: torch.Tensor, name: str) -> int:
    try:
        return _INDEX[t.dtype]
    except KeyError:
        raise TypeError(f"{name} must be int32 or int64, got {t.dtype}") from None


def _tensor(t, name: str, index: int = -1, dtype: Optional[torch.dtype] = None, shape=None) -> int:
    """Address of a contiguous device tensor, on device `index` and of that
    dtype and shape where given."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    on = t.get_device() if t.is_cuda else -1
    if on < 0:
        raise ValueError(f"{name} must be a device tensor")
    if index >= 0 and on != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


_fns = {}


def _run(name: str, index: int, stream, *args) -> None:
    """One C call on device `index`: the library works on the current device."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_lib.load(), name)
    if stream is None:
        handle = _raw_stream(index)
    elif stream.device.index != index:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to cuda:{index}")
    else:
        handle = stream.cuda_stream
    if index == torch.cuda.current_device():
        st = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            st = fn(*args, handle)
    if st:
        check(st, name)


def _query(name: str, *args) -> int:
    out = ctypes.c_size_t(0)
    check(getattr(_lib.load(), name)(*args, ctypes.byref(out)), name)
    return out.value


def _workspace(given: Optional[torch.Tensor], need: int, index: int, stream) -> Tuple[Optional[torch.Tensor], int, int]:
    """(workspace allocated here or None, address, bytes)."""
    if given is not None:
        if not given.is_cuda or given.get_device() != index or given.dtype != torch.uint8 or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
        return None, given.data_ptr(), given.numel()
    if need == 0:
        return None, 0, 0
    device = torch.device("cuda", index)
    ws = alloc_workspace(need, device) if stream is None else _alloc_workspace(stream, need, device)
    return ws, ws.data_ptr(), ws.numel()


# ---------------------------------------------------------------- embedding
def embedding(table: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0,
              out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """dmuon_embedding_forward: scale * table[tokens], of shape tokens.shape +
    (dim,) and dtype `out_dtype` (default: the table's).  A token outside
    [0, vocab) gives a zero row.  Outside autograd: its gradient is
    embedding_grad."""
    src = _tensor(table, "table")
    if table.dim() != 2:
        raise ValueError(f"table must be 2-D, got shape {tuple(table.shape)}")
    dev = table.get_device()
    tok = _tensor(tokens, "tokens", dev)
    vocab, dim = table.shape
    if out is None:
        new, shape, dt = table.new_empty, (*tokens.shape, dim), out_dtype or table.dtype
        out = new(shape, dtype=dt) if stream is None else _alloc(stream, new, shape, dtype=dt)
        dst = out.data_ptr()
    else:
        dst = _tensor(out, "out", dev, out_dtype, (*tokens.shape, dim))
    _run("dmuon_embedding_forward", dev, stream, src, vocab, dim, dtype_code(table.dtype), tok, tokens.numel(),
         _index_code(tokens, "tokens"), scale, dst, dtype_code(out.dtype))
    return out


class EmbeddingPlan:
    """Sorted order of one batch's tokens (dmuon_embedding_plan), in device
    int32 tensors: `order`, `slot` (n), `rows` (min(n, vocab)), `row_index`
    (vocab) and `count` (1)."""

    def __init__(self, n: int, vocab: int, device, stream=None):
        self.n, self.vocab, self.cap = n, vocab, min(n, vocab)
        # each on its own 256 bytes
        a = n + 63 & ~63
        b = a + a
        c = b + (self.cap + 63 & ~63)
        d = c + (vocab + 63 & ~63)
        self._at = (0, n), (a, n), (b, self.cap), (c, vocab), (d, 1)
        self._buf = _alloc(stream, torch.empty, d + 64, dtype=torch.int32, device=device)
        self.device, self._index = self._buf.device, self._buf.get_device()
        p = self._buf.data_ptr()
        self._ptrs = p, p + 4 * a, p + 4 * b, p + 4 * c, p + 4 * d

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
    tok = _tensor(tokens, "tokens")
    code, n, dev, vocab = _index_code(tokens, "tokens"), tokens.numel(), tokens.get_device(), int(vocab)
    need = embedding_plan_workspace_bytes(n, vocab)   # also the check of n and vocab
    if plan is None:
        plan = EmbeddingPlan(n, vocab, tokens.device, stream)
    elif (plan.n, plan.vocab, plan._index) != (n, vocab, dev):
        raise ValueError(f"plan is for {plan.n} tokens of {plan.vocab} on {plan.device}, not {n} of {vocab} on cuda:{dev}")
    _ws, ptr, nbytes = _workspace(workspace, need, dev, stream)
    _run("dmuon_embedding_plan", dev, stream, tok, n, code, vocab, *plan._ptrs, ptr, nbytes)
    if stream is not None:
        _used_on(stream, plan._buf)
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
    dev = plan._index
    src = _tensor(dout, "dout", dev)
    if dout.dim() < 2:
        raise ValueError(f"dout must have the tokens' shape and a last dimension, got {tuple(dout.shape)}")
    dim = dout.shape[-1]
    if dim == 0 or dout.numel() // dim != plan.n:
        raise ValueError(f"dout has shape {tuple(dout.shape)}, the plan {plan.n} tokens")
    shape = (plan.cap if form == "rows" else plan.vocab, dim)
    if out is None:
        if form == "add":
            raise ValueError("form 'add' needs out")
        new, dt = dout.new_empty, dtype or dout.dtype
        out = new(shape, dtype=dt) if stream is None else _alloc(stream, new, shape, dtype=dt)
        dst = out.data_ptr()
    else:
        dst = _tensor(out, "out", dev, dtype, shape)
    code = dtype_code(dout.dtype)
    need = _query("dmuon_embedding_backward_workspace_bytes", plan.n, dim, code)
    _ws, ptr, nbytes = _workspace(workspace, need, dev, stream)
    _run("dmuon_embedding_backward", dev, stream, src, plan.n, dim, code, scale, *plan._ptrs, plan.vocab, _FORMS[form],
         dst, dtype_code(out.dtype), ptr, nbytes)
    if stream is not None:
        _used_on(stream, plan._buf)
    return out


# ---------------------------------------------------------------- AdamW, gradient as rows
def _adamw_rows_args(param, grad_rows, row_index, exp_avg, exp_avg_sq, step, lr, betas, eps, weight_decay):
    """(device index, arguments of dmuon_adamw_rows_step up to the stream)."""
    p = _tensor(param, "param")
    if param.dim() != 2:
        raise ValueError(f"param must be 2-D, got shape {tuple(param.shape)}")
    dev, (rows, dim) = param.get_device(), param.shape
    g = _tensor(grad_rows, "grad_rows", dev, param.dtype)
    if grad_rows.dim() != 2 or grad_rows.shape[1] != dim:
        raise ValueError(f"grad_rows has shape {tuple(grad_rows.shape)}, expected (n, {dim})")
    index = _tensor(row_index, "row_index", dev, torch.int32, (rows,))
    m = _tensor(exp_avg, "exp_avg", dev, torch.float32, param.shape)
    v = _tensor(exp_avg_sq, "exp_avg_sq", dev, torch.float32, param.shape)
    b1, b2 = betas
    return dev, (p, g, grad_rows.shape[0], index, m, v, rows, dim, dtype_code(param.dtype), int(step), lr, b1, b2, eps,
                 weight_decay)


def adamw_rows_step_(param: torch.Tensor, grad_rows: torch.Tensor, row_index: torch.Tensor, exp_avg: torch.Tensor,
                     exp_avg_sq: torch.Tensor, step: int, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                     weight_decay: float = 0.01, stream=None) -> None:
    """dmuon_adamw_rows_step: one AdamW step of a (rows, dim) table in place.
    Row r has the gradient grad_rows[row_index[r]], or zero where row_index[r]
    names none: embedding_grad(plan, ..., form="rows") with plan.row_index.
    Defaults as in adamw_step_."""
    dev, args = _adamw_rows_args(param, grad_rows, row_index, exp_avg, exp_avg_sq, step, lr, betas, eps, weight_decay)
    _run("dmuon_adamw_rows_step", dev, stream, *args)


def adamw_rows_prepared(stream, *args):
    """The same step, checked now and taken by the call that is returned:
    several tables can be turned down before the first is changed."""
    dev, args = _adamw_rows_args(*args)
    check(_lib.load().dmuon_adamw_rows_check(*args), "dmuon_adamw_rows_step")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream belongs to {stream.device}, the tensors to cuda:{dev}")
    return lambda: _run("dmuon_adamw_rows_step", dev, stream, *args)


# ---------------------------------------------------------------- distillation loss
def distill_loss_workspace_bytes(n: int, vocab: int) -> int:
    return _query("dmuon_distill_loss_workspace_bytes", n, vocab)


def _rows(t, name: str, like: Optional[torch.Tensor] = None) -> int:
    """Stride between the rows of a 2-D device tensor with contiguous rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2 or not t.is_cuda or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D device tensor with contiguous rows")
    if like is not None and (t.dtype != like.dtype or t.get_device() != like.get_device() or t.shape != like.shape):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected {like.dtype} "
                         f"{tuple(like.shape)} on {like.device}")
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

    logits (n, vocab), rows contiguous; teacher_index (n, k) int32 or int64,
    entries outside the vocabulary left out, and teacher_logits (n, k) float32,
    or both None for the label's term alone (kd_weight 0); labels (n) of the
    indices' type, those outside the vocabulary ignored; row_weight (n) float32,
    rows of weight 0 skipped.  dlogits may be logits itself: the gradient then
    takes its place.  Outside autograd: the losses do not lead back to the
    logits, the gradient is returned beside them."""
    stride = _rows(logits, "logits")
    dev, (n, vocab) = logits.get_device(), logits.shape
    if (teacher_index is None) != (teacher_logits is None):
        raise ValueError("teacher_index and teacher_logits come together")
    k, iptr, tptr, code = 0, 0, 0, _lib.DMUON_I64
    if teacher_index is not None:
        iptr = _tensor(teacher_index, "teacher_index", dev)
        if teacher_index.dim() != 2 or teacher_index.shape[0] != n:
            raise ValueError(f"teacher_index has shape {tuple(teacher_index.shape)}, expected ({n}, k)")
        k, code = teacher_index.shape[1], _index_code(teacher_index, "teacher_index")
        tptr = _tensor(teacher_logits, "teacher_logits", dev, torch.float32, teacher_index.shape)
    lptr = 0
    if labels is not None:
        lptr = _tensor(labels, "labels", dev, None if teacher_index is None else teacher_index.dtype, (n,))
        code = _index_code(labels, "labels")
    wptr = 0 if row_weight is None else _tensor(row_weight, "row_weight", dev, torch.float32, (n,))
    dptr = dstride = 0
    if losses is None:
        new = logits.new_empty
        losses = new((n,), dtype=torch.float32) if stream is None else _alloc(stream, new, (n,), dtype=torch.float32)
    else:
        _tensor(losses, "losses", dev, torch.float32, (n,))
    if not grad:
        dlogits = None
    elif dlogits is None:
        new = logits.new_empty
        dlogits = new((n, vocab)) if stream is None else _alloc(stream, new, (n, vocab))
        dptr, dstride = dlogits.data_ptr(), vocab
    else:
        dstride = _rows(dlogits, "dlogits", logits)
        dptr = dlogits.data_ptr()
    _ws, ptr, nbytes = _workspace(workspace, distill_loss_workspace_bytes(n, vocab), dev, stream)
    _run("dmuon_distill_loss", dev, stream, logits.data_ptr(), n, vocab, stride, dtype_code(logits.dtype), iptr, code,
         tptr, k, lptr, temperature, kd_weight, ce_weight, wptr, grad_scale, losses.data_ptr(), dptr, dstride, ptr,
         nbytes)
    return losses, dlogits


# ---------------------------------------------------------------- query / key norm
def rope_table(max_pos: int, rot_dim: int, theta: float = 10000.0, device=None) -> torch.Tensor:
    """Rotation table for qk_norm_rope: float32 (max_pos, rot_dim), the cosines
    of position * theta^(-2 i / rot_dim), then the sines; angles in float64.
    rot_dim is even; device: the current GPU by default."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and >= 0, got {rot_dim}")
    freq = theta ** (-torch.arange(rot_dim // 2, dtype=torch.float64) * 2 / rot_dim)
    angle = torch.arange(max_pos, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to("cuda" if device is None else device)


def _heads(t, name: str, like: Optional[torch.Tensor] = None) -> Tuple[int, int]:
    """Address of (tokens, heads, dim) with contiguous heads, and the stride
    between its tokens; of `like`'s type, device and shape if that is given."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a (tokens, heads, head_dim) device tensor")
    if like is not None and (t.dtype != like.dtype or t.get_device() != like.get_device() or t.shape != like.shape):
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} on {t.device}, expected {like.dtype} "
                         f"{tuple(like.shape)} on {like.device}")
    st, sh, sd = t.stride()
    _, h, d = t.shape
    if (sd != 1 and d > 1) or (sh != d and h > 1):
        raise ValueError(f"{name}'s heads must lie next to each other (strides {t.stride()})")
    return t.data_ptr(), st


def _qk_args(q, k, q_weight, k_weight, positions, rope, eps, interleaved, weight_offset):
    """(device index, dmuon_qk_shape, [q, stride, k, stride, gains, positions, rope]) of a call."""
    args = [*_heads(q, "q"), *_heads(k, "k")]
    dev, (n, qh, d), (nk, kh, dk) = q.get_device(), q.shape, k.shape
    if nk != n or dk != d or k.dtype != q.dtype or k.get_device() != dev:
        raise ValueError(f"q is {q.dtype} {tuple(q.shape)} on {q.device}, k {k.dtype} {tuple(k.shape)} on {k.device}")
    wdt = None
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is None:
            args.append(0)
        else:
            args.append(_tensor(w, name, dev, wdt, (d,)))
            wdt = w.dtype
    max_pos = rot = pos_dtype = pos = table = 0
    if rope is not None:
        table = _tensor(rope, "rope", dev, torch.float32)
        if rope.dim() != 2:
            raise ValueError(f"rope must be (max_pos, rot_dim), got shape {tuple(rope.shape)}")
        max_pos, rot = rope.shape
    if positions is not None or rot:
        pos = _tensor(positions, "positions", dev, None, (n,))
        pos_dtype = _index_code(positions, "positions")
    s = _lib.QkShape(n, qh, kh, d, rot, 1 if interleaved else 0, max_pos, eps, weight_offset, dtype_code(q.dtype),
                     dtype_code(wdt or q.dtype), pos_dtype)
    args += [pos, table]
    return dev, s, args


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
    out, and positions are then needed only for padding.  Outside autograd: the
    gradients are qk_norm_rope_grad's.  q_out, k_out may be q and k themselves."""
    dev, s, args = _qk_args(q, k, q_weight, k_weight, positions, rope, eps, interleaved, weight_offset)
    outs = []
    for out, x, name in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        if out is None:
            out = x.new_empty(x.shape) if stream is None else _alloc(stream, x.new_empty, x.shape)
            args += [out.data_ptr(), x.shape[1] * x.shape[2]]
        else:
            args += _heads(out, name, x)
        outs.append(out)
    _run("dmuon_qk_norm_rope_forward", dev, stream, s, *args)
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
    dev, s, args = _qk_args(q, k, q_weight, k_weight, positions, rope, eps, interleaved, weight_offset)
    head = [*_heads(dq_out, "dq_out", q), *_heads(dk_out, "dk_out", k)]
    outs = []
    for out, x, name in ((dq, q, "dq"), (dk, k, "dk")):
        if out is None:
            out = x.new_empty(x.shape) if stream is None else _alloc(stream, x.new_empty, x.shape)
            args += [out.data_ptr(), x.shape[1] * x.shape[2]]
        else:
            args += _heads(out, name, x)
        outs.append(out)
    need = 0
    for w in (q_weight, k_weight):
        if w is None:
            outs.append(None)
            args.append(0)
        else:
            dw = torch.empty_like(w) if stream is None else _alloc(stream, torch.empty_like, w)
            outs.append(dw)
            args.append(dw.data_ptr())
            need = need or _query("dmuon_qk_norm_rope_backward_workspace_bytes", s)
    _ws, ptr, nbytes = _workspace(workspace, need, dev, stream)
    _run("dmuon_qk_norm_rope_backward", dev, stream, s, *head, *args, ptr, nbytes)
    return tuple(outs)
