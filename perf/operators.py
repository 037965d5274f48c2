"""Cases of the operators that feed the non-matrix parameters of a training step.

Embedding lookup and its gradient by sorted tokens, AdamW on a table whose
gradient comes as rows, the distillation loss with its gradient, and the norm
of queries and keys with the position rotation, forward and backward.  `run`
computes them in plain torch operations, or, with `own` set, through the
framework's entry points.
"""
import math

import torch

own = False


def _f32(x):
    """x as the float32 the optimizer's interface takes."""
    return float(torch.tensor(x, dtype=torch.float32))


LR, BETA1, BETA2, ADAM_EPS, DECAY = _f32(1e-3), _f32(0.9), _f32(0.999), _f32(1e-8), _f32(0.01)
STEP = 100
NORM_EPS = _f32(1e-6)
DT = {"f32": torch.float32, "bf16": torch.bfloat16}

VOCAB, DIM = 128256, 4096          # token embedding and head of the Llama-3-8B set
SMALL_VOCAB, HYBRID_DIM, TINY_DIM = 32000, 2048, 512


def listed():
    return [
        # one decoding step of four sequences: launch latency
        dict(name="embed decode", op="embed", n=4, vocab=VOCAB, dim=DIM, dtype="bf16", out="bf16", scale=1.0, pad=0.0),
        # 8 sequences of 8192 tokens, float32 master table, bf16 activations, sqrt(dim) scaling
        dict(name="embed batch", op="embed", n=65536, vocab=VOCAB, dim=DIM, dtype="f32", out="bf16", scale=64.0, pad=0.0),
        # a micro-batch of a smaller float32 model, the whole table's gradient
        dict(name="embed grad dense", op="embed_grad", n=16384, vocab=SMALL_VOCAB, dim=HYBRID_DIM, dtype="f32",
             out="f32", scale=1.0, pad=0.0, form="dense"),
        # a large batch with padded sequences, the gradient as one row per distinct token
        dict(name="embed grad rows", op="embed_grad", n=65536, vocab=VOCAB, dim=DIM, dtype="bf16", out="bf16",
             scale=64.0, pad=0.03, form="rows"),
        # a small float32 model's table after a short batch
        dict(name="adamw rows small", op="adamw_rows", n=1001, vocab=SMALL_VOCAB, dim=TINY_DIM, dtype="f32"),
        # the large bf16 table after an 8192-token batch
        dict(name="adamw rows table", op="adamw_rows", n=8192, vocab=VOCAB, dim=DIM, dtype="bf16"),
        # scoring a few rows of float32 logits: the loss alone, a ragged vocabulary
        dict(name="distill few rows", op="distill", n=7, vocab=32003, k=20, dtype="f32", temperature=1.0, ce=0.0,
             grad=False, masked=0.0),
        # a training batch: bf16 logits of the large vocabulary, mixed with the labels, prompt rows masked
        dict(name="distill batch", op="distill", n=8192, vocab=VOCAB, k=64, dtype="bf16", temperature=2.0, ce=0.5,
             grad=True, masked=0.1),
        # a decoding step of sixteen sequences on the packed projection's output
        dict(name="qk decode", op="qk", n=16, qh=32, kh=8, d=128, rot=128, inter=False, offset=0.0, dtype="bf16"),
        # a float32 prompt with a partial interleaved rotation and gains around zero
        dict(name="qk prompt f32", op="qk", n=8191, qh=16, kh=16, d=80, rot=32, inter=True, offset=1.0, dtype="f32"),
        # the backward pass of a short ragged batch
        dict(name="qk grad short", op="qk_grad", n=777, qh=6, kh=3, d=64, rot=64, inter=False, offset=1.0, dtype="f32"),
        # the backward pass of a 32768-token batch
        dict(name="qk grad batch", op="qk_grad", n=32768, qh=32, kh=8, d=128, rot=128, inter=False, offset=0.0,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "adamw_rows", "distill", "qk", "qk_grad"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("embed", "embed_grad"):
        c = dict(op=op, n=_log(rng, 1, 65536), vocab=_log(rng, 500, VOCAB), dim=_log(rng, 64, DIM), dtype=dtype,
                 out=rng.choice(["f32", "bf16"]), scale=rng.choice([1.0, 0.125, 22.5]),
                 pad=rng.choice([0.0, 0.05, 0.5]))
        if rng.random() < 0.7:
            c["dim"] = c["dim"] // 8 * 8
        if op == "embed_grad":
            c["form"] = rng.choice(["dense", "rows"])
        return c
    if op == "adamw_rows":
        dim = _log(rng, 64, DIM)
        if rng.random() < 0.7:
            dim = dim // 8 * 8
        return dict(op=op, n=_log(rng, 1, 32768), vocab=_log(rng, 500, VOCAB), dim=dim, dtype=dtype)
    if op == "distill":
        vocab = _log(rng, 500, VOCAB)
        return dict(op=op, n=_log(rng, 1, max(2, min(8192, (1 << 29) // vocab))), vocab=vocab, k=_log(rng, 1, 128), dtype=dtype,
                    temperature=rng.choice([1.0, 2.0, 0.7]), ce=rng.choice([0.0, 0.3]), grad=rng.random() < 0.7,
                    masked=rng.choice([0.0, 0.4]))
    d = rng.choice([40, 64, 80, 96, 128, 192, 256])
    kh = rng.choice([1, 2, 4, 8])
    return dict(op=op, n=_log(rng, 1, 16384), qh=kh * rng.choice([1, 2, 4]), kh=kh, d=d,
                rot=d if rng.random() < 0.6 else d // 16 * 8, inter=rng.random() < 0.4,
                offset=rng.choice([0.0, 1.0]), dtype=dtype)


# ---------------------------------------------------------------- inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, std, dtype):
    out = torch.empty(shape, device="cuda", dtype=dtype)
    return out.normal_(0.0, std, generator=g)


def _tokens(g, n, vocab, pad):
    """Word-like frequencies (the r-th most frequent token ~ 1 / r) under
    shuffled ids; a `pad` share at the end holds -1."""
    rank = torch.exp(torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(vocab)).long() - 1
    ids = torch.randperm(vocab, generator=g, device="cuda")[rank.clamp(0, vocab - 1)]
    ids[n - int(n * pad):] = -1
    return ids


def prepare(case, seed):
    g = _generator(seed)
    c, op = case, case["op"]
    dt = DT[c["dtype"]]
    s = dict(case=c, op=op)
    if op == "embed":
        s["table"] = _normal(g, (c["vocab"], c["dim"]), 0.02, dt)
        s["tokens"] = _tokens(g, c["n"], c["vocab"], c["pad"])
    elif op == "embed_grad":
        s["tokens"] = _tokens(g, c["n"], c["vocab"], c["pad"])
        s["dout"] = _normal(g, (c["n"], c["dim"]), 1e-3, dt)
    elif op == "adamw_rows":
        shape = (c["vocab"], c["dim"])
        touched = torch.zeros(c["vocab"], dtype=torch.bool, device="cuda")
        touched[_tokens(g, c["n"], c["vocab"], 0.0)] = True
        s["row_index"] = torch.where(touched, touched.cumsum(0) - 1, -1).int()
        s["grad_rows"] = _normal(g, (min(c["n"], c["vocab"]), c["dim"]), 1e-3, dt)
        s["param"] = _normal(g, shape, 0.02, dt)
        s["exp_avg"] = _normal(g, shape, 1e-4, torch.float32)
        s["exp_avg_sq"] = _normal(g, shape, 1e-4, torch.float32).square_()
    elif op == "distill":
        n, vocab, k = c["n"], c["vocab"], c["k"]
        # the teacher's entries lie in k strata of the vocabulary, the student partly agrees with them
        strata = torch.arange(k, device="cuda") * vocab // k
        s["index"] = strata + torch.randint(0, vocab // k, (n, k), generator=g, device="cuda")
        s["teacher"] = (_normal(g, (n, k), 2.0, torch.float32) + 6.0).sort(1, descending=True).values
        s["logits"] = _normal(g, (n, vocab), 2.0, dt)
        s["logits"].scatter_add_(1, s["index"], (s["teacher"] + 2.0 * _normal(g, (n, k), 1.0, torch.float32)).to(dt))
        s["labels"] = s["index"][:, 0].clone()
        s["labels"][torch.rand(n, generator=g, device="cuda") < 0.05] = -100
        s["weight"] = (torch.rand(n, generator=g, device="cuda") >= c["masked"]).float()
        s["scale"] = 1.0 / n
    else:
        n, qh, kh, d = c["n"], c["qh"], c["kh"], c["d"]
        packed = _normal(g, (n, (qh + 2 * kh) * d), 1.5, dt)   # a fused projection's output
        s["q"] = packed[:, :qh * d].unflatten(1, (qh, d))
        s["k"] = packed[:, qh * d:(qh + kh) * d].unflatten(1, (kh, d))
        s["qw"], s["kw"] = (_normal(g, (d,), 0.1, torch.float32).add_(1.0 - c["offset"]).to(dt) for _ in range(2))
        first = torch.randint(0, 4096, (1,), generator=g, device="cuda")
        s["positions"] = (first + torch.arange(n, device="cuda")) % 8192
        freq = 500000.0 ** (-torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64) * 2 / c["rot"])
        angle = torch.arange(8192, device="cuda", dtype=torch.float64)[:, None] * freq
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()   # (positions, rot): cosines, then sines
        if op == "qk_grad":
            s["dq"] = _normal(g, (n, qh, d), 1e-2, dt)
            s["dk"] = _normal(g, (n, kh, d), 1e-2, dt)
    return s


# ---------------------------------------------------------------- plain forms
def _embed(s):
    c, tok = s["case"], s["tokens"]
    rows = s["table"][tok.clamp(min=0)].float() * c["scale"]
    return torch.where((tok >= 0)[:, None], rows, 0.0).to(DT[c["out"]])


def _embed_grad(s):
    c, tok, dout = s["case"], s["tokens"], s["dout"]
    n, vocab = c["n"], c["vocab"]
    if c["form"] == "dense":
        acc = torch.zeros(vocab + 1, c["dim"], device="cuda")
        acc.index_add_(0, torch.where(tok >= 0, tok, vocab), dout.float())
        return (acc[:vocab] * c["scale"]).to(DT[c["out"]])
    cap = min(n, vocab)
    key, order = torch.where(tok >= 0, tok, vocab).sort(stable=True)
    head = torch.ones(n, dtype=torch.bool, device="cuda")
    head[1:] = key[1:] != key[:-1]
    head &= key < vocab
    slot = torch.where(key < vocab, head.cumsum(0) - 1, cap)
    rows = torch.full((cap + 1,), -1, dtype=torch.int64, device="cuda").scatter_(0, slot, key)[:cap]
    index = torch.full((vocab + 1,), -1, dtype=torch.int64, device="cuda").scatter_(0, key, slot)[:vocab]
    acc = torch.zeros(cap + 1, c["dim"], device="cuda").index_add_(0, slot, dout[order].float())
    # slots behind the last distinct token hold no row
    used = torch.arange(cap, device="cuda") < head.sum()
    return ((acc[:cap] * c["scale"]).to(DT[c["out"]]), torch.where(used, rows, -1).int(), index.int(),
            head.sum().int().reshape(1))


def _adamw_rows(s):
    p, m, v, index = s["param"], s["exp_avg"], s["exp_avg_sq"], s["row_index"].long()
    g = torch.where((index >= 0)[:, None], s["grad_rows"][index.clamp(min=0)].float(), 0.0)
    m.mul_(BETA1).add_(g * (1 - BETA1))
    v.mul_(BETA2).add_(g * g * (1 - BETA2))
    denom = v.sqrt() / math.sqrt(1 - BETA2 ** STEP) + ADAM_EPS
    new = p.float() * (1 - LR * DECAY) - (LR / (1 - BETA1 ** STEP)) * (m / denom)
    p.copy_(new)
    return p, m, v


def _distill(s):
    c = s["case"]
    z, t, w = s["logits"].float(), c["temperature"], s["weight"]
    q = torch.softmax(s["teacher"] / t, 1)
    logq = torch.log_softmax(s["teacher"] / t, 1)
    top = z.amax(1, keepdim=True)
    et = torch.exp((z - top) / t)
    st = et.sum(1, keepdim=True)
    logp = (z.gather(1, s["index"]) - top) / t - st.log()
    loss = t * t * (q * (logq - logp)).sum(1)
    has = s["labels"] >= 0
    label = s["labels"].clamp(min=0)[:, None]
    if c["ce"]:
        e1 = torch.exp(z - top)
        s1 = e1.sum(1, keepdim=True)
        nll = (s1.log() + top - z.gather(1, label)).squeeze(1)
        loss = loss + c["ce"] * torch.where(has, nll, 0.0)
    loss = torch.where(w != 0, w * loss, 0.0)
    if not c["grad"]:
        return loss
    dz = (et / st).scatter_add_(1, s["index"], -q) * t
    if c["ce"]:
        dz += c["ce"] * torch.where(has[:, None], (e1 / s1).scatter_add_(1, label, -torch.ones_like(st)), 0.0)
    dz *= (w * s["scale"])[:, None]
    return loss, dz.to(s["logits"].dtype)


def _rotate(x, cos, sin, inter, rot):
    """x (n, heads, d) rotated by the angles of cos, sin (n, rot / 2)."""
    cos, sin = cos[:, None], sin[:, None]
    if inter:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _angles(s):
    rot = s["case"]["rot"]
    table = s["rope"][s["positions"]]
    return table[:, :rot // 2], table[:, rot // 2:]


def _norm_rope(s, x, w):
    c = s["case"]
    cos, sin = _angles(s)
    x32 = x.float()
    y = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + NORM_EPS) * (c["offset"] + w.float())
    return _rotate(y, cos, sin, c["inter"], c["rot"]).to(x.dtype)


def _norm_rope_grad(s, dy, x, w):
    c = s["case"]
    cos, sin = _angles(s)
    x32 = x.float()
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + NORM_EPS)
    xh = x32 * r
    dn = _rotate(dy.float(), cos, -sin, c["inter"], c["rot"])
    dw = (dn * xh).sum((0, 1))
    g = dn * (c["offset"] + w.float())
    dx = r * (g - xh * (g * xh).mean(-1, keepdim=True))
    return dx.to(x.dtype), dw.to(w.dtype)


def _plain(s):
    op = s["op"]
    if op == "embed":
        return _embed(s)
    if op == "embed_grad":
        return _embed_grad(s)
    if op == "adamw_rows":
        return _adamw_rows(s)
    if op == "distill":
        return _distill(s)
    if op == "qk":
        return _norm_rope(s, s["q"], s["qw"]), _norm_rope(s, s["k"], s["kw"])
    dq, dqw = _norm_rope_grad(s, s["dq"], s["q"], s["qw"])
    dk, dkw = _norm_rope_grad(s, s["dk"], s["k"], s["kw"])
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import newton_schulz_08_amd as nsa

    c, op = s["case"], s["op"]
    if op == "embed":
        return nsa.embedding(s["table"], s["tokens"], scale=c["scale"], out_dtype=DT[c["out"]])
    if op == "embed_grad":
        plan = nsa.embedding_plan(s["tokens"], c["vocab"])
        grad = nsa.embedding_grad(plan, s["dout"], scale=c["scale"], form=c["form"], dtype=DT[c["out"]])
        return grad if c["form"] == "dense" else (grad, plan.rows, plan.row_index, plan.count)
    if op == "adamw_rows":
        nsa.adamw_rows_step_(s["param"], s["grad_rows"], s["row_index"], s["exp_avg"], s["exp_avg_sq"], STEP, lr=LR,
                             betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=DECAY)
        return s["param"], s["exp_avg"], s["exp_avg_sq"]
    if op == "distill":
        loss, dz = nsa.distill_loss(s["logits"], s["index"], s["teacher"], s["labels"], temperature=c["temperature"],
                                    ce_weight=c["ce"], row_weight=s["weight"], grad=c["grad"], grad_scale=s["scale"])
        return (loss, dz) if c["grad"] else loss
    kw = dict(eps=NORM_EPS, interleaved=c["inter"], weight_offset=c["offset"])
    if op == "qk":
        return nsa.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["positions"], s["rope"], **kw)
    return nsa.qk_norm_rope_grad(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["positions"], s["rope"], **kw)


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass needs
def _distinct(c):
    """Expected number of distinct tokens of _tokens."""
    n = c["n"] - int(c["n"] * c.get("pad", 0.0))
    p = torch.log1p(1.0 / torch.arange(1, c["vocab"] + 1, dtype=torch.float64)) / math.log(c["vocab"])
    return max(1, int((1.0 - (1.0 - p) ** n).sum()))


def work(case):
    c, op = case, case["op"]
    e = {"f32": 4, "bf16": 2}
    size = e[c["dtype"]]
    if op == "embed":
        # a table row is read once however often its token occurs
        return {"bytes": c["dim"] * (_distinct(c) * size + c["n"] * e[c["out"]]) + 8 * c["n"], "flops": c["n"] * c["dim"]}
    if op == "embed_grad":
        rows = c["vocab"] if c["form"] == "dense" else min(c["n"], c["vocab"])
        return {"bytes": c["dim"] * (int(c["n"] * (1 - c["pad"])) * size + rows * e[c["out"]]) + 8 * c["n"],
                "flops": c["n"] * c["dim"]}
    if op == "adamw_rows":
        # param and both moments read and written, the distinct tokens' gradient rows read
        return {"bytes": c["vocab"] * c["dim"] * (2 * size + 16) + _distinct(c) * c["dim"] * size,
                "flops": 12 * c["vocab"] * c["dim"]}
    if op == "distill":
        rows = c["n"] * (1 - c["masked"])
        return {"bytes": rows * c["vocab"] * size + (c["n"] * c["vocab"] * size if c["grad"] else 0)
                + c["n"] * (12 * c["k"] + 16), "flops": (8 if c["grad"] else 4) * rows * c["vocab"]}
    elems = c["n"] * (c["qh"] + c["kh"]) * c["d"]
    return {"bytes": elems * size * (3 if op == "qk_grad" else 2) + c["n"] * 4 * c["rot"],
            "flops": elems * (16 if op == "qk_grad" else 8)}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "embed":
        known = s["tokens"] >= 0
        out = torch.zeros(c["n"], c["dim"], dtype=torch.float64, device="cuda")
        out[known] = s["table"][s["tokens"][known]].double() * c["scale"]
        return out
    if op == "embed_grad":
        known = s["tokens"] >= 0
        tok, dout = s["tokens"][known], s["dout"][known].double()
        if c["form"] == "dense":
            out = torch.zeros(c["vocab"], c["dim"], dtype=torch.float64, device="cuda")
            return out.index_add_(0, tok, dout, alpha=c["scale"])
        _, back = torch.unique(tok, return_inverse=True)
        out = torch.zeros(min(c["n"], c["vocab"]), c["dim"], dtype=torch.float64, device="cuda")
        return out.index_add_(0, back, dout, alpha=c["scale"]), None, None, None
    if op == "adamw_rows":
        g = torch.zeros(c["vocab"], c["dim"], dtype=torch.float64, device="cuda")
        touched = s["row_index"] >= 0
        g[touched] = s["grad_rows"][s["row_index"][touched].long()].double()
        m = BETA1 * s["exp_avg"].double() + (1 - BETA1) * g
        v = BETA2 * s["exp_avg_sq"].double() + (1 - BETA2) * g ** 2
        del g
        m_hat, v_hat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
        return s["param"].double() * (1 - LR * DECAY) - LR * m_hat / (v_hat ** 0.5 + ADAM_EPS), m, v
    if op == "distill":
        z, t = s["logits"].double(), c["temperature"]
        logq = torch.log_softmax(s["teacher"].double() / t, 1)
        logp = torch.log_softmax(z / t, 1)
        loss = t * t * (logq.exp() * (logq - logp.gather(1, s["index"]))).sum(1)
        on = torch.nonzero(s["labels"] >= 0).squeeze(1)
        lab = s["labels"][on]
        if c["ce"]:
            log1 = torch.log_softmax(z, 1)
            loss[on] -= c["ce"] * log1[on, lab]
        w = s["weight"].double()
        if not c["grad"]:
            return w * loss
        dz = logp.exp_().scatter_add_(1, s["index"], -logq.exp()) * t
        if c["ce"]:
            log1.exp_()
            log1[on, lab] -= 1.0
            log1[s["labels"] < 0] = 0.0
            dz.add_(log1, alpha=c["ce"])
        return w * loss, dz * (w * s["scale"])[:, None]

    # the rotation as a matrix per position on pairs (i, j): [[cos, -sin], [sin, cos]]
    rot, d = c["rot"], c["d"]
    half = torch.arange(rot // 2, device="cuda")
    i, j = (2 * half, 2 * half + 1) if c["inter"] else (half, half + rot // 2)
    at = s["rope"].double()[s["positions"]]
    cos, sin = at[:, None, :rot // 2], at[:, None, rot // 2:]

    def normed(x):
        return x / (x.pow(2).sum(-1, keepdim=True) / d + NORM_EPS).sqrt()

    def forward(x, w):
        y = normed(x.double()) * (c["offset"] + w.double())
        out = y.clone()
        out[..., i] = cos * y[..., i] - sin * y[..., j]
        out[..., j] = sin * y[..., i] + cos * y[..., j]
        return out

    def backward(dy, x, w):
        dy, x = dy.double(), x.double()
        dn = dy.clone()
        dn[..., i] = cos * dy[..., i] + sin * dy[..., j]
        dn[..., j] = cos * dy[..., j] - sin * dy[..., i]
        n = normed(x)
        g = dn * (c["offset"] + w.double())
        along = (g * n).sum(-1, keepdim=True) / d
        dx = (g - n * along) / (x.pow(2).sum(-1, keepdim=True) / d + NORM_EPS).sqrt()
        return dx, (dn * n).flatten(0, 1).sum(0)

    if op == "qk":
        return forward(s["q"], s["qw"]), forward(s["k"], s["kw"])
    dq, dqw = backward(s["dq"], s["q"], s["qw"])
    dk, dkw = backward(s["dk"], s["k"], s["kw"])
    return dq, dk, dqw, dkw
