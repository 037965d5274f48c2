"""Cases of the operators between a decoder block's projections.

Attention over packed sequences with its gradient, the norms around a block
with its gate and residual scale and their gradient, and the gated feed-forward
product with the gradients that the Muon step takes.  `run` computes them in
plain torch operations, or, with `own` set, through the framework's entry
points.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
NORM_EPS = float(torch.tensor(1e-6, dtype=torch.float32))
RES_SCALE = float(torch.tensor(0.8, dtype=torch.float32))

WIDE, HIDDEN = 4096, 14336         # width and hidden width of the Llama-3-8B set
TINY, TINY_HIDDEN = 512, 2048      # of the TinyMLP set


def listed():
    return [
        # scoring a short ragged batch with a small float32 model: launch latency
        dict(name="attend short", op="attend", n=203, batch=3, past=0, qh=6, kh=3, d=64, window=0, dtype="f32"),
        # one new token of each of eight sequences over what they have seen so far
        dict(name="attend token", op="attend", n=8, batch=8, past=65536, qh=32, kh=8, d=128, window=0, dtype="bf16"),
        # a training batch: two packed sequences of unequal length, 16384 tokens in all
        dict(name="attend batch", op="attend", n=16384, batch=2, past=0, qh=32, kh=8, d=128, window=0, dtype="bf16"),
        # the gradient of a short float32 batch with odd heads and a sliding window
        dict(name="attend grad short", op="attend_grad", n=777, batch=3, past=0, qh=16, kh=16, d=80, window=100,
             dtype="f32"),
        # the gradient of the training batch
        dict(name="attend grad batch", op="attend_grad", n=16384, batch=2, past=0, qh=32, kh=8, d=128, window=0,
             dtype="bf16"),
        # a decoding step of sixteen sequences: the norm before the next block, the branch added
        dict(name="norm step", op="norm", n=16, dim=WIDE, post=False, gate=False, dtype="bf16", branch="bf16"),
        # the gradient of a short float32 batch of odd width, every part of it
        dict(name="norm grad short", op="norm_grad", n=777, dim=1001, post=True, gate=True, dtype="f32", branch="f32"),
        # the gradient of a 32768-token batch: a float32 residual stream, bf16 branches
        dict(name="norm grad batch", op="norm_grad", n=32768, dim=WIDE, post=True, gate=True, dtype="f32",
             branch="bf16"),
        # a decoding step of four sequences: the weights are read once
        dict(name="ffn step", op="ffn", n=4, dim=WIDE, hidden=HIDDEN, act="silu", dtype="bf16"),
        # the forward pass of an 8192-token batch
        dict(name="ffn batch", op="ffn", n=8192, dim=WIDE, hidden=HIDDEN, act="silu", dtype="bf16"),
        # the gradient of a small float32 model after a batch of odd size
        dict(name="ffn grad short", op="ffn_grad", n=1001, dim=TINY, hidden=TINY_HIDDEN, act="gelu", dtype="f32"),
        # the gradient of the 8192-token batch
        dict(name="ffn grad batch", op="ffn_grad", n=8192, dim=WIDE, hidden=HIDDEN, act="silu", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend_grad", "norm", "norm_grad", "ffn", "ffn_grad"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    if op in ("attend", "attend_grad"):
        kh = rng.choice([1, 2, 4, 8])
        c = dict(op=op, n=_log(rng, 1, 8192 if dtype == "bf16" else 2048), batch=rng.choice([1, 1, 2, 3, 7, 16]), past=0,
                 qh=kh * rng.choice([1, 2, 3, 4]), kh=kh, d=rng.choice([32, 64, 72, 80, 96, 128, 128, 192, 256]),
                 window=rng.choice([0, 0, 0, 64, 1000]), dtype=dtype)
        if op == "attend" and rng.random() < 0.5:
            c["past"] = _log(rng, 1, 32768)
            c["n"] = min(c["n"], 512)
        return c
    if op in ("norm", "norm_grad"):
        dim = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            dim = dim // 8 * 8
        return dict(op=op, n=_log(rng, 1, min(32768, (1 << 26) // dim)), dim=dim, post=rng.random() < 0.6,
                    gate=rng.random() < 0.6, dtype=dtype, branch="bf16" if dtype == "bf16" else rng.choice(["f32", "bf16"]))
    dim, hidden = _log(rng, 64, WIDE), _log(rng, 64, HIDDEN)
    if rng.random() < 0.7:
        dim, hidden = dim // 8 * 8, hidden // 8 * 8
    n = _log(rng, 1, 8192 if dtype == "bf16" else max(16, min(2048, (1 << 33) // (dim * hidden))))
    return dict(op=op, n=n, dim=dim, hidden=hidden, act=rng.choice(["silu", "gelu"]), dtype=dtype)


# ---------------------------------------------------------------- inputs
def _lengths(total, batch, key):
    """`batch` unequal lengths that sum to `total`, the same for every seed."""
    rng = random.Random(total * 1000 + batch * 10 + key)
    share = [rng.uniform(0.5, 1.5) for _ in range(batch)]
    cut = [round(total * sum(share[:i]) / sum(share)) for i in range(batch + 1)]
    return [b - a for a, b in zip(cut, cut[1:])]


def _spans(c):
    """(queries, keys) of every sequence: its new tokens, and those behind what it has seen."""
    new = _lengths(c["n"], c["batch"], 0)
    past = _lengths(c["past"], c["batch"], 1) if c["past"] else [0] * c["batch"]
    return [(a, a + b) for a, b in zip(new, past)]


def _normal(g, shape, std, dtype):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0.0, std, generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, op, dt = case, case["op"], DT[case["dtype"]]
    s = dict(case=c, op=op)
    if op in ("attend", "attend_grad"):
        spans, qh, kh, d = _spans(c), c["qh"], c["kh"], c["d"]
        keys = sum(b for _, b in spans)
        s["q"] = _normal(g, (c["n"], qh, d), 1.5, dt)
        packed = _normal(g, (keys, 2 * kh, d), 1.0, dt)       # keys and values side by side
        s["k"], s["v"] = packed[:, :kh], packed[:, kh:]
        # keys of a sequence have something in common, as trained ones do
        s["k"] += _normal(g, (1, kh, d), 0.5, dt)
        s["spans"] = spans
        for name, which in (("q_offsets", 0), ("k_offsets", 1)):
            ends = torch.tensor([0] + [sp[which] for sp in spans]).cumsum(0)
            s[name] = ends.int().cuda()
        if op == "attend_grad":
            s["dout"] = _normal(g, (c["n"], qh, d), 1e-2, dt)
            out, lse = _attend({**s, "op": "attend"})         # what the forward pass has left
            s["out"], s["lse"] = out, lse
    elif op in ("norm", "norm_grad"):
        n, dim, bt = c["n"], c["dim"], DT[c["branch"]]
        s["x"] = _normal(g, (n, dim), 2.0, dt)                # the residual stream (behind the block for the gradient)
        s["h"] = _normal(g, (n, dim), 0.5, bt)                # the block's output
        s["post"] = _normal(g, (dim,), 0.1, torch.float32).add_(1.0).to(bt) if c["post"] else None
        s["gate"] = _normal(g, (dim,), 0.2, torch.float32).add_(0.5).to(bt) if c["gate"] else None
        s["pre"] = _normal(g, (dim,), 0.1, torch.float32).add_(1.0).to(bt)
        if op == "norm_grad":
            s["dx"] = _normal(g, (n, dim), 1e-2, dt)
            s["dy"] = _normal(g, (n, dim), 1e-2, bt)
    else:
        n, dim, hidden = c["n"], c["dim"], c["hidden"]
        s["x"] = _normal(g, (n, dim), 1.0, dt)
        s["wg"] = _normal(g, (hidden, dim), 1.2 * dim ** -0.5, dt)
        s["wu"] = _normal(g, (hidden, dim), 1.0 * dim ** -0.5, dt)
        if op == "ffn_grad":
            s["dh"] = _normal(g, (n, hidden), 1e-2, dt)
    return s


# ---------------------------------------------------------------- plain forms
def _seen(first, rows, lk, lq, window, device):
    """Truth values (rows, lk): which keys the queries first .. first + rows - 1 see."""
    i = torch.arange(first, first + rows, device=device)[:, None] + (lk - lq)
    j = torch.arange(lk, device=device)
    see = j <= i
    return see & (j > i - window) if window else see


def _parts(s):
    """(query rows, key rows, first query, lengths) of every sequence, in runs of
    queries whose scores of one key head stay below 2^28."""
    q0 = k0 = 0
    group = s["case"]["qh"] // s["case"]["kh"]
    for lq, lk in s["spans"]:
        step = max(1, (1 << 28) // max(1, lk * group))
        for a in range(0, lq, step):
            b = min(lq, a + step)
            yield slice(q0 + a, q0 + b), slice(k0, k0 + lk), a, lq, lk
        q0, k0 = q0 + lq, k0 + lk


def _head_runs(kh, size):
    """Key heads that are worked on at once: few where one alone has much."""
    step = max(1, min(kh, (1 << 28) // max(1, size)))
    return [slice(a, min(kh, a + step)) for a in range(0, kh, step)]


def _attend(s):
    c = s["case"]
    qh, kh, d = c["qh"], c["kh"], c["d"]
    g, scale = qh // kh, d ** -0.5
    q = s["q"].float().view(-1, kh, g, d)
    k, v = s["k"].float(), s["v"].float()
    out = torch.zeros(q.shape, device="cuda")
    lse = torch.zeros((kh, g, c["n"]), device="cuda")
    for rq, rk, a, lq, lk in _parts(s):
        rows = rq.stop - rq.start
        see = _seen(a, rows, lk, lq, c["window"], "cuda")
        for h in _head_runs(kh, rows * lk * g):
            qs = q[rq, h].permute(1, 2, 0, 3)                                     # heads, group, rows, d
            z = (qs.flatten(1, 2) @ k[rk, h].permute(1, 2, 0).contiguous()).unflatten(1, (g, rows)) * scale
            z = torch.where(see, z, float("-inf"))
            top = z.amax(-1, keepdim=True)
            e = torch.exp(z - top)
            total = e.sum(-1, keepdim=True)
            o = ((e / total).flatten(1, 2) @ v[rk, h].transpose(0, 1).contiguous()).unflatten(1, (g, rows))
            out[rq, h] = o.permute(2, 0, 1, 3)
            lse[h, :, rq] = (total.log() + top).squeeze(-1)
    return out.view(-1, qh, d).to(s["q"].dtype), lse.flatten(0, 1)


def _attend_grad(s):
    c = s["case"]
    qh, kh, d = c["qh"], c["kh"], c["d"]
    g, scale = qh // kh, d ** -0.5
    q, do, o = (s[name].float().view(-1, kh, g, d) for name in ("q", "dout", "out"))
    k, v = s["k"].float(), s["v"].float()
    lse = s["lse"].view(kh, g, -1)
    dq, dk, dv = torch.zeros_like(q), torch.zeros(k.shape, device="cuda"), torch.zeros(k.shape, device="cuda")
    for rq, rk, a, lq, lk in _parts(s):
        rows = rq.stop - rq.start
        see = _seen(a, rows, lk, lq, c["window"], "cuda")
        for h in _head_runs(kh, rows * lk * g):
            pick = lambda t: t[rq, h].permute(1, 2, 0, 3).flatten(1, 2)  # noqa: E731  heads, group * rows, d
            qs, dos, os_ = pick(q), pick(do), pick(o)
            ks, vs = k[rk, h].transpose(0, 1).contiguous(), v[rk, h].transpose(0, 1).contiguous()
            z = (qs @ ks.transpose(1, 2).contiguous()).unflatten(1, (g, rows)) * scale
            p = torch.where(see, torch.exp(z - lse[h, :, rq, None]), 0.0).flatten(1, 2)
            dp = dos @ vs.transpose(1, 2).contiguous()
            ds = p * (dp - (dos * os_).sum(-1, keepdim=True)) * scale
            dq[rq, h] = (ds @ ks).unflatten(1, (g, rows)).permute(2, 0, 1, 3)
            dk[rk, h] += (ds.transpose(1, 2).contiguous() @ qs).transpose(0, 1)
            dv[rk, h] += (p.transpose(1, 2).contiguous() @ dos).transpose(0, 1)
    t = s["q"].dtype
    return dq.view(-1, qh, d).to(t), dk.to(t), dv.to(t)


def _norm(s):
    c, x = s["case"], s["x"].float()
    b = s["h"].float()
    if c["post"]:
        b = b * torch.rsqrt(b.square().mean(-1, keepdim=True) + NORM_EPS) * s["post"].float()
    if c["gate"]:
        b = b * s["gate"].float()
    x = (x + RES_SCALE * b).to(s["x"].dtype)     # the stream is stored, and the next norm reads what was stored
    x32 = x.float()
    y = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + NORM_EPS) * s["pre"].float()
    return x, y.to(s["h"].dtype)


def _rms_grad(dn, x, w):
    """(dx, dw) of x / rms(x) * w."""
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + NORM_EPS)
    xh = x * r
    t = dn * w
    return r * (t - xh * (t * xh).mean(-1, keepdim=True)), (dn * xh).sum(0)


def _norm_grad(s):
    c, x, h = s["case"], s["x"].float(), s["h"].float()
    dx, dpre = _rms_grad(s["dy"].float(), x, s["pre"].float())
    dx = dx + s["dx"].float()
    db = RES_SCALE * dx
    gate = s["gate"].float() if c["gate"] else torch.ones((), device="cuda")
    dgate = dpost = None
    if c["post"]:
        w = s["post"].float()
        if c["gate"]:
            dgate = (db * h * torch.rsqrt(h.square().mean(-1, keepdim=True) + NORM_EPS) * w).sum(0)
        dh, dpost = _rms_grad(db * gate, h, w)
    else:
        dh = db * gate
        if c["gate"]:
            dgate = (db * h).sum(0)
    out = [dx.to(s["x"].dtype), dh.to(s["h"].dtype), dpre.to(s["pre"].dtype)]
    return out + [t.to(s["pre"].dtype) for t in (dpost, dgate) if t is not None]


GELU_C, GELU_A = math.sqrt(2.0 / math.pi), 0.044715


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    t = torch.tanh(GELU_C * (g + GELU_A * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * GELU_C * (1.0 + 3.0 * GELU_A * g * g)


def _ffn(s):
    x = s["x"].float()
    a, _ = _act(x @ s["wg"].float().T, s["case"]["act"])
    return (a * (x @ s["wu"].float().T)).to(s["x"].dtype)


def _ffn_grad(s):
    x, wg, wu, dh = (s[name].float() for name in ("x", "wg", "wu", "dh"))
    a, da = _act(x @ wg.T, s["case"]["act"])
    dg = dh * (x @ wu.T) * da
    du = dh * a
    return tuple(t.to(s["x"].dtype) for t in (dg @ wg + du @ wu, dg.T @ x, du.T @ x))


PLAIN = {"attend": _attend, "attend_grad": _attend_grad, "norm": _norm, "norm_grad": _norm_grad, "ffn": _ffn,
         "ffn_grad": _ffn_grad}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    import newton_schulz_08_amd as nsa

    c, op = s["case"], s["op"]
    if op == "attend":
        return nsa.attention(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], window=c["window"])
    if op == "attend_grad":
        return nsa.attention_grad(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["q_offsets"], s["k_offsets"],
                                  window=c["window"])
    kw = dict(eps=NORM_EPS, residual_scale=RES_SCALE, post_norm=c["post"]) if op in ("norm", "norm_grad") else {}
    if op == "norm":
        return nsa.block_norm(s["x"], s["h"], s["pre"], s["post"], s["gate"], **kw)
    if op == "norm_grad":
        dx, dh, dpre, dpost, dgate = nsa.block_norm_grad(s["dx"], s["dy"], s["x"], s["h"], s["pre"], s["post"], s["gate"],
                                                         **kw)
        return [t for t in (dx, dh, dpre, dpost, dgate) if t is not None]
    if op == "ffn":
        return nsa.gated_ffn(s["x"], s["wg"], s["wu"], activation=c["act"])
    return nsa.gated_ffn_grad(s["dh"], s["x"], s["wg"], s["wu"], activation=c["act"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ---------------------------------------------------------------- what a pass needs
def _pairs(c):
    """Visible (query, key) pairs of all sequences."""
    total = 0
    for lq, lk in _spans(c):
        first = lk - lq + 1                       # keys that the first query could see
        if not c["window"]:
            total += lq * first + lq * (lq - 1) // 2
            continue
        grow = max(0, min(lq, c["window"] - first))   # queries that still see everything before them
        total += grow * first + grow * (grow - 1) // 2 + (lq - grow) * min(c["window"], max(first, c["window"]))
    return total


def work(case):
    c, op = case, case["op"]
    e = {"f32": 4, "bf16": 2}
    size = e[c["dtype"]]
    if op in ("attend", "attend_grad"):
        keys = sum(b for _, b in _spans(c))
        rows, cols = c["n"] * c["qh"] * c["d"] * size, keys * c["kh"] * c["d"] * size
        back = op == "attend_grad"
        return {"bytes": rows * (4 if back else 2) + cols * (4 if back else 2) + 4 * c["n"] * c["qh"],
                "flops": (10 if back else 4) * c["d"] * c["qh"] * _pairs(c)}
    if op in ("norm", "norm_grad"):
        elems = c["n"] * c["dim"]
        per = (3 if op == "norm_grad" else 2) * (size + e[c["branch"]])
        return {"bytes": elems * per, "flops": elems * (24 if op == "norm_grad" else 10)}
    n, dim, hidden = c["n"], c["dim"], c["hidden"]
    weights, acts = 2 * hidden * dim * size, n * (dim + hidden) * size
    # the gradient forms both projections again, then dx and both weights' gradients
    if op == "ffn":
        return {"bytes": weights + acts, "flops": 4 * n * dim * hidden}
    return {"bytes": 2 * weights + acts + n * dim * size, "flops": 12 * n * dim * hidden}


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_attend(s, back):
    """One query head at a time: softmax over the keys that each query sees."""
    c = s["case"]
    qh, kh, d = c["qh"], c["kh"], c["d"]
    f64 = dict(dtype=torch.float64, device="cuda")
    out, lse = torch.zeros(c["n"], qh, d, **f64), torch.zeros(qh, c["n"], **f64)
    dq, dk, dv = torch.zeros(c["n"], qh, d, **f64), torch.zeros(s["k"].shape, **f64), torch.zeros(s["k"].shape, **f64)
    q0 = k0 = 0
    for lq, lk in s["spans"]:
        for h in range(qh if lq else 0):
            kv = h // (qh // kh)
            q, k, v = s["q"][q0:q0 + lq, h].double(), s["k"][k0:k0 + lk, kv].double(), s["v"][k0:k0 + lk, kv].double()
            score = torch.mm(q, k.T) / math.sqrt(d)
            for a in range(0, lq, 4096):      # the mask by blocks of queries
                b = min(lq, a + 4096)
                score[a:b].masked_fill_(~_seen(a, b - a, lk, lq, c["window"], "cuda"), -math.inf)
            norm = torch.logsumexp(score, 1)
            if not back:
                lse[h, q0:q0 + lq] = norm
                out[q0:q0 + lq, h] = torch.mm(score.softmax(1), v)
                continue
            # the forward pass's stored results are inputs of the gradient
            prob = score.sub_(s["lse"][h, q0:q0 + lq].double()[:, None]).exp_()
            do = s["dout"][q0:q0 + lq, h].double()
            dv[k0:k0 + lk, kv] += torch.mm(prob.T, do)
            along = (do * s["out"][q0:q0 + lq, h].double()).sum(1, keepdim=True)
            prob *= torch.mm(do, v.T).sub_(along)
            dq[q0:q0 + lq, h] = torch.mm(prob, k) / math.sqrt(d)
            dk[k0:k0 + lk, kv] += torch.mm(prob.T, q) / math.sqrt(d)
        q0, k0 = q0 + lq, k0 + lk
    return (dq, dk, dv) if back else (out, lse)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op in ("attend", "attend_grad"):
        return _exact_attend(s, op == "attend_grad")
    if op in ("norm", "norm_grad"):
        n, dim = c["n"], c["dim"]
        sums = [torch.zeros(dim, dtype=torch.float64, device="cuda") for _ in range(3)]
        first = torch.empty(n, dim, dtype=torch.float64, device="cuda")
        second = torch.empty_like(first)
        pre = s["pre"].double()
        post = s["post"].double() if c["post"] else 1.0
        gate = s["gate"].double() if c["gate"] else 1.0

        def length(t):
            return (t.pow(2).sum(1, keepdim=True) / dim + NORM_EPS).sqrt()

        for a in range(0, n, 4096):      # rows at a time
            r = slice(a, min(n, a + 4096))
            x, h = s["x"][r].double(), s["h"][r].double()
            unit = h / length(h) if c["post"] else h
            if op == "norm":
                first[r] = x + RES_SCALE * gate * post * unit
                stored = first[r].to(s["x"].dtype).double()     # the next norm reads the stored stream
                second[r] = stored / length(stored) * pre
                continue
            along = x / length(x)
            dy, dx = s["dy"][r].double(), s["dx"][r].double()
            inner = (dy * pre * along).sum(1, keepdim=True) / dim
            dx = dx + (dy * pre - along * inner) / length(x)
            first[r] = dx
            sums[0] += (dy * along).sum(0)
            sums[1] += RES_SCALE * (dx * gate * unit).sum(0)
            sums[2] += RES_SCALE * (dx * post * unit).sum(0)
            dn = RES_SCALE * dx * gate
            if c["post"]:
                dn = dn * post
                dn = (dn - unit * (dn * unit).sum(1, keepdim=True) / dim) / length(h)
            second[r] = dn
        if op == "norm":
            return first, second
        return [first, second, sums[0]] + [t for t, has in ((sums[1], c["post"]), (sums[2], c["gate"])) if has]
    x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
    g, u = torch.mm(x, wg.T), torch.mm(x, wu.T)
    if c["act"] == "silu":
        sig = torch.sigmoid(g)
        a, da = g * sig, sig + g * sig * (1.0 - sig)
    else:
        inner = GELU_C * (g + GELU_A * g.pow(3))
        a = g * (1.0 - 1.0 / (torch.exp(2.0 * inner) + 1.0))
        da = a / g + 0.5 * g / torch.cosh(inner).pow(2) * GELU_C * (1.0 + 3.0 * GELU_A * g.pow(2))
        da = torch.where(g == 0, 0.5, da)
    if op == "ffn":
        return a * u
    dh = s["dh"].double()
    du = dh * a
    dg = dh * u * da
    del a, da, u, g, dh
    return torch.mm(dg, wg) + torch.mm(du, wu), torch.mm(dg.T, x), torch.mm(du.T, x)
