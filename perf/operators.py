"""The training operators around the optimizer step: what is measured, and in which cases.

Three operators, each with its gradient.  Their bf16 gradients are what the
optimizer accumulates.

  distill   loss of a student's logits against the top logits that a teacher
            left for each token (and, if wanted, against the token's label),
            and its gradient;
  norm      a block's output, normalised, gated and scaled, added to the
            residual stream, and the norm that feeds the next block; and the
            gradient of all of it;
  balance   a router's choice of k experts for each token, the experts'
            counts, the balance loss and the z-loss; and their gradient.

`run` computes them in their plain form (elementary torch operations in 32
bits, rounded once at the end), or, where `own` is true, by the calls that a
training program makes of the package.
"""
import math

import torch

own = False

NEG = float("-inf")
F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"bf16": BF16, "f32": F32}
BYTES = {"bf16": 2, "f32": 4}

VOCAB = 250880          # the vocabulary of the scaled-down workload
SEQ = 2048              # its tokens per sequence
HIDDEN, WIDE = 2048, 14336   # hidden sizes of the scaled-down and the full model


# ---------------------------------------------------------------- the cases

def _distill(way, rows, vocab, k, dtype, temperature, ce, full=False, masked=0.0, padded=0):
    """`full`: the teacher's normaliser came with its top logits.  `masked`:
    share of rows that count for nothing (padding tokens).  `padded`: vocabulary
    entries at the end that no token uses (logit -inf)."""
    return dict(op="distill", way=way, rows=rows, vocab=vocab, k=k, dtype=dtype, temperature=temperature, ce=ce,
                full=full, masked=masked, padded=padded)


def _norm(way, rows, hidden, branch, stream, weight, pre, post, gates, act, rs=1.0, bs=1.0):
    """`branch`, `stream`: types of the block's tensors and of the residual
    stream.  `gates`: gate rows (0: none); rows / gates consecutive rows share one."""
    return dict(op="norm", way=way, rows=rows, hidden=hidden, branch=branch, stream=stream, weight=weight, pre=pre,
                post=post, gates=gates, act=act, rs=rs, bs=bs)


def _balance(way, tokens, experts, k, dtype, groups=1, masked=0.0, renorm=True, z=1e-3):
    return dict(op="balance", way=way, tokens=tokens, experts=experts, k=k, dtype=dtype, groups=groups, masked=masked,
                renorm=renorm, z=z)


def listed():
    cases = [
        # a few tokens with a small odd vocabulary: a unit test's or a probe's step, latency only
        ("distill_few_tokens", _distill("step", 6, 2053, 4, "bf16", 1.0, 0.0)),
        # one sequence of the scaled-down workload: the loss and its gradient as a training step takes them
        ("distill_sequence", _distill("step", SEQ, VOCAB, 64, "bf16", 2.0, 0.5, masked=0.05, padded=200)),
        # held-out loss against a teacher whose normaliser was stored too
        ("distill_evaluation", _distill("forward", 512, VOCAB, 128, "bf16", 1.0, 0.0, full=True)),
        # the gradient by itself, as autograd asks for it, 32-bit logits, an odd number of tokens, an odd vocabulary
        ("distill_gradient_f32", _distill("backward", 1021, 32003, 20, "f32", 1.5, 1.0, masked=0.1)),
        # one token between two blocks
        ("norm_one_token", _norm("forward", 1, HIDDEN, "bf16", "bf16", "bf16", "rms", "rms", 0, "none")),
        # the full model's hidden size, a 32-bit residual stream, one learned gate vector
        ("norm_wide_f32_stream", _norm("forward", 4096, WIDE, "bf16", "f32", "bf16", "rms", "rms", 1, "none")),
        # a micro-batch of four sequences, layer norms with biases, a gate for each sequence
        ("norm_gradient_sequences", _norm("backward", 4 * SEQ, HIDDEN, "bf16", "bf16", "bf16", "layer", "layer", 4, "none", rs=0.5)),
        # the full model's hidden size
        ("norm_gradient_wide", _norm("backward", 4096, WIDE, "bf16", "bf16", "bf16", "layer", "rms", 0, "none", bs=0.25)),
        # odd sizes and a gate of its own for each token
        ("norm_gradient_odd", _norm("backward", 1543, 1537, "bf16", "f32", "f32", "rms", "layer", 1543, "sigmoid")),
        # a few tokens, a few experts: latency only
        ("balance_few_tokens", _balance("step", 16, 8, 2, "f32")),
        # eight sequences balanced each for itself, padding masked
        ("balance_sequences", _balance("step", 8 * SEQ, 64, 6, "f32", groups=8, masked=0.1)),
        # a large batch and many experts, bf16 logits with their ties
        ("balance_many_experts", _balance("step", 262144, 256, 8, "bf16", renorm=False)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["distill", "norm", "balance"])
    if op == "distill":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        vocab = _spread(rng, 512, VOCAB)
        rows = _spread(rng, 1, min(4 * SEQ, max(1, SEQ * VOCAB * 2 // (vocab * BYTES[dtype]) // 2)))
        ce = rng.choice([0.0, 0.3, 1.0])
        return _distill(rng.choice(["step", "forward", "backward"]), rows, vocab, _spread(rng, 1, 128), dtype,
                        rng.choice([1.0, 1.5, 2.0, 4.0]), ce, full=rng.random() < 0.3,
                        masked=rng.choice([0.0, 0.2]) if rows > 8 else 0.0,
                        padded=rng.choice([0, vocab // 50]))
    if op == "norm":
        hidden = _spread(rng, 64, WIDE)
        hidden = hidden if rng.random() < 0.3 else max(64, hidden // 16 * 16)
        rows = _spread(rng, 1, min(8 * SEQ, 4096 * WIDE // (hidden * 2)))
        many = rng.choice([0, 1, 4, rows])
        rows, gates = (max(many, rows // many * many), many) if many else (rows, 0)
        branch, stream = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        pre, post = rng.choice([("rms", "rms"), ("layer", "layer"), ("layer", "rms"), ("rms", "none"), ("none", "layer")])
        return _norm(rng.choice(["forward", "backward"]), rows, hidden, branch, stream, rng.choice(["bf16", "f32"]),
                     pre, post, gates, rng.choice(["none", "sigmoid"]) if gates else "none",
                     rs=rng.choice([1.0, 0.7]), bs=rng.choice([1.0, 0.3]))
    experts = _spread(rng, 4, 256)
    groups = rng.choice([1, 1, 4, 16])
    return _balance(rng.choice(["step", "forward"]), groups * _spread(rng, 1, 262144 // groups),
                    experts, _spread(rng, 1, min(8, experts)), rng.choice(["bf16", "f32"]), groups=groups,
                    masked=rng.choice([0.0, 0.15]), renorm=rng.random() < 0.5, z=rng.choice([0.0, 1e-3]))


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    return dict(case=case, **{"distill": _inputs_distill, "norm": _inputs_norm, "balance": _inputs_balance}[case["op"]](case, g))


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _rand(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def _inputs_distill(c, g):
    """Logits with a few tall ones in each row; the teacher sees the same
    tokens a little otherwise and keeps its k largest, in descending order, the
    last of them missing here and there."""
    rows, vocab, k = c["rows"], c["vocab"], min(c["k"], c["vocab"] - c["padded"])
    logits = torch.empty(rows, vocab, dtype=TYPES[c["dtype"]], device="cuda")
    ids = torch.empty(rows, k, dtype=torch.int32, device="cuda")
    top = torch.empty(rows, k, dtype=TYPES[c["dtype"]], device="cuda")
    lse = torch.empty(rows, device="cuda")
    for a in range(0, rows, 512):
        b = min(rows, a + 512)
        z = _randn(g, b - a, vocab).mul_(1.5)
        tall = torch.randint(0, vocab, (b - a, 1), device="cuda", generator=g) + torch.arange(24, device="cuda") * (vocab // 24)
        z.scatter_add_(1, tall % vocab, 12 * _rand(g, b - a, 24))
        if c["padded"]:
            z[:, vocab - c["padded"]:] = NEG
        logits[a:b] = z
        z.add_(_randn(g, b - a, vocab).mul_(0.5))
        t, i = z.topk(k, dim=1)
        ids[a:b], top[a:b] = i.int(), t.to(top.dtype)
        lse[a:b] = torch.logsumexp(z / c["temperature"], 1)
    ids[:, k // 2 + 1:][_rand(g, rows, max(0, k - k // 2 - 1)) < 0.05] = -1
    s = dict(logits=logits, ids=ids, top=top, teacher_lse=lse if c["full"] else None, labels=None, weight=None, saved=None, dloss=None)
    if c["ce"]:
        s["labels"] = torch.randint(0, vocab - c["padded"], (rows,), device="cuda", generator=g)
        s["labels"][_rand(g, rows) < 0.03] = -100
    if c["masked"]:
        s["weight"] = (_rand(g, rows) >= c["masked"]).float() / rows
    if c["way"] == "backward":   # what the forward pass left: the log-sum-exps at the temperature and at 1
        saved = torch.empty(rows, 2, device="cuda")
        for a in range(0, rows, 512):
            z = logits[a:a + 512].float()
            saved[a:a + 512, 0] = torch.logsumexp(z / c["temperature"], 1)
            saved[a:a + 512, 1] = torch.logsumexp(z, 1)
        s["saved"], s["dloss"] = saved, 0.5 + _rand(g, rows)
    return s


def _inputs_norm(c, g):
    rows, h, tb, ts, tw = c["rows"], c["hidden"], TYPES[c["branch"]], TYPES[c["stream"]], TYPES[c["weight"]]
    s = dict(x=None, r=None, stats=None, dr=None, dh=None, gate=None)
    s["y"] = (_randn(g, rows, h) * (0.5 + _rand(g, rows, 1)) + 0.1).to(tb)
    for n in ("pre", "post"):
        s[n + "_weight"] = (1 + 0.2 * _randn(g, h)).to(tw) if c[n] != "none" else None
        s[n + "_bias"] = (0.1 * _randn(g, h)).to(tw) if c[n] == "layer" else None
    if c["gates"]:
        s["gate"] = (0.6 + 0.5 * _randn(g, c["gates"], h)).to(tb)
    stream = (2 * _randn(g, rows, h) - 0.2).to(ts)
    if c["way"] == "forward":
        s["x"] = stream
    else:   # the forward pass left the new stream and each row's mean and 1/deviation, of the stream and of y
        s["r"] = stream
        s["stats"] = torch.cat([_moments(stream.float(), c["pre"]), _moments(s["y"].float(), c["post"])], 1)
        s["dr"] = (0.01 * _randn(g, rows, h)).to(ts)
        s["dh"] = (0.02 * _randn(g, rows, h)).to(tb) if c["pre"] != "none" else None
    return s


def _inputs_balance(c, g):
    t, e = c["tokens"], c["experts"]
    z = _randn(g, t, e) + torch.linspace(0.8, -0.8, e, device="cuda")    # some experts are liked more
    s = dict(logits=z.to(TYPES[c["dtype"]]), mask=None, dweights=None)
    if c["masked"]:
        s["mask"] = _rand(g, t) >= c["masked"]
    if c["way"] == "step":
        s["dweights"] = 0.01 * _randn(g, t, c["k"])
    return s


# ----------------------------------------------------------------- the work

def work(case):
    c = case
    if c["op"] == "distill":
        n, live = c["rows"] * c["vocab"], 1.0 - c["masked"]
        moved = {"forward": live, "backward": live + 1, "step": live + 1}[c["way"]]   # a masked row's gradient is zeros
        exps = (2 if c["way"] == "step" else 1) * (2 if c["ce"] and c["temperature"] != 1 else 1)
        return dict(bytes=n * BYTES[c["dtype"]] * moved + c["rows"] * c["k"] * (4 + BYTES[c["dtype"]]),
                    flops=n * live * 3 * exps)
    if c["op"] == "norm":
        n, b, s = c["rows"] * c["hidden"], BYTES[c["branch"]], BYTES[c["stream"]]
        pre, each, h = c["pre"] != "none", c["gates"] * c["hidden"], c["hidden"] * BYTES[c["weight"]]
        vectors = h * ((c["pre"] != "none") + (c["pre"] == "layer") + (c["post"] != "none") + (c["post"] == "layer"))
        if c["way"] == "forward":
            return dict(bytes=n * (2 * s + b + b * pre) + each * b + vectors, flops=14 * n)
        return dict(bytes=n * ((2 if pre else 1) * s + s + 2 * b + b * pre) + 2 * each * b + 2 * vectors, flops=36 * n)
    n, b = c["tokens"] * c["experts"], BYTES[c["dtype"]]
    step = c["way"] == "step"
    return dict(bytes=n * b * (2 if step else 1) + c["tokens"] * c["k"] * (16 if step else 8), flops=(20 if step else 12) * n)


# ------------------------------------------------------------------ the run

def run(state):
    c = state["case"]
    return {"distill": _run_distill, "norm": _run_norm, "balance": _run_balance}[c["op"]](c, state)


def _run_distill(c, s):
    if own:
        from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
        how = dict(temperature=c["temperature"], ce_weight=c["ce"], labels=s["labels"], row_weight=s["weight"],
                   teacher_lse=s["teacher_lse"])
        if c["way"] == "forward":
            loss, lse = ops.distill_forward(s["logits"], s["ids"], s["top"], **how)
            return dict(loss=loss, lse=lse)
        if c["way"] == "backward":
            return dict(dlogits=ops.distill_backward(s["logits"], s["ids"], s["top"], s["saved"], s["dloss"], **how))
        loss, dlogits = ops.distill_loss_grad(s["logits"], s["ids"], s["top"], **how)
        return dict(loss=loss, dlogits=dlogits)

    temp, rows = c["temperature"], s["logits"].shape[0]
    z = s["logits"].float()
    w = s["weight"] if s["weight"] is not None else torch.ones(rows, device=z.device)
    live = w != 0
    valid = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    t = torch.where(valid, s["top"].float() / temp, torch.full_like(s["top"], NEG, dtype=F32))
    if s["teacher_lse"] is None:
        high = t.amax(1, keepdim=True).clamp(min=-1e30)
        total = (t - high).exp().sum(1, keepdim=True)
        logp = t - high - total.log()
    else:
        logp = t - s["teacher_lse"][:, None]
    p = torch.where(valid, logp.exp(), torch.zeros_like(t))
    mass = p.sum(1)
    has_label = s["labels"] >= 0 if s["labels"] is not None else torch.zeros(rows, dtype=torch.bool, device=z.device)
    label = s["labels"].clamp(min=0) if s["labels"] is not None else None
    if s["saved"] is None:
        top = z.amax(1, keepdim=True)
        lse_t = (top / temp + ((z - top) / temp).exp_().sum(1, keepdim=True).log()).squeeze(1)
        if temp == 1.0 or not c["ce"]:
            lse_1 = lse_t
        else:
            lse_1 = (top + (z - top).exp_().sum(1, keepdim=True).log()).squeeze(1)
    else:
        lse_t, lse_1 = s["saved"][:, 0], s["saved"][:, 1]
    out = {}
    if c["way"] != "backward":
        there = z.gather(1, at) / temp
        terms = torch.where(p > 0, p * (logp - there + lse_t[:, None]), torch.zeros_like(p))
        loss = temp * temp * terms.sum(1)
        if label is not None:
            loss = loss + c["ce"] * torch.where(has_label, lse_1 - z.gather(1, label[:, None]).squeeze(1), torch.zeros_like(lse_1))
        out["loss"] = torch.where(live, w * loss, torch.zeros_like(loss))
    if c["way"] == "forward":
        lse = torch.stack([lse_t, lse_1], 1)
        out["lse"] = torch.where(live[:, None], lse, torch.zeros_like(lse))
        return out
    scale = torch.where(live, w * s["dloss"] if s["dloss"] is not None else w, torch.zeros_like(w))
    grad = (z / temp - lse_t[:, None]).exp_().mul_((scale * temp * mass)[:, None])
    if label is not None:
        hard = c["ce"] * scale * has_label
        grad += (z - lse_1[:, None]).exp_().mul_(hard[:, None])
        grad.scatter_add_(1, label[:, None], -hard[:, None])
    grad.scatter_add_(1, at, -(scale * temp)[:, None] * p)
    out["dlogits"] = grad.to(s["logits"].dtype)
    return out


EPS = 1e-5


def _moments(x, kind):
    """Each row's mean (0 for an rms norm) and 1 / sqrt(mean square of the rest + eps)."""
    if kind == "none":
        return torch.zeros(x.shape[0], 2, device=x.device)
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros(x.shape[0], 1, device=x.device)
    rest = x - mean
    return torch.cat([mean, (rest.square().mean(1, keepdim=True) + EPS).rsqrt()], 1)


def _norm_gradient(upstream, hat, rstd, weight, kind):
    """Gradients of an input, a weight and a bias from that of (hat * weight + bias)."""
    a = upstream * weight
    dx = a - hat * (a * hat).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - a.mean(1, keepdim=True)
    return dx * rstd, (upstream * hat).sum(0), upstream.sum(0)


def _run_norm(c, s):
    if own:
        from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
        how = dict(pre=c["pre"], post=c["post"], pre_weight=s["pre_weight"], pre_bias=s["pre_bias"],
                   post_weight=s["post_weight"], post_bias=s["post_bias"], gate=s["gate"], gate_act=c["act"],
                   residual_scale=c["rs"], branch_scale=c["bs"], eps=EPS)
        if c["way"] == "forward":
            r, h, stats = ops.norm_gate_forward(s["x"], s["y"], **how)
            return dict(r=r, h=h, stats=stats)
        return ops.norm_gate_backward(s["dr"], s["dh"], s["r"], s["y"], s["stats"], **how)

    rows, h, gates = c["rows"], c["hidden"], c["gates"]
    y = s["y"].float()
    gate = None
    if gates:
        gate = s["gate"].float()
        gate = (gate.sigmoid() if c["act"] == "sigmoid" else gate)[:, None, :].expand(gates, rows // gates, h).reshape(rows, h)
    weight = {n: s[n + "_weight"].float() if c[n] != "none" else None for n in ("pre", "post")}
    if c["way"] == "forward":
        post = _moments(y, c["post"])
        u = y
        if c["post"] != "none":
            u = (y - post[:, :1]) * post[:, 1:] * weight["post"]
            u = u + s["post_bias"].float() if c["post"] == "layer" else u
        u = u * c["bs"] if gate is None else u * gate * c["bs"]
        r = s["x"].float() * c["rs"] + u
        pre = _moments(r, c["pre"])
        out = dict(r=r.to(s["x"].dtype), h=None, stats=torch.cat([pre, post], 1))
        if c["pre"] != "none":
            v = (r - pre[:, :1]) * pre[:, 1:] * weight["pre"]
            v = v + s["pre_bias"].float() if c["pre"] == "layer" else v
            out["h"] = v.to(s["y"].dtype)
        return out

    out = dict(dx=None, dy=None, dgate=None, dpre_weight=None, dpre_bias=None, dpost_weight=None, dpost_bias=None)
    flow = s["dr"].float()
    if c["pre"] != "none":
        hat = (s["r"].float() - s["stats"][:, 0:1]) * s["stats"][:, 1:2]
        dr, dw, db = _norm_gradient(s["dh"].float(), hat, s["stats"][:, 1:2], weight["pre"], c["pre"])
        flow = flow + dr
        out["dpre_weight"] = dw.to(s["pre_weight"].dtype)
        out["dpre_bias"] = db.to(s["pre_bias"].dtype) if c["pre"] == "layer" else None
    out["dx"] = (flow * c["rs"]).to(s["r"].dtype)
    flow = flow * c["bs"]
    hat, u = None, y
    if c["post"] != "none":
        hat = (y - s["stats"][:, 2:3]) * s["stats"][:, 3:4]
        u = hat * weight["post"]
        u = u + s["post_bias"].float() if c["post"] == "layer" else u
    if gates:
        dgate = (flow * u).reshape(gates, rows // gates, h).sum(1)
        if c["act"] == "sigmoid":
            a = s["gate"].float().sigmoid()
            dgate = dgate * a * (1 - a)
        out["dgate"] = dgate.to(s["gate"].dtype)
        flow = flow * gate
    if c["post"] != "none":
        flow, dw, db = _norm_gradient(flow, hat, s["stats"][:, 3:4], weight["post"], c["post"])
        out["dpost_weight"] = dw.to(s["post_weight"].dtype)
        out["dpost_bias"] = db.to(s["post_bias"].dtype) if c["post"] == "layer" else None
    out["dy"] = flow.to(s["y"].dtype)
    return out


BALANCE = 1e-2


def _run_balance(c, s):
    if own:
        from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
        how = dict(mask=s["mask"], groups=c["groups"], balance_weight=BALANCE, z_weight=c["z"], renormalise=c["renorm"])
        ids, weights, counts, loss, saved = ops.balance_forward(s["logits"], c["k"], **how)
        out = dict(ids=ids, weights=weights, counts=counts, loss=loss)
        if c["way"] == "step":
            out["dlogits"] = ops.balance_backward(s["logits"], ids, counts, saved, s["dweights"], **how)
        return out

    t, e, k, groups = c["tokens"], c["experts"], c["k"], c["groups"]
    z = s["logits"].float()
    live = s["mask"] if s["mask"] is not None else torch.ones(t, dtype=torch.bool, device=z.device)
    ids = z.sort(dim=1, descending=True, stable=True).indices[:, :k]
    lse = z.amax(1, keepdim=True)
    lse = lse + (z - lse).exp().sum(1, keepdim=True).log()
    p = (z - lse).exp() * live[:, None]
    chosen = torch.zeros_like(z).scatter_(1, ids, 1.0) * live[:, None]
    weights = p.gather(1, ids)
    if c["renorm"]:
        weights = weights / torch.where(live[:, None], weights.sum(1, keepdim=True), torch.ones_like(lse))
    counts = chosen.reshape(groups, t // groups, e).sum(1)
    n = live.reshape(groups, -1).sum(1).float().clamp(min=1)[:, None]
    f = counts * (e / k) / n
    mean = p.reshape(groups, t // groups, e).sum(1) / n
    squares = (lse.squeeze(1).square() * live).reshape(groups, -1).sum(1) / n.squeeze(1)
    loss = (BALANCE * (f * mean).sum(1) + c["z"] * squares).sum() / groups
    out = dict(ids=torch.where(live[:, None], ids, torch.full_like(ids, -1)).int(), weights=weights, counts=counts.int(), loss=loss)
    if c["way"] == "step":
        each = (t // groups, e)
        f, n = (v[:, None, :].expand(groups, *each[:1], v.shape[1]).reshape(t, -1) for v in (f, n))
        grad = BALANCE * p * (f - (f * p).sum(1, keepdim=True)) + c["z"] * 2 * lse * p
        grad = grad / (n * groups)
        up = torch.zeros_like(z).scatter_(1, ids, s["dweights"])
        if c["renorm"]:
            w = torch.zeros_like(z).scatter_(1, ids, weights)
            grad = grad + w * (up - (up * w).sum(1, keepdim=True))
        else:
            grad = grad + p * (up - (up * p).sum(1, keepdim=True))
        out["dlogits"] = (grad * live[:, None]).to(s["logits"].dtype)
    return out


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"distill": _exact_distill, "norm": _exact_norm, "balance": _exact_balance}[case["op"]](case, s)


def _exact_distill(c, s):
    """Row by row blocks; the gradient is autograd's."""
    temp, rows = c["temperature"], c["rows"]
    losses, lses, grads = [], [], []
    for a in range(0, rows, 128):
        b = slice(a, min(rows, a + 128))
        z = s["logits"][b].double().requires_grad_(True)
        with torch.enable_grad():
            student = torch.log_softmax(z / temp, 1)
            valid = s["ids"][b] >= 0
            t = s["top"][b].double() / temp
            if s["teacher_lse"] is None:
                logp = torch.log_softmax(t.masked_fill(~valid, -1e300), 1)
            else:
                logp = t - s["teacher_lse"][b].double()[:, None]
            p = logp.exp() * valid
            q = student.gather(1, s["ids"][b].clamp(min=0).long())
            loss = temp ** 2 * torch.where(p > 0, p * (logp - q), torch.zeros_like(p)).sum(1)
            if s["labels"] is not None:
                loss = loss + c["ce"] * torch.nn.functional.nll_loss(torch.log_softmax(z, 1), s["labels"][b], ignore_index=-100, reduction="none")
            w = s["weight"][b].double() if s["weight"] is not None else torch.ones_like(loss)
            loss = loss * w
            up = s["dloss"][b].double() if s["dloss"] is not None else torch.ones_like(loss)
            if c["way"] != "forward":
                grads.append(torch.autograd.grad((loss * up).sum(), z)[0])
        losses.append(loss.detach())
        both = torch.stack([torch.logsumexp(z.detach() / temp, 1), torch.logsumexp(z.detach(), 1)], 1)
        if temp != 1 and not c["ce"]:
            both[:, 1] = both[:, 0]
        lses.append(both * (w != 0)[:, None])
    if c["way"] == "forward":
        return dict(loss=torch.cat(losses), lse=torch.cat(lses))
    if c["way"] == "backward":
        return dict(dlogits=torch.cat(grads))
    return dict(loss=torch.cat(losses), dlogits=torch.cat(grads))


def _exact_norm(c, s):
    def normed(v, n):
        w, b = (None if s[n + k] is None else leaf[n + k] for k in ("_weight", "_bias"))
        if c[n] == "none":
            return v
        if c[n] == "layer":
            return torch.nn.functional.layer_norm(v, v.shape[1:], w, b, EPS)
        return v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w

    def stat(v, kind):
        if kind == "none":
            return torch.zeros_like(v[:, :2])
        var, mean = torch.var_mean(v, 1, correction=0) if kind == "layer" else ((v * v).mean(1), torch.zeros_like(v[:, 0]))
        return torch.stack([mean, 1 / torch.sqrt(var + EPS)], 1)

    leaf = {n: v.double().requires_grad_(True) for n, v in s.items()
            if torch.is_tensor(v) and n in ("y", "x", "r", "gate", "pre_weight", "pre_bias", "post_weight", "post_bias")}
    with torch.enable_grad():
        u = normed(leaf["y"], "post")
        if c["gates"]:
            gate = torch.sigmoid(leaf["gate"]) if c["act"] == "sigmoid" else leaf["gate"]
            u = u * gate.repeat_interleave(c["rows"] // c["gates"], 0)
        if c["way"] == "forward":
            r = c["rs"] * leaf["x"] + c["bs"] * u
            h = normed(r, "pre").detach() if c["pre"] != "none" else None
            r = r.detach()
            return dict(r=r, h=h, stats=torch.cat([stat(r, c["pre"]), stat(leaf["y"].detach(), c["post"])], 1))
        out = dict(dpre_weight=None, dpre_bias=None, dpost_weight=None, dpost_bias=None, dgate=None)
        flow = s["dr"].double()
        if c["pre"] != "none":
            names = [n for n in ("r", "pre_weight", "pre_bias") if n in leaf]
            got = dict(zip(names, torch.autograd.grad(normed(leaf["r"], "pre"), [leaf[n] for n in names], s["dh"].double())))
            flow = flow + got.pop("r")
            out.update({"d" + n: v for n, v in got.items()})
        names = [n for n in ("y", "gate", "post_weight", "post_bias") if n in leaf]
        got = torch.autograd.grad(u, [leaf[n] for n in names], flow * c["bs"])
        out.update({"d" + n: v for n, v in zip(names, got)})
    return dict(out, dx=flow * c["rs"])


def _exact_balance(c, s):
    t, e, k, groups = c["tokens"], c["experts"], c["k"], c["groups"]
    z = s["logits"].double().requires_grad_(True)
    live = s["mask"] if s["mask"] is not None else torch.ones(t, dtype=torch.bool, device=z.device)
    order = torch.argsort(-z.detach(), dim=1, stable=True)[:, :k]
    with torch.enable_grad():
        p = torch.softmax(z, 1)
        weights = p.gather(1, order)
        weights = weights / weights.sum(1, keepdim=True) if c["renorm"] else weights
        weights = weights.masked_fill(~live[:, None], 0.0)
        loss, counts = torch.zeros((), dtype=torch.float64, device=z.device), []
        for i in range(groups):
            at = torch.arange(i * (t // groups), (i + 1) * (t // groups), device=z.device)
            at = at[live[at]]
            counts.append(torch.bincount(order[at].flatten(), minlength=e))
            if len(at):
                f = counts[-1].double() * e / (k * len(at))
                loss = loss + BALANCE * (f * p[at].mean(0)).sum() + c["z"] * torch.logsumexp(z[at], 1).square().mean()
        loss = loss / groups
        out = dict(ids=order.masked_fill(~live[:, None], -1).int(), weights=weights.detach(), counts=torch.stack(counts).int(), loss=loss.detach())
        if c["way"] == "step":
            whole = loss + (weights * s["dweights"].double()).sum()
            out["dlogits"] = torch.autograd.grad(whole, z)[0]
    return out
