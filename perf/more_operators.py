"""Operators of a fine-tuning step beside the ones of `operators.py`: what is measured, and in which cases.

Five operators, each in both directions:

  policy      clipped policy loss with a KL term from a model's logits at the
              tokens that were sampled, its gradient, and the log-probabilities
              that it (or a frozen reference) gives to them;
  preference  loss of pairs of answers, one preferred to the other, from the sums of
              their tokens' log-probabilities against a reference's, and its gradient;
  glu8        the feed-forward block's activation (gated or not), whose inputs
              are kept in 8 bits for the backward pass, which works on what was kept;
  pack8       any activation kept in 8 bits and read back;
  rotary      positions turned into the queries and keys, and out of their gradients.

The 8 bits: runs of 32 columns of a row share a power of two 2^(b - 127), the
smallest by which the run's largest magnitude is at most 448 (b, one byte, is at least 0);
each value is divided by it and rounded to the nearest e4m3 number.

`run` computes them in their plain form (elementary torch operations in 32
bits, rounded once at the end), or, where `own` is true, by the calls that a
training program makes of the package.
"""
import math

import torch

own = False

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
TYPES = {"bf16": BF16, "f32": F32}
BYTES = {"bf16": 2, "f32": 4}

VOCAB = 250880          # the vocabulary of the scaled-down workload
SEQ = 2048              # its tokens per sequence
HIDDEN, WIDE = 2048, 14336   # hidden sizes of the scaled-down and the full model
RUN = 32                # columns that share a scale


# ---------------------------------------------------------------- the cases

def _policy(way, rows, vocab, dtype, old=True, ref=True, kl=0.02, temperature=1.0, masked=0.0, padded=0):
    """`old`: the sampler's log-probabilities are there (else the tokens are this
    model's own: ratio 1).  `masked`: share of rows that count for nothing.
    `padded`: vocabulary entries at the end that no token uses (logit -inf)."""
    return dict(op="policy", way=way, rows=rows, vocab=vocab, dtype=dtype, old=old, ref=ref, kl=kl,
                temperature=temperature, masked=masked, padded=padded)


def _preference(way, pairs, length, vocab, dtype, kind="sigmoid", beta=0.1, smoothing=0.0, margin=0.0, mean=False, spare=0):
    """`length`: longest sequence; they are between a quarter of it and all of
    it, a third of each a prompt.  `spare`: rows behind the last sequence."""
    return dict(op="preference", way=way, pairs=pairs, length=length, vocab=vocab, dtype=dtype, kind=kind, beta=beta,
                smoothing=smoothing, margin=margin, mean=mean, spare=spare)


def _glu8(way, rows, columns, dtype, act, gated=True, halves=False):
    """`halves`: gate and up are the two halves of one projection's rows."""
    return dict(op="glu8", way=way, rows=rows, columns=columns, dtype=dtype, act=act, gated=gated, halves=halves)


def _pack8(rows, columns, dtype):
    return dict(op="pack8", rows=rows, columns=columns, dtype=dtype)


def _rotary(way, tokens, heads, kv, dim, turned, dtype, layout, scaling="none", factor=1.0, far=0, fused=False):
    """`turned`: leading elements of each head that positions turn.  `far`: 0,
    sequences of up to SEQ tokens one after another; else every token somewhere below
    it (single tokens of many sequences).  `fused`: q and k are parts of one projection's rows."""
    return dict(op="rotary", way=way, tokens=tokens, heads=heads, kv=kv, dim=dim, turned=turned, dtype=dtype,
                layout=layout, scaling=scaling, factor=factor, far=far, fused=fused)


def listed():
    cases = [
        # a few tokens with a small odd vocabulary: a unit test's or a probe's step, latency only
        ("policy_few_tokens", _policy("step", 7, 2053, "bf16", ref=False, kl=0.0)),
        # one sequence of the scaled-down workload: loss and gradient as a training step takes them
        ("policy_sequence", _policy("step", SEQ, VOCAB, "bf16", masked=0.1, padded=200)),
        # the gradient by itself, as autograd asks for it, 32-bit logits, an odd vocabulary
        ("policy_gradient_f32", _policy("backward", 1021, 32003, "f32", temperature=0.8)),
        # a reference's log-probabilities of a batch of answers
        ("policy_reference_logp", _policy("logp", 4 * SEQ, 32000, "bf16", temperature=1.0, masked=0.2)),
        # one short pair: latency, and the sums' order of launches
        ("preference_short_pair", _preference("step", 1, 24, 2053, "f32", kind="ipo")),
        # a micro-batch of pairs at the workload's vocabulary, some rows unused
        ("preference_pairs", _preference("step", 4, 380, VOCAB, "bf16", smoothing=0.1, spare=41)),
        # a few rows with an odd width, no gate
        ("glu8_odd_rows", _glu8("step", 9, 1367, "f32", "gelu", gated=False)),
        # the full model's width, both halves of one projection, forward and backward
        ("glu8_wide", _glu8("step", SEQ, 4 * WIDE, "bf16", "silu", halves=True)),
        # the backward pass of four sequences of the scaled-down model
        ("glu8_gradient", _glu8("backward", 4 * SEQ, 4 * HIDDEN, "bf16", "gelu")),
        # a block's input of four sequences, kept and read back
        ("pack8_block_input", _pack8(4 * SEQ, WIDE, "bf16")),
        # single tokens of sixteen long sequences, positions scaled
        ("rotary_single_tokens", _rotary("forward", 16, 16, 16, 128, 128, "bf16", "half", "yarn", 16.0, far=500000)),
        # gradients of four sequences at the full model's heads, parts of one projection
        ("rotary_gradient_wide", _rotary("backward", 4 * SEQ, 112, 16, 128, 64, "bf16", "interleaved", fused=True)),
    ]
    return [dict(c, name=name) for name, c in cases]


def _spread(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["policy", "policy", "preference", "glu8", "glu8", "pack8", "rotary"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "policy":
        vocab = _spread(rng, 512, VOCAB)
        rows = _spread(rng, 1, min(4 * SEQ, SEQ * VOCAB * 2 // (vocab * BYTES[dtype]) // 2))
        kl = rng.choice([0.0, 0.01, 0.1])
        return _policy(rng.choice(["step", "step", "forward", "backward", "logp"]), rows, vocab, dtype, old=rng.random() < 0.8,
                       ref=kl > 0, kl=kl, temperature=rng.choice([1.0, 1.0, 0.7, 1.3]),
                       masked=rng.choice([0.0, 0.25]) if rows > 8 else 0.0, padded=rng.choice([0, vocab // 50]))
    if op == "preference":
        vocab = _spread(rng, 512, VOCAB)
        pairs = _spread(rng, 1, 32)
        length = _spread(rng, 4, max(4, min(SEQ, 2 * 380 * 4 * VOCAB * 2 // (vocab * BYTES[dtype] * 2 * pairs) // 2)))
        return _preference(rng.choice(["step", "step", "forward"]), pairs, length, vocab, dtype,
                           kind=rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"]), beta=rng.choice([0.05, 0.1, 0.5]),
                           smoothing=rng.choice([0.0, 0.1]), margin=rng.choice([0.0, 0.5]), mean=rng.random() < 0.3,
                           spare=rng.choice([0, 13]))
    if op == "glu8":
        columns = _spread(rng, 32, 4 * WIDE)
        columns = columns if rng.random() < 0.3 else max(32, columns // 16 * 16)
        rows = _spread(rng, 1, max(1, min(8 * SEQ, SEQ * 4 * WIDE * 2 // (columns * BYTES[dtype]) // 2)))
        gated = rng.random() < 0.7
        return _glu8(rng.choice(["step", "backward"]), rows, columns, dtype, rng.choice(["silu", "gelu"]), gated=gated,
                     halves=gated and rng.random() < 0.4)
    if op == "pack8":
        columns = _spread(rng, 32, WIDE)
        columns = columns if rng.random() < 0.3 else max(32, columns // 16 * 16)
        return _pack8(_spread(rng, 1, max(1, min(8 * SEQ, 4 * SEQ * WIDE * 2 // (columns * BYTES[dtype]) // 2))), columns, dtype)
    dim = rng.choice([32, 64, 80, 96, 128, 256])
    heads = rng.choice([1, 4, 16, 32, 112])
    kv = rng.choice([h for h in (1, 4, 16) if heads % h == 0] + [heads])
    scaling, factor = rng.choice([("none", 1.0), ("none", 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 16.0)])
    most = 4 * SEQ * 128 * 128 * 2 // ((heads + kv) * dim * BYTES[dtype])
    return _rotary(rng.choice(["forward", "backward"]), _spread(rng, 1, min(16 * SEQ, most)), heads, kv, dim,
                   rng.choice([dim, dim, dim // 2, max(4, dim // 4)]), dtype, rng.choice(["half", "interleaved"]), scaling,
                   factor, far=rng.choice([0, 0, 4000000]), fused=rng.random() < 0.4)


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2 + 1)
    make = {"policy": _inputs_policy, "preference": _inputs_preference, "glu8": _inputs_glu8, "pack8": _inputs_pack8,
            "rotary": _inputs_rotary}
    return dict(case=case, **make[case["op"]](case, g))


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _rand(g, *shape):
    return torch.rand(*shape, device="cuda", generator=g)


def _logits(g, rows, vocab, padded, dtype, temperature=1.0):
    """Logits with a few tall ones in each row, the tokens that were sampled from
    them (mostly tall ones) and those tokens' log-probabilities."""
    live = vocab - padded
    logits = torch.empty(rows, vocab, dtype=TYPES[dtype], device="cuda")
    labels = torch.empty(rows, dtype=torch.int64, device="cuda")
    logp = torch.empty(rows, device="cuda")
    for a in range(0, rows, 512):
        b = min(rows, a + 512)
        z = _randn(g, b - a, vocab).mul_(1.5)
        tall = (torch.randint(0, live, (b - a, 1), device="cuda", generator=g) + torch.arange(24, device="cuda") * (live // 24)) % live
        height = 14 * _rand(g, b - a, 24)
        z.scatter_add_(1, tall, height)
        pick = (height + 2 * _randn(g, b - a, 24)).argmax(1, keepdim=True)
        other = torch.randint(0, live, (b - a, 1), device="cuda", generator=g)
        label = torch.where(_rand(g, b - a, 1) < 0.9, tall.gather(1, pick), other)
        if padded:
            z[:, live:] = float("-inf")
        z = z.to(logits.dtype)
        logits[a:b] = z
        z = z.float() / temperature
        labels[a:b] = label.squeeze(1)
        logp[a:b] = z.gather(1, label).squeeze(1) - torch.logsumexp(z, 1)
    return logits, labels, logp


CLIP = (0.2, 0.28)   # the ratio's lower and upper clip


def _inputs_policy(c, g):
    """Old log-probabilities some updates away (not within a thousandth of a clip's
    border, where 32 bits say either), a reference's a little further, and
    advantages of whole answers."""
    rows = c["rows"]
    logits, labels, logp = _logits(g, rows, c["vocab"], c["padded"], c["dtype"], c["temperature"])
    s = dict(logits=logits, labels=labels, old=None, ref=None, weight=None, saved=None, dloss=None)
    if c["old"]:
        moved = 0.15 * _randn(g, rows)
        for border in (1 - CLIP[0], 1 + CLIP[1]):
            moved = torch.where((moved - math.log(border)).abs() < 1e-3, torch.zeros_like(moved), moved)
        s["old"] = logp - moved
    if c["ref"]:
        s["ref"] = logp + 0.3 * _randn(g, rows)
    answers = max(1, rows // 256)
    s["advantage"] = _randn(g, answers).repeat_interleave(-(-rows // answers))[:rows].contiguous()
    if c["masked"]:
        s["weight"] = (_rand(g, rows) >= c["masked"]).float() / rows
    if c["way"] == "backward":   # what the forward pass left of each row: largest logit, sum, loss by log-probability, index
        saved = torch.empty(rows, 4, device="cuda")
        for a in range(0, rows, 512):
            z = logits[a:a + 512].float()
            saved[a:a + 512, 0] = z.amax(1)
            saved[a:a + 512, 1] = ((z - saved[a:a + 512, :1]) / c["temperature"]).exp().sum(1)
        slope = _policy_terms(c, s, logp)[1]
        live = s["weight"] != 0 if s["weight"] is not None else torch.ones(rows, dtype=torch.bool, device="cuda")
        saved[:, 2] = torch.where(live, slope, torch.zeros_like(slope))
        saved.view(torch.int32)[:, 3] = torch.where(live, torch.arange(rows, device="cuda"), -1).int()
        saved[:, :2] *= live[:, None]
        s["saved"], s["dloss"] = saved, 0.5 + _rand(g, rows)
    return s


def _inputs_preference(c, g):
    pairs, longest = c["pairs"], c["length"]
    low = max(2, longest // 4)
    lengths = torch.randint(low, max(low, longest) + 1, (2 * pairs,), device="cuda", generator=g)
    offsets = torch.zeros(2 * pairs + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = lengths.cumsum(0)
    # the batch's rows are fixed by the plan (the longest that it may be), the sequences fill them from the front
    rows = 2 * pairs * longest + c["spare"]
    logits, labels, logp = _logits(g, rows, c["vocab"], 0, c["dtype"])
    row = torch.arange(rows, device="cuda")
    which = torch.searchsorted(offsets[1:].long(), row, right=True).clamp(max=2 * pairs - 1)
    prompt = row - offsets[which] < lengths[which] // 3
    labels[prompt | (row >= offsets[-1])] = -100
    counted = labels >= 0
    sums = torch.zeros(2 * pairs, dtype=F64, device="cuda").index_add_(0, which[counted], logp[counted].double())
    if c["mean"]:
        n = torch.zeros(2 * pairs, dtype=F64, device="cuda").index_add_(0, which[counted], torch.ones_like(logp[counted], dtype=F64))
        sums = sums / n.clamp(min=1)
    ref = (sums + (1.0 if c["mean"] else 8.0) * _randn(g, 2 * pairs)).float()
    return dict(logits=logits, labels=labels, offsets=offsets, ref=ref)


def _codes(x):
    """(codes, scales) of [rows, columns], as the package keeps them: bytes [rows, 32 runs] and [rows, runs]."""
    values, exponent = _kept(x.float())
    rows, columns = x.shape
    runs = exponent.shape[1]
    codes = torch.zeros(rows, runs * RUN, dtype=torch.uint8, device=x.device)
    codes[:, :columns] = values[:, :columns].to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (exponent + 127).to(torch.uint8)


def _power(exponent):
    """2^exponent in 32 bits, exactly (the GPU's powers are not), from -127 on."""
    bits = torch.where(exponent > -127, (exponent + 127) << 23, torch.full_like(exponent, 1 << 22))
    return bits.int().view(F32)


def _kept(x):
    """What e4m3 holds of [rows, columns] (columns filled up to whole runs), and each run's exponent."""
    rows, columns = x.shape
    runs = -(-columns // RUN)
    full = torch.zeros(rows, runs * RUN, dtype=x.dtype, device=x.device)
    full[:, :columns] = x
    fraction, exponent = torch.frexp(full.reshape(rows, runs, RUN).abs().amax(2))
    exponent = torch.where(fraction > 0.875, exponent - 8, exponent - 9)
    exponent = torch.where(fraction == 0, torch.full_like(exponent, -127), exponent).clamp(min=-127)
    scaled = full.reshape(rows, runs, RUN) * _power(-exponent)[:, :, None]
    return scaled.to(torch.float8_e4m3fn).to(x.dtype).reshape(rows, runs * RUN), exponent


def _read(values, exponent, columns):
    rows, runs = exponent.shape
    return (values.reshape(rows, runs, RUN) * _power(exponent)[:, :, None]).reshape(rows, runs * RUN)[:, :columns]


def _inputs_glu8(c, g):
    rows, n, t = c["rows"], c["columns"], TYPES[c["dtype"]]
    wide = 1 + c["halves"]
    both = torch.empty(rows, wide * n, dtype=t, device="cuda")
    for a in range(0, rows, 1024):    # activations with columns and rows that are larger than the others
        x = _randn(g, min(1024, rows - a), wide * n)
        x *= 0.3 + 2 * _rand(g, x.shape[0], 1)
        both[a:a + 1024] = x
    gate = both[:, :n]
    up = None
    if c["gated"]:
        up = both[:, n:] if c["halves"] else (1.5 * _randn(g, rows, n)).to(t)
    s = dict(gate=gate, up=up, dh=(0.02 * _randn(g, rows, n)).to(t), codes=None, scales=None)
    if c["way"] == "backward":
        parts = [_codes(x) for x in ([gate, up] if c["gated"] else [gate])]
        s["codes"], s["scales"] = (torch.stack([p[i] for p in parts]) for i in range(2))
        s["gate"] = s["up"] = None
    return s


def _inputs_pack8(c, g):
    x = _randn(g, c["rows"], c["columns"])
    x *= torch.exp(_randn(g, 1, c["columns"]))
    return dict(x=x.to(TYPES[c["dtype"]]))


def _inputs_rotary(c, g):
    t, h, kv, d, dtype = c["tokens"], c["heads"], c["kv"], c["dim"], TYPES[c["dtype"]]
    if c["fused"]:
        rows = _randn(g, t, h + 2 * kv, d).to(dtype)
        q, k = rows[:, :h], rows[:, h:h + kv]
    else:
        q, k = _randn(g, t, h, d).to(dtype), _randn(g, t, kv, d).to(dtype)
    if c["far"]:
        positions = torch.randint(0, c["far"], (t,), device="cuda", generator=g)
    else:
        ends = torch.randint(1, SEQ + 1, (t // 64 + 2,), device="cuda", generator=g).cumsum(0)
        row = torch.arange(t, device="cuda")
        which = torch.searchsorted(ends, row, right=True).clamp(max=len(ends) - 1)
        positions = row - torch.where(which > 0, ends[(which - 1).clamp(min=0)], torch.zeros_like(row))
    return dict(q=q, k=k, positions=positions)


# ----------------------------------------------------------------- the work

def work(case):
    c = case
    if c["op"] == "policy":
        n, live = c["rows"] * c["vocab"], 1.0 - c["masked"]
        moved = {"logp": live, "forward": live, "backward": live + 1, "step": live + 1}[c["way"]]   # a masked row's gradient is zeros
        return dict(bytes=n * BYTES[c["dtype"]] * moved + c["rows"] * 24, flops=n * live * (6 if c["way"] == "step" else 3))
    if c["op"] == "preference":
        rows = 2 * c["pairs"] * c["length"] + c["spare"]
        live = 2 * c["pairs"] * c["length"] * (1 + max(2, c["length"] // 4) / c["length"]) / 2 * 2 / 3   # on average: the rest is prompt, or unused
        n = c["vocab"] * BYTES[c["dtype"]]
        return dict(bytes=n * (live + rows * (c["way"] == "step")) + rows * 16, flops=c["vocab"] * live * (6 if c["way"] == "step" else 3))
    if c["op"] == "glu8":
        n, b, parts = c["rows"] * c["columns"], BYTES[c["dtype"]], 1 + c["gated"]
        kept = parts * (1 + 1 / RUN)
        forward, backward = parts * b + b + kept, b + kept + parts * b
        return dict(bytes=n * (backward + (forward if c["way"] == "step" else 0)), flops=n * 20 * parts)
    if c["op"] == "pack8":
        return dict(bytes=c["rows"] * c["columns"] * (2 * BYTES[c["dtype"]] + 2 * (1 + 1 / RUN)), flops=8 * c["rows"] * c["columns"])
    n = c["tokens"] * (c["heads"] + c["kv"]) * c["dim"]
    return dict(bytes=2 * n * BYTES[c["dtype"]] + 8 * c["tokens"], flops=3 * n)


# ------------------------------------------------------------------ the run

def run(state):
    c = state["case"]
    go = {"policy": _run_policy, "preference": _run_preference, "glu8": _run_glu8, "pack8": _run_pack8, "rotary": _run_rotary}
    return go[c["op"]](c, state)


def _policy_terms(c, s, logp):
    """Each row's loss and its derivative by the row's log-probability, the row's weight in both."""
    ratio = (logp - s["old"]).exp() if s["old"] is not None else torch.ones_like(logp)
    adv = s["advantage"].to(logp.dtype)
    kept = torch.where(adv >= 0, ratio.clamp(max=1 + CLIP[1]), ratio.clamp(min=1 - CLIP[0]))
    loss = -kept * adv
    slope = torch.where(kept == ratio, -ratio * adv, torch.zeros_like(adv))
    if s["ref"] is not None:
        d = s["ref"] - logp
        loss = loss + c["kl"] * (d.expm1() - d)
        slope = slope - c["kl"] * d.expm1()
    if s["weight"] is not None:
        loss, slope = loss * s["weight"], slope * s["weight"]
    return loss, slope


def _sums(z, temperature):
    top = z.amax(1, keepdim=True)
    return top.squeeze(1), ((z - top) / temperature).exp_().sum(1)


def _softmax_gradient(z, top, total, labels, scale, temperature):
    """scale / temperature ([j = label] - softmax(z / temperature)_j)"""
    scale = scale / temperature
    grad = ((z - top[:, None]) / temperature).exp_().mul_((-scale / total)[:, None])
    return grad.scatter_add_(1, labels.clamp(min=0)[:, None], scale[:, None])


def _run_policy(c, s):
    if own:
        from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
        how = dict(temperature=c["temperature"], row_weight=s["weight"])
        if c["way"] == "logp":
            logp, saved = ops.token_logp_forward(s["logits"], s["labels"], **how)
            return dict(logp=logp, top=saved[:, 0], sum=saved[:, 1])
        if c["way"] == "backward":
            return dict(dlogits=ops.token_logp_backward(s["logits"], s["labels"], s["saved"], s["dloss"], temperature=c["temperature"]))
        how.update(old_logp=s["old"], ref_logp=s["ref"], clip_low=CLIP[0], clip_high=CLIP[1], kl_weight=c["kl"])
        if c["way"] == "forward":
            loss, logp, saved = ops.policy_forward(s["logits"], s["labels"], s["advantage"], **how)
            return dict(loss=loss, logp=logp, top=saved[:, 0], sum=saved[:, 1], slope=saved[:, 2])
        loss, logp, dlogits = ops.policy_loss_grad(s["logits"], s["labels"], s["advantage"], **how)
        return dict(loss=loss, logp=logp, dlogits=dlogits)

    z, temp = s["logits"].float(), c["temperature"]
    if c["way"] == "backward":
        top, total, slope = s["saved"][:, 0], s["saved"][:, 1], s["saved"][:, 2]
        grad = _softmax_gradient(z, top, total.clamp(min=1), s["labels"], slope * s["dloss"], temp)
        return dict(dlogits=grad.to(s["logits"].dtype))
    live = s["weight"] != 0 if s["weight"] is not None else torch.ones(c["rows"], dtype=torch.bool, device=z.device)
    zero = torch.zeros(c["rows"], device=z.device)
    top, total = _sums(z, temp)
    logp = (z.gather(1, s["labels"][:, None]).squeeze(1) - top) / temp - total.log()
    if c["way"] == "logp":
        return dict(logp=torch.where(live, logp, zero), top=torch.where(live, top, zero), sum=torch.where(live, total, zero))
    loss, slope = _policy_terms(c, s, logp)
    loss, slope, logp = torch.where(live, loss, zero), torch.where(live, slope, zero), torch.where(live, logp, zero)
    if c["way"] == "forward":
        return dict(loss=loss, logp=logp, top=torch.where(live, top, zero), sum=torch.where(live, total, zero), slope=slope)
    grad = _softmax_gradient(z, top, total, s["labels"], slope, temp)
    return dict(loss=loss, logp=logp, dlogits=grad.to(s["logits"].dtype))


def _pair_terms(c, m):
    """A pair's loss and its derivative by what it is of: h (ipo) or the margin m."""
    if c["kind"] == "ipo":
        d = m - 0.5 / c["beta"]
        return d * d, 2 * d
    if c["kind"] == "hinge":
        return (1 - m).clamp(min=0), -(m < 1).to(m.dtype)
    e = c["smoothing"]
    soft = torch.log1p(torch.exp(-m.abs()))
    loss = (1 - e) * (soft + (-m).clamp(min=0)) + e * (soft + m.clamp(min=0))
    return loss, e * torch.sigmoid(m) - (1 - e) * torch.sigmoid(-m)


def _run_preference(c, s):
    if own:
        from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
        how = dict(ref_logp=s["ref"], kind=c["kind"], beta=c["beta"], label_smoothing=c["smoothing"], margin=c["margin"],
                   length_normalise=c["mean"])
        loss, logp, saved = ops.preference_forward(s["logits"], s["labels"], s["offsets"], **how)
        out = dict(loss=loss, logp=logp)
        if c["way"] == "step":
            out["dlogits"] = ops.token_logp_backward(s["logits"], s["labels"], saved)
        return out

    pairs, z = c["pairs"], s["logits"].float()
    rows = z.shape[0]
    row = torch.arange(rows, device=z.device)
    which = torch.searchsorted(s["offsets"][1:].long(), row, right=True)
    counted = (which < 2 * pairs) & (s["labels"] >= 0)
    which = which.clamp(max=2 * pairs - 1)
    top, total = _sums(z, 1.0)
    each = (z.gather(1, s["labels"].clamp(min=0)[:, None]).squeeze(1) - top).double() - total.double().log()   # long sums: in 64 bits
    each = torch.where(counted, each, torch.zeros_like(each))
    logp = torch.zeros(2 * pairs, dtype=F64, device=z.device).index_add_(0, which, each)
    share = torch.ones_like(logp)
    if c["mean"]:
        share = 1 / torch.zeros_like(logp).index_add_(0, which, counted.double()).clamp(min=1)
    logp = logp * share
    rel = logp - s["ref"].double()
    h = rel[:pairs] - rel[pairs:]
    inner = 1.0 if c["kind"] == "ipo" else c["beta"]
    loss, slope = _pair_terms(c, inner * h - c["margin"])
    out = dict(loss=loss.float(), logp=logp.float())
    if c["way"] == "step":
        slope = torch.cat([slope, -slope]) * inner * share
        scale = torch.where(counted, slope[which], torch.zeros_like(each)).float()
        out["dlogits"] = _softmax_gradient(z, top, total, s["labels"], scale, 1.0).to(s["logits"].dtype)
    return out


ROOT = math.sqrt(2 / math.pi)


def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = g.sigmoid()
        return g * s, s * (1 + g * (1 - s))
    t = torch.tanh(ROOT * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * ROOT * (1 + 3 * 0.044715 * g * g)


def _run_glu8(c, s):
    if own:
        from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
        if c["way"] == "backward":
            dgate, dup = ops.glu8_backward(s["dh"], s["codes"], s["scales"], act=c["act"])
            return dict(dgate=dgate, dup=dup)
        h, codes, scales = ops.glu8_forward(s["gate"], s["up"], act=c["act"])
        dgate, dup = ops.glu8_backward(s["dh"], codes, scales, act=c["act"])
        return dict(h=h, dgate=dgate, dup=dup)

    n, t, out, up = c["columns"], s["dh"].dtype, {}, None
    if c["way"] == "backward":
        exponents = s["scales"].int() - 127
        gate = _read(s["codes"][0].view(torch.float8_e4m3fn).float(), exponents[0], n)
        if c["gated"]:
            up = _read(s["codes"][1].view(torch.float8_e4m3fn).float(), exponents[1], n)
    else:
        a = _act(s["gate"].float(), c["act"])[0]
        out["h"] = (a * s["up"].float() if c["gated"] else a).to(t)
        gate = _read(*_kept(s["gate"].float()), n)
        if c["gated"]:
            up = _read(*_kept(s["up"].float()), n)
    a, da = _act(gate, c["act"])
    dh = s["dh"].float()
    out["dgate"] = (dh * up * da if c["gated"] else dh * da).to(t)
    out["dup"] = (dh * a).to(t) if c["gated"] else None
    return out


def _run_pack8(c, s):
    if own:
        from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
        codes, scales = ops.pack8(s["x"])
        return dict(x=ops.unpack8(codes, scales, c["columns"], dtype=s["x"].dtype))
    return dict(x=_read(*_kept(s["x"].float()), c["columns"]).to(s["x"].dtype))


BASE = 10000.0


def _frequencies(c):
    """Radians per position of each turned pair (64 bits, on the GPU), and the factor on the turned pairs' length."""
    d = c["turned"]
    base = BASE * c["factor"] ** (d / (d - 2)) if c["scaling"] == "ntk" else BASE
    f = base ** (-torch.arange(0, d, 2, dtype=F64, device="cuda") / d)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "yarn":   # pairs that turn often in a sequence keep their frequency, those that hardly turn are slowed
        keep = ((SEQ * f / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
        f = f * (keep + (1 - keep) / c["factor"])
    return f, 0.1 * math.log(c["factor"]) + 1 if c["scaling"] == "yarn" else 1.0


def _run_rotary(c, s):
    if own:
        from mixed_precision_optimizer_bf16_gb300 import train_ops as ops
        how = dict(rotary_dim=c["turned"], layout=c["layout"], base=BASE, scaling=c["scaling"], factor=c["factor"], original_length=SEQ)
        q, k = (ops.rotary_forward if c["way"] == "forward" else ops.rotary_backward)(s["q"], s["k"], s["positions"], **how)
        return dict(q=q, k=k)

    f, length = _frequencies(c)
    angle = s["positions"].double()[:, None] * f            # far positions: in 64 bits
    cos, sin = (length * angle.cos()).float()[:, None, :], (length * angle.sin()).float()[:, None, :]
    sin = sin if c["way"] == "forward" else -sin
    n, out = c["turned"], {}
    for name in ("q", "k"):
        x = s[name].float()
        if c["layout"] == "half":
            a, b = x[..., :n // 2], x[..., n // 2:n]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:n:2], x[..., 1:n:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out[name] = torch.cat([turned, x[..., n:]], -1).to(s[name].dtype)
    return out


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    go = {"policy": _exact_policy, "preference": _exact_preference, "glu8": _exact_glu8, "pack8": _exact_pack8, "rotary": _exact_rotary}
    return go[case["op"]](case, s)


def _exact_policy(c, s):
    """Row by row blocks; the gradients are autograd's."""
    rows, parts = c["rows"], {}
    for a in range(0, rows, 128):
        b = slice(a, min(rows, a + 128))
        z = s["logits"][b].double().requires_grad_(True)
        w = s["weight"][b].double() if s["weight"] is not None else torch.ones(z.shape[0], dtype=F64, device=z.device)
        with torch.enable_grad():
            logp = torch.log_softmax(z / c["temperature"], 1).gather(1, s["labels"][b][:, None]).squeeze(1)
            if c["way"] == "logp":
                loss = logp
            else:
                old = s["old"][b].double() if s["old"] is not None else logp.detach()
                ratio, adv = torch.exp(logp - old), s["advantage"][b].double()
                loss = -torch.minimum(ratio * adv, ratio.clamp(1 - CLIP[0], 1 + CLIP[1]) * adv)
                if s["ref"] is not None:
                    d = s["ref"][b].double() - logp
                    loss = loss + c["kl"] * (torch.exp(d) - 1 - d)
                loss = loss * w
            if c["way"] == "backward":   # by what the forward pass left: its slope, its sums
                given = s["saved"][b].double()
                q = torch.exp((z.detach() - given[:, :1]) / c["temperature"]) / given[:, 1:2].clamp(min=1)
                one = torch.nn.functional.one_hot(s["labels"][b], c["vocab"])
                got = dict(dlogits=(one - q) * (given[:, 2] * s["dloss"][b].double() / c["temperature"])[:, None])
            elif c["way"] == "step":
                got = dict(loss=loss.detach(), logp=logp.detach() * (w != 0), dlogits=torch.autograd.grad(loss.sum(), z)[0])
            else:
                top = z.detach().amax(1)
                got = dict(logp=logp.detach() * (w != 0), top=top * (w != 0),
                           sum=torch.exp(torch.logsumexp(z.detach() / c["temperature"], 1) - top / c["temperature"]) * (w != 0))
                if c["way"] == "forward":
                    got.update(loss=loss.detach(), slope=torch.autograd.grad(loss.sum(), logp)[0])
        for n, v in got.items():
            parts.setdefault(n, []).append(v)
    return {n: torch.cat(v) for n, v in parts.items()}


def _exact_preference(c, s):
    pairs, ends = c["pairs"], s["offsets"].tolist()
    logits, labels = s["logits"], s["labels"]
    sums, blocks = [], []
    for i in range(2 * pairs):
        at = torch.arange(ends[i], ends[i + 1], device=logits.device)
        at = at[labels[at] >= 0]
        total = torch.zeros((), dtype=F64, device=logits.device)
        for part in at.split(128):
            total = total + torch.log_softmax(logits[part].double(), 1).gather(1, labels[part][:, None]).sum()
        sums.append(total / max(1, len(at)) if c["mean"] else total)
        blocks.append(at)
    logp = torch.stack(sums).requires_grad_(True)
    with torch.enable_grad():
        rel = logp - s["ref"].double()
        h = rel[:pairs] - rel[pairs:]
        if c["kind"] == "ipo":
            loss = (h - c["margin"] - 1 / (2 * c["beta"])) ** 2
        elif c["kind"] == "hinge":
            loss = torch.relu(1 - (c["beta"] * h - c["margin"]))
        else:
            m = c["beta"] * h - c["margin"]
            loss = -(1 - c["smoothing"]) * torch.nn.functional.logsigmoid(m) - c["smoothing"] * torch.nn.functional.logsigmoid(-m)
        slope = torch.autograd.grad(loss.sum(), logp)[0]
    out = dict(loss=loss.detach(), logp=logp.detach())
    if c["way"] == "step":
        grad = torch.zeros(logits.shape, dtype=F64 if logits.numel() < 1 << 28 else F32, device=logits.device)
        for i, at in enumerate(blocks):
            for part in at.split(128):
                one = torch.nn.functional.one_hot(labels[part], c["vocab"])
                scale = slope[i] / len(at) if c["mean"] else slope[i]
                grad[part] = (scale * (one - torch.softmax(logits[part].double(), 1))).to(grad.dtype)
        out["dlogits"] = grad
    return out


def _exact_values(x):
    """What 8 bits hold of [rows, columns]: to the nearest of three significant bits behind the first, ties to the even one."""
    def power(v):   # of two, at most v > 0
        return ((v.view(torch.int64) >> 52) << 52).view(F64)

    rows, columns = x.shape
    runs = -(-columns // RUN)
    x = torch.nn.functional.pad(x.double(), (0, runs * RUN - columns)).reshape(rows, runs, RUN)
    most = x.abs().amax(2, keepdim=True)
    scale = power((most / 448).clamp(min=2.0 ** -127))
    scale = torch.where(scale * 448 < most, 2 * scale, scale)
    y = x / scale
    step = power(y.abs().clamp(min=2.0 ** -6)) / 8
    return (torch.round(y / step) * step * scale).reshape(rows, -1)[:, :columns]


def _exact_glu8(c, s):
    def plain(g, u):
        a = torch.nn.functional.silu(g) if c["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        return a * u if u is not None else a

    parts = {}
    for a in range(0, c["rows"], 512):
        b = slice(a, a + 512)
        if c["way"] == "backward":
            scale = ((s["scales"][:, b].long() - 127 + 1023) << 52).view(F64).repeat_interleave(RUN, 2)
            kept = [v[:, :c["columns"]] for v in s["codes"][:, b].view(torch.float8_e4m3fn).double() * scale]
            got = {}
        else:
            given = [s["gate"][b]] + ([s["up"][b]] if c["gated"] else [])
            got = dict(h=plain(given[0].double(), given[1].double() if c["gated"] else None))
            kept = [_exact_values(x) for x in given]
        kept = [v.requires_grad_(True) for v in kept]
        with torch.enable_grad():
            grads = torch.autograd.grad(plain(kept[0], kept[1] if c["gated"] else None), kept, s["dh"][b].double())
        got.update(dgate=grads[0], dup=grads[1] if c["gated"] else None)
        for n, v in got.items():
            parts.setdefault(n, []).append(v)
    return {n: torch.cat(v) if v[0] is not None else None for n, v in parts.items()}


def _exact_pack8(c, s):
    return dict(x=torch.cat([_exact_values(x) for x in s["x"].split(1024)]))


def _exact_rotary(c, s):
    """As products of complex numbers."""
    f, length = _frequencies(c)
    out = {}
    for name in ("q", "k"):
        whole = []
        for x, p in zip(s[name].split(1024), s["positions"].split(1024)):
            x, n = x.double(), c["turned"]
            turn = torch.polar(torch.full((len(p), n // 2), length, dtype=F64, device=x.device), p.double()[:, None] * f)
            turn = (turn if c["way"] == "forward" else turn.conj())[:, None, :]
            pairs = x[..., :n].unflatten(-1, (2, n // 2)).transpose(-1, -2) if c["layout"] == "half" else x[..., :n].unflatten(-1, (n // 2, 2))
            got = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            got = got.transpose(-1, -2) if c["layout"] == "half" else got
            whole.append(torch.cat([got.reshape(*x.shape[:-1], n), x[..., n:]], -1))
        out[name] = torch.cat(whole)
    return out
