"""The token losses, the 8-bit activations and the rotary positions in 64 bits, from their formulas: plain, slow,
and sharing nothing with the library.  Results are float64 on the inputs' device."""
import math

import torch

INF = float("inf")
F64 = torch.float64


def logp(z, labels, temperature=1.0):
    """(logp [rows], softmax [rows, vocab], label's place [rows, vocab]) of rows whose labels lie in the vocabulary."""
    z = z.double() / temperature
    at = labels.long()[:, None]
    top = z.amax(1, keepdim=True)
    empty = (top == -INF)
    base = torch.where(empty, torch.zeros_like(top), top)
    e = (z - base).exp()
    total = e.sum(1, keepdim=True)
    p = torch.where(empty, torch.zeros_like(z), e / total)
    value = torch.where(empty, torch.full_like(top, -INF), z.gather(1, at) - base - total.log()).squeeze(1)
    return value, p, torch.zeros_like(z).scatter_(1, at, 1.0)


def counts(labels, vocab, row_weight=None):
    ok = (labels >= 0) & (labels < vocab)
    return ok if row_weight is None else ok & (row_weight != 0)


def token_logp(z, labels, temperature=1.0, row_weight=None, dloss=None):
    """(logp, dz, scale): scale bounds the magnitudes behind each dz."""
    live = counts(labels, z.shape[1], row_weight)
    v, p, one = logp(z, labels.clamp(0, z.shape[1] - 1), temperature)
    up = torch.ones_like(v) if dloss is None else dloss.double()
    return torch.where(live, v, torch.zeros_like(v)), *gradient(live, up, p, one, temperature)


def gradient(live, c, p, one, temperature):
    c = torch.where(live, c, torch.zeros_like(c))[:, None] / temperature
    none = c == 0
    dz = torch.where(none, torch.zeros_like(p), c * (one - p))
    return dz, torch.where(none, torch.zeros_like(p), c.abs() * (one + p))


def policy(z, labels, advantage, old_logp=None, ref_logp=None, clip_low=0.2, clip_high=0.2, kl_weight=0.0, temperature=1.0,
           row_weight=None, dloss=None):
    """(loss, logp, slope, dz, scale)."""
    live = counts(labels, z.shape[1], row_weight)
    v, p, one = logp(z, labels.clamp(0, z.shape[1] - 1), temperature)
    a = advantage.double()
    ratio = torch.exp(v - (v if old_logp is None else old_logp.double()))
    inside = torch.minimum(torch.maximum(ratio, torch.as_tensor(1 - clip_low, device=z.device)), torch.as_tensor(1 + clip_high, device=z.device))
    loss = -torch.minimum(ratio * a, inside * a)
    slope = torch.where(ratio * a <= inside * a, -ratio * a, torch.zeros_like(a))
    if ref_logp is not None and kl_weight:
        d = ref_logp.double() - v
        loss = loss + kl_weight * torch.where(d == INF, d, d.expm1() - d)
        slope = slope - kl_weight * d.expm1()
    w = row_weight.double() if row_weight is not None else torch.ones_like(a)
    loss, slope = (torch.where(live, x * w, torch.zeros_like(x)) for x in (loss, slope))
    up = slope if dloss is None else slope * dloss.double()
    return loss, torch.where(live, v, torch.zeros_like(v)), slope, *gradient(live, up, p, one, temperature)


def preference(z, labels, offsets, ref_logp=None, kind="sigmoid", beta=0.1, label_smoothing=0.0, margin=0.0, length_normalise=False,
               temperature=1.0, dloss=None):
    """(loss [pairs], logp [2 pairs], dz, scale)."""
    rows, vocab = z.shape
    given = [min(max(int(o), 0), rows) for o in offsets.tolist()]
    ends, most = [], 0
    for o in given:
        most = max(most, o)
        ends.append(min(most, given[-1]))
    pairs = len(ends) // 2
    ok = counts(labels, vocab)
    v, p, one = logp(z, labels.clamp(0, vocab - 1), temperature)
    total, share = [], []
    for i in range(2 * pairs):
        live = ok[ends[i]:ends[i + 1]]
        n = max(1, int(live.sum())) if length_normalise else 1
        total.append(v[ends[i]:ends[i + 1]][live].sum() / n)
        share.append(1.0 / n)
    total = torch.stack(total) if total else v[:0]
    ref = ref_logp.double() if ref_logp is not None else torch.zeros_like(total)
    h = (total - ref)[:pairs] - (total - ref)[pairs:]
    if kind == "ipo":
        d = h - margin - 1 / (2 * beta)
        loss, slope = d * d, 2 * d
    else:
        m = beta * h - margin
        if kind == "hinge":
            loss, slope = torch.relu(1 - m), -beta * (m < 1).double()
        else:
            e = label_smoothing
            loss = (1 - e) * torch.nn.functional.softplus(-m) + e * torch.nn.functional.softplus(m)
            slope = beta * (e * torch.sigmoid(m) - (1 - e) * torch.sigmoid(-m))
    up = slope if dloss is None else slope * dloss.double()
    c, live = torch.zeros_like(v), torch.zeros_like(ok)
    for i in range(2 * pairs):
        c[ends[i]:ends[i + 1]] = (up[i] if i < pairs else -up[i - pairs]) * share[i]
        live[ends[i]:ends[i + 1]] = ok[ends[i]:ends[i + 1]]
    return loss, total, *gradient(live, c, p, one, temperature)


# ------------------------------------------------------------------ 8 bits

def e4m3_numbers():
    """The 127 numbers from 0 to 448, by their codes."""
    return torch.tensor([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127], dtype=F64)


def pack(x):
    """(codes, scales) by search among e4m3's numbers; x [rows, columns]."""
    rows, columns = x.shape
    runs = (columns + 31) // 32
    full = torch.zeros(rows, 32 * runs, dtype=F64, device=x.device)
    full[:, :columns] = x.double()
    full = full.reshape(rows, runs, 32)
    fine = torch.isfinite(full)
    most = torch.where(fine, full.abs(), torch.zeros_like(full)).amax(2)
    powers = torch.tensor([2.0 ** (b - 127) for b in range(255)], dtype=F64, device=x.device)
    byte = torch.searchsorted(448 * powers, most)            # the first whose 448 scales reach it
    y = full / powers[byte][:, :, None]
    numbers = e4m3_numbers().to(x.device)
    up = torch.searchsorted(numbers, y.abs().nan_to_num(0, 0, 0)).clamp(max=126)
    down = (up - 1).clamp(min=0)
    over, under = numbers[up] - y.abs(), y.abs() - numbers[down]
    code = torch.where((over < under) | ((over == under) & (up % 2 == 0)), up, down)
    code = torch.where((numbers[code] * powers[byte][:, :, None] >= 2.0 ** 128), code - 1, code)    # no FP32 number
    code = code + 128 * torch.signbit(full).long()
    code = torch.where(fine, code, torch.full_like(code, 127))
    return code.reshape(rows, -1).to(torch.uint8), byte.to(torch.uint8)


def unpack(codes, scales, columns):
    numbers = torch.cat([e4m3_numbers(), torch.tensor([math.nan], dtype=F64)])
    numbers = torch.cat([numbers, -numbers]).to(codes.device)
    powers = torch.tensor([2.0 ** (b - 127) for b in range(256)], dtype=F64, device=codes.device)
    rows, runs = scales.shape
    return (numbers[codes.long()].reshape(rows, runs, 32) * powers[scales.long()][:, :, None]).reshape(rows, -1)[:, :columns]


def act(g, kind):
    """(act(g), act'(g), the sigmoid's argument) of finite g; a NaN stays one."""
    y = g if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    dy = torch.ones_like(g) if kind == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    s, rest = torch.sigmoid(y), torch.sigmoid(-y)
    return g * s, s + torch.where(s * rest == 0, torch.zeros_like(g), g * dy * s * rest) + 0 * g, y


# ------------------------------------------------------------------ rotary positions

def frequencies(dim, base=10000.0, scaling=None, factor=1.0, original_length=2048, slow=1.0, fast=32.0):
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    f = [base ** (-2 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        f = [v / factor for v in f]
    if scaling == "yarn":
        for i, v in enumerate(f):
            turns = original_length * v / (2 * math.pi)
            keep = 0.0 if turns < slow else 1.0 if turns > fast else (turns - slow) / (fast - slow)
            f[i] = (1 - keep) * v / factor + keep * v
    return f, 0.1 * math.log(factor) + 1 if scaling == "yarn" and factor > 1 else 1.0


def rotary(x, positions, rotary_dim, layout, inverse=False, **how):
    """x [batch, tokens, heads, dim], positions [batch, tokens]."""
    f, scale = frequencies(rotary_dim, **how)
    out = x.double().clone()
    angle = positions.double()[:, :, None] * torch.tensor(f, dtype=F64, device=x.device)
    c, s = (scale * angle.cos())[:, :, None], (scale * angle.sin())[:, :, None] * (-1 if inverse else 1)
    half = rotary_dim // 2
    first = slice(0, half) if layout == "half" else slice(0, rotary_dim, 2)
    second = slice(half, rotary_dim) if layout == "half" else slice(1, rotary_dim, 2)
    a, b = x.double()[..., first], x.double()[..., second]
    out[..., first] = a * c - b * s
    out[..., second] = b * c + a * s
    return out
