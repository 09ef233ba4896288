"""The training operators in 64 bits, from their formulas: plain, slow, and
sharing nothing with the library.  Inputs are torch tensors of any float type
on any device; results are float64 on the same device.  The edge rules (rows
without entries, masked vocabulary, experts that are off) are spelt out."""
import torch

INF = float("inf")


def _soft(z, dim=1):
    """softmax that gives 0 everywhere where all of z is -inf; (p, lse)."""
    lse = torch.logsumexp(z, dim, keepdim=True)
    p = torch.where(z == -INF, torch.zeros_like(z), torch.exp(z - torch.where(lse == -INF, torch.zeros_like(lse), lse)))
    return p, lse.squeeze(dim)


def distill(z, ids, top, temperature=1.0, kl_weight=1.0, ce_weight=0.0, labels=None, row_weight=None, teacher_lse=None,
            dloss=None):
    """(loss, dz, scale): scale bounds the sum of magnitudes behind each dz."""
    z, top = z.double(), top.double()
    rows, vocab = z.shape
    w = row_weight.double() if row_weight is not None else torch.ones(rows, dtype=torch.float64, device=z.device)
    up = w * (dloss.double() if dloss is not None else 1.0)
    q, lse_t = _soft(z / temperature)
    s, lse_1 = _soft(z)
    there = (ids >= 0) & (ids < vocab) & (top != -INF)
    at = torch.where(there, ids, torch.zeros_like(ids)).long()
    x = torch.where(there, top / temperature, torch.full_like(top, -INF))
    p, norm = _soft(x) if ids.shape[1] else (x, torch.full((rows,), -INF, dtype=torch.float64, device=z.device))
    if teacher_lse is not None:
        norm = teacher_lse.double()
        p = torch.where(there, torch.exp(x - norm[:, None]), torch.zeros_like(x))
    mass = p.sum(1)
    empty = (z == -INF).all(1)
    loss = torch.zeros(rows, dtype=torch.float64, device=z.device)
    for r in range(rows):     # term by term, so that 0 * inf never appears
        kl = 0.0
        if kl_weight:
            t = there[r] & (p[r] != 0)
            if empty[r]:
                kl = INF if bool(t.any()) else 0.0
            else:
                kl = (p[r][t] * ((x[r][t] - norm[r]) - (z[r][at[r][t]] / temperature - lse_t[r]))).sum()
        ce = 0.0
        if ce_weight and labels is not None and 0 <= int(labels[r]) < vocab:
            ce = INF if empty[r] else lse_1[r] - z[r, int(labels[r])]
        loss[r] = w[r] * (kl_weight * temperature ** 2 * kl + ce_weight * ce)
    soft = (up * kl_weight * temperature)[:, None]
    take = torch.zeros_like(z).scatter_add_(1, at, p) if ids.shape[1] else torch.zeros_like(z)
    dz, scale = soft * (mass[:, None] * q - take), soft.abs() * (mass[:, None] * q + take)
    if ce_weight and labels is not None:
        ok = (labels >= 0) & (labels < vocab)
        one = torch.zeros_like(z)
        one[torch.arange(rows, device=z.device)[ok], labels[ok].long()] = 1.0
        hard = (up * ce_weight * ok)[:, None]
        dz = dz + hard * (s - one)
        scale = scale + hard.abs() * (s + one)
    dead = (w == 0)
    for v in (loss, dz, scale):
        v[dead] = 0.0
    lse = torch.stack([lse_t, lse_1], 1)
    lse[dead] = 0.0
    return loss, dz, scale, lse


def _norm(v, kind, eps):
    """(hat, mean, rstd) of rows."""
    if kind in (None, "none"):
        return v, torch.zeros_like(v[:, :1]), torch.ones_like(v[:, :1])
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(v[:, :1])
    rstd = 1.0 / torch.sqrt(((v - mean) ** 2).mean(1, keepdim=True) + eps)
    return (v - mean) * rstd, mean, rstd


def _d(t):
    return t.double() if t is not None else None


def _act(gate, act, rows):
    if gate is None:
        return 1.0, 0.0
    g = gate.double().repeat_interleave(rows // gate.shape[0], 0)
    if act == "sigmoid":
        a = torch.sigmoid(g)
        return a, a * (1 - a)
    return g, torch.ones_like(g)


def norm_gate(x, y, pre, post, pre_weight=None, pre_bias=None, post_weight=None, post_bias=None, gate=None, gate_act="none",
              residual_scale=1.0, branch_scale=1.0, eps=1e-5):
    x, y = x.double(), y.double()
    one = torch.ones(x.shape[1], dtype=torch.float64, device=x.device)
    hat, m2, s2 = _norm(y, post, eps)
    u = hat * (_d(post_weight) if post_weight is not None else one) + (_d(post_bias) if post_bias is not None else 0 * one)
    a, _ = _act(gate, gate_act, x.shape[0])
    r = residual_scale * x + branch_scale * a * u
    h = None
    m1, s1 = torch.zeros_like(m2), torch.zeros_like(s2)
    if pre not in (None, "none"):
        hat, m1, s1 = _norm(r, pre, eps)
        h = hat * (_d(pre_weight) if pre_weight is not None else one) + (_d(pre_bias) if pre_bias is not None else 0 * one)
    if post in (None, "none"):
        m2, s2 = torch.zeros_like(m2), torch.zeros_like(s2)
    return r, h, torch.cat([m1, s1, m2, s2], 1)


def norm_gate_backward(dr, dh, r, y, pre, post, pre_weight=None, pre_bias=None, post_weight=None, post_bias=None, gate=None,
                       gate_act="none", residual_scale=1.0, branch_scale=1.0, eps=1e-5):
    """dict of gradients, and under "sums" the sums of magnitudes behind each."""
    rows, n = y.shape
    y = y.double()
    flow = dr.double() if dr is not None else torch.zeros_like(y)
    size = flow.abs()
    out, sums = {}, {}

    def through(hat, rstd, kind, weight, g, size):
        w = weight.double() if weight is not None else 1.0
        a, b = g * w, size * abs(w)
        d = a - hat * (a * hat).mean(1, keepdim=True)
        e = b + hat.abs() * (b * hat.abs()).mean(1, keepdim=True)
        if kind == "layer":
            d, e = d - a.mean(1, keepdim=True), e + b.mean(1, keepdim=True)
        return d * rstd, e * rstd

    if pre not in (None, "none") and dh is not None:
        hat, _, rstd = _norm(r.double(), pre, eps)
        g = dh.double()
        d, e = through(hat, rstd, pre, pre_weight, g, g.abs())
        flow, size = flow + d, size + e
        out["dpre_weight"], sums["dpre_weight"] = (g * hat).sum(0), (g * hat).abs().sum(0)
        out["dpre_bias"], sums["dpre_bias"] = g.sum(0), g.abs().sum(0)
    else:
        out["dpre_weight"] = out["dpre_bias"] = sums["dpre_weight"] = sums["dpre_bias"] = torch.zeros(n, dtype=torch.float64, device=y.device)
    out["dx"], sums["dx"] = residual_scale * flow, abs(residual_scale) * size
    flow, size = branch_scale * flow, abs(branch_scale) * size
    hat, _, rstd = _norm(y, post, eps)
    u = hat * (_d(post_weight) if post_weight is not None else 1.0) + (_d(post_bias) if post_bias is not None else 0.0)
    a, slope = _act(gate, gate_act, rows)
    if gate is not None:
        out["dgate"] = (flow * u * slope).reshape(gate.shape[0], -1, n).sum(1)
        sums["dgate"] = (size * u * slope).abs().reshape(gate.shape[0], -1, n).sum(1)
    flow, size = flow * a, size * abs(a)
    if post not in (None, "none"):
        out["dpost_weight"], sums["dpost_weight"] = (flow * hat).sum(0), (size * hat.abs()).sum(0)
        out["dpost_bias"], sums["dpost_bias"] = flow.sum(0), size.sum(0)
        flow, size = through(hat, rstd, post, post_weight, flow, size)
    out["dy"], sums["dy"] = flow, size
    out["sums"] = sums
    return out


def balance(z, k, mask=None, groups=1, balance_weight=1e-2, z_weight=0.0, renormalise=True, dweights=None, dloss=1.0):
    """(ids, weights, counts, loss, dz), token by token."""
    z = z.double().cpu()
    tokens, experts = z.shape
    per = tokens // groups if groups else 0
    live = mask.cpu().bool() if mask is not None else torch.ones(tokens, dtype=torch.bool)
    live = live & ~(z == -INF).all(1)
    ids = torch.full((tokens, k), -1, dtype=torch.int32)
    weights = torch.zeros(tokens, k, dtype=torch.float64)
    counts = torch.zeros(groups, experts, dtype=torch.int32)
    p, lse = _soft(z)
    for t in range(tokens):
        if not live[t]:
            continue
        order = sorted((e for e in range(experts) if z[t, e] != -INF),
                       key=lambda e: (0, -float(z[t, e]), e) if z[t, e] == z[t, e] else (1, 0.0, e))[:k]
        ids[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
        w = p[t, order]
        weights[t, :len(order)] = w / w.sum() if renormalise else w
        for e in order:
            counts[t // per, e] += 1
    loss = torch.zeros((), dtype=torch.float64)
    dz = torch.zeros_like(z)
    for g in range(groups):
        at = torch.arange(g * per, (g + 1) * per)
        at = at[live[at]]
        n = len(at)
        if n == 0:
            continue
        f = counts[g].double() * experts / (k * n)
        loss = loss + balance_weight * (f * p[at].mean(0)).sum() + z_weight * (lse[at] ** 2).mean()
        inner = (p[at] * f).sum(1, keepdim=True)
        dz[at] = dloss / (groups * n) * (balance_weight * p[at] * (f - inner) + 2 * z_weight * lse[at][:, None] * p[at])
    if dweights is not None:
        up = dweights.double().cpu()
        for t in range(tokens):
            if not live[t]:
                continue
            e = [int(i) for i in ids[t] if i >= 0]
            u = up[t, :len(e)]
            w = weights[t, :len(e)]
            if renormalise:
                dz[t, e] += w * (u - (w * u).sum())
            else:
                dz[t] -= p[t] * (w * u).sum()
                dz[t, e] += w * u
    return ids, weights, counts, loss / max(groups, 1), dz
