"""The training operators on the GPU against their formulas in 64 bits.

Tolerances come from the arithmetic: an output of u bits' rounding is within
2^-9 (bf16; 2^-8 is allowed) or 2^-24 of the exact value, and what is summed in
FP32 is within 2e-5 of the sum of the magnitudes that went in (a few hundred
roundings of 2^-24 one after another, or a function's error of a few units).
"""
import math

import pytest

torch = pytest.importorskip("torch")

import train_ops_reference as R  # noqa: E402
from mixed_precision_optimizer_bf16_gb300 import train_ops as ops  # noqa: E402
from mixed_precision_optimizer_bf16_gb300 import bf16opt as C  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def close(got, ref, sums, what):
    """|got - ref| within the output type's rounding of ref and 2e-5 of the
    magnitudes summed; infinities and NaN alike."""
    u = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -20
    got, ref = got.double(), ref.double().to(got.device)
    sums = torch.as_tensor(sums, dtype=torch.float64, device=got.device)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    odd = ~torch.isfinite(ref)
    assert torch.equal(got[odd & ~torch.isnan(ref)], ref[odd & ~torch.isnan(ref)]), what
    err = (got - ref).abs()
    bound = u * ref.abs() + 2e-5 * sums + 1e-30
    bad = (err > bound) & ~odd
    assert not bool(bad.any()), (what, int(bad.sum()), float((err - bound)[~odd].max()))


# ------------------------------------------------------------------ distillation

def distill_case(rows, vocab, k, dtype, seed=0, labels=False, weights=False, full=False, temperature=1.0):
    g = gen(seed)
    z = (3 * randn(g, rows, vocab)).to(dtype)
    t = z.float() + 0.5 * randn(g, rows, vocab)
    top, ids = t.topk(k, 1) if k else (t[:, :0], torch.zeros(rows, 0, dtype=torch.int64, device="cuda"))
    how = dict(temperature=temperature)
    if labels:
        how["labels"] = torch.randint(-1, vocab, (rows,), device="cuda", generator=g)
        how["ce_weight"] = 0.7
    if weights:
        how["row_weight"] = torch.where(torch.rand(rows, device="cuda", generator=g) < 0.4, 0.0, 0.5 + torch.rand(rows, device="cuda", generator=g))
    if full:
        how["teacher_lse"] = torch.logsumexp(t / temperature, 1)
    return z, ids.int(), top.to(dtype), how


def loss_scale(z, top, how):
    t = how.get("temperature", 1.0)
    big = lambda v: torch.where(torch.isfinite(v.float()), v.float().abs(), torch.zeros_like(v, dtype=F32)).amax(1) if v.shape[1] else 0.0  # noqa: E731
    w = how["row_weight"].abs() if how.get("row_weight") is not None else 1.0
    return w * (t * t + 1) * (12 + 2 * big(z) * max(1, 1 / t) + 2 * big(top) / t)


def check_distill(z, ids, top, how, dloss=None):
    loss_r, dz_r, scale, lse_r = R.distill(z, ids, top, dloss=dloss, **how)
    loss_only, lse = ops.distill_forward(z, ids, top, **how)
    back = ops.distill_backward(z, ids, top, lse, dloss, **how)
    loss, dz = ops.distill_loss_grad(z, ids, top, dloss, **how)
    close(loss_only, loss_r, loss_scale(z, top, how), "loss of the forward call")   # (its sums have another order)
    close(loss, loss_r, loss_scale(z, top, how), "loss")
    close(lse[:, 0], lse_r[:, 0], 1 + lse_r[:, 0].abs().nan_to_num(0, 0, 0), "lse")
    close(dz, dz_r, scale, "dlogits")
    close(back, dz_r, scale, "dlogits of the backward call")
    return loss, dz


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (3, 7, 2), (2, 8, 8), (5, 9, 3), (4, 31, 0), (300, 1000, 16), (7, 2053, 1),
                                          (3, 33000, 64), (2, 70001, 129), (160, 4096, 1024), (2, 250880, 64)])
def test_distill_sizes(rows, vocab, k, dtype):
    check_distill(*distill_case(rows, vocab, k, dtype, labels=k % 2 == 0, temperature=1.0 if k == 16 else 2.0))


@pytest.mark.parametrize("labels", [False, True])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 3.0])
def test_distill_terms(labels, weights, full, temperature):
    z, ids, top, how = distill_case(9, 1537, 20, F32, 3, labels, weights, full, temperature)
    check_distill(z, ids, top, how, dloss=torch.rand(9, device="cuda") - 0.3)


def test_distill_label_alone_and_no_terms():
    z, ids, top, how = distill_case(6, 515, 4, BF16, 1, labels=True, temperature=2.0)
    how["kl_weight"] = 0.0
    loss_r, dz_r, scale, _ = R.distill(z, ids, top, **how)
    loss, dz = ops.distill_loss_grad(z, ids, top, **how)
    close(loss, loss_r, loss_scale(z, top, how), "loss")
    close(dz, dz_r, scale, "dlogits")
    loss, dz = ops.distill_loss_grad(z, ids, top, kl_weight=0.0)
    assert not loss.any() and not dz.any()


def test_distill_edges():
    """Rows without entries, ids outside, repeated ids, a teacher's -inf, masked
    vocabulary, an all-masked row, labels outside."""
    rows, vocab, k = 12, 100, 6
    z, ids, top, how = distill_case(rows, vocab, k, F32, 5, labels=True, temperature=2.0)
    ids[0] = -1                                    # no entries
    ids[1, 3:] = vocab + 5                         # outside
    ids[2] = 17                                    # one id six times
    ids[3, 1] = ids[3, 4]                          # a repeated one
    top[4, 2] = -INF                               # an entry with no probability
    top[5] = -INF
    z[6, 50:] = -INF                               # masked vocabulary, the teacher's entries elsewhere
    ids[6] = torch.arange(6, device="cuda", dtype=torch.int32)
    how["labels"][6] = 3
    z[7] = -INF                                    # nothing left
    z[8] = -INF
    ids[8] = -1
    how["labels"][8] = -100
    z[9, 30:] = -INF                               # an entry on masked vocabulary
    ids[9, 0] = 40
    how["labels"][9] = -100
    how["labels"][10] = vocab
    ids[11, 2] = how["labels"][11] = 8             # the label is an entry too
    loss, dz = check_distill(z, ids, top, how)
    assert loss[7] == INF and loss[8] == 0 and loss[9] == INF
    assert not dz[8].any() and bool(torch.isfinite(dz).all())


@pytest.mark.parametrize("temperature", [1.0, 2.0, 1.5])
@pytest.mark.parametrize("away", [-300.0, 300.0, -1000.0, "lowest", "largest"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_distill_rows_far_from_zero(dtype, away, temperature):
    """Adding a number to a row's logits, the student's or the teacher's, changes neither loss nor
    gradient, up to the number that the type can still tell apart: not either where every logit is
    the type's lowest or largest."""
    rows, vocab, k = 5, 6007, 37
    z, ids, top, how = distill_case(rows, vocab, k, dtype, 11, labels=True, temperature=temperature)
    if isinstance(away, str):
        away = (-1 if away == "lowest" else 1) * torch.finfo(dtype).max
    z, top = (z.float() + away).to(dtype), (top.float() + away / 2).to(dtype)
    near, near_top = z.double() - away, top.double() - torch.tensor(away / 2).to(dtype).double().item()
    loss_r, dz_r, scale, _ = R.distill(near, ids, near_top, **how)
    loss, dz = ops.distill_loss_grad(z, ids, top, **how)
    close(loss, loss_r, loss_scale(near, near_top, how), "loss")
    close(dz, dz_r, scale, "dlogits")
    only, lse = ops.distill_forward(z, ids, top, **how)
    close(only, loss_r, loss_scale(near, near_top, how), "loss of the forward call")
    assert bool(torch.isfinite(lse).all())
    assert bool(torch.isfinite(ops.distill_backward(z, ids, top, lse, **how)).all())


def test_distill_nan_and_inf_stay_in_their_row():
    z, ids, top, how = distill_case(6, 3000, 8, F32, 2)
    clean_loss, clean = ops.distill_loss_grad(z, ids, top, **how)
    z2, top2 = z.clone(), top.clone()
    z2[1, 77] = float("nan")
    z2[3, 2999] = INF
    top2[4, 0] = float("nan")
    loss, dz = ops.distill_loss_grad(z2, ids, top2, **how)
    for r in (1, 3, 4):
        assert torch.isnan(loss[r]) and torch.isnan(dz[r]).all()
    keep = [0, 2, 5]
    assert torch.equal(loss[keep], clean_loss[keep]) and torch.equal(dz[keep], clean[keep])
    w = torch.ones(6, device="cuda")
    w[[1, 3, 4]] = 0                               # a row of weight 0 is not read
    loss, dz = ops.distill_loss_grad(z2, ids, top2, row_weight=w, **how)
    assert bool(torch.isfinite(loss).all()) and not dz[[1, 3, 4]].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset,pad", [(1, 3), (3, 8), (0, 5)])
def test_distill_strided_rows_and_index_types(dtype, offset, pad):
    rows, vocab, k = 5, 2051, 12
    z0, ids, top, how = distill_case(rows, vocab, k, dtype, 7, labels=True, weights=True)
    base = torch.full((rows * (vocab + pad) + offset,), 55.0, device="cuda", dtype=dtype)
    z = base[offset:].view(rows, vocab + pad)[:, :vocab]
    z.copy_(z0)
    wide = torch.full((rows, 2 * k), -7, device="cuda", dtype=torch.int64)
    wide[:, :k] = ids
    how["labels"] = how["labels"].int()
    a = ops.distill_loss_grad(z0, ids, top, **how)
    b = ops.distill_loss_grad(z, wide[:, :k], top.float(), **how)
    close(b[0], a[0], loss_scale(z0, top, how), "loss")
    close(b[1], a[1], 1.0, "dlogits")
    res = ops.distill_loss_grad(z, wide[:, :k], top.float(), out=z, **how)[1]          # in place, rows apart
    assert res.data_ptr() == z.data_ptr() and torch.equal(res, b[1])
    left = base[offset:].view(rows, vocab + pad)[:, vocab:]
    assert bool((left == 55).all())                                                   # between the rows: untouched


@pytest.mark.parametrize("dtype,vocab", [(BF16, 4000), (F32, 33001), (F32, 500000)])
def test_distill_in_place_is_the_same(dtype, vocab):
    """(500000 FP32 logits do not fit the CTAs' shared memory: the slice is read twice.)"""
    z, ids, top, how = distill_case(5, vocab, 40, dtype, 4, labels=True, temperature=2.0)
    loss, dz = ops.distill_loss_grad(z, ids, top, **how)
    lse = ops.distill_forward(z, ids, top, **how)[1]
    back = ops.distill_backward(z, ids, top, lse, **how)
    z1, z2 = z.clone(), z.clone()
    loss1, dz1 = ops.distill_loss_grad(z1, ids, top, out=z1, **how)
    assert torch.equal(loss, loss1) and torch.equal(dz, dz1)
    assert torch.equal(ops.distill_backward(z2, ids, top, lse, out=z2, **how), back)
    close(dz, R.distill(z, ids, top, **how)[1], R.distill(z, ids, top, **how)[2], "dlogits")


def test_distill_rows_beyond_32_bit_offsets():
    stride = 2 ** 32 + 8
    base = torch.empty(stride + 4096, dtype=BF16, device="cuda")
    z = base.as_strided((2, 3001), (stride, 1))
    small, ids, top, how = distill_case(2, 3001, 9, BF16, 8)
    near = torch.empty(2, 3008, dtype=BF16, device="cuda")[:, :3001]   # rows aligned as z's: the same order of sums
    z.copy_(small)
    near.copy_(small)
    small = near
    loss, dz = ops.distill_loss_grad(z, ids, top, **how)
    loss1, dz1 = ops.distill_loss_grad(small, ids, top, **how)
    assert torch.equal(loss, loss1) and torch.equal(dz, dz1)
    ops.distill_loss_grad(z, ids, top, out=z, **how)
    assert torch.equal(z, dz)


def test_distill_gradient_against_differences():
    z, ids, top, how = distill_case(3, 403, 11, F32, 9, labels=True, full=True, temperature=1.5)
    v = torch.randn(z.shape, dtype=torch.float64, device="cuda", generator=gen(1))
    h = 1e-5
    up = (R.distill(z.double() + h * v, ids, top, **how)[0].sum() - R.distill(z.double() - h * v, ids, top, **how)[0].sum()) / (2 * h)
    _, dz = ops.distill_loss_grad(z, ids, top, **how)
    # h^2 of the difference's own error, 1e-5 of the gradient's
    assert abs(float((dz.double() * v).sum() - up)) <= 1e-5 * float((dz.double() * v).abs().sum())


def test_distill_autograd_and_determinism():
    z, ids, top, how = distill_case(64, 50001, 32, BF16, 6, labels=True, temperature=2.0)
    z.requires_grad_(True)
    loss = ops.distill_loss(z, ids, top, **how)
    (loss * torch.arange(64, device="cuda")).sum().backward()
    _, dz_r, scale, _ = R.distill(z.detach(), ids, top, dloss=torch.arange(64, device="cuda").float(), **how)
    close(z.grad, dz_r, scale, "dlogits")
    a = ops.distill_loss_grad(z.detach(), ids, top, **how)
    for _ in range(3):
        b = ops.distill_loss_grad(z.detach(), ids, top, **how)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------------- gated norms

def norm_case(rows, hidden, branch, stream, weight, pre, post, gates, seed=0):
    g = gen(seed)
    x = (2 * randn(g, rows, hidden) + 0.3).to(stream)
    y = (randn(g, rows, hidden) - 0.2).to(branch)
    how = dict(pre=pre, post=post)
    for n, kind in (("pre", pre), ("post", post)):
        if kind != "none":
            how[n + "_weight"] = (1 + 0.3 * randn(g, hidden)).to(weight)
        if kind == "layer":
            how[n + "_bias"] = (0.2 * randn(g, hidden)).to(weight)
    if gates:
        how["gate"] = randn(g, gates, hidden).to(branch)
    return x, y, how


def rowmax(t):
    return t.abs().amax(1, keepdim=True) if t.numel() else t


def check_norm(x, y, how, dr_none=False, dh_none=False, seed=1):
    r, h, stats = ops.norm_gate_forward(x, y, **how)
    r_r, h_r, stats_r = R.norm_gate(x, y, **how)
    close(r, r_r, rowmax(r_r), "r")
    close(stats, stats_r, 1 + stats_r.abs(), "stats")
    if h_r is None:
        assert h is None
    else:
        close(h, h_r, rowmax(h_r), "h")
    g = gen(seed)
    dr = None if dr_none else randn(g, *x.shape).to(x.dtype)
    dh = None if dh_none or h_r is None else randn(g, *y.shape).to(y.dtype)
    # the backward call takes the stored stream and the statistics of that
    _, _, stats = ops.norm_gate_forward(r, torch.zeros_like(y), **{**how, "residual_scale": 1.0, "branch_scale": 0.0})
    stats[:, 2:] = stats_r[:, 2:].float()
    got = ops.norm_gate_backward(dr, dh, r, y, stats, **how)
    ref = R.norm_gate_backward(dr, dh, r, y, **how)
    for n in ("dx", "dy"):
        close(got[n], ref[n], rowmax(ref["sums"][n]), n)
    for n in ("dgate", "dpre_weight", "dpre_bias", "dpost_weight", "dpost_bias"):
        if how.get(n[1:]) is None:
            assert got[n] is None
        else:
            close(got[n], ref[n], ref["sums"][n], n)
    return got


@pytest.mark.parametrize("branch,stream,weight", [(BF16, BF16, BF16), (BF16, F32, F32), (F32, F32, BF16)])
@pytest.mark.parametrize("rows,hidden", [(1, 1), (3, 7), (1, 8), (2, 64), (5, 257), (700, 512), (9, 1537), (33, 2048), (400, 4096),
                                         (6, 4104), (310, 8200), (7, 14336), (2, 16384), (3, 16383)])
def test_norm_sizes(rows, hidden, branch, stream, weight):
    x, y, how = norm_case(rows, hidden, branch, stream, weight, "layer", "rms", 0)
    check_norm(x, y, dict(how, residual_scale=0.7, branch_scale=1.3))


@pytest.mark.parametrize("pre,post", [("rms", "rms"), ("layer", "layer"), ("rms", "none"), ("none", "layer"), ("none", "none")])
@pytest.mark.parametrize("gates", [0, 1, 6, 36])
@pytest.mark.parametrize("act", ["none", "sigmoid"])
def test_norm_kinds_and_gates(pre, post, gates, act):
    x, y, how = norm_case(36, 1032, BF16, F32, F32, pre, post, gates)
    check_norm(x, y, dict(how, gate_act=act, branch_scale=0.5))


@pytest.mark.parametrize("rows,gates,hidden", [(3000, 1000, 72), (3000, 7 * 100, 64), (4500, 3, 96), (4500, 450, 40), (1216, 608, 2048), (900, 2, 4200)])
def test_norm_gates_that_straddle_the_teams(rows, gates, hidden):
    rows = rows // gates * gates
    x, y, how = norm_case(rows, hidden, F32, F32, F32, "rms", "layer", gates)
    check_norm(x, y, dict(how, gate_act="sigmoid"))


def test_norm_missing_gradients_and_weights():
    x, y, how = norm_case(40, 520, BF16, BF16, BF16, "layer", "layer", 1)
    check_norm(x, y, how, dr_none=True)
    check_norm(x, y, how, dh_none=True)
    bare = dict(pre="layer", post="rms")
    check_norm(x, y, bare)


def test_norm_constant_and_large_rows():
    x, y, how = norm_case(6, 300, F32, F32, F32, "layer", "layer", 0)
    y[1] = 5.0                                    # no variance
    y[2] = 1e4 + y[2]                             # a large mean: the variance may not cancel
    y[3] = 0.0
    x[4] *= 1e15
    r, h, stats = ops.norm_gate_forward(x, y, **how)
    r_r, h_r, stats_r = R.norm_gate(x, y, **how)
    assert bool(torch.isfinite(r).all() and torch.isfinite(h).all())
    rows = [0, 1, 3, 4, 5]
    close(r[rows], r_r[rows], rowmax(r_r[rows]), "r")
    close(h[rows], h_r[rows], rowmax(h_r[rows]), "h")
    # row 2: a mean of 1e4 is off by 1e4 2^-24, which the deviation of 1 shows undivided
    close(r[2:3], r_r[2:3], 1e4 * 2.0 ** -24 / 2e-5 * 4, "r at a large mean")


def test_norm_nan_stays_in_its_row():
    x, y, how = norm_case(8, 900, BF16, BF16, BF16, "layer", "rms", 0)
    clean = ops.norm_gate_forward(x, y, **how)
    y2 = y.clone()
    y2[3, 5] = float("nan")
    got = ops.norm_gate_forward(x, y2, **how)
    keep = [0, 1, 2, 4, 5, 6, 7]
    for a, b in zip(clean, got):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(got[0][3]).all() and torch.isnan(got[1][3]).all()


@pytest.mark.parametrize("branch,stream", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("rows,hidden,gates", [(90, 2, 0), (61, 9, 61), (33, 13, 0), (700, 31, 7), (40, 250, 40), (24, 1031, 2), (16, 4097, 0),
                                               (5, 9001, 5), (3, 14333, 1)])
def test_norm_rows_between_boundaries(rows, hidden, gates, branch, stream):
    """Rows that begin anywhere between two 16-byte boundaries, each tensor at a place of its own: no row sees its
    neighbours' elements, which are NaN in one row of all inputs."""
    x, y, how = norm_case(rows, hidden, branch, stream, F32, "layer", "rms", gates, 7)
    if gates:
        how["gate_act"] = "sigmoid"
    check_norm(x, y, how)

    def placed(t, offset):
        return torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")[offset:].view(t.shape).copy_(t)
    g = gen(8)
    r, h, stats = ops.norm_gate_forward(x, y, **how)
    dr, dh = randn(g, rows, hidden).to(stream), randn(g, rows, hidden).to(branch)
    clean = ops.norm_gate_backward(dr, dh, r, y, stats, **how)
    spoilt = [t.clone() for t in (dr, dh, r, y)]
    for t in spoilt:
        t[rows // 2] = float("nan")
    got = ops.norm_gate_backward(*[placed(t, i) for i, t in zip((1, 3, 2, 5), spoilt)], stats,
                                 **{**how, **({"gate": placed(how["gate"], 7)} if gates else {})})
    keep = torch.arange(rows, device="cuda") != rows // 2
    for n in ("dx", "dy") + (("dgate",) if gates == rows else ()):
        size = clean[n].double().abs().max()
        close(got[n][keep], clean[n][keep], 40 * size, n)
        assert bool(torch.isnan(got[n][rows // 2]).all())


@pytest.mark.parametrize("offset", [0, 1])
def test_norm_in_place_and_unaligned(offset):
    rows, hidden = 50, 1048
    x, y, how = norm_case(rows, hidden, BF16, BF16, BF16, "rms", "layer", 5)
    def shifted(t):
        b = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
        v = b[offset:].view(t.shape)
        return v.copy_(t)
    r, h, stats = ops.norm_gate_forward(x, y, **how)
    xs, ys = shifted(x), shifted(y)
    r2, h2, stats2 = ops.norm_gate_forward(xs, ys, out_r=xs, out_h=ys, **how)
    assert r2.data_ptr() == xs.data_ptr() and h2.data_ptr() == ys.data_ptr()
    close(r2, r, rowmax(r.double()), "r")
    close(h2, h, rowmax(h.double()), "h")
    dr, dh = torch.randn_like(r), torch.randn_like(h)
    a = ops.norm_gate_backward(dr, dh, r, y, stats, **how)
    b = ops.norm_gate_backward(shifted(dr), shifted(dh), shifted(r), shifted(y), stats, **how)
    for n in a:
        if a[n] is not None:
            close(b[n], a[n], 40 * a[n].double().abs().max(), n)


def test_norm_no_rows():
    x = torch.empty(0, 128, dtype=BF16, device="cuda")
    how = dict(pre="rms", post="rms", pre_weight=torch.ones(128, dtype=BF16, device="cuda"),
               post_weight=torch.ones(128, dtype=BF16, device="cuda"))
    r, h, stats = ops.norm_gate_forward(x, x, **how)
    assert r.shape == h.shape == (0, 128)
    got = ops.norm_gate_backward(x, x, x, x, stats, **how)
    assert not got["dpre_weight"].any() and not got["dpost_weight"].any()


def test_norm_gradient_against_differences():
    x, y, how = norm_case(12, 264, F32, F32, F32, "layer", "rms", 4, seed=3)
    how = dict(how, gate_act="sigmoid", residual_scale=0.8, branch_scale=1.2)
    x, y = x.requires_grad_(True), y.requires_grad_(True)
    leaves = {n: v.requires_grad_(True) for n, v in how.items() if torch.is_tensor(v)}
    g = gen(4)
    cr, ch = randn(g, 12, 264), randn(g, 12, 264)
    r, h = ops.norm_gate(x, y, **how)
    ((r * cr).sum() + (h * ch).sum()).backward()

    def value(s, which):
        moved = {n: v.detach().double() + (s * dirs[n] if n == which else 0) for n, v in {"x": x, "y": y, **leaves}.items()}
        rest = {n: v for n, v in how.items() if not torch.is_tensor(v)}
        rr, hh, _ = R.norm_gate(moved.pop("x"), moved.pop("y"), **rest, **moved)
        return (rr * cr.double()).sum() + (hh * ch.double()).sum()

    everything = {"x": x, "y": y, **leaves}
    dirs = {n: torch.randn(v.shape, dtype=torch.float64, device="cuda", generator=g) for n, v in everything.items()}
    for n, v in everything.items():
        d = (value(1e-5, n) - value(-1e-5, n)) / 2e-5
        along = v.grad.double() * dirs[n]
        assert abs(float(along.sum() - d)) <= 1e-5 * float(along.abs().sum()) + 1e-6, n


# ----------------------------------------------------------------- expert balance

def check_balance(z, k, dloss=None, up=True, **how):
    tokens = z.shape[0]
    dw = torch.randn(tokens, k, device="cuda", generator=gen(11)) if up else None
    ids, weights, counts, loss, saved = ops.balance_forward(z, k, **how)
    dz = ops.balance_backward(z, ids, counts, saved, dw, dloss, **how)
    r = R.balance(z, k, dweights=dw, dloss=1.0 if dloss is None else float(dloss), **how)
    assert torch.equal(ids.cpu(), r[0]) and torch.equal(counts.cpu(), r[2])
    close(weights, r[1], 1.0 * (r[1] != 0), "weights")
    close(loss, r[3], r[3].abs(), "loss")
    close(dz, r[4], 0.2 * rowmax(r[4]) + (rowmax(dw.double()).cpu() if up else 0), "dlogits")
    return ids, weights, counts, loss, dz


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (5, 3, 2), (64, 8, 2), (130, 33, 4), (1000, 64, 6), (77, 100, 8), (300, 256, 8),
                                              (40, 1000, 3), (20, 1024, 32), (2500, 16, 16)])
def test_balance_sizes(tokens, experts, k, dtype):
    z = (2 * randn(gen(tokens), tokens, experts)).to(dtype)
    check_balance(z, k, balance_weight=0.5, z_weight=0.1)


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("groups", [1, 4, 33, 660])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_groups_and_masks(renormalise, groups, masked):
    tokens, experts = 1980, 24
    g = gen(groups)
    mask = torch.rand(tokens, device="cuda", generator=g) < 0.6 if masked else None
    if masked:
        mask[: tokens // groups] = False              # a group with no live token
    check_balance(randn(g, tokens, experts), 3, groups=groups, mask=mask, renormalise=renormalise, balance_weight=0.3,
                  z_weight=0.01, dloss=torch.tensor(1.7, device="cuda"))


def test_balance_ties_off_experts_and_nan():
    tokens, experts = 200, 40
    z = torch.randint(-2, 3, (tokens, experts), device="cuda", generator=gen(2)).float()
    z[z == 0] *= torch.where(torch.rand(int((z == 0).sum()), device="cuda") < 0.5, -1.0, 1.0)   # both zeros are one number
    check_balance(z, 5, balance_weight=0.1)
    z[3, 2:] = -INF                                   # fewer than k
    z[4] = -INF                                       # none
    z[5, ::2] = -INF
    ids = check_balance(z, 5, balance_weight=0.1)[0]
    assert ids[3].tolist()[2:] == [-1] * 3 and ids[4].tolist() == [-1] * 5
    bad = z.clone()
    bad[10, 7] = float("nan")
    ids2, w, counts, loss, saved = ops.balance_forward(bad, 5)
    assert torch.isnan(w[10]).all() and torch.isnan(loss)
    assert len(set(ids2[10].tolist())) == 5 and torch.equal(ids2[:10], ids[:10]) and torch.equal(ids2[11:], ids[11:])
    assert bool(torch.isfinite(w[:10]).all())
    none = torch.full((70, 9), -INF, device="cuda")
    ids, w, counts, loss, saved = ops.balance_forward(none, 2, z_weight=1.0)
    assert bool((ids == -1).all()) and not w.any() and not counts.any() and float(loss) == 0
    assert not ops.balance_backward(none, ids, counts, saved, torch.ones(70, 2, device="cuda"), z_weight=1.0).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_balance_strides_in_place_and_determinism(dtype):
    tokens, experts, k = 900, 64, 4
    z0 = randn(gen(5), tokens, experts).to(dtype)
    wide = torch.full((tokens, experts + 5), 9.0, device="cuda", dtype=dtype)
    z = wide[:, 1:1 + experts]
    z.copy_(z0)
    dw = torch.randn(tokens, k, device="cuda")
    a = ops.balance_forward(z0, k, z_weight=0.1)
    b = ops.balance_forward(z, k, z_weight=0.1)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    da = ops.balance_backward(z0, a[0], a[2], a[4], dw, z_weight=0.1)
    db = ops.balance_backward(z, b[0], b[2], b[4], dw, z_weight=0.1, out=z)
    assert torch.equal(da, db) and bool((wide[:, 0] == 9).all() and (wide[:, 1 + experts:] == 9).all())
    for _ in range(3):
        for s, t in zip(a, ops.balance_forward(z0, k, z_weight=0.1)):
            assert torch.equal(s, t)


def test_balance_no_tokens():
    ids, w, counts, loss, saved = ops.balance_forward(torch.empty(0, 8, device="cuda"), 2)
    assert ids.shape == (0, 2) and not counts.any() and float(loss) == 0


def test_balance_gradient_against_differences():
    """The counts do not move under a small change, so differences see the
    gradient that holds them fixed."""
    z = randn(gen(8), 60, 12)
    mask = torch.rand(60, device="cuda", generator=gen(9)) < 0.8
    how = dict(mask=mask, groups=3, balance_weight=0.4, z_weight=0.05)
    zz = z.clone().requires_grad_(True)
    ids, w, counts, loss = ops.balance(zz, 3, **how)
    c = torch.randn(60, 3, device="cuda", generator=gen(10))
    (loss * 2 + (w * c).sum()).backward()
    v = torch.randn(60, 12, dtype=torch.float64)
    h = 1e-6

    def value(s):
        _, w2, cnt, l2, _ = R.balance(z.double().cpu() + s * v, 3, **how)
        assert torch.equal(cnt, counts.cpu())
        return l2 * 2 + (w2 * c.double().cpu()).sum()

    along = zz.grad.double().cpu() * v
    assert abs(float(along.sum() - (value(h) - value(-h)) / (2 * h))) <= 1e-5 * float(along.abs().sum())


# ------------------------------------------------------------- streams and graphs

def test_other_stream_and_graph():
    z, ids, top, how = distill_case(16, 5000, 8, BF16, 1)
    x, y, nh = norm_case(64, 512, BF16, BF16, BF16, "rms", "rms", 0)
    zb = randn(gen(3), 512, 16)
    torch.cuda.synchronize()

    def everything(stream=None):
        loss, dz = ops.distill_loss_grad(z, ids, top, stream=stream, **how)
        r, h, stats = ops.norm_gate_forward(x, y, stream=stream, **nh)
        g = ops.norm_gate_backward(r, h, r, y, stats, stream=stream, **nh)
        b = ops.balance_forward(zb, 2, stream=stream)
        d = ops.balance_backward(zb, b[0], b[2], b[4], b[1], stream=stream)
        return [loss, dz, r, h, stats, *[v for v in g.values() if v is not None], *b, d]

    want = [t.clone() for t in everything()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    z.copy_(z.flip(0).clone())
    graph.replay()
    for a, b in zip(everything(), got):
        assert torch.equal(a, b)


def test_refusals_on_the_gpu():
    z, ids, top, how = distill_case(4, 100, 3, BF16)
    for bad in (lambda: ops.distill_forward(z.half(), ids, top), lambda: ops.distill_forward(z.t(), ids, top),
                lambda: ops.distill_forward(z, ids[:3], top), lambda: ops.distill_forward(z, ids.short(), top),
                lambda: ops.distill_forward(z.cpu(), ids, top), lambda: ops.distill_forward(z[:1].expand(4, 100), ids, top)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.distill_forward(z, ids, top, temperature=0.0), lambda: ops.distill_forward(z, ids, top, ce_weight=-1.0),
                lambda: ops.distill_loss_grad(z, ids, top, temperature=float("nan")),
                lambda: ops.balance_forward(z, 101), lambda: ops.balance_forward(z, 2, groups=3),
                lambda: ops.norm_gate_forward(z, z, gate=z[:3])):
        with pytest.raises(C.Bf16OptError):
            bad()
    base = torch.zeros(4 * 100 + 50, dtype=BF16, device="cuda")
    with pytest.raises(C.Bf16OptError):               # an output that overlaps, but is not, the input
        ops.distill_loss_grad(base[:400].view(4, 100), ids, top, out=base[50:450].view(4, 100))
