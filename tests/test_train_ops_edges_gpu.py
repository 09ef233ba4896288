"""The training operators on the GPU where they are easily wrong: rows far from zero, norms without weights,
tokens that are off, and what autograd and streams ask of them.

Tolerances as in test_train_ops_gpu.py: an output's own rounding, and 2e-5 of the magnitudes summed in FP32.
"""
import pytest

torch = pytest.importorskip("torch")

import train_ops_reference as R  # noqa: E402
from mixed_precision_optimizer_bf16_gb300 import train_ops as ops  # noqa: E402
from test_train_ops_gpu import (BF16, F32, INF, check_balance, check_distill, check_norm, close, distill_case, gen,  # noqa: E402
                                loss_scale, norm_case, randn, rowmax)

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]


# ------------------------------------------------------------------- gated norms

BARE = pytest.mark.parametrize("hidden", [1, 7, 40, 257, 264, 500, 1031, 2049, 4104, 9001])


def bare(hidden, branch, stream, gate, bias):
    x, y, how = norm_case(6, hidden, branch, stream, F32, "layer", "layer", 3 if gate else 0)
    how = {n: v for n, v in how.items() if not n.endswith("_weight") and (bias or not n.endswith("_bias"))}
    return x, y, dict(how, gate_act=gate or "none")


@pytest.mark.parametrize("branch,stream", [(BF16, BF16), (BF16, F32), (F32, F32)])
@BARE
@pytest.mark.parametrize("gate", [None, "none", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_norm_layer_norms_without_weights(hidden, branch, stream, gate, bias):
    """Both norms subtract a mean and have no weight: what lies beyond a row's end in its threads counts for nothing."""
    x, y, how = bare(hidden, branch, stream, gate, bias)
    r, h, stats = ops.norm_gate_forward(x, y + 3, **how)
    for got, want, n in zip((r, h, stats), R.norm_gate(x, y + 3, **how), ("r", "h", "stats")):
        close(got, want, rowmax(want) if n != "stats" else 1 + want.abs(), n)


@pytest.mark.parametrize("branch,stream", [(BF16, BF16), (BF16, F32), (F32, F32)])
@BARE
@pytest.mark.parametrize("gate", [None, "sigmoid"])
def test_norm_layer_norms_without_weights_backward(hidden, branch, stream, gate):
    check_norm(*bare(hidden, branch, stream, gate, False))


# ------------------------------------------------------------------ distillation

@pytest.mark.parametrize("temperature", [1.5, 0.7, 2.0])
@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("away", [1e4, -1e4, 1e6])
def test_distill_teacher_far_from_zero(away, full, temperature):
    """Distinct teacher's logits far from zero: their softmax comes from differences."""
    z, ids, top, how = distill_case(5, 3001, 21, F32, 12, labels=True, temperature=temperature)
    top = top + away
    if full:    # the normaliser as an FP32 number, whatever it comes to: the formula takes it as it is
        how["teacher_lse"] = torch.logsumexp(top.double() / temperature, 1).float()
    exact = dict(how, temperature=torch.tensor(temperature).item())      # the number that the call takes: FP32
    loss_r, dz_r, scale, _ = R.distill(z, ids, top, **exact)
    loss, dz = ops.distill_loss_grad(z, ids, top, **how)
    close(loss, loss_r, loss_scale(z, top - away, how), "loss")
    close(dz, dz_r, scale, "dlogits")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_distill_teacher_at_the_types_ends(sign, dtype):
    """t / T does not fit FP32 at T = 0.5: the largest entry alone has a probability."""
    z, ids, top, how = distill_case(4, 515, 6, F32, 13, labels=True, temperature=0.5)
    top = (sign * torch.finfo(dtype).max * (1 - torch.arange(6, device="cuda") / 16.0)).to(dtype).expand(4, 6).contiguous()
    loss_r, dz_r, scale, _ = R.distill(z, ids, top, **how)
    loss, dz = ops.distill_loss_grad(z, ids, top, **how)
    close(loss, loss_r, loss_scale(z, torch.zeros_like(top), how), "loss")
    close(dz, dz_r, scale, "dlogits")


def far_case(rows, vocab, k, dtype, away, temperature, weights=False):
    z, ids, top, how = distill_case(rows, vocab, k, dtype, 11, labels=True, weights=weights, temperature=temperature)
    if isinstance(away, str):
        away = (-1 if away == "lowest" else 1) * torch.finfo(dtype).max
    z = (z.float() + away).to(dtype)
    return z, z.double() - away, ids, top, how


@pytest.mark.parametrize("temperature", [1.0, 2.0, 1.5, 0.5])
@pytest.mark.parametrize("away", [300.0, -300.0, 1e4, -1e6, "lowest", "largest"])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_distill_backward_far_from_zero(dtype, away, temperature):
    """The gradient from saved log-sum-exps, whose FP32 number has no room for the sum's logarithm beside a far maximum."""
    z, near, ids, top, how = far_case(5, 6007, 37, dtype, away, temperature)
    _, dz_r, scale, _ = R.distill(near, ids, top, **how)
    dloss = torch.ones(5, device="cuda")
    lse = ops.distill_forward(z, ids, top, **how)[1]
    back = ops.distill_backward(z, ids, top, lse, dloss, **how)
    close(back, dz_r, scale, "dlogits of the backward call")
    leaf = z.clone().requires_grad_(True)
    ops.distill_loss(leaf, ids, top, **how).sum().backward()
    assert torch.equal(leaf.grad, back)
    assert torch.equal(ops.distill_backward(z, ids, top, lse, dloss, out=z, **how), back)    # in place


@pytest.mark.parametrize("dtype,rows,vocab", [(F32, 330, 40001), (BF16, 3, 250880), (BF16, 310, 70001), (F32, 700, 2051)])
@pytest.mark.parametrize("temperature", [1.0, 4.0])
def test_distill_backward_far_and_near_rows(dtype, rows, vocab, temperature):
    """Rows far from zero among others and rows of weight 0, several to each cluster of CTAs; an all-masked row."""
    z, near, ids, top, how = far_case(rows, vocab, 9, dtype, 0.0, temperature, weights=True)
    z[1::3] = (z[1::3].float() - 5000).to(dtype)
    near[1::3] = z[1::3].double() + 5000
    how["row_weight"][0] = 1.0
    z[0], near[0], ids[0], how["labels"][0] = -INF, -INF, -1, -1
    _, dz_r, scale, _ = R.distill(near, ids, top, **how)
    lse = ops.distill_forward(z, ids, top, **how)[1]
    back = ops.distill_backward(z, ids, top, lse, **how)
    close(back, dz_r, scale, "dlogits of the backward call")
    assert not back[0].any()
    for _ in range(2):
        assert torch.equal(ops.distill_backward(z, ids, top, lse, **how), back)


@pytest.mark.parametrize("dtype,rows,vocab", [(BF16, 400, 130001), (F32, 330, 40001)])
def test_distill_rows_of_weight_zero_in_clusters(dtype, rows, vocab):
    """Several CTAs to a row and several rows to a cluster, some of weight 0."""
    z, ids, top, how = distill_case(rows, vocab, 9, dtype, 14, labels=True, weights=True, temperature=2.0)
    check_distill(z, ids, top, how)


# ----------------------------------------------------------------- expert balance

def from_top(z):
    """Logits less their token's largest, in 64 bits: the same softmax, where the type's lowest would leave the
    logarithm of a sum no room in 64 bits either.  (Not with a z-loss.)"""
    top = z.double().amax(1, keepdim=True)
    return z.double() - torch.where(torch.isfinite(top), top, torch.zeros_like(top))


def check_balance_far(z, k, **how):
    """check_balance without a z-loss, for logits anywhere."""
    dw = torch.randn(z.shape[0], k, device="cuda", generator=gen(11))
    ids, weights, counts, loss, saved = ops.balance_forward(z, k, **how)
    dz = ops.balance_backward(z, ids, counts, saved, dw, **how)
    r = R.balance(from_top(z), k, dweights=dw, **how)
    assert torch.equal(ids.cpu(), r[0]) and torch.equal(counts.cpu(), r[2])
    close(weights, r[1], 1.0 * (r[1] != 0), "weights")
    close(loss, r[3], r[3].abs(), "loss")
    close(dz, r[4], 0.2 * rowmax(r[4]) + rowmax(dw.double()).cpu(), "dlogits")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tokens,groups", [(70, 2), (4000, 1), (4000, 4), (4000, 100)])
def test_balance_loss_of_the_lowest_logits(tokens, groups, dtype):
    """Without the z-loss the square of a far log-sum-exp, which FP32 cannot hold, is no part of the loss."""
    z = randn(gen(6), tokens, 16).to(dtype)
    z[::9] = torch.finfo(dtype).min
    got = ops.balance_forward(z, 2, groups=groups, balance_weight=0.5)
    want = R.balance(from_top(z), 2, groups=groups, balance_weight=0.5)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[2].cpu(), want[2])
    close(got[1], want[1], 1.0 * (want[1] != 0), "weights")
    close(got[3], want[3], want[3].abs(), "loss")


@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("dtype,experts", [(F32, 8), (BF16, 24), (BF16, 64), (BF16, 200), (F32, 256), (F32, 600)])
@pytest.mark.parametrize("away", [20.0, -300.0, 1e4, -1e6, "lowest", "largest"])
def test_balance_far_from_zero(dtype, experts, away, renormalise):
    """Adding a number to a token's logits changes neither its weights nor, without the z-loss, loss and gradient."""
    if isinstance(away, str):
        away = (-1 if away == "lowest" else 1) * torch.finfo(dtype).max
    z = (2 * randn(gen(3), 70, experts) + away).to(dtype)
    check_balance_far(z, 3, balance_weight=0.5, renormalise=renormalise, groups=2)


def test_balance_nan_backward_stays_in_its_token():
    """A NaN makes its token's gradient NaN; the counts, which the others' depend on, stay whole numbers."""
    for dtype, experts in ((F32, 40), (BF16, 64), (BF16, 256)):
        z = randn(gen(4), 130, experts).to(dtype)
        z[10, 7] = z[77, 0] = float("nan")
        up = torch.randn(130, 5, device="cuda", generator=gen(5))
        how = dict(balance_weight=0.3, z_weight=0.1, groups=2)
        ids, w, counts, loss, saved = ops.balance_forward(z, 5, **how)
        dz = ops.balance_backward(z, ids, counts, saved, up, **how)
        want = R.balance(z, 5, dweights=up, **how)
        assert torch.equal(ids.cpu(), want[0]) and torch.equal(counts.cpu(), want[2]) and bool(torch.isnan(loss))
        keep = torch.ones(130, dtype=torch.bool)
        keep[[10, 77]] = False
        assert bool(torch.isnan(dz[[10, 77]]).all()) and bool(torch.isnan(w[[10, 77]]).all())
        close(dz.cpu()[keep], want[4][keep], 0.2 * want[4][keep].abs().amax(1, keepdim=True) + up.double().cpu()[keep].abs().amax(1, keepdim=True),
              "dlogits")


@pytest.mark.parametrize("experts", [33, 40, 64, 100, 128, 200, 256])
@pytest.mark.parametrize("k", [1, 5, 8, 9, 32])
def test_balance_bf16_ties_off_experts_and_nan(experts, k):
    """The choice from sorted keys of 16 bits: many ties, both zeros, experts that are off, NaN, more than eight choices."""
    tokens = 60
    z = torch.randint(-2, 3, (tokens, experts), device="cuda", generator=gen(experts)).bfloat16()
    zero = (z == 0) & (torch.rand(tokens, experts, device="cuda", generator=gen(1)) < 0.5)
    z[zero] = -0.0
    z[3, min(2, k):] = -INF                           # two experts on, or as many as are chosen
    z[4] = -INF
    z[5, ::2] = -INF
    z[6] = torch.finfo(BF16).min                      # a number like any other
    z[7, 1:] = torch.finfo(BF16).min
    z[8, 1:] = -INF
    check_balance_far(z, k, balance_weight=0.1)
    bad = z.clone()
    bad[10, 7] = float("nan")
    bad[11, : experts - 1] = float("nan")             # one number, the rest NaN
    bad[12, 1::2] = -INF
    bad[12, 0] = -float("nan")
    bad[13] = float("nan")
    got = ops.balance_forward(bad, k)
    want = R.balance(from_top(bad), k)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[2].cpu(), want[2])
    odd = [10, 11, 12, 13]
    there = got[0][odd] >= 0
    assert bool(torch.isnan(got[1][odd][there]).all()) and not got[1][odd][~there].any() and bool(torch.isnan(got[3]))
    keep = [t for t in range(tokens) if t not in odd]
    close(got[1].cpu()[keep], want[1][keep], 1.0 * (want[1][keep] != 0), "weights")


@pytest.mark.parametrize("dtype,experts", [(F32, 1), (F32, 9), (BF16, 48), (F32, 119), (BF16, 256), (F32, 600)])
def test_balance_one_choice_has_all_the_weight(dtype, experts):
    """Renormalised, a single choice's weight is 1 whatever the logits are: nothing comes back through it, not even a
    rounding, which would be large beside the balance loss's own gradient over many tokens."""
    z = randn(gen(10), 500, experts).to(dtype)
    up = torch.randn(500, 1, device="cuda", generator=gen(11))
    ids, w, counts, loss, saved = ops.balance_forward(z, 1)
    close(w, torch.ones_like(w), 0.0, "weights")
    assert torch.equal(ops.balance_backward(z, ids, counts, saved, up), ops.balance_backward(z, ids, counts, saved))
    z[:, 1:] = -INF                                   # or the only expert that is on
    if experts > 1:
        ids, w, counts, loss, saved = ops.balance_forward(z, 2)
        up = torch.randn(500, 2, device="cuda", generator=gen(11))
        assert torch.equal(ops.balance_backward(z, ids, counts, saved, up), ops.balance_backward(z, ids, counts, saved))


def balance_plain(z, k, mask, groups, balance_weight, z_weight, renormalise, dweights, dloss):
    """R.balance for many tokens: by whole tensors, on their device, without NaN."""
    z = z.double()
    tokens, experts = z.shape
    live = (mask.bool() & ~(z == -INF).all(1))[:, None]
    p, lse = R._soft(z)
    order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :k]
    there = live & (z.gather(1, order) != -INF)
    w = torch.where(there, p.gather(1, order), 0.0)
    weights = w / torch.where(live, w.sum(1, keepdim=True), 1.0) if renormalise else w
    sent = torch.zeros_like(z).scatter_add_(1, order, there.double())
    counts = sent.reshape(groups, -1, experts).sum(1)
    n = live.double().reshape(groups, -1).sum(1, keepdim=True)
    f = (counts * experts / (k * n.clamp(min=1))).repeat_interleave(tokens // groups, 0)
    per = (dloss / (groups * n.clamp(min=1))).repeat_interleave(tokens // groups, 0)
    lse = torch.where(live, lse[:, None], 0.0)
    dz = per * (balance_weight * p * (f - (p * f).sum(1, keepdim=True)) + 2 * z_weight * lse * p)
    if dweights is not None:
        u = torch.where(there, dweights.double(), 0.0)
        dot = (weights * u).sum(1, keepdim=True)
        dz = dz.scatter_add(1, order, weights * (u - dot) if renormalise else weights * u) - (0.0 if renormalise else p * dot)
    return torch.where(there, order, -1).int(), weights, counts.int(), torch.where(live, dz, 0.0)


@pytest.mark.parametrize("experts", [136, 200, 256])
@pytest.mark.parametrize("groups", [1, 6, 900])
@pytest.mark.parametrize("renormalise", [True, False])
def test_balance_backward_ring(experts, groups, renormalise):
    """bf16 and 129 to 256 experts, several tokens to a warp: groups, masked tokens, experts that are off, rows apart, in place."""
    tokens, k = 19800, 7
    g = gen(groups)
    z = randn(g, tokens, experts).bfloat16()
    z[torch.rand(tokens, experts, device="cuda", generator=g) < 0.05] = -INF
    z[3, 4:] = -INF                                   # fewer than k
    z[5::50] = -INF
    mask = torch.rand(tokens, device="cuda", generator=g) < 0.7
    mask[tokens // groups: 2 * (tokens // groups)] = False
    mask[:4] = True
    how = dict(groups=groups, mask=mask, renormalise=renormalise, balance_weight=0.3, z_weight=0.01)
    up = torch.randn(tokens, k, device="cuda", generator=gen(11))
    dloss = torch.tensor(0.6, device="cuda")
    ids, w, counts, loss, saved = ops.balance_forward(z, k, **how)
    dz = ops.balance_backward(z, ids, counts, saved, up, dloss, **how)
    want = balance_plain(z, k, dweights=up, dloss=0.6, **how)
    assert torch.equal(ids, want[0]) and torch.equal(counts, want[2])
    close(w, want[1], 1.0 * (want[1] != 0), "weights")
    close(dz, want[3], 0.2 * rowmax(want[3]) + rowmax(up.double()), "dlogits")
    wide = torch.full((tokens, experts + 16), 5.0, dtype=BF16, device="cuda")
    apart = wide[:, 8:8 + experts]
    apart.copy_(z)
    got = ops.balance_backward(apart, ids, counts, saved, up, dloss, out=apart, **how)
    assert torch.equal(got, dz) and bool((wide[:, :8] == 5).all() and (wide[:, 8 + experts:] == 5).all())
    alone = ops.balance_backward(z, ids, counts, saved, None, **how)
    want = balance_plain(z, k, dweights=None, dloss=1.0, **how)
    close(alone, want[3], 0.2 * rowmax(want[3]), "dlogits without the weights' gradients")


def test_balance_plain_against_the_reference():
    """The form for many tokens is the one token by token."""
    z = randn(gen(7), 120, 24).bfloat16()
    z[torch.rand(120, 24, device="cuda", generator=gen(8)) < 0.2] = -INF
    z[5] = z[40, 2:] = -INF
    mask = torch.rand(120, device="cuda", generator=gen(9)) < 0.7
    mask[24:48] = False
    up = torch.randn(120, 3, device="cuda", generator=gen(11))
    for renormalise in (True, False):
        how = dict(mask=mask, groups=5, balance_weight=0.3, z_weight=0.01, renormalise=renormalise, dweights=up, dloss=0.6)
        got, want = balance_plain(z, 3, **how), R.balance(z, 3, **how)
        assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[2].cpu(), want[2])
        assert float((got[1].cpu() - want[1]).abs().max()) < 1e-13 and float((got[3].cpu() - want[4]).abs().max()) < 1e-13


# -------------------------------------------------------- autograd, outputs, streams

def graphs():
    """Each operator on leaves of its own: (leaf, outputs)."""
    z, ids, top, how = distill_case(6, 300, 5, F32, 1, labels=True, temperature=2.0)
    z.requires_grad_(True)
    yield "distill", z, ops.distill_loss(z, ids, top, **how).sum()
    x, y, nh = norm_case(6, 72, F32, F32, F32, "rms", "layer", 1)
    y.requires_grad_(True)
    r, h = ops.norm_gate(x, y, **nh)
    yield "norm", y, (r * r).sum() + (h * h * h).sum()
    z = randn(gen(2), 24, 8).requires_grad_(True)
    ids, w, counts, loss = ops.balance(z, 2, z_weight=0.1)
    yield "balance", z, (w * w).sum() + loss


def test_gradients_of_gradients_are_refused():
    """create_graph keeps the gradients themselves; going through them once more is an error, not a constant."""
    for name, leaf, value in graphs():
        plain, = torch.autograd.grad(value, leaf, retain_graph=True)
        first, = torch.autograd.grad(value, leaf, create_graph=True)
        assert torch.equal(first, plain), name
        with pytest.raises(RuntimeError, match="train_ops"):
            (value + first.square().sum()).backward()


def test_written_tensors_are_marked_as_written():
    z, ids, top, how = distill_case(6, 300, 5, BF16, 1, labels=True)
    lse = ops.distill_forward(z, ids, top, **how)[1]
    for call in (lambda o: ops.distill_backward(z, ids, top, lse, out=o, **how),
                 lambda o: ops.distill_loss_grad(z, ids, top, out=o, **how)):
        o = torch.empty_like(z)
        before = o._version
        call(o)
        assert o._version > before
    zb = randn(gen(2), 24, 8)
    b = ops.balance_forward(zb, 2)
    o = torch.empty_like(zb)
    before = o._version
    ops.balance_backward(zb, b[0], b[2], b[4], out=o)
    assert o._version > before
    x, y, nh = norm_case(6, 72, BF16, BF16, BF16, "rms", "rms", 0)
    xv, yv = x._version, y._version
    ops.norm_gate_forward(x, y, out_r=x, out_h=y, **nh)
    assert x._version > xv and y._version > yv
    with torch.inference_mode():                       # such tensors have no version
        ops.distill_loss_grad(z.clone(), ids, top, out=torch.empty_like(z), **how)


def test_a_saved_tensor_that_was_overwritten_is_an_error():
    """A loss by autograd, then both at once over the same logits in place, then the first one's backward."""
    z, ids, top, how = distill_case(6, 300, 5, F32, 1, labels=True)
    leaf = z.clone().requires_grad_(True)
    logits = leaf * 1.0
    loss = ops.distill_loss(logits, ids, top, **how)
    _, dlogits = ops.distill_loss_grad(logits, ids, top, out=logits, **how)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()
    logits = leaf + 1.0                                # nothing saved: the gradient goes on from where the logits were
    _, dlogits = ops.distill_loss_grad(logits, ids, top, out=logits, **how)
    logits.backward(dlogits.detach().clone())
    assert torch.equal(leaf.grad, ops.distill_loss_grad(z + 1.0, ids, top, **how)[1])


def test_a_leaf_that_requires_a_gradient_is_not_written():
    z, ids, top, how = distill_case(6, 300, 5, F32, 1, labels=True)
    lse = ops.distill_forward(z, ids, top, **how)[1]
    zb = randn(gen(2), 24, 8)
    b = ops.balance_forward(zb, 2)
    x, y, nh = norm_case(6, 72, F32, F32, F32, "rms", "rms", 0)
    calls = [(z, lambda o: ops.distill_loss_grad(z, ids, top, out=o, **how)), (z, lambda o: ops.distill_backward(z, ids, top, lse, out=o, **how)),
             (zb, lambda o: ops.balance_backward(zb, b[0], b[2], b[4], out=o)), (x, lambda o: ops.norm_gate_forward(x, y, out_r=o, **nh)),
             (y, lambda o: ops.norm_gate_forward(x, y, out_h=o, **nh))]
    for like, call in calls:
        for leaf in (torch.zeros_like(like).requires_grad_(True), torch.zeros_like(like).requires_grad_(True)[:]):
            with pytest.raises(ValueError, match="requires a gradient"):
                call(leaf)
            assert not leaf.any()
        with torch.no_grad():
            call(leaf)
        assert bool(leaf.any())


def test_frozen_weights_cost_nothing(monkeypatch):
    """Gradients that nobody asked for are not computed."""
    x, y, nh = norm_case(24, 264, F32, F32, F32, "layer", "layer", 3)
    names = ["gate", "pre_weight", "pre_bias", "post_weight", "post_bias"]
    asked = []
    backward = ops.C.bf16opt_norm_gate_backward

    def recorded(d, dr, dh, r, yy, stats, dx, dy, *weights):
        asked.append([bool(w) for w in weights[:5]])
        return backward(d, dr, dh, r, yy, stats, dx, dy, *weights)
    monkeypatch.setattr(ops.C, "bf16opt_norm_gate_backward", recorded)

    def grads(wanted):
        leaves = {n: nh[n].clone().requires_grad_(n in wanted) for n in names}
        yy = y.clone().requires_grad_(True)
        r, h = ops.norm_gate(x, yy, **{**nh, **leaves})
        ((r * r).sum() + h.square().sum()).backward()
        return {"y": yy.grad, **{n: leaves[n].grad for n in names}}
    everything = grads(names)
    for wanted in ([], ["gate"], ["pre_bias"], ["post_weight"], ["gate", "pre_weight", "post_bias"]):
        got = grads(wanted)
        assert asked[-1] == [n in wanted for n in names]
        for n, v in got.items():
            assert (v is None) == (n != "y" and n not in wanted)
            if v is not None:
                assert torch.equal(v, everything[n]), n


def test_a_row_weight_that_requires_a_gradient_is_refused():
    z, ids, top, how = distill_case(6, 300, 5, F32, 1, labels=True, weights=True)
    how["row_weight"].requires_grad_(True)
    with pytest.raises(ValueError, match="row_weight"):
        ops.distill_loss(z.requires_grad_(True), ids, top, **how)
    with torch.no_grad():
        assert ops.distill_loss(z, ids, top, **how).shape == (6,)


def test_tensors_by_name():
    z, ids, top, how = distill_case(6, 300, 5, F32, 1, labels=True)
    named = dict(logits=z, teacher_ids=ids, teacher_logits=top, **how)
    loss, lse = ops.distill_forward(**named)
    for a, b in zip((loss, lse), ops.distill_forward(z, ids, top, **how)):
        assert torch.equal(a, b)
    assert torch.equal(ops.distill_backward(lse=lse, **named), ops.distill_backward(z, ids, top, lse, **how))
    assert torch.equal(ops.distill_loss_grad(**named)[1], ops.distill_loss_grad(z, ids, top, **how)[1])
    x, y, nh = norm_case(6, 72, F32, F32, F32, "rms", "rms", 0)
    r, h, stats = ops.norm_gate_forward(x=x, y=y, **nh)
    got, want = ops.norm_gate_backward(dr=r, dh=h, r=r, y=y, stats=stats, **nh), ops.norm_gate_backward(r, h, r, y, stats, **nh)
    assert torch.equal(got["dy"], want["dy"]) and torch.equal(got["dpre_weight"], want["dpre_weight"])
    zb = randn(gen(2), 24, 8)
    b = ops.balance_forward(logits=zb, k=2)
    assert torch.equal(ops.balance_backward(logits=zb, ids=b[0], counts=b[2], saved=b[4]), ops.balance_backward(zb, b[0], b[2], b[4]))


@pytest.mark.parametrize("named", [False, True])
def test_a_stream_is_taken_where_the_first_tensors_are_not_there(named, monkeypatch):
    """norm_gate_backward without dr, or with every tensor by name, launches on the stream that it was given."""
    x, y, nh = norm_case(24, 264, F32, F32, F32, "rms", "layer", 0)
    r, h, stats = ops.norm_gate_forward(x, y, **nh)
    want = ops.norm_gate_backward(None, h, r, y, stats, **nh)
    streams = []
    backward = ops.C.bf16opt_norm_gate_backward
    monkeypatch.setattr(ops.C, "bf16opt_norm_gate_backward", lambda *a: streams.append(a[-1]) or backward(*a))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    how = dict(dh=h, r=r, y=y, stats=stats, stream=side, **nh)
    got = ops.norm_gate_backward(dr=None, **how) if named else ops.norm_gate_backward(None, **how)
    torch.cuda.synchronize()
    assert streams == [side.cuda_stream]
    for n in ("dx", "dy", "dpre_weight"):
        assert torch.equal(got[n], want[n])


# ----------------------------------------------------------------------- many rows

def test_norm_more_rows_than_a_grid_has_blocks_for():
    """2^33 and a few rows of one column, the stream in place: 34 GB."""
    rows = 2 ** 33 + 7
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("34 GB of device memory wanted")
    x = torch.empty(rows, 1, dtype=BF16, device="cuda")
    y = torch.empty(rows, 1, dtype=BF16, device="cuda")
    for a in range(0, rows, 1 << 30):
        b = min(rows, a + (1 << 30))
        y[a:b] = torch.randint(-100, 100, (b - a, 1), device="cuda", dtype=torch.int8)
        x[a:b] = 8.0
    d = ops.C.bf16opt_norm_gate_t(rows, 1, 0, 0, 0, 0, 0, 0, 0, 0, None, None, None, None, None, 1.0, 1.0, 1e-5)
    ops.C.check(ops.C.bf16opt_norm_gate_forward(d, x.data_ptr(), y.data_ptr(), x.data_ptr(), None, None, torch.cuda.current_stream().cuda_stream))
    for a in range(0, rows, 1 << 30):
        b = min(rows, a + (1 << 30))
        assert torch.equal(x[a:b], y[a:b] + 8.0)       # whole numbers below 2^8: exact
