"""The fine-tuning operators on the GPU against their formulas in 64 bits.

Tolerances come from the arithmetic.  A rounding is off by at most half a step: 2^-9 of a bf16 value (2^-8 is
allowed), 2^-24 of an FP32 one.  The exponential of an exponent x (in powers of two) is off by 2^-22 (the function)
and 2^-23 |x| (x's own rounding and that of its factor); a sum of n terms by n 2^-24 of it."""
import math

import pytest

torch = pytest.importorskip("torch")

import tuning_reference as R  # noqa: E402
from mixed_precision_optimizer_bf16_gb300 import train_ops as ops  # noqa: E402
from mixed_precision_optimizer_bf16_gb300 import bf16opt as C  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
INF, NAN = float("inf"), float("nan")


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def close(got, ref, slack, what):
    """|got - ref| within the output type's rounding of ref (and its smallest normal number's) and `slack`; infinities and NaN alike."""
    u = 2.0 ** -8 if got.dtype == BF16 else 2.0 ** -23
    got, ref = got.double(), ref.double().to(got.device)
    slack = torch.as_tensor(slack, dtype=F64, device=got.device)
    assert got.shape == ref.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), (what, "NaN")
    odd = ~torch.isfinite(ref)
    assert torch.equal(got[odd & ~torch.isnan(ref)], ref[odd & ~torch.isnan(ref)]), (what, "infinities")
    err = torch.where(odd, torch.zeros_like(ref), (got - ref).abs())
    bound = torch.where(odd, torch.ones_like(ref), u * ref.abs() + slack + 2.0 ** -126)
    assert not bool((err > bound).any()), (what, int((err > bound).sum()), float((err / bound).max()))


# ------------------------------------------------------------------ token losses

def sum_error(vocab):
    """Of a row's sum, relative: the exponentials, their exponents (weighed, at most log2 of their number), the additions."""
    return 2.0 ** -21 + (vocab / 512 + 24 + 2 * math.log2(vocab + 1)) * 2.0 ** -24


def gradient_slack(scale, vocab):
    """Of dz: the sum's and the exponential's errors in q, and the slope's, all relative to what goes in; q |x| is at most 0.6.
    An exponential below 2^-126 is 0: dz is off by that times c / T, which is at most the row's largest scale (the label's)."""
    return (2 * sum_error(vocab) + 2.0 ** -20) * scale + 2.0 ** -126 * scale.amax(1, keepdim=True)


def rows_case(rows, vocab, dtype, seed=0, spread=3.0, away=0.0, pad=0, shift=0):
    """Logits whose rows lie `pad` further apart than they are long and begin `shift` elements from a boundary."""
    g = gen(seed)
    stride = vocab + pad
    flat = torch.zeros(rows * stride + shift + 8, dtype=dtype, device="cuda")
    z = flat[shift:shift + rows * stride].view(rows, stride)[:, :vocab]
    z.copy_(spread * randn(g, rows, vocab) + away)
    labels = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    return z, labels, g


def check_logp(z, labels, temperature=1.0, row_weight=None, dloss=None):
    vocab = z.shape[1]
    logp, saved = ops.token_logp_forward(z, labels, temperature=temperature, row_weight=row_weight)
    want, dz, scale = R.token_logp(z, labels, temperature, row_weight, dloss)
    close(logp, want, sum_error(vocab) + 2.0 ** -23 * want.abs().nan_to_num(0, 0, 0), "logp")
    got = ops.token_logp_backward(z, labels, saved, dloss, temperature=temperature)
    close(got, dz, gradient_slack(scale.nan_to_num(0, 0, 0), vocab), "dlogits")
    return logp, saved, got


SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 31), (300, 257), (40, 2053), (9, 4096), (700, 1000), (310, 12000), (3, 33000), (2, 70001), (2, 250880)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_logp_sizes(rows, vocab, dtype):
    z, labels, _ = rows_case(rows, vocab, dtype, rows + vocab)
    check_logp(z, labels)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,shift", [(0, 1), (1, 0), (3, 5), (8, 4), (5, 7)])
@pytest.mark.parametrize("vocab", [5, 40, 1001, 9001])
def test_logp_rows_anywhere(vocab, pad, shift, dtype):
    """Rows that begin between boundaries; what lies between them is left as it was."""
    z, labels, _ = rows_case(6, vocab, dtype, 3, pad=pad, shift=shift)
    logp, saved, dz = check_logp(z, labels.int(), 0.7)
    out = torch.full((6, vocab + 11), 5.0, dtype=dtype, device="cuda")
    ops.token_logp_backward(z, labels, saved, temperature=0.7, out=out[:, 3:3 + vocab])
    assert torch.equal(out[:, 3:3 + vocab], dz) and bool((out[:, :3] == 5).all()) and bool((out[:, 3 + vocab:] == 5).all())
    ops.token_logp_backward(z, labels, saved, temperature=0.7, out=z)       # in place
    assert torch.equal(z, dz)


@pytest.mark.parametrize("temperature", [1.0, 0.25, 2.0, 30.0])
@pytest.mark.parametrize("away", [-300.0, 300.0, 1e4, -1e4])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logp_far_from_zero(dtype, away, temperature):
    for vocab in (700, 9000, 40000):
        z, labels, _ = rows_case(5, vocab, dtype, 7, spread=4.0, away=away)
        check_logp(z, labels, temperature)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [3, 100, 5000, 33000])
def test_logp_masks_and_ends_of_the_type(vocab, dtype):
    """-inf, the type's lowest and largest values, whole rows of them, and where a thread sees them first."""
    low = torch.finfo(dtype).min
    z, labels, _ = rows_case(14, vocab, dtype, 11)
    z[0], labels[0] = -INF, 0
    z[1], labels[1] = low, vocab - 1
    z[2], labels[2] = -low, vocab // 2
    z[3, 1:], labels[3] = low, 0                       # one logit and masks
    z[4, :-1], labels[4] = -INF, vocab - 1
    z[5, :vocab // 2], labels[5] = low, vocab - 1      # masks first, logits behind
    z[6, :vocab // 2], labels[6] = -INF, vocab - 1
    z[7, vocab // 2:], labels[7] = -INF, vocab - 1     # the label is masked
    z[8] *= 1e30
    z[9, 0], labels[9] = -low, 0                       # one far above the rest
    z[10], z[10, 0], labels[10] = low, 0.5 * low, 0
    z[11] = -2e37 - z[11].abs() * 1e34
    z[12, 0], labels[12] = 1e20, vocab - 1
    z[13] -= 3e3
    logp, saved, dz = check_logp(z, labels)
    assert logp[0] == -INF and not dz[0, 1:].any() and dz[0, 0] == 1
    assert abs(float(logp[1]) + math.log(vocab)) < 1e-5 and abs(float(logp[2]) + math.log(vocab)) < 1e-5
    check_logp(z[8:], labels[8:], 0.01)
    check_logp(z[:8], labels[:8], 1e6)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [9, 2000, 33000])
def test_logp_nan_and_inf_stay_in_their_rows(vocab, dtype):
    z, labels, _ = rows_case(6, vocab, dtype, 13)
    clean = z.clone()
    z[1, vocab // 3] = NAN
    z[2, vocab - 1] = INF
    z[4] = NAN
    logp, saved = ops.token_logp_forward(z, labels)
    dz = ops.token_logp_backward(z, labels, saved)
    wrong = torch.tensor([False, True, True, False, True, False], device="cuda")
    want, more = ops.token_logp_forward(clean, labels)
    assert torch.equal(torch.isnan(logp), wrong) and torch.equal(logp[~wrong], want[~wrong])
    assert bool(torch.isnan(dz[wrong]).all()) and torch.equal(dz[~wrong], ops.token_logp_backward(clean, labels, more)[~wrong])


@pytest.mark.parametrize("rows,vocab", [(12, 300), (5, 40000)])
def test_logp_rows_that_do_not_count(rows, vocab):
    """Weight 0, labels outside: not read (NaN there), 0 everywhere."""
    z, labels, _ = rows_case(rows, vocab, BF16, 17)
    w = torch.ones(rows, device="cuda")
    w[1], labels[2], labels[3] = 0, -100, vocab
    clean = z.clone()
    z[1:4] = NAN
    logp, saved, dz = check_logp(clean, labels, 1.0, w)
    got, kept = ops.token_logp_forward(z, labels, row_weight=w)
    assert torch.equal(got, logp) and torch.equal(kept.view(torch.int32), saved.view(torch.int32)) and not got[1:4].any()
    assert bool((saved.view(torch.int32)[1:4, 3] == -1).all()) and not saved[1:4, :3].any()
    assert torch.equal(ops.token_logp_backward(z, labels, kept), dz) and not dz[1:4].any()
    dloss = torch.ones(rows, device="cuda")
    dloss[0] = 0                                     # and a row that nothing asks for
    z[0] = NAN
    assert not ops.token_logp_backward(z, labels, kept, dloss)[0].any()


def policy_case(rows, vocab, dtype, seed=0, old=True, ref=True, weights=False, temperature=1.0, **more):
    z, labels, g = rows_case(rows, vocab, dtype, seed, **more)
    logp = R.logp(z, labels, temperature)[0]
    moved = 0.3 * randn(g, rows).double()
    for border in (0.8, 1.25):                        # within 1e-3 of a border 32 bits may say either
        moved = torch.where((moved - math.log(border)).abs() < 1e-3, moved + 4e-3, moved)
    how = dict(temperature=temperature, clip_low=0.2, clip_high=0.25)
    how["old_logp"] = (logp - moved).float() if old else None
    if ref:
        how.update(ref_logp=(logp + 0.4 * randn(g, rows)).float(), kl_weight=0.05)
    if weights:
        how["row_weight"] = torch.where(torch.rand(rows, device="cuda", generator=g) < 0.3, 0.0, torch.rand(rows, device="cuda", generator=g) + 0.1)
    return z, labels, randn(g, rows), how


def check_policy(z, labels, adv, how, dloss=None):
    vocab = z.shape[1]
    loss_r, logp_r, slope_r, dz_r, scale = R.policy(z, labels, adv, dloss=dloss, **how)
    # the ratio and exp(ref - logp) are off by the log-probability's error and the exponential's, relative
    off = sum_error(vocab) + 2.0 ** -21
    w = how["row_weight"].double() if how.get("row_weight") is not None else 1.0
    back = torch.exp(how["ref_logp"].double() - logp_r) if how.get("ref_logp") is not None else 0.0
    size = w * (slope_r.abs() + adv.abs().double() * 1.25 + how.get("kl_weight", 0.0) * (1 + back))
    loss, logp, saved = ops.policy_forward(z, labels, adv, **how)
    close(loss, loss_r, off * size, "loss")
    close(logp, logp_r, sum_error(vocab), "logp")
    close(saved[:, 2], slope_r, off * size, "slope")
    # (a slope's error weighs with the softmax, and with 1 at the label: scale / |c| is that)
    slack = gradient_slack(scale, vocab) + torch.where(slope_r != 0, off * size / slope_r.abs().clamp(min=1e-300), torch.zeros_like(slope_r))[:, None] * scale
    got = ops.token_logp_backward(z, labels, saved, dloss, temperature=how["temperature"])
    close(got, dz_r, slack, "dlogits of the backward call")
    both = ops.policy_loss_grad(z, labels, adv, dloss, **how)
    close(both[0], loss_r, off * size, "loss of the single pass")
    close(both[1], logp_r, sum_error(vocab), "logp of the single pass")
    close(both[2], dz_r, slack, "dlogits of the single pass")
    return loss, both


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_policy_sizes(rows, vocab, dtype):
    z, labels, adv, how = policy_case(rows, vocab, dtype, rows + vocab, weights=rows > 4)
    check_policy(z, labels, adv, how)


@pytest.mark.parametrize("old", [False, True])
@pytest.mark.parametrize("ref", [False, True])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("temperature", [1.0, 0.6, 2.0])
def test_policy_terms(old, ref, weights, temperature):
    z, labels, adv, how = policy_case(64, 1537, F32, 5, old, ref, weights, temperature, pad=2, shift=3)
    g = gen(2)
    loss, both = check_policy(z, labels, adv, how, dloss=torch.rand(64, device="cuda", generator=g) - 0.3)
    if not old and not ref and not weights:
        assert torch.equal(loss, -adv)


@pytest.mark.parametrize("rows,vocab", [(30, 900), (4, 40000)])
def test_policy_clips(rows, vocab):
    """Clipped tokens have no gradient and are not read backward; ratios beyond exp's range, advantages of 0, no upper clip."""
    z, labels, adv, how = policy_case(rows, vocab, F32, 9, ref=False)
    logp = R.logp(z, labels)[0]
    how["old_logp"] = (logp - torch.linspace(-100, 100, rows, device="cuda")).float()
    adv[0], adv[rows - 1] = -1.5, 2.0
    adv[rows // 2] = 0
    loss, both = check_policy(z, labels, adv, how)
    assert not both[2][0].any() and not both[2][rows - 1].any()
    assert abs(float(loss[rows - 1]) + 2.0 * 1.25) < 1e-5 and abs(float(loss[0]) - 1.5 * 0.8) < 1e-5
    how["clip_high"] = INF
    how["old_logp"] = (logp - 3).float()
    adv = adv.abs() + 0.1
    check_policy(z, labels, adv, how)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab", [(20, 515), (3, 50001), (400, 8192)])
def test_policy_in_place(rows, vocab, dtype):
    z, labels, adv, how = policy_case(rows, vocab, dtype, 21, weights=True, pad=5, shift=2)
    want = ops.policy_loss_grad(z, labels, adv, **how)
    got = ops.policy_loss_grad(z, labels, adv, out=z, **how)
    assert got[2] is z and all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("vocab,dtype,pad,shift", [(20011, BF16, 1, 3), (36000, BF16, 0, 0), (12345, F32, 0, 0), (40009, BF16, 0, 0), (36872, BF16, 8, 0), (100003, BF16, 3, 5), (131072, BF16, 0, 0), (24577, F32, 0, 1), (66001, F32, 0, 0)])
def test_policy_many_long_rows(vocab, dtype, pad, shift):
    """More rows than the SMs, longer than shared memory's part of them: masked ones side by side, clipped ones, far ones, masks, NaN, in place."""
    rows = 640
    z, labels, adv, how = policy_case(rows, vocab, dtype, vocab % 97, weights=True, pad=pad, shift=shift)
    how["row_weight"][150:310] = 0                     # whole CTAs' turns
    labels[400:402] = -100
    how["old_logp"][410:415] -= 3                     # clipped where the advantage is positive
    how["ref_logp"][410:415] = R.logp(z[410:415], labels[410:415])[0].float()
    how["kl_weight"] = 0.0
    z[500] *= 1e6
    z[501] = torch.finfo(dtype).min
    z[502, vocab // 2:] = -INF
    for r in (500, 501, 502):
        labels[r] = 3
        how["row_weight"][r] = 0.5
        how["old_logp"][r] = (R.logp(z[r:r + 1], labels[r:r + 1])[0] - 0.05).float()
    loss_r, logp_r, slope_r, dz_r, scale = (x[480:] for x in R.policy(z, labels, adv, **how))
    off = sum_error(vocab) + 2.0 ** -21
    got = ops.policy_loss_grad(z, labels, adv, **how)
    loss, logp, saved = ops.policy_forward(z, labels, adv, **how)
    back = ops.token_logp_backward(z, labels, saved, temperature=how["temperature"])
    close(got[0][480:], loss_r, off * 2 * (loss_r.abs() + slope_r.abs()), "loss")
    close(got[1][480:], logp_r, sum_error(vocab) + 2.0 ** -23 * logp_r.abs(), "logp")
    close(got[2][480:], dz_r, gradient_slack(scale, vocab) + 2 * off * scale, "dlogits")
    # the other rows against the two calls: the same sums in another order, so a step of the type apart at most, and what the sums are off by
    assert torch.equal(got[2] == 0, back == 0)
    u = 2.0 ** -7 if dtype == BF16 else 2.0 ** -22
    assert bool(((got[2].double() - back.double()).abs() <= u * back.double().abs() + 4 * off * back.double().abs().amax(1, keepdim=True) + 2.0 ** -126).all())
    assert not got[2][150:310].any() and not got[2][400:402].any()
    z[320, 7], z[321, 0] = NAN, INF
    how["row_weight"][319:323] = 1.0
    how["old_logp"][319:323] = logp[319:323] if bool(logp[319:323].all()) else how["old_logp"][319:323]
    again = ops.policy_loss_grad(z, labels, adv, out=z, **how)
    assert bool(torch.isnan(again[2][320:322]).all()) and bool(torch.isnan(again[0][320:322]).all())
    same = torch.ones(rows, dtype=torch.bool, device="cuda")
    same[319:323] = False
    assert all(torch.equal(a[same], b[same]) for a, b in zip(got, again))


def test_policy_a_masked_label_and_rows_of_nothing():
    z, labels, adv, how = policy_case(4, 600, F32, 23)
    z[0, 300:], labels[0] = -INF, 400
    z[1] = -INF
    how.update(ref_logp=None, kl_weight=0.0)
    loss, both = check_policy(z, labels, adv, how)
    assert torch.isfinite(both[2]).all()
    how.update(ref_logp=torch.full((4,), -2.0, device="cuda"), kl_weight=0.1)
    loss, _, _ = ops.policy_forward(z, labels, adv, **how)
    assert loss[0] == INF and loss[1] == INF and bool(torch.isfinite(loss[2:]).all())


def preference_case(lengths, vocab, dtype, seed=0, spare=3, before=0, **more):
    pairs, rows = len(lengths) // 2, sum(lengths) + spare + before
    z, labels, g = rows_case(rows, vocab, dtype, seed, **more)
    ends = torch.tensor([before] + lengths, device="cuda").cumsum(0)
    labels[torch.rand(rows, device="cuda", generator=g) < 0.3] = -100
    return z, labels, ends, randn(g, 2 * pairs) - 3.0 * torch.tensor(lengths, device="cuda"), g


def check_preference(z, labels, ends, ref, dloss=None, **how):
    vocab = z.shape[1]
    loss_r, logp_r, dz_r, scale = R.preference(z, labels, ends, ref, dloss=dloss, **how)
    loss, logp, saved = ops.preference_forward(z, labels, ends, ref_logp=ref, **how)
    n = float(len(z)) if not how.get("length_normalise") else 1.0
    off = n * sum_error(vocab)                       # of a sum of log-probabilities
    close(logp, logp_r, off, "logp")
    beta, kind = how.get("beta", 0.1), how.get("kind", "sigmoid")
    d = (loss_r.sqrt() if kind == "ipo" else torch.zeros_like(loss_r)).nan_to_num(0, 0, 0)
    size = (logp_r.abs().sum() + ref.abs().sum().double() if ref is not None else logp_r.abs().sum()).nan_to_num(0, 0, 0)
    slope_off = 2 * (2 * off + 2.0 ** -23 * (d + 1 / beta)) if kind == "ipo" else beta * beta * 2 * off + beta * 2.0 ** -20 + beta * beta * size * 2.0 ** -23
    loss_off = 2 * d * (2 * off) + 4 * off * off + 2.0 ** -20 * d * d if kind == "ipo" else beta * 2 * off + 2.0 ** -21 * (1 + beta * size)
    close(loss, loss_r, loss_off, "loss")
    got = ops.token_logp_backward(z, labels, saved, dloss)
    up = 1.0 if dloss is None else float(dloss.abs().max())
    close(got, dz_r, gradient_slack(scale, vocab) + up * float(torch.as_tensor(slope_off).max()) * 2 * (scale > 0), "dlogits")   # the largest pair's
    return loss, logp, got


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths,vocab", [([3, 5], 40), ([1, 1, 0, 7], 2053), ([40, 3, 90, 600, 2, 77], 300), ([4, 6], 40000), ([0, 0], 9)])
def test_preference(lengths, vocab, dtype, mean, kind):
    z, labels, ends, ref, g = preference_case(lengths, vocab, dtype, 31, spread=1.0)
    how = dict(kind=kind, length_normalise=mean, beta=0.3, margin=0.2, label_smoothing=0.1 if kind == "sigmoid" else 0.0)
    dloss = torch.rand(len(lengths) // 2, device="cuda", generator=g) + 0.2
    check_preference(z, labels, ends.int(), ref, dloss, **how)
    check_preference(z, labels, ends, None, **how)


def test_preference_rows_outside_the_sequences():
    """Rows before the first and behind the last sequence are not read and have no gradient."""
    z, labels, ends, ref, _ = preference_case([6, 4, 9, 2], 700, BF16, 33, spare=5, before=4)
    want = check_preference(z, labels, ends, ref)
    first, last = int(ends[0]), int(ends[-1])
    z[:first], z[last:] = NAN, NAN
    loss, logp, saved = ops.preference_forward(z, labels, ends, ref_logp=ref)
    dz = ops.token_logp_backward(z, labels, saved)
    assert torch.equal(loss, want[0]) and torch.equal(logp, want[1]) and torch.equal(dz, want[2])
    assert not dz[:first].any() and not dz[last:].any()


@pytest.mark.parametrize("given", [[0, 9, 4, 12, 20], [-5, 3, 8, 99, 300], [7, 3, 2, 1, 0], [0, 25, 2, 25, 14], [20, 20, 20, 20, 20], [1 << 40, 0, 5, -(1 << 40), 11]])
def test_preference_offsets_that_are_no_offsets(given):
    z, labels, _, _, _ = preference_case([6, 6, 6, 2], 130, F32, 35, spare=0)
    ends = torch.tensor(given, device="cuda")
    check_preference(z, labels, ends, torch.randn(4, device="cuda", generator=gen(1)))


def test_preference_without_pairs_or_rows():
    z, labels, _, _, _ = preference_case([6, 6], 130, F32, 35)
    loss, logp, saved = ops.preference_forward(z, labels, torch.tensor([3], device="cuda"))
    assert loss.numel() == 0 and logp.numel() == 0 and not ops.token_logp_backward(z, labels, saved).any()
    loss, logp, saved = ops.preference_forward(z[:0], labels[:0], torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert torch.allclose(loss, torch.full_like(loss, math.log(2))) and not logp.any()
    assert ops.token_logp_forward(z[:0], labels[:0])[0].numel() == 0
    assert ops.policy_loss_grad(z[:0], labels[:0], z[:0, 0])[2].shape == (0, 130)


def test_policy_log_probabilities_at_the_ends():
    """A sampler's or a reference's -inf: the formula's value, in that row alone."""
    z, labels, adv, how = policy_case(6, 300, F32, 27)
    adv[:] = torch.tensor([1.0, -1.0, 1.0, 1.0, -1.0, 0.5], device="cuda")
    how["old_logp"][0], how["old_logp"][1], how["ref_logp"][2], how["ref_logp"][3] = -INF, -INF, -INF, INF
    loss, logp, saved = ops.policy_forward(z, labels, adv, **how)
    want = R.policy(z, labels, adv, **how)
    assert loss[1] == INF and loss[2] == INF and loss[3] == INF and bool(torch.isfinite(loss[[0, 4, 5]]).all())
    assert abs(float(loss[0] - want[0][0])) < 1e-5 and torch.equal(torch.isfinite(saved[:, 2]), torch.isfinite(want[2]))


def test_preference_extremes():
    """Margins far beyond exp's range, and a label on masked vocabulary."""
    z, labels, ends, ref, _ = preference_case([6, 6, 5, 5], 130, F32, 37)
    for beta in (50.0, 1e4):
        check_preference(z, labels, ends, ref, beta=beta)
    labels[labels < 0] = 0
    z[2, 7], labels[2] = -INF, 7
    loss, logp, saved = ops.preference_forward(z, labels, ends, ref_logp=ref)
    assert logp[0] == -INF and loss[0] == INF and bool(torch.isfinite(loss[1]))
    z[2, 8] = NAN
    loss, logp, saved = ops.preference_forward(z, labels, ends, ref_logp=ref)
    assert torch.isnan(loss[0]) and bool(torch.isfinite(loss[1]))
    dz = ops.token_logp_backward(z, labels, saved)
    in_pair = torch.zeros(len(z), dtype=torch.bool, device="cuda")
    for i in (0, 2):
        in_pair[int(ends[i]):int(ends[i + 1])] = True
    assert torch.equal(torch.isnan(dz).any(1), in_pair)


def test_saved_numbers_of_elsewhere():
    """An index that no loss belongs to counts as none."""
    z, labels, _ = rows_case(8, 500, BF16, 39)
    logp, saved = ops.token_logp_forward(z, labels)
    assert not ops.token_logp_backward(z, labels, saved, torch.ones(3, device="cuda"))[3:].any()
    saved.view(torch.int32)[:, 3] = torch.tensor([0, -7, 2 ** 31 - 1, 8, 7, -2 ** 31, 1, 2], device="cuda", dtype=torch.int32)
    dz = ops.token_logp_backward(z, labels, saved, torch.ones(8, device="cuda"))
    assert torch.equal(dz.any(1), torch.tensor([1, 0, 0, 0, 1, 0, 1, 1], device="cuda").bool())
    labels[0] = 10 ** 12                              # (a label that went away after the forward call)
    assert bool(torch.isfinite(ops.token_logp_backward(z, labels, saved)).all())


@pytest.mark.parametrize("what", ["logp", "policy", "preference"])
def test_token_losses_autograd(what):
    z, labels, adv, how = policy_case(24, 900, F32, 41)
    leaf = z.clone().requires_grad_(True)
    up = torch.rand(24, device="cuda", generator=gen(3))
    if what == "logp":
        loss = ops.token_logp(leaf * 1.0, labels, temperature=0.8)
        want = R.token_logp(z, labels, 0.8, dloss=up)[1]
    elif what == "policy":
        loss, logp = ops.policy_loss(leaf * 1.0, labels, adv, **how)
        assert not logp.requires_grad
        want = R.policy(z, labels, adv, dloss=up, **how)[3]
    else:
        ends, up = torch.tensor([0, 5, 11, 17, 22], device="cuda"), up[:2]
        loss, logp = ops.preference_loss(leaf * 1.0, labels, ends, beta=0.4)
        assert not logp.requires_grad
        want = R.preference(z, labels, ends, beta=0.4, dloss=up)[2]
    (loss * up).sum().backward()
    assert (leaf.grad.double() - want).abs().max() < 1e-5
    leaf.grad = None
    summed = (ops.token_logp(leaf, labels) if what == "logp" else ops.policy_loss(leaf, labels, adv, **how)[0] if what == "policy"
              else ops.preference_loss(leaf, labels, ends)[0]).sum()       # an expanded gradient
    (first,) = torch.autograd.grad(summed, leaf, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        first.square().sum().backward()


def test_token_losses_differences():
    """Directional differences of the 32-bit losses themselves."""
    z, labels, adv, how = policy_case(16, 300, F32, 43)
    ends = torch.tensor([0, 3, 8, 12, 16], device="cuda")
    d = randn(gen(4), *z.shape)
    for f in (lambda x: ops.token_logp(x, labels, temperature=1.4), lambda x: ops.policy_loss(x, labels, adv, **{**how, "clip_low": 1.0, "clip_high": INF})[0],
              lambda x: ops.preference_loss(x, labels, ends, beta=0.2)[0]):
        leaf = z.clone().requires_grad_(True)
        (grad,) = torch.autograd.grad(f(leaf).double().sum(), leaf)
        along = float((grad.double() * d.double()).sum())
        h = 2.0 ** -7
        got = float((f(z + h * d).double() - f(z - h * d).double()).sum()) / (2 * h)
        # third-order term h^2 of size and 2^-21 of each loss over h
        assert abs(got - along) < 0.03 * (1 + abs(along)), (got, along)


def test_token_losses_refusals():
    z, labels, adv, how = policy_case(6, 100, BF16, 45)
    ends = torch.tensor([0, 3, 6], device="cuda")
    for call, word in (
            (lambda: ops.token_logp_forward(z.half(), labels), "dtype"), (lambda: ops.token_logp_forward(z.t(), labels), "contiguous"),
            (lambda: ops.token_logp_forward(z, labels[:5]), "shape"), (lambda: ops.token_logp_forward(z, labels.float()), "dtype"),
            (lambda: ops.token_logp_forward(z, labels.cpu()), "CUDA"), (lambda: ops.token_logp_forward(z[0], labels), "two dimensions"),
            (lambda: ops.token_logp_forward(z, labels, row_weight=adv.double()), "dtype"), (lambda: ops.policy_forward(z, labels, adv[:3]), "shape"),
            (lambda: ops.policy_forward(z, labels, adv, old_logp=adv.bfloat16()), "dtype"), (lambda: ops.policy_forward(z, labels, adv[::1].expand(2, 6).t()[:, 0], ref_logp=adv[:1].expand(6)), "contiguous"),
            (lambda: ops.preference_forward(z, labels, ends[:2]), "2 pairs"), (lambda: ops.preference_forward(z, labels, ends.float()), "dtype"),
            (lambda: ops.preference_forward(z, labels, ends, kind="other"), "kind"), (lambda: ops.preference_forward(z, labels, ends, ref_logp=adv), "shape"),
            (lambda: ops.token_logp_backward(z, labels, torch.zeros(6, 3, device="cuda")), "shape"),
            (lambda: ops.token_logp_backward(z, labels, torch.zeros(6, 4, device="cuda"), adv[:, None]), "shape"),
            (lambda: ops.token_logp_backward(z, labels, torch.zeros(6, 4, device="cuda"), out=z.float()), "dtype"),
            (lambda: ops.policy_loss(z, labels, adv.requires_grad_(True)), "requires a gradient"),
            (lambda: ops.token_logp_backward(z, labels, torch.zeros(6, 4, device="cuda"), out=z.clone().requires_grad_(True)), "leaf")):
        with pytest.raises(ValueError, match=word):
            call()
    adv = adv.detach()
    for call in (lambda: ops.token_logp_forward(z, labels, temperature=0.0), lambda: ops.policy_forward(z, labels, adv, clip_low=2.0),
                 lambda: ops.preference_forward(z, labels, ends, beta=0.0), lambda: ops.policy_loss_grad(z, labels, adv, kl_weight=-1.0),
                 lambda: ops.token_logp_backward(z[:3], labels[:3], torch.zeros(3, 4, device="cuda"), out=z[1:4])):
        with pytest.raises(C.Bf16OptError):
            call()


# ------------------------------------------------------------------ 8 bits

def activations(rows, columns, dtype, seed=0, pad=0, shift=0):
    g = gen(seed)
    stride = columns + pad
    flat = torch.zeros(rows * stride + shift + 8, dtype=dtype, device="cuda")
    x = flat[shift:shift + rows * stride].view(rows, stride)[:, :columns]
    x.copy_(randn(g, rows, columns) * torch.exp(2 * randn(g, rows, 1)) * torch.exp(randn(g, 1, columns)))
    return x


COLUMNS = [1, 7, 8, 31, 32, 33, 100, 255, 256, 257, 1367, 4104, 8192]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("columns", COLUMNS)
@pytest.mark.parametrize("rows,pad,shift", [(1, 0, 0), (5, 8, 0), (37, 3, 1)])
def test_pack(rows, columns, pad, shift, dtype):
    x = activations(rows, columns, dtype, columns, pad, shift)
    codes, scales = ops.pack8(x)
    want = R.pack(x)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
    for t in (BF16, F32):
        assert torch.equal(ops.unpack8(codes, scales, columns, dtype=t), R.unpack(*want, columns).to(t))
    out = torch.full((rows, columns + 9), 7.0, dtype=dtype, device="cuda")
    ops.unpack8(codes, scales, columns, dtype=dtype, out=out[:, 4:4 + columns])
    assert torch.equal(out[:, 4:4 + columns].double(), R.unpack(*want, columns)) and bool((out[:, :4] == 7).all()) and bool((out[:, 4 + columns:] == 7).all())


@pytest.mark.parametrize("columns,pad", [(128, 0), (131, 0), (128, 1)])
def test_pack_ends_of_the_type(columns, pad):
    """Every bf16 value there is, runs of one size each, FP32's smallest and largest, NaN and infinities."""
    bits = torch.arange(1 << 16, device="cuda", dtype=torch.int32).to(torch.int16)
    x = torch.zeros(512, columns + pad, dtype=BF16, device="cuda")[:, :columns]
    x[:, :128] = bits.view(BF16).view(512, 128)
    codes, scales = ops.pack8(x)
    want = R.pack(x)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
    g = gen(1)
    y = torch.zeros(512, columns + pad, device="cuda")[:, :columns]
    y.copy_(torch.exp2(torch.randint(-149, 128, (512, 1), device="cuda", generator=g).double() + torch.rand(512, columns, device="cuda", generator=g).double()
                       * torch.randint(-3, 2, (512, columns), device="cuda", generator=g)).float())
    y[0], y[1, 3], y[2, 40], y[3] = 0, INF, NAN, -INF
    y[4] = torch.finfo(F32).max
    y[5] = 2.0 ** -149
    y[6, 5], y[6, 37] = -0.0, 448.0
    codes, scales = ops.pack8(y)
    want = R.pack(y)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
    back, ref = ops.unpack8(codes, scales, columns, dtype=F32), R.unpack(*want, columns)
    assert torch.equal(torch.isnan(back), torch.isnan(ref)) and torch.equal(back.nan_to_num(0), ref.float().nan_to_num(0))
    # the error that is promised: half a step of three bits, or of the smallest one
    fine = torch.isfinite(y.double())
    limit = torch.maximum(y.double().abs() * 2.0 ** -4, torch.exp2(scales.double() - 127 - 10).repeat_interleave(32, 1)[:, :columns])
    assert bool(((back.double() - y.double()).abs() <= limit)[fine].all())


def glu_slack(y, value, factor=1.0):
    """Of value = g (a sigmoid of y) times an exact factor: the exponential's error, y's own (three products of 2^-24), the
    division.  A sigmoid below 2^-126 is 0, and |g| times it is then at most 88 2^-126 (|g| exp(-|g|) falls; gelu's less)."""
    return value.abs() * (2.0 ** -20 + y.abs().nan_to_num(0, 0, 0) * 2.0 ** -21) + 2.0 ** -119 * torch.as_tensor(factor, device=value.device).abs()


def check_glu(gate, up, act, dh, **outs):
    h, codes, scales = ops.glu8_forward(gate, up, act=act)
    parts = [gate] if up is None else [gate, up]
    a, _, y = R.act(gate.double(), act)
    want = a if up is None else a * up.double()
    close(h, want, glu_slack(y, want, 1.0 if up is None else up.double()), "h")
    for i, x in enumerate(parts):
        c, s = R.pack(x)
        assert torch.equal(codes[i], c) and torch.equal(scales[i], s)
    kept = [R.unpack(codes[i], scales[i], gate.shape[1]) for i in range(len(parts))]
    a, slope, y = R.act(kept[0], act)
    u = kept[1] if up is not None else torch.ones_like(a)
    d = dh.double()
    again = torch.empty_like(dh)
    dgate, dup = ops.glu8_backward(dh, codes, scales, act=act, out_h=again, **outs)
    s = torch.sigmoid(y)
    dy = 1.0 if act == "silu" else 1.5957691216 * (1 + 3 * 0.044715 * kept[0] ** 2)
    terms = s + (torch.where(s * torch.sigmoid(-y) == 0, torch.zeros_like(y), kept[0] * dy * s * torch.sigmoid(-y))).abs()
    close(dgate, d * u * slope, glu_slack(2 * y, d * u * terms, d * u * 8), "dgate")   # (its sigmoids come with up to three more factors of gelu's slope)
    close(again, a * u, glu_slack(y, a * u, u), "h of what was kept")
    if up is not None:
        close(dup, d * a, glu_slack(y, d * a, d), "dup")
    else:
        assert dup is None
    return h, codes, scales, dgate, dup, again


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,columns,pad,shift", [(1, 1, 0, 0), (3, 31, 0, 0), (9, 1367, 0, 0), (4, 256, 8, 8), (5, 264, 1, 3), (70, 2048, 0, 0), (2, 8200, 4, 1)])
def test_glu(rows, columns, pad, shift, gated, act, dtype):
    gate = activations(rows, columns, dtype, 1, pad, shift)
    up = activations(rows, columns, dtype, 2, shift, pad) if gated else None
    check_glu(gate, up, act, activations(rows, columns, dtype, 3))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("columns", [48, 72, 515])
def test_glu_halves_of_one_projection(columns, dtype):
    both, grad = activations(6, 2 * columns, dtype, 4), torch.full((6, 2 * columns + 3), 9.0, dtype=dtype, device="cuda")
    gate, up, dh = both[:, :columns], both[:, columns:], activations(6, columns, dtype, 5)
    *_, dgate, dup, _ = check_glu(gate, up, "silu", dh)
    h, codes, scales = ops.glu8_forward(gate, up)
    got = ops.glu8_backward(dh, codes, scales, out_gate=grad[:, :columns], out_up=grad[:, columns:2 * columns])
    assert torch.equal(got[0], dgate) and torch.equal(got[1], dup) and bool((grad[:, 2 * columns:] == 9).all())
    # in place: h over a half, gradients over dh
    assert torch.equal(ops.glu8_forward(gate, up, out=up)[0], h)
    mine = dh.clone()
    assert torch.equal(ops.glu8_backward(mine, codes, scales, out_up=mine)[1], dup) and torch.equal(mine, dup)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_ends_of_the_type(act, dtype):
    big = torch.finfo(dtype).max
    v = [0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 87.0, -87.0, 89.0, -89.0, 130.0, -130.0, 1e10, -1e10, 1e18, -1e18, big, -big, 5.0, -5.0, 63.0, -65.0]
    gate = torch.tensor([v], device="cuda").to(dtype).t().contiguous().repeat(1, 40)
    for up in (None, torch.ones_like(gate)):
        h, codes, scales, dgate, dup, again = check_glu(gate, up, act, torch.full_like(gate, 0.5))
        assert bool(torch.isfinite(h).all()) and bool(torch.isfinite(dgate).all())
    gate[0, :3] = torch.tensor([NAN, INF, -INF])
    h, codes, scales = ops.glu8_forward(gate, act=act)
    dgate, _ = ops.glu8_backward(torch.ones_like(gate), codes, scales, act=act)
    assert bool(torch.isnan(dgate[0, :3]).all()) and bool(torch.isfinite(dgate[0, 3:]).all()) and bool(torch.isnan(h[0, 0]))
    assert bool(torch.isfinite(h[0, 3:]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("columns", [5, 8, 9, 31, 250, 256, 263, 520])
def test_glu_rows_anywhere(columns, dtype):
    """Each tensor's rows begin somewhere else between boundaries; results are those of aligned rows, and nothing beside the rows is written."""
    rows, places = 5, 8 if dtype == BF16 else 4

    def placed(x, at, pad):
        flat = torch.full((rows * (columns + pad) + 16,), 3.0, dtype=dtype, device="cuda")
        view = flat[at:at + rows * (columns + pad)].view(rows, columns + pad)[:, :columns]
        if x is not None:
            view.copy_(x)
        return flat, view

    def untouched(flat, view):
        return int((flat == 3.0).sum()) == flat.numel() - rows * columns + int((view == 3.0).sum())

    gate, up, dh = (activations(rows, columns, dtype, i) for i in range(3))
    wide = [torch.zeros(rows, 2 * columns + 16, dtype=dtype, device="cuda")[:, :columns] for _ in range(3)]   # aligned rows
    for w, x in zip(wide, (gate, up, dh)):
        w.copy_(x)
    h, codes, scales = ops.glu8_forward(wide[0], wide[1], act="gelu")
    dgate, dup = ops.glu8_backward(wide[2], codes, scales, act="gelu")
    again = torch.empty_like(h)
    ops.glu8_backward(wide[2], codes, scales, act="gelu", out_h=again)
    for at in range(places):
        for pad in (0, 1, 3):
            a, b, d = (placed(x, (at * k + k) % places, pad + k) for k, x in ((0, gate), (1, up), (3, dh)))
            outs = [placed(None, (at + 2 * k + 1) % places, pad + 2 * k) for k in range(4)]
            got = ops.glu8_forward(a[1], b[1], act="gelu", out=outs[0][1])
            assert torch.equal(outs[0][1], h) and torch.equal(got[1], codes) and torch.equal(got[2], scales)
            ops.glu8_backward(d[1], codes, scales, act="gelu", out_gate=outs[1][1], out_up=outs[2][1], out_h=outs[3][1])
            assert torch.equal(outs[1][1], dgate) and torch.equal(outs[2][1], dup) and torch.equal(outs[3][1], again)
            assert all(untouched(*o) for o in outs), (at, pad)
            assert torch.equal(ops.unpack8(codes[0], scales[0], columns, dtype=dtype, out=a[1]), ops.unpack8(codes[0], scales[0], columns, dtype=dtype))
            assert untouched(*a)


def test_glu_keeps_nothing_on_request_and_no_rows():
    gate, up = activations(5, 100, BF16, 6), activations(5, 100, BF16, 7)
    h, codes, scales = ops.glu8_forward(gate, up, keep=False)
    assert codes is None and scales is None and torch.equal(h, ops.glu8_forward(gate, up)[0])
    h, codes, scales = ops.glu8_forward(gate[:0], up[:0])
    assert h.shape == (0, 100) and ops.glu8_backward(h, codes, scales)[0].shape == (0, 100)
    assert ops.unpack8(*ops.pack8(gate[:0]), 100).shape == (0, 100)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("gated", [False, True])
def test_glu_autograd(act, gated):
    gate = activations(12, 96, F32, 8).requires_grad_(True)
    up = activations(12, 96, F32, 9).requires_grad_(True) if gated else None
    d = activations(12, 96, F32, 10)
    (ops.glu8(gate, up, act=act) * d).sum().backward()
    h, codes, scales = ops.glu8_forward(gate.detach(), up.detach() if gated else None, act=act)
    dgate, dup = ops.glu8_backward(d, codes, scales, act=act)
    assert torch.equal(gate.grad, dgate) and (up is None or torch.equal(up.grad, dup))
    # of what was kept, in 64 bits
    kept = [R.unpack(codes[i], scales[i], 96).requires_grad_(True) for i in range(1 + gated)]
    plain = torch.nn.functional.silu(kept[0]) if act == "silu" else torch.nn.functional.gelu(kept[0], approximate="tanh")
    want = torch.autograd.grad((plain * (kept[1] if gated else 1.0) * d.double()).sum(), kept)
    assert ((dgate.double() - want[0]).abs() <= 1e-5 * (want[0].abs() + d.abs() * (kept[1].detach().abs() if gated else 1))).all()
    gate.grad = None
    ops.glu8(gate, up.detach() if gated else None, act=act).sum().backward()     # an expanded gradient, a constant up
    assert gate.grad is not None
    (first,) = torch.autograd.grad(ops.glu8(gate, up, act=act).sum(), gate, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        first.sum().backward()


def test_glu_refusals():
    x = activations(4, 64, BF16)
    h, codes, scales = ops.glu8_forward(x, x.clone())
    for call, word in ((lambda: ops.pack8(x.half()), "dtype"), (lambda: ops.pack8(x.t()), "contiguous"), (lambda: ops.pack8(x[0]), "two dimensions"),
                       (lambda: ops.unpack8(codes[0], scales[0], 65), "shape"), (lambda: ops.unpack8(codes[0], scales[0], 64, dtype=torch.half), "dtype"),
                       (lambda: ops.unpack8(codes[0], scales[0], 64, out=x.float()), "dtype"), (lambda: ops.glu8_forward(x, x.float()), "dtype"),
                       (lambda: ops.glu8_forward(x, x[:3]), "shape"), (lambda: ops.glu8_forward(x, act="relu"), "act"),
                       (lambda: ops.glu8_backward(h, codes[0], scales[0]), "shape"), (lambda: ops.glu8_backward(h[:, :32], codes, scales), "shape"),
                       (lambda: ops.glu8_backward(h, codes[:1], scales[:1], out_up=x), "no up"), (lambda: ops.glu8_backward(h, codes.int(), scales), "dtype"),
                       (lambda: ops.glu8_backward(h, codes, scales, out_gate=x[:2]), "shape")):
        with pytest.raises(ValueError, match=word):
            call()
    for call in (lambda: ops.glu8_backward(h, codes, scales, out_gate=x, out_up=x),
                 lambda: ops.glu8_forward(x[:2], out=x[1:3])):
        with pytest.raises(C.Bf16OptError, match="overlap"):
            call()


# ------------------------------------------------------------------ rotary positions

def turned(x, positions, how, inverse=False):
    four = x if x.dim() == 4 else x[None]
    p = positions if positions.dim() == 2 else positions[None].expand(four.shape[:2])
    dim = how.get("rotary_dim") or x.shape[-1]
    more = {k: v for k, v in how.items() if k in ("base", "scaling", "factor", "original_length")}
    y = R.rotary(four, p + how.get("offset", 0), dim, how.get("layout", "half"), inverse, **more)
    return y.view(x.shape) if x.dim() == 4 else y[0]


def rotary_slack(x, how):
    """An angle's rounding, the sine's and the products': 2^-22 of the pair's magnitudes (twice the larger of a head at most) each."""
    scale = R.frequencies(64, scaling=how.get("scaling"), factor=how.get("factor", 1.0))[1]
    return 2.0 ** -21 * 2 * scale * x.double().abs().nan_to_num(0, 0, 0).amax(-1, keepdim=True).expand(x.shape)


def check_rotary(q, k, positions, **how):
    p = positions if positions is not None else torch.arange(q.shape[-3], device="cuda")
    for call, inverse in ((ops.rotary_forward, False), (ops.rotary_backward, True)):
        got = call(q, k, positions, **how)
        for x, y, what in ((q, got[0], "q"), (k, got[1], "k")):
            if x is None:
                assert y is None
                continue
            close(y, turned(x, p, how, inverse), rotary_slack(x, how), (what, inverse))
            n = how.get("rotary_dim") or x.shape[-1]
            assert torch.equal(y[..., n:], x[..., n:])
    return ops.rotary_forward(q, k, positions, **how)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,part", [(2, 2), (6, 4), (16, 16), (64, 32), (80, 20), (80, 80), (96, 96), (128, 64), (128, 128), (256, 256), (300, 10), (7, 6), (1031, 256)])
@pytest.mark.parametrize("tokens,heads,kv", [(1, 1, 1), (5, 3, 1), (67, 8, 2)])
def test_rotary_sizes(tokens, heads, kv, dim, part, layout, dtype):
    g = gen(dim)
    q, k = randn(g, tokens, heads, dim).to(dtype), randn(g, tokens, kv, dim).to(dtype)
    positions = torch.randint(0, 5000, (tokens,), device="cuda", generator=g)
    check_rotary(q, k, positions, layout=layout, rotary_dim=part)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("how", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=16.0, original_length=4096),
                                 dict(base=500000.0, offset=17), dict(offset=-3, layout="interleaved")])
def test_rotary_far_positions(how, dtype):
    """Positions up to 2^28 and below 0, whose angles a product in 32 bits would lose altogether.  (The reference's own angle is off by 2^-53 of 2^28.)"""
    g = gen(2)
    q, k = randn(g, 40, 4, 64).to(dtype), randn(g, 40, 2, 64).to(dtype)
    positions = torch.randint(-(1 << 28), 1 << 28, (40,), device="cuda", generator=g)
    check_rotary(q, k, positions, **how)
    check_rotary(q, k, positions.int(), **how)
    check_rotary(q, k, None, **how)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_strides(layout, dtype):
    g = gen(3)
    how = dict(layout=layout, rotary_dim=32)
    for tokens, heads, kv, dim in ((33, 6, 2, 64), (9, 3, 1, 50)):
        rows = randn(g, tokens, (heads + 2 * kv), dim).to(dtype)
        q, k = rows[:, :heads], rows[:, heads:heads + kv]
        want = check_rotary(q, k, None, **how)
        same = rows.clone()                           # parts of one projection, in place: v stays
        a, b = same[:, :heads], same[:, heads:heads + kv]
        got = ops.rotary_forward(a, b, None, out_q=a, out_k=b, **how)
        assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(same[:, heads + kv:], rows[:, heads + kv:])
        # batch, and heads before tokens
        x, y = randn(g, 2, heads, tokens, dim).to(dtype), randn(g, 2, kv, tokens, dim).to(dtype)
        for positions in (torch.randint(0, 99, (2, tokens), device="cuda", generator=g), torch.arange(5, 5 + tokens, device="cuda")):
            check_rotary(x.transpose(1, 2), y.transpose(1, 2), positions, **how)
        check_rotary(q, None, None, **how)
        check_rotary(rows[:, :1].expand(tokens, heads, dim), None, None, **how)
        # rows that begin between boundaries, an output with room around
        odd = randn(g, tokens * heads * dim + 1).to(dtype)[1:].view(tokens, heads, dim)
        check_rotary(odd, k, None, **how)
        wide = torch.full((tokens, heads, dim + 3), 4.0, dtype=dtype, device="cuda")
        got = ops.rotary_forward(q, None, None, out_q=wide[..., 1:1 + dim], **how)[0]
        assert torch.equal(got, want[0]) and bool((wide[..., 0] == 4).all()) and bool((wide[..., 1 + dim:] == 4).all())


def test_rotary_turns_back_and_nothing():
    g = gen(5)
    q, k = randn(g, 2, 11, 4, 64), randn(g, 2, 11, 4, 64)
    positions = torch.randint(0, 1 << 20, (2, 11), device="cuda", generator=g)
    a, b = ops.rotary_forward(q, k, positions)
    back = ops.rotary_backward(a, b, positions)
    assert (back[0] - q).abs().max() < 4e-6 and (back[1] - k).abs().max() < 4e-6
    assert ops.rotary_forward(q[:, :0], k[:, :0], positions[:, :0])[0].shape == (2, 0, 4, 64)
    assert ops.rotary_forward(q[:0], k[:0])[0].shape == (0, 11, 4, 64)
    none, kk = ops.rotary_forward(q[:, :, :0], k, positions)
    assert none.shape == (2, 11, 0, 64) and torch.equal(kk, b)
    qq, none = ops.rotary_forward(q, k[:, :, :0], positions)
    assert none.shape == (2, 11, 0, 64) and torch.equal(qq, a)
    q[0, 0, 0, 40] = NAN                             # NaN and infinities where nothing turns pass; where it does they stay in their pair
    got = ops.rotary_forward(q, None, positions, rotary_dim=32)[0]
    assert int(torch.isnan(got).sum()) == 1
    q[0, 0, 0, 3] = INF
    got = ops.rotary_forward(q, None, positions, rotary_dim=32)[0]
    assert int((~torch.isfinite(got)).sum()) <= 3


def test_rotary_autograd():
    g = gen(6)
    q, k = (randn(g, 9, h, 32).requires_grad_(True) for h in (4, 2))
    positions = torch.randint(0, 1000, (9,), device="cuda", generator=g)
    how = dict(layout="interleaved", rotary_dim=16, scaling="yarn", factor=4.0)
    a, b = ops.rotary(q, k, positions, **how)
    da, db = randn(g, 9, 4, 32), randn(g, 9, 2, 32)
    ((a * da).sum() + (b * db).sum()).backward()
    close(q.grad, turned(da, positions, how, True), rotary_slack(da, how), "dq")
    close(k.grad, turned(db, positions, how, True), rotary_slack(db, how), "dk")
    e = randn(g, 9, 4, 32)                           # linear: a difference is the derivative
    along = float((ops.rotary_forward(q.detach() + e, None, positions, **how)[0].double() * da).sum() - (a.detach().double() * da).sum())
    assert abs(along - float((q.grad.double() * e).sum())) < 1e-3
    q.grad = k.grad = None
    ops.rotary(q, k, positions, **how)[1].sum().backward()      # k alone, an expanded gradient
    assert q.grad is None or not q.grad.any()
    close(k.grad, turned(torch.ones_like(db), positions, how, True), rotary_slack(torch.ones_like(db), how), "dk alone")
    q.grad = None
    ops.rotary(q, None, positions, **how)[0].sum().backward()
    assert q.grad is not None
    (first,) = torch.autograd.grad(ops.rotary(q, k, positions, **how)[0].square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        first.sum().backward()


def test_rotary_refusals():
    q, k = torch.zeros(4, 3, 32, device="cuda"), torch.zeros(4, 1, 32, device="cuda")
    p = torch.arange(4, device="cuda")
    for call, word in ((lambda: ops.rotary_forward(q[0]), r"\[tokens"), (lambda: ops.rotary_forward(q.half()), "must be"), (lambda: ops.rotary_forward(q.transpose(1, 2)), "contiguous"),
                       (lambda: ops.rotary_forward(q, k.bfloat16()), "must be"), (lambda: ops.rotary_forward(q, k[:3]), "does not go"), (lambda: ops.rotary_forward(q, k[..., :16]), "does not go"),
                       (lambda: ops.rotary_forward(q, k, p[:3]), "shape"), (lambda: ops.rotary_forward(q, k, p.float()), "dtype"), (lambda: ops.rotary_forward(q, layout="other"), "layout"),
                       (lambda: ops.rotary_forward(q, rotary_dim=31), "rotary_dim"), (lambda: ops.rotary_forward(q, scaling="other"), "scaling"),
                       (lambda: ops.rotary_forward(q, out_k=k), "no k"), (lambda: ops.rotary_forward(q, out_q=k), "shape"), (lambda: ops.rotary_forward(q, out_q=q.clone().requires_grad_(True)), "leaf")):
        with pytest.raises(ValueError, match=word):
            call()
    for call, word in ((lambda: ops.rotary_forward(q, rotary_dim=34), "rotary_dim"), (lambda: ops.rotary_forward(q, out_q=q[:, :1].expand(4, 3, 32)), "twice"),
                       (lambda: ops.rotary_forward(q, q.clone(), out_q=q, out_k=q), "overlap")):
        with pytest.raises(C.Bf16OptError, match=word):
            call()


# ------------------------------------------------------------------ all of them

def every_call(seed=0):
    """One call of each forward and backward, as closures over their own inputs."""
    z, labels, adv, how = policy_case(60, 5000, BF16, 50 + seed, weights=True)
    ends = torch.tensor([0, 12, 20, 41, 55], device="cuda")
    gate, up, dh = (activations(50, 700, BF16, 60 + seed + i) for i in range(3))
    g = gen(70 + seed)
    q, k = randn(g, 50, 6, 64).bfloat16(), randn(g, 50, 2, 64).bfloat16()
    positions = torch.randint(0, 9999, (50,), device="cuda", generator=g)

    def policy():
        loss, logp, saved = ops.policy_forward(z, labels, adv, **how)
        return loss, logp, ops.token_logp_backward(z, labels, saved), *ops.policy_loss_grad(z, labels, adv, **how)

    def prefer():
        loss, logp, saved = ops.preference_forward(z, labels, ends)
        return loss, logp, saved, ops.token_logp_backward(z, labels, saved)

    def glu():
        h, codes, scales = ops.glu8_forward(gate, up)
        return h, codes, scales, *ops.glu8_backward(dh, codes, scales), ops.unpack8(*ops.pack8(gate), 700)

    return [policy, prefer, glu, lambda: ops.rotary_forward(q, k, positions), lambda: ops.rotary_backward(q, k, positions, layout="interleaved"),
            lambda: ops.token_logp_forward(z, labels)]


def bits(x):
    return x.view(torch.uint8) if x.dtype != torch.uint8 else x


def test_calls_repeat_on_other_streams_and_side_by_side():
    calls, others = every_call(), every_call(7)
    want, more = [c() for c in calls], [c() for c in others]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [[], []]
        for c, o in zip(calls, others):
            for s, f, into in ((streams[0], c, got[0]), (streams[1], o, got[1])):
                with torch.cuda.stream(s):
                    into.append(f())
        torch.cuda.synchronize()
        for a, b in ((want, got[0]), (more, got[1])):
            for x, y in zip(a, b):
                assert all(torch.equal(bits(u), bits(v)) for u, v in zip(x, y))


def test_stream_argument():
    z, labels, _ = rows_case(20, 3000, BF16, 80)
    side = torch.cuda.Stream()
    want = ops.token_logp_forward(z, labels)[0]
    torch.cuda.synchronize()
    got = ops.token_logp_forward(z, labels, stream=side)[0]
    turned = ops.rotary_forward(z.view(20, 30, 100), stream=side)[0]
    h = ops.glu8_forward(z, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(turned, ops.rotary_forward(z.view(20, 30, 100))[0]) and torch.equal(h, ops.glu8_forward(z)[0])


def test_captured_graphs_share_no_state():
    """Two graphs of the same calls, replayed in turn while eager calls run between them, with new inputs in place."""
    z, labels, adv, how = policy_case(60, 5000, BF16, 90)
    gate, dh = activations(50, 700, BF16, 91), activations(50, 700, BF16, 92)
    q = randn(gen(93), 50, 6, 64).bfloat16()

    def step():
        loss, logp, saved = ops.policy_forward(z, labels, adv, **how)
        h, codes, scales = ops.glu8_forward(gate)
        return [loss, logp, ops.token_logp_backward(z, labels, saved), *ops.policy_loss_grad(z, labels, adv, **how)[:3], h,
                ops.glu8_backward(dh, codes, scales)[0], ops.rotary_forward(q)[0],
                *ops.preference_forward(z, labels, torch_ends)[:2]]

    torch_ends = torch.tensor([0, 12, 20, 41, 55], device="cuda")
    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        step()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step())
        graphs.append(graph)
    for i in range(4):
        z.copy_(z.flip(0)), gate.copy_(gate.flip(1)), q.copy_(q.flip(0))
        want = step()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs[i % 2]))


def test_a_captured_backward_beside_an_eager_graph():
    """Forward and backward captured from leaves of their own while an eager graph of other leaves lives."""
    z, labels, adv, how = policy_case(40, 900, F32, 95)
    q = randn(gen(96), 40, 9, 100)
    eager = z.clone().requires_grad_(True)
    alive = ops.policy_loss(eager, labels, adv, **how)[0].sum()
    leaf, x = z.clone().requires_grad_(True), q.clone().requires_grad_(True)

    def step():
        loss = ops.policy_loss(leaf, labels, adv, **how)[0].sum()
        turned = ops.rotary(x)[0]
        return torch.autograd.grad(loss + ops.glu8(turned.reshape(40, 900)).sum(), [leaf, x])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    alive.backward()
    assert torch.equal(eager.grad, want[0])


def test_offsets_beyond_32_bits():
    """Rows more than 2^32 bytes (and 2^31 elements) apart."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    far = (1 << 32) + 24
    flat = torch.empty(far + 4096, dtype=BF16, device="cuda")
    z = flat.as_strided((2, 2053), (far, 1))
    small, labels, g = rows_case(2, 2053, BF16, 97)
    z.copy_(small)
    logp, saved = ops.token_logp_forward(z, labels)
    assert torch.equal(logp, ops.token_logp_forward(small, labels)[0])
    assert torch.equal(ops.token_logp_backward(z, labels, saved), ops.token_logp_backward(small, labels, saved))
    adv = torch.ones(2, device="cuda")
    want = ops.policy_loss_grad(small, labels, adv)
    got = ops.policy_loss_grad(z, labels, adv, out=z)
    assert torch.equal(got[0], want[0]) and torch.equal(z, want[2])
    z.copy_(small)
    h, codes, scales = ops.glu8_forward(z)
    want = ops.glu8_forward(small)
    assert torch.equal(h, want[0]) and torch.equal(codes, want[1])
    ops.glu8_backward(small, codes, scales, out_gate=z)
    assert torch.equal(z, ops.glu8_backward(small, codes, scales)[0])
    q = flat.as_strided((2, 4, 64), (far, 64, 1))
    x = randn(g, 2, 4, 64).bfloat16()
    q.copy_(x)
    ops.rotary_forward(q, out_q=q)
    assert torch.equal(q, ops.rotary_forward(x)[0])
