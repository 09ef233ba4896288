"""The fine-tuning operators on the GPU where they are easily wrong: tokens that the vocabulary masks, sums of many
small log-probabilities, sigmoids at the end of FP32, positions beyond 2^32, and calls so large that a kernel's threads walk on.

Tolerances as in test_tuning_ops_gpu.py."""
import decimal
import math

import pytest

torch = pytest.importorskip("torch")

import tuning_reference as R  # noqa: E402
from mixed_precision_optimizer_bf16_gb300 import train_ops as ops  # noqa: E402
from test_tuning_ops_gpu import (BF16, F32, F64, INF, NAN, activations, check_glu, check_logp, close, gen, gradient_slack,  # noqa: E402
                                 randn, rotary_slack, rows_case, sum_error, turned)

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]


# ------------------------------------------------------------------ token losses

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,vocab", [(6, 600), (6, 1500), (700, 3001), (6, 12000), (700, 20011), (6, 70001)])
def test_policy_of_its_own_tokens_is_a_constant_ratio(rows, vocab, dtype):
    """Without a sampler's log-probabilities the ratio is 1, whatever the log-probability: a masked label's and an empty row's loss
    and gradient are finite; a NaN or +inf in the row is NaN."""
    z, labels, g = rows_case(rows, vocab, dtype, vocab)
    z[0, vocab // 2:], labels[0] = -INF, vocab - 1
    z[1] = -INF
    z[2, 1], z[3, vocab - 1] = NAN, INF
    labels[4] = -100
    adv = randn(g, rows)
    w, up = torch.rand(rows, device="cuda", generator=g) + 0.2, torch.rand(rows, device="cuda", generator=g) + 0.1
    v, p, one = R.logp(z, labels.clamp(min=0))
    live = R.counts(labels, vocab, w)
    ratio = torch.where(torch.isnan(v), v, torch.ones_like(v))
    slope = torch.where(live, -ratio * adv.double() * w.double(), torch.zeros_like(v))
    dz, scale = R.gradient(live, slope * up.double(), p, one, 1.0)
    slack = gradient_slack(scale.nan_to_num(0, 0, 0), vocab)
    loss, logp, saved = ops.policy_forward(z, labels, adv, row_weight=w)
    assert logp[0] == -INF and logp[1] == -INF and logp[4] == 0
    close(loss, slope, 0.0, "loss")                   # (w times A is rounded once)
    close(saved[:, 2], slope, 0.0, "slope")
    close(ops.token_logp_backward(z, labels, saved, up), dz, slack, "dlogits of the backward call")
    both = ops.policy_loss_grad(z, labels, adv, up, row_weight=w)
    close(both[0], slope, 0.0, "loss of the single pass")
    close(both[2], dz, slack, "dlogits of the single pass")
    assert bool(torch.isfinite(both[2][:2]).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("vocab", [7, 3000, 33000])
@pytest.mark.parametrize("temperature", [4.0, 65536.0])
def test_logp_of_differences_that_no_number_holds(temperature, vocab, dtype):
    """The type's lowest value beside its largest: their difference is infinite in FP32, divided by the temperature it is not."""
    z, labels, g = rows_case(4, vocab, dtype, vocab)
    big = torch.finfo(dtype).max
    z[0, 1], z[0, 0], labels[0] = big, -big, 0
    z[1], z[1, vocab - 1], labels[1] = -big, big, 2
    z[2, 1], z[2, 0], labels[2] = big, -INF, 0
    check_logp(z, labels, temperature)
    loss = ops.policy_loss_grad(z, labels, torch.ones(4, device="cuda"), temperature=temperature)
    assert torch.equal(loss[1], ops.token_logp_forward(z, labels, temperature=temperature)[0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lengths", [(2048, 1500), (65536, 60001), (3, 40000)])
def test_preference_sums_of_small_log_probabilities(lengths, dtype):
    """Tokens that the model is sure of: the label has the largest logit and the sum of exponentials lies in [1, 1.29], so a log-probability is
    one FP32 number, -log of it, and the sequence's sum is the 64-bit sum of those numbers within 2^-40 of it.  (Of 65536 such, a plain FP32
    sum is 8e-4 off.)  The loss h^2 beside 1 shows that: ref_logp is the sum rounded to FP32."""
    rows = sum(lengths)
    g = gen(rows)
    z = (-3.2 - 1.8 * torch.rand(rows, 8, device="cuda", generator=g)).to(dtype)
    labels = torch.randint(0, 8, (rows,), device="cuda", generator=g)
    z.scatter_(1, labels[:, None], 0.0)
    each, saved = ops.token_logp_forward(z, labels)
    ends = torch.tensor([0, *lengths], device="cuda").cumsum(0)
    total = torch.stack([x.double().sum() for x in each.split(list(lengths))])
    ref = total.float()
    loss, logp, kept = ops.preference_forward(z, labels, ends, ref_logp=ref, kind="ipo", beta=0.5)
    assert torch.equal(kept[:, :2], saved[:, :2])
    close(logp, total, 2.0 ** -40 * total.abs(), "logp")
    off = total - ref.double()
    d = off[0] - off[1] - 1.0
    close(loss, (d * d)[None], 2 * d.abs() * 2.0 ** -40 * total.abs().sum(), "loss")


@pytest.mark.parametrize("pairs", [257, 2100])
@pytest.mark.parametrize("mean", [False, True])
def test_preference_of_many_pairs(pairs, mean):
    """More pairs than a CTA has threads, sequences of no or a few tokens, some offsets that descend."""
    g = gen(pairs)
    lengths = torch.randint(0, 7, (2 * pairs,), device="cuda", generator=g)
    ends = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), lengths.cumsum(0)])
    rows, vocab = int(ends[-1]) + 5, 50
    z, labels, g = rows_case(rows, vocab, F32, 3, spread=1.0)
    labels[torch.rand(rows, device="cuda", generator=g) < 0.3] = -100
    down = torch.randint(1, 2 * pairs, (pairs // 8,), device="cuda", generator=g)
    ends[down] -= 4
    how = dict(beta=0.3, label_smoothing=0.1, margin=0.2, length_normalise=mean)
    dloss = torch.rand(pairs, device="cuda", generator=g) + 0.2
    ref = randn(g, 2 * pairs) - 10.0
    loss_r, logp_r, dz_r, scale = R.preference(z, labels, ends, ref, dloss=dloss, **how)
    loss, logp, saved = ops.preference_forward(z, labels, ends.int(), ref_logp=ref, **how)
    most = int(ends.cummax(0).values.clamp(max=int(ends[-1])).diff().max())
    off = most * sum_error(vocab)                     # of a sequence's sum
    size = (logp_r.abs() + ref.abs().double()).view(2, pairs).sum(0)
    close(logp, logp_r, off, "logp")
    close(loss, loss_r, 0.3 * 2 * off + 2.0 ** -21 * (1 + 0.3 * size), "loss")
    slope_off = 0.3 * 0.3 * 2 * off + 0.3 * 2.0 ** -20 + 0.3 * 0.3 * float(size.max()) * 2.0 ** -23
    close(ops.token_logp_backward(z, labels, saved, dloss), dz_r, gradient_slack(scale, vocab) + 1.2 * slope_off * 2 * (scale > 0), "dlogits")


# ------------------------------------------------------------------ 8 bits

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act,low,high", [("silu", -88.7, -80.0), ("gelu", -10.05, -9.5)])
def test_glu_sigmoids_below_the_smallest_normal_number(act, low, high, dtype):
    """Down to 2^-128 a sigmoid counts: times its input it is a normal number."""
    gate = torch.linspace(low, high, 40 * 33, device="cuda").view(40, 33).to(dtype)
    gate = gate.clamp(min=low) if dtype == F32 else torch.where(gate.double() < low, torch.full_like(gate, high), gate)
    gate[0, 0] = -88.0 if act == "silu" else -10.0
    up = 1.0 + torch.rand(40, 33, device="cuda", generator=gen(1)).to(dtype)
    dh = torch.ones_like(gate)

    def slack(y, value, sigmoids):                    # the exponential's and its argument's errors, and a subnormal sigmoid's rounding
        return value.abs() * (2.0 ** -20 + y.abs() * 2.0 ** -21) + sigmoids.abs() * 2.0 ** -148

    a, _, y = R.act(gate.double(), act)
    want = a * up.double()
    h, codes, scales = ops.glu8_forward(gate, up, act=act)
    assert bool((want.abs() > 2.0 ** -126).all())
    got = h.double()
    u = 2.0 ** -8 if dtype == BF16 else 2.0 ** -23
    assert bool(((got - want).abs() <= u * want.abs() + slack(y, want, gate.double() * up.double())).all()), float(((got - want) / want).abs().max())
    g, v = (R.unpack(codes[i], scales[i], 33) for i in range(2))
    fine = torch.sigmoid(R.act(g, act)[2]) > 2.0 ** -127.9
    a, slope, y = R.act(g, act)
    dgate, dup = (x.double() for x in ops.glu8_backward(dh, codes, scales, act=act))
    steep = (g * (1 if act == "silu" else 1.6 * (1 + 0.135 * g * g))).abs() + 1
    for got, want, terms in ((dgate, v * slope, v * steep), (dup, a, g)):
        assert bool(((got - want).abs() <= u * want.abs() + slack(2 * y, want, terms))[fine].all())
    assert bool(fine.any()) and bool(((torch.sigmoid(y) < 2.0 ** -126) & fine).any() or act == "gelu")


LARGE = [(50003, 40, 0, 0), (3001, 2056, 8, 0), (1501, 8200, 0, 0), (9001, 45, 3, 1), (3001, 2053, 0, 0), (1501, 8200, 3, 1)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,columns,pad,shift", LARGE)
def test_glu_more_rows_than_are_resident(rows, columns, pad, shift, gated, dtype):
    """Threads that walk down several rows, the next ones on their way, with a remainder; in place too; twice the same bits."""
    act = "gelu" if pad else "silu"
    gate = activations(rows, columns, dtype, 1, pad, shift)
    up = activations(rows, columns, dtype, 2, pad, shift) if gated else None
    dh = activations(rows, columns, dtype, 3, pad, shift)
    h, codes, scales, dgate, dup, again = check_glu(gate, up, act, dh)
    for _ in range(2):
        got = ops.glu8_backward(dh, codes, scales, act=act)
        assert torch.equal(got[0], dgate) and (not gated or torch.equal(got[1], dup))
    for out in ("out_gate", "out_h", *(["out_up"] if gated else [])):
        mine = activations(rows, columns, dtype, 3, pad, shift)
        got = ops.glu8_backward(mine, codes, scales, act=act, **{out: mine})
        assert torch.equal(mine, {"out_gate": dgate, "out_up": dup, "out_h": again}[out])
        assert out == "out_gate" or torch.equal(got[0], dgate)
    for k, x in enumerate([gate, up] if gated else [gate]):
        mine = activations(rows, columns, dtype, 1 + k, pad, shift)
        got = ops.glu8_forward(*([mine] if not gated else [mine, up] if k == 0 else [gate, mine]), act=act, out=mine)
        assert torch.equal(mine, h) and torch.equal(got[1], codes) and torch.equal(got[2], scales)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,columns,pad,shift", LARGE)
def test_pack_more_rows_than_are_resident(rows, columns, pad, shift, dtype):
    x = activations(rows, columns, dtype, 5, pad, shift)
    codes, scales = ops.pack8(x)
    want = R.pack(x)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
    for t in (BF16, F32):
        out = torch.full((rows, columns + pad), 7.0, dtype=t, device="cuda")
        ops.unpack8(codes, scales, columns, dtype=t, out=out[:, :columns])
        assert torch.equal(out[:, :columns], R.unpack(*want, columns).to(t)) and bool((out[:, columns:] == 7).all())


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tokens,heads,kv,dim,part", [(40009, 1, 1, 128, 128), (20011, 8, 2, 128, 64), (1503, 112, 16, 128, 128), (9001, 3, 1, 50, 20), (30011, 2, 5, 31, 30)])
def test_rotary_more_tokens_than_are_resident(tokens, heads, kv, dim, part, layout, dtype):
    """CTAs that walk from one group of tokens to the next, from q's to k's, with tables and positions of their own each time; in place too."""
    g = gen(tokens)
    rows = randn(g, tokens, heads + 2 * kv, dim).to(dtype)
    q, k = rows[:, :heads], rows[:, heads:heads + kv]
    positions = torch.randint(0, 100000, (tokens,), device="cuda", generator=g)
    how = dict(layout=layout, rotary_dim=part)
    for call, inverse in ((ops.rotary_forward, False), (ops.rotary_backward, True)):
        got = call(q, k, positions, **how)
        for x, y in zip((q, k), got):
            close(y, turned(x, positions, how, inverse), rotary_slack(x, how), (layout, inverse))
            assert torch.equal(y[..., part:], x[..., part:])
        same = rows.clone()
        call(same[:, :heads], same[:, heads:heads + kv], positions, out_q=same[:, :heads], out_k=same[:, heads:heads + kv], **how)
        assert torch.equal(same[:, :heads], got[0]) and torch.equal(same[:, heads:heads + kv], got[1]) and torch.equal(same[:, heads + kv:], rows[:, heads + kv:])
        one = rows.clone()[:, heads:heads + kv]        # k by itself, in place of q
        assert torch.equal(call(one, None, positions, **how)[0], got[1])


TURN = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194988918461563281257")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("far", [31, 36, 40])
def test_rotary_positions_beyond_32_bits(far, layout):
    """The angle is the position times the frequency (a number of 64 bits), whose whole turns are exact: against decimal arithmetic.  A frequency in
    2^-64 turns is off by half a unit, which a position multiplies."""
    g = gen(far)
    tokens, heads, dim = 24, 3, 64
    q = randn(g, tokens, heads, dim)
    positions = torch.randint(-(1 << far), 1 << far, (tokens,), device="cuda", generator=g)
    f = R.frequencies(dim)[0]
    with decimal.localcontext() as ctx:
        ctx.prec = 90
        left = [[float((decimal.Decimal(p) * decimal.Decimal(v) / TURN) % 1) for v in f] for p in positions.tolist()]
    angle = 2 * math.pi * torch.tensor(left, dtype=F64, device="cuda")
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    first, second = (slice(0, 32), slice(32, 64)) if layout == "half" else (slice(0, 64, 2), slice(1, 64, 2))
    a, b = q.double()[..., first], q.double()[..., second]
    want = torch.empty(tokens, heads, dim, dtype=F64, device="cuda")
    want[..., first], want[..., second] = a * c - b * s, b * c + a * s
    slack = rotary_slack(q, {}) + 2.0 ** (far - 65) * 2 * math.pi * 1.5 * q.double().abs().amax(-1, keepdim=True)
    close(ops.rotary_forward(q, None, positions, layout=layout)[0], want, slack, "q")
    close(ops.rotary_forward(q, None, positions - (1 << 35), layout=layout, offset=1 << 35)[0], want, slack, "q by an offset")
