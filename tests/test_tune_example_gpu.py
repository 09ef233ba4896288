"""The fine-tuning operators and the optimizer together, as a user runs them: examples/tune_policy.py."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

import tuning_reference as R  # noqa: E402

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("tune_policy", os.path.join(ROOT, "examples", "tune_policy.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs_and_repeats():
    m = example()
    rewards, losses = m.tune(steps=3, seed=3)
    assert len(rewards) == len(losses) == 3 and all(math.isfinite(v) for v in rewards + losses) and all(0 <= r <= 1 for r in rewards)
    assert m.tune(steps=3, seed=3) == (rewards, losses)


class Gated(torch.autograd.Function):
    """silu(gate) up; its gradients those at gate and up as 8 bits keep them."""
    @staticmethod
    def forward(ctx, gate, up):
        ctx.save_for_backward(*(R.unpack(*R.pack(v.bfloat16()), v.shape[1]) for v in (gate, up)))
        return torch.nn.functional.silu(gate) * up

    @staticmethod
    def backward(ctx, dh):
        gate, up = ctx.saved_tensors
        a, slope, _ = R.act(gate, "silu")
        return dh * up * slope, dh * a


class Down(torch.autograd.Function):
    """h w, w's gradient at the h that is computed again from what was kept."""
    @staticmethod
    def forward(ctx, h, w, gate, up):
        gate, up = (R.unpack(*R.pack(v.detach().bfloat16()), v.shape[1]) for v in (gate, up))
        ctx.save_for_backward(torch.nn.functional.silu(gate) * up, w)
        return h @ w

    @staticmethod
    def backward(ctx, dy):
        h, w = ctx.saved_tensors
        return dy @ w.t(), h.t() @ dy, None, None


def plain_logits(m, model, tokens):
    """The decoder in 64 bits from formulas."""
    n, t = tokens.shape
    w = {k: p.detach().double().requires_grad_(True) for k, p in model.named_parameters()}

    def norm(v, weight):
        return v / (v.square().mean(1, keepdim=True) + 1e-5).sqrt() * weight

    def turned(v):
        f, scale = R.frequencies(m.ROTARY["rotary_dim"], scaling="yarn", factor=m.ROTARY["factor"], original_length=m.ROTARY["original_length"])
        angle = torch.arange(t, device="cuda", dtype=torch.float64)[:, None] * torch.tensor(f, device="cuda", dtype=torch.float64)
        c, s, half = scale * angle.cos()[:, None], scale * angle.sin()[:, None], len(f)
        a, b = v[..., :half], v[..., half:2 * half]
        return torch.cat([a * c - b * s, b * c + a * s, v[..., 2 * half:]], -1)

    x = h = w["embedding"][tokens.reshape(-1)]
    for b in range(m.BLOCKS):
        qkv = (h @ w[f"qkv.{b}"]).view(n, t, m.HEADS + 2 * m.KV, m.DIM)
        q, k, v = turned(qkv[:, :, :m.HEADS]), turned(qkv[:, :, m.HEADS:m.HEADS + m.KV]), qkv[:, :, m.HEADS + m.KV:]
        k, v = (y.repeat_interleave(m.HEADS // m.KV, 2) for y in (k, v))
        z = torch.einsum("nqhd,nkhd->nhqk", q, k) / math.sqrt(m.DIM)
        z = z.masked_fill(torch.ones(t, t, device="cuda", dtype=torch.bool).triu(1), -math.inf)
        y = torch.einsum("nhqk,nkhd->nqhd", torch.softmax(z, -1), v).reshape(n * t, -1) @ w[f"out.{b}"]
        x = x + norm(y, w[f"post.{2 * b}"])
        h = norm(x, w[f"pre.{2 * b}"])
        both = h @ w[f"w_in.{b}"]
        gate, up = both[:, :m.WIDE], both[:, m.WIDE:]
        x = x + norm(Down.apply(Gated.apply(gate, up), w[f"w_out.{b}"], gate, up), w[f"post.{2 * b + 1}"])
        h = norm(x, w[f"pre.{2 * b + 1}"])
    return h @ w["embedding"].t(), w


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_a_step_gradient_against_plain_autograd(which):
    """One step's gradients through the operators against the same model in 64 bits: bf16 matrix products and roundings on one
    side, some twenty of 2^-9 on an activation's way and as many on a gradient's, and now and then another of 8 bits' neighbours
    where an activation lies between them (2^-4 apart; a bf16 error of 2^-8 moves one in sixteen).  8 % of the whole is ample."""
    m = example()
    gen = torch.Generator(device="cuda").manual_seed(1)
    model = m.Decoder(gen)
    tokens, labels = m.answers(model, gen)
    logits, w = plain_logits(m, model, tokens)
    live = labels >= 0
    logp = torch.log_softmax(logits, 1).gather(1, labels.clamp(min=0)[:, None]).squeeze(1)
    if which == "policy":
        advantage = torch.randn(m.ANSWERS, device="cuda", generator=gen)
        noise = 0.05 * torch.randn(len(labels), device="cuda", generator=gen)      # no token near a clip
        with torch.no_grad():
            mine = m.ops.token_logp_forward(model(tokens), labels)[0]
        m.policy_step_loss(model, tokens, labels, advantage, mine - noise, mine + 4 * noise).backward()
        now = logp.detach()
        ratio = torch.exp(logp - (now - noise))
        d = now + 4 * noise - logp
        loss = ((-ratio * advantage.double().repeat_interleave(m.LENGTH) + 0.02 * (torch.exp(d) - 1 - d)) * live).sum() / live.sum()
    else:
        ref = torch.randn(m.ANSWERS, device="cuda", generator=gen)
        with torch.no_grad():
            ref = ref + m.ops.token_logp_forward(model(tokens), labels)[0].view(m.ANSWERS, -1).sum(1)
        m.preference_step_loss(model, tokens, labels, ref).backward()
        total = (logp * live).view(m.ANSWERS, -1).sum(1) - ref
        half = m.ANSWERS // 2
        loss = torch.nn.functional.softplus(-0.2 * (total[:half] - total[half:])).mean()
    want = dict(zip(w, torch.autograd.grad(loss, list(w.values()))))
    off = sum((p.grad.double() - want[n]).square().sum() for n, p in model.named_parameters())
    whole = sum(g.square().sum() for g in want.values())
    assert float((off / whole).sqrt()) < 0.08
