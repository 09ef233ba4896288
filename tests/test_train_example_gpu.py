"""The training operators and the optimizer together, as a user runs them: examples/distill_student.py."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no CUDA device")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("distill_student", os.path.join(ROOT, "examples", "distill_student.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_student_learns_and_repeats():
    m = example()
    losses, counts = m.train(steps=30, seed=3)
    assert all(v == v and v < float("inf") for v in losses)
    assert sum(losses[-5:]) < 0.8 * sum(losses[:5]), losses
    for n in counts:                                   # every token went to CHOSEN experts
        assert n.shape == (m.SEQUENCES, m.EXPERTS) and bool((n.sum(1) == m.TOKENS * m.CHOSEN).all())


def test_a_step_gradient_against_plain_autograd(monkeypatch):
    """One micro-batch's gradients through the operators against the same model with
    plain formulas in 32 bits, the experts' choice taken over: bf16 matrix products and
    roundings on both sides, about ten of 2^-9 on a gradient's way, so 4 % of the whole is ample."""
    m = example()
    choices, balance = [], m.ops.balance

    def recorded(*args, **more):
        out = balance(*args, **more)
        choices.append(out[0].long())
        return out

    monkeypatch.setattr(m.ops, "balance", recorded)
    gen = torch.Generator(device="cuda").manual_seed(1)
    student = m.Student(gen)
    table = 4 * torch.randn(64, m.VOCAB, device="cuda", generator=gen)
    tokens, ids, top, labels = m.teacher_batch(table, gen)
    logits, aux, _ = student(tokens)
    (m.ops.distill_loss(logits, ids, top, temperature=m.TEMPERATURE, ce_weight=0.2, labels=labels).mean() + aux).backward()
    got = {n: p.grad.double().clone() for n, p in student.named_parameters()}
    student.zero_grad()

    def norm(v, w):
        return v / (v.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.float()

    x = torch.nn.functional.embedding(tokens, student.embedding).float()
    h, aux = x, 0.0
    for b in range(m.BLOCKS):
        z = (h.bfloat16() @ student.routers[b]).float()
        p = torch.softmax(z, 1)
        choice = choices[b]
        w = p.gather(1, choice)
        f = torch.zeros_like(p).scatter_(1, choice, 1.0).reshape(m.SEQUENCES, m.TOKENS, -1).mean(1) * m.EXPERTS / m.CHOSEN
        aux = aux + (1e-2 * (f * p.reshape(m.SEQUENCES, m.TOKENS, -1).mean(1)).sum(1)).mean() + 1e-4 * torch.logsumexp(z, 1).square().mean()
        every = torch.einsum("ehw,nh->new", student.up[b], h.bfloat16())
        every = torch.einsum("ewh,new->neh", student.down[b], torch.nn.functional.gelu(every))
        chosen = every.gather(1, choice[:, :, None].expand(-1, -1, m.HIDDEN))
        y = (chosen * (w / w.sum(1, keepdim=True))[:, :, None].bfloat16()).sum(1).float()
        x = x.bfloat16().float() + student.gates[b].float() * norm(y, student.post[b])
        h = norm(x, student.pre[b])
    z = (h.bfloat16() @ student.embedding.t()).float()
    q = torch.log_softmax(z / m.TEMPERATURE, 1).gather(1, ids.long())
    t = torch.log_softmax(top.float() / m.TEMPERATURE, 1)
    rows = m.TEMPERATURE ** 2 * (t.exp() * (t - q)).sum(1) + 0.2 * torch.nn.functional.cross_entropy(z, labels, reduction="none")
    (rows.mean() + aux).backward()
    for n, p in student.named_parameters():
        off = float((got[n] - p.grad.double()).norm() / p.grad.double().norm())
        assert off < 0.04, (n, off)
