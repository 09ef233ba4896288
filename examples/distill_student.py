"""A small mixture-of-experts student learns from a teacher's stored top logits.

Everything that the library adds to a training step, together: each block's
router chooses and balances its experts (train_ops.balance), the block's output joins
the residual stream through its norms and gate (train_ops.norm_gate), the head
learns from the teacher's top logits and the labels (train_ops.distill_loss), and the bf16
gradients that autograd leaves go into the optimizer's FP32 accumulator, which
clips them and applies AdamW (optimizer.BF16Optimizer).

    python examples/distill_student.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixed_precision_optimizer_bf16_gb300 import train_ops as ops  # noqa: E402
from mixed_precision_optimizer_bf16_gb300.optimizer import BF16Optimizer  # noqa: E402

VOCAB, HIDDEN, WIDE, EXPERTS, CHOSEN, BLOCKS, KEPT = 2053, 128, 256, 8, 2, 2, 16
TEMPERATURE, GAS, SEQUENCES, TOKENS = 2.0, 2, 4, 64


class Student(torch.nn.Module):
    def __init__(self, gen):
        super().__init__()

        def weight(*shape, scale):
            return torch.nn.Parameter((scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16())

        def vector(value):
            return torch.nn.Parameter(torch.full((HIDDEN,), value, device="cuda", dtype=torch.bfloat16))

        self.embedding = weight(VOCAB, HIDDEN, scale=0.5)
        self.routers = torch.nn.ParameterList([weight(HIDDEN, EXPERTS, scale=HIDDEN ** -0.5) for _ in range(BLOCKS)])
        self.up = torch.nn.ParameterList([weight(EXPERTS, HIDDEN, WIDE, scale=HIDDEN ** -0.5) for _ in range(BLOCKS)])
        self.down = torch.nn.ParameterList([weight(EXPERTS, WIDE, HIDDEN, scale=WIDE ** -0.5) for _ in range(BLOCKS)])
        self.post = torch.nn.ParameterList([vector(1.0) for _ in range(BLOCKS)])
        self.pre = torch.nn.ParameterList([vector(1.0) for _ in range(BLOCKS)])
        self.gates = torch.nn.ParameterList([torch.nn.Parameter(torch.full((1, HIDDEN), 0.5, device="cuda", dtype=torch.bfloat16))
                                             for _ in range(BLOCKS)])

    def forward(self, tokens):
        """Logits of flat tokens, the blocks' balance losses, and their experts' counts."""
        x = torch.nn.functional.embedding(tokens, self.embedding)
        h, aux, counts = x, [], []
        for b in range(BLOCKS):
            ids, weights, n, loss = ops.balance(h @ self.routers[b], CHOSEN, groups=SEQUENCES, z_weight=1e-4)
            every = torch.einsum("ehw,nh->new", self.up[b], h)
            every = torch.einsum("ewh,new->neh", self.down[b], torch.nn.functional.gelu(every))
            chosen = every.gather(1, ids.long()[:, :, None].expand(-1, -1, HIDDEN))
            y = (chosen * weights[:, :, None].bfloat16()).sum(1)
            x, h = ops.norm_gate(x, y, pre="rms", post="rms", pre_weight=self.pre[b], post_weight=self.post[b],
                                 gate=self.gates[b])
            aux.append(loss)
            counts.append(n)
        return h @ self.embedding.t(), torch.stack(aux).sum(), counts


def teacher_batch(table, gen):
    """Tokens, the teacher's KEPT largest logits after each with their ids, and labels drawn from them."""
    tokens = torch.randint(0, VOCAB, (SEQUENCES * TOKENS,), device="cuda", generator=gen)
    top, ids = table[tokens % table.shape[0]].topk(KEPT, dim=1)
    labels = ids.gather(1, torch.multinomial(torch.softmax(top, 1), 1, generator=gen)).squeeze(1)
    return tokens, ids.int(), top.bfloat16(), labels


def train(steps=40, seed=0):
    """The mean loss of each step, and the last step's counts."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    student = Student(gen)
    table = 4 * torch.randn(64, VOCAB, device="cuda", generator=gen)       # the teacher: 64 kinds of token
    vectors = [p for n, p in student.named_parameters() if n.split(".")[0] in ("post", "pre", "gates")]
    matrices = [p for n, p in student.named_parameters() if n.split(".")[0] not in ("post", "pre", "gates")]
    opt = BF16Optimizer.from_parameters([{"params": matrices, "weight_decay": 0.01}, {"params": vectors}], lr=4e-3,
                                        max_grad_norm=1.0)
    losses, counts = [], []
    for _ in range(steps):
        total = torch.zeros((), device="cuda")
        for k in range(GAS):
            opt.zero_grad()
            tokens, ids, top, labels = teacher_batch(table, gen)
            logits, aux, counts = student(tokens)
            rows = ops.distill_loss(logits, ids, top, temperature=TEMPERATURE, ce_weight=0.2, labels=labels)
            loss = rows.mean() + aux
            loss.backward()
            opt.accumulate(first=k == 0, last=k == GAS - 1, defer=k == GAS - 1)
            total += loss.detach() / GAS
        opt.grad_norm()
        opt.step()
        losses.append(total)
    losses = torch.stack(losses).tolist()
    opt.close()
    return losses, counts


if __name__ == "__main__":
    got, used = train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
    for i, v in enumerate(got):
        if i % 5 == 0 or i + 1 == len(got):
            print(f"step {i:4d}  loss {v:.4f}")
    print("tokens per expert, last block, by sequence:", used[-1].tolist())
