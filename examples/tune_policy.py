"""A small decoder is tuned by its own answers, then by pairs of them.

The fine-tuning operators together, next to the norms and the optimizer: positions are turned
into queries and keys (train_ops.rotary), the feed-forward blocks keep what their backward pass needs
in 8 bits (train_ops.glu8_forward / glu8_backward), the block's outputs join the residual stream
through train_ops.norm_gate, the sampler's and a frozen reference's log-probabilities come from
train_ops.token_logp_forward, and the model learns by train_ops.policy_loss from rewards, then by
train_ops.preference_loss from its best and worst answers.  The bf16 gradients go into the
optimizer's FP32 accumulator (optimizer.BF16Optimizer).

    python examples/tune_policy.py [steps]
"""
import copy
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixed_precision_optimizer_bf16_gb300 import train_ops as ops  # noqa: E402
from mixed_precision_optimizer_bf16_gb300.optimizer import BF16Optimizer  # noqa: E402

VOCAB, HIDDEN, HEADS, KV, DIM, WIDE, BLOCKS = 517, 128, 4, 2, 32, 320, 2
ANSWERS, PROMPT, LENGTH = 16, 4, 20          # sequences, their given tokens, all of their tokens
ROTARY = dict(layout="half", rotary_dim=16, scaling="yarn", factor=4.0, original_length=16)
EPOCHS = 2                                   # updates on one set of answers


class FeedForward(torch.autograd.Function):
    """silu(x G) (x U) D, of which autograd keeps x and, in 8 bits, x G and x U; h is computed again from those for D's gradient."""

    @staticmethod
    def forward(ctx, x, w_in, w_out):
        both = x @ w_in
        h, codes, scales = ops.glu8_forward(both[:, :WIDE], both[:, WIDE:])
        ctx.save_for_backward(x, w_in, w_out, codes, scales)
        return h @ w_out

    @staticmethod
    def backward(ctx, dy):
        x, w_in, w_out, codes, scales = ctx.saved_tensors
        dh = dy @ w_out.t()
        dboth, h = dh.new_empty(dh.shape[0], 2 * WIDE), torch.empty_like(dh)
        ops.glu8_backward(dh, codes, scales, out_gate=dboth[:, :WIDE], out_up=dboth[:, WIDE:], out_h=h)
        return dboth @ w_in.t(), x.t() @ dboth, h.t() @ dy


class Decoder(torch.nn.Module):
    def __init__(self, gen):
        super().__init__()

        def weight(*shape, scale):
            return torch.nn.Parameter((scale * torch.randn(*shape, device="cuda", generator=gen)).bfloat16())

        def vectors():
            return torch.nn.ParameterList([torch.nn.Parameter(torch.ones(HIDDEN, device="cuda", dtype=torch.bfloat16)) for _ in range(2 * BLOCKS)])

        self.embedding = weight(VOCAB, HIDDEN, scale=0.5)
        self.qkv = torch.nn.ParameterList([weight(HIDDEN, (HEADS + 2 * KV) * DIM, scale=HIDDEN ** -0.5) for _ in range(BLOCKS)])
        self.out = torch.nn.ParameterList([weight(HEADS * DIM, HIDDEN, scale=HIDDEN ** -0.5) for _ in range(BLOCKS)])
        self.w_in = torch.nn.ParameterList([weight(HIDDEN, 2 * WIDE, scale=HIDDEN ** -0.5) for _ in range(BLOCKS)])
        self.w_out = torch.nn.ParameterList([weight(WIDE, HIDDEN, scale=WIDE ** -0.5) for _ in range(BLOCKS)])
        self.pre, self.post = vectors(), vectors()

    def forward(self, tokens):
        """Logits [sequences * tokens, VOCAB] of [sequences, tokens]."""
        n, t = tokens.shape
        x = torch.nn.functional.embedding(tokens.reshape(-1), self.embedding)
        h = x
        for b in range(BLOCKS):
            qkv = (h @ self.qkv[b]).view(n, t, HEADS + 2 * KV, DIM)
            q, k = ops.rotary(qkv[:, :, :HEADS], qkv[:, :, HEADS:HEADS + KV], **ROTARY)
            k, v = (y.repeat_interleave(HEADS // KV, 2).transpose(1, 2) for y in (k, qkv[:, :, HEADS + KV:]))
            y = torch.nn.functional.scaled_dot_product_attention(q.transpose(1, 2), k, v, is_causal=True)
            y = y.transpose(1, 2).reshape(n * t, HEADS * DIM) @ self.out[b]
            x, h = ops.norm_gate(x, y, pre_weight=self.pre[2 * b], post_weight=self.post[2 * b])
            y = FeedForward.apply(h, self.w_in[b], self.w_out[b])
            x, h = ops.norm_gate(x, y, pre_weight=self.pre[2 * b + 1], post_weight=self.post[2 * b + 1])
        return h @ self.embedding.t()


@torch.no_grad()
def answers(model, gen):
    """(tokens [ANSWERS, LENGTH], labels [ANSWERS * LENGTH]: the next token, -100 where none was sampled)."""
    tokens = torch.randint(0, VOCAB, (ANSWERS, PROMPT), device="cuda", generator=gen)
    while tokens.shape[1] < LENGTH:
        last = model(tokens).view(ANSWERS, -1, VOCAB)[:, -1].float()
        tokens = torch.cat([tokens, torch.multinomial(torch.softmax(last, 1), 1, generator=gen)], 1)
    labels = torch.full_like(tokens, -100)
    labels[:, PROMPT - 1:-1] = tokens[:, PROMPT:]
    return tokens, labels.reshape(-1)


def rewards(tokens):
    """The share of small even tokens in each answer."""
    answer = tokens[:, PROMPT:]
    return ((answer % 2 == 0) & (answer < VOCAB // 2)).float().mean(1)


def policy_step_loss(model, tokens, labels, advantage, old_logp, ref_logp):
    """Mean over the sampled tokens."""
    weight = (labels >= 0).float()
    loss, _ = ops.policy_loss(model(tokens), labels, advantage.repeat_interleave(LENGTH), old_logp=old_logp, ref_logp=ref_logp,
                              clip_high=0.28, kl_weight=0.02, row_weight=weight / weight.sum())
    return loss.sum()


def preference_step_loss(model, tokens, labels, ref_logp):
    """tokens: preferred answers, then the others, pair by pair."""
    offsets = torch.arange(0, tokens.numel() + 1, LENGTH, device="cuda", dtype=torch.int32)
    loss, _ = ops.preference_loss(model(tokens), labels, offsets, ref_logp=ref_logp, beta=0.2)
    return loss.mean()


def tune(steps=10, seed=0):
    """The rewards of each step's answers, and the losses of the pairs that follow."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Decoder(gen)
    reference = copy.deepcopy(model).requires_grad_(False)
    vectors = [p for p in model.parameters() if p.dim() == 1]
    opt = BF16Optimizer.from_parameters([{"params": [p for p in model.parameters() if p.dim() > 1], "weight_decay": 0.01}, {"params": vectors}],
                                        lr=2e-3, max_grad_norm=1.0)

    def update(loss):
        opt.zero_grad()
        loss().backward()
        opt.accumulate(first=True, last=True, defer=True)
        opt.grad_norm()
        opt.step()

    got, losses = [], []
    for _ in range(steps):
        tokens, labels = answers(model, gen)
        with torch.no_grad():
            old_logp, ref_logp = (ops.token_logp_forward(m(tokens), labels)[0] for m in (model, reference))
        reward = rewards(tokens)
        advantage = (reward - reward.mean()) / (reward.std() + 1e-4)
        got.append(reward.mean())
        for _ in range(EPOCHS):
            update(lambda: policy_step_loss(model, tokens, labels, advantage, old_logp, ref_logp))
        order = reward.argsort(descending=True, stable=True)                     # the best answers against the worst
        order = torch.cat([order[:ANSWERS // 2], order[ANSWERS // 2:].flip(0)])
        tokens, labels = tokens[order], labels.view(ANSWERS, LENGTH)[order].reshape(-1)
        with torch.no_grad():
            logp = ops.token_logp_forward(reference(tokens), labels)[0].view(ANSWERS, LENGTH).sum(1)
        update(lambda: losses.append(preference_step_loss(model, tokens, labels, logp)) or losses[-1])
    got, losses = torch.stack(got).tolist(), torch.stack([v.detach() for v in losses]).tolist()
    opt.close()
    return got, losses


if __name__ == "__main__":
    got, losses = tune(int(sys.argv[1]) if len(sys.argv) > 1 else 10)
    for i, (r, v) in enumerate(zip(got, losses)):
        print(f"step {i:3d}  mean reward {r:.4f}  loss of the pairs {v:.4f}")
