"""Private distillation of a small decoder: the sequence operators around clipped linear layers.

A student of a few pre-norm blocks (frozen token embedding, trainable linear layers) learns
from a teacher's top logits.  Each step is one ordinary forward and backward pass:

    rotary -> attention -> linear layers -> distillation loss (one per example)

through the package's operators, and PrivacyEngine turns the captured activations and output
gradients of the linear layers into the privatised gradient (per-example clipping, noise,
1/B).  The operators have no parameters and never mix examples, so clipping the linear layers
bounds everything that an example contributes.

    python examples/private_distillation.py --steps 20
"""
import argparse
import os
import sys

import torch
import torch.nn as nn

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import example_gradient_clipping_gb300 as dp  # noqa: E402


class Block(nn.Module):
    def __init__(self, width: int, heads: int, kv_heads: int, head: int):
        super().__init__()
        self.heads, self.kv_heads, self.head = heads, kv_heads, head
        self.qkv = nn.Linear(width, (heads + 2 * kv_heads) * head)
        self.out = nn.Linear(heads * head, width)
        self.up, self.down = nn.Linear(width, 4 * width), nn.Linear(4 * width, width)

    @staticmethod
    def norm(x):
        return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)

    def forward(self, x, table, lens, ops):
        B, T, _ = x.shape
        # q, k and v are read from the one projection by their strides
        qkv = self.qkv(self.norm(x)).view(B, T, self.heads + 2 * self.kv_heads, self.head)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=2)
        q, k = ops.rotary(q, k, table)
        o = ops.attention(q, k, v, causal=True, q_lens=lens, k_lens=lens)
        x = x + self.out(o.reshape(B, T, -1))
        return x + self.down(nn.functional.gelu(self.up(self.norm(x))))


class Student(nn.Module):
    """ops: where rotary and attention come from (the package)."""

    def __init__(self, vocab: int, width=64, heads=4, kv_heads=2, head=16, layers=2, context=512, ops=dp):
        super().__init__()
        self.ops = ops
        self.embed = nn.Embedding(vocab, width)
        self.embed.weight.requires_grad_(False)
        self.blocks = nn.ModuleList([Block(width, heads, kv_heads, head) for _ in range(layers)])
        self.lm_head = nn.Linear(width, vocab, bias=False)
        self.context, self.rotated = context, head
        self.table = None

    def forward(self, tokens, lens):
        if self.table is None:   # built once
            self.table = dp.rotary_table(self.rotated, self.context, device=str(tokens.device))
        x = self.embed(tokens)
        for b in self.blocks:
            x = b(x, self.table, lens, self.ops)
        return self.lm_head(Block.norm(x))


def synthetic_batch(B, T, vocab, K, seed, device="cuda"):
    """Tokens of ragged examples, a teacher's top K logits per position, labels and token weights."""
    g = torch.Generator(device=device).manual_seed(seed)
    tokens = torch.randint(0, vocab, (B, T), generator=g, device=device)
    lens = torch.randint(max(1, T // 2), T + 1, (B,), generator=g, device=device, dtype=torch.int32)
    # the teacher prefers a fixed map of the token, so there is something to learn
    first = (tokens * 7 + 3) % vocab
    indices = (first.unsqueeze(-1) + torch.arange(K, device=device)) % vocab
    teacher = 4.0 - torch.arange(K, device=device).float().expand(B, T, K)
    weights = (torch.arange(T, device=device)[None] < lens[:, None]).float()
    return tokens, lens, indices.int(), teacher.contiguous(), first, weights


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--length", type=int, default=48)
    ap.add_argument("--vocab", type=int, default=256)
    ap.add_argument("--sigma", type=float, default=0.2)
    ap.add_argument("--clip", type=float, default=1.0)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args(argv)
    torch.manual_seed(0)
    student = Student(a.vocab).to("cuda", torch.bfloat16)
    engine = dp.PrivacyEngine(student, C=a.clip, sigma=a.sigma)
    opt = torch.optim.SGD([p for p in student.parameters() if p.requires_grad], lr=a.lr)
    losses = []
    for step in range(a.steps):
        tokens, lens, indices, teacher, labels, weights = synthetic_batch(a.batch, a.length, a.vocab, 8, seed=step)
        loss, _ = dp.distill_loss(student(tokens, lens), indices, teacher, labels=labels, weights=weights,
                                  temperature=2.0, alpha=0.2)
        loss.sum().backward()          # the sum: every example's G is its own gradient
        engine.privatise(seed=step)    # .grad <- (sum_i c_i g_i + sigma C z) / B
        opt.step()
        losses.append((loss.sum() / weights.sum()).item())
        print(f"step {step:3d}  loss per token {losses[-1]:.4f}")
    if dp.dp_check_status() != dp.DP_OK:
        raise SystemExit("a device-side condition was raised")
    return losses


if __name__ == "__main__":
    main()
