"""The example's training step: the sequence operators between clipped linear layers.

GPU: the privatised gradient of the example's student equals the naive per-example loop
(batch size 1, autograd per example, plain torch operators) clipped and averaged; and the
example's own training loop learns.
"""
import math
import os
import sys

import numpy as np
import pytest

from helpers import rel_flat

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:Full backward hook is firing")]


@pytest.fixture()
def example(lib):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import private_distillation
    return private_distillation


class _Plain:
    """rotary and attention in plain torch."""

    @staticmethod
    def rotary(q, k, table):
        R = table.shape[1]
        c, s = (t[None, :q.shape[1], None] for t in (table[:, :R // 2].to(q.dtype), table[:, R // 2:].to(q.dtype)))

        def turn(x):
            a, b = x[..., :R // 2], x[..., R // 2:R]
            import torch
            return torch.cat([a * c - b * s, b * c + a * s, x[..., R:]], dim=-1)
        return turn(q), turn(k)

    @staticmethod
    def attention(q, k, v, causal, q_lens, k_lens):
        import torch
        B, T, H, D = q.shape
        n = int(q_lens[0])
        k, v = (x.repeat_interleave(H // x.shape[2], dim=2) for x in (k, v))
        s = torch.einsum("bthd,bshd->bhts", q, k) / math.sqrt(D)
        i = torch.arange(T, device=q.device)
        see = (i[None, :] <= i[:, None]) & (i[None, :] < n)
        p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
        o = torch.einsum("bhts,bshd->bthd", p, v)
        return torch.where((i < n)[None, :, None, None], o, 0.0)


def test_privatised_gradient_equals_the_per_example_loop(lib, example):
    import torch
    torch.backends.cuda.matmul.allow_tf32 = False
    B, T, V, C = 5, 19, 40, 0.7
    torch.manual_seed(1)
    student = example.Student(V, width=32, heads=4, kv_heads=2, head=8, context=32).cuda()
    tokens, lens, idx, teacher, labels, w = example.synthetic_batch(B, T, V, 6, seed=3)
    kw = dict(temperature=2.0, alpha=0.3)
    engine = lib.PrivacyEngine(student, C=C, sigma=0.0)
    loss, _ = lib.distill_loss(student(tokens, lens), idx, teacher, labels=labels, weights=w, **kw)
    loss.sum().backward()
    flat = engine.privatise(seed=0).cpu().numpy()
    engine.detach()

    student = student.double()
    student.ops = _Plain
    want = 0.0
    for i in range(B):
        student.zero_grad()
        z = student(tokens[i:i + 1], lens[i:i + 1])[0]
        logq, logp = torch.log_softmax(z / 2.0, -1), torch.log_softmax(z, -1)
        p = torch.softmax(teacher[i].double() / 2.0, -1)
        kl = (p * (torch.log(p) - torch.gather(logq, 1, idx[i].long()))).sum(-1)
        row = 0.7 * 4.0 * kl - 0.3 * logp[torch.arange(T), labels[i]]
        l = (row * w[i]).sum()
        assert abs(l.item() - loss[i].item()) <= 1e-5 * (1 + abs(l.item()))
        l.backward()
        g = np.concatenate([np.concatenate([m.weight.grad.cpu().numpy().ravel()] +
                                           ([m.bias.grad.cpu().numpy().ravel()] if m.bias is not None else []))
                            for m in engine.layers])
        want = want + g * min(1.0, C / np.linalg.norm(g)) / B

    class Blk:
        def __init__(self, m):
            self.p, self.D, self.has_bias = m.weight.shape[0], m.weight.shape[1], m.bias is not None
    # fp32 layers and operators through two blocks: each stays within the fp32 tolerance of 1e-5,
    # and about ten of them follow one another
    assert rel_flat(flat, want, [Blk(m) for m in engine.layers]) <= 1e-4
    assert lib.dp_check_status() == lib.DP_OK


def test_example_learns(lib, example):
    losses = example.main(["--steps", "12"])
    assert all(np.isfinite(losses)) and losses[-1] < 0.9 * losses[0]
