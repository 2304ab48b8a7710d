"""Embeddings and layer norms clipped per example beside linear layers: ClipStep, VirtualStep and PrivacyEngine against
the naive per-example loop, and the teacher's alternatives into the distillation loss."""
import numpy as np
import pytest
import torch
import torch.nn as nn

import oracle
from helpers import TOL, rel_elem, rel_rows

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:Full backward hook is firing")]

B, T, V, D, P = 6, 37, 90, 48, 20


def _inputs(lib, dtype, seed=0, b=B):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def n(*s):
        return torch.randn(*s, generator=g, device="cuda").to(dt)
    tokens = torch.randint(0, V, (b, T), generator=g, device="cuda")
    tokens[:, T // 2:] = 3
    scale = 10.0 ** torch.linspace(-1, 1, b, device="cuda")[:, None, None]   # some examples below the bound, some above
    x, dy, a, gl = n(b, T, D), (n(b, T, D) * scale).to(dt), n(b, T, D), (n(b, T, P) * scale).to(dt)
    w = n(D)
    _, mean, rstd = lib.layer_norm_forward(x, w, w)
    _, each = lib.layer_norm_backward(dy, x, w, mean, rstd, per_example=True)
    return [(tokens, dy), (each, None), (a, gl)]


def _descs(lib, dtype, b=B):
    dt = lib.DP_BF16 if dtype == "bf16" else lib.DP_FP32
    return [lib.embedding_desc(dt, B=b, T=T, V=V, D=D, scale=2.0, padding=5, index_i64=True),
            lib.kept_desc(B=b, p=D, has_bias=True), lib.layer_desc(lib.DP_LINEAR, dt, B=b, p=P, T=T, d=D)]


def _each(inputs):
    """Per-example gradients by layer, float64 [B, n_l]."""
    (tokens, dy), (kept, _), (a, g) = inputs
    b = tokens.shape[0]
    emb = torch.zeros(b, V, D, dtype=torch.float64, device="cuda")
    for i in range(b):
        keep = tokens[i] != 5
        emb[i].index_add_(0, tokens[i][keep], 2.0 * dy[i][keep].double())
    lin = torch.cat([torch.einsum("btp,btd->bpd", g.double(), a.double()).flatten(1), g.double().sum(1)], 1)
    return [emb.flatten(1).cpu().numpy(), kept.double().cpu().numpy(), lin.cpu().numpy()]


def _clipped(each, C, per_layer):
    norms = [np.sqrt((e * e).sum(1)) for e in each]
    if not per_layer:
        norms = [np.sqrt(sum(n * n for n in norms))] * len(each)
    f = [np.minimum(1.0, C / n) for n in norms]
    return np.concatenate([(c[:, None] * e).sum(0) for c, e in zip(f, each)])


def _rows_off(got, want):
    """rel_rows of each block: the embedding's rows, the layer norm's vector, the linear layer's rows."""
    worst, o = 0.0, 0
    for n, row in ((V * D, D), (2 * D, 2 * D), (P * D, D), (P, P)):
        g, w = got[o:o + n], want[o:o + n]
        worst, o = max(worst, rel_rows(g, w, row)), o + n
    assert o == got.size == want.size
    return worst


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("per_layer", [False, True])
def test_step(lib, dtype, per_layer):
    inputs = _inputs(lib, dtype)
    each = _each(inputs)
    C, sigma = 30.0, 0.5
    step = lib.ClipStep(_descs(lib, dtype), C=C, sigma=0.0, per_layer=per_layer)
    flat = step.run(inputs, seed=0).double().cpu().numpy() * B
    for l, e in enumerate(each):
        assert rel_elem(step.sqnorms[l].cpu().numpy(), (e * e).sum(1)) <= TOL[dtype]
    want = _clipped(each, C, per_layer)
    assert _rows_off(flat, want) <= TOL[dtype]
    # noise: the two-call form bit for bit, the oracle's, and a captured step with changed inputs
    noisy = lib.ClipStep(_descs(lib, dtype), C=C, sigma=sigma, per_layer=per_layer)
    got = noisy.run(inputs, seed=11).clone()
    plain = lib.ClipStep(_descs(lib, dtype), C=C, sigma=sigma, per_layer=per_layer, fuse_noise=False)
    assert torch.equal(plain.run(inputs, seed=11), got)
    z = got.double().cpu().numpy() - flat / B
    want_z = oracle.add_noise(np.zeros_like(flat), sigma, C, B, 11)
    # normals of the hardware's sine (4e-6 absolute each) and three roundings of the sums, which stand in one entry
    assert np.abs(z - want_z).max() <= (1e-5 * 6 + 4e-6) * sigma * C / B + 8 * 2.0 ** -24 * np.abs(flat).max() / B
    noisy.capture(inputs)
    other = _inputs(lib, dtype, seed=1)
    for (a, g), (a2, g2) in zip(inputs, other):
        a.copy_(a2)
        if g is not None:
            g.copy_(g2)
    replayed = noisy.replay(12).clone()
    assert torch.equal(replayed, plain.run(other, seed=12))
    assert lib.dp_check_status() == lib.DP_OK


def test_virtual_step_and_pipeline(lib):
    inputs = _inputs(lib, "fp32")
    C = 30.0
    want = _clipped(_each(inputs), C, False) / B
    vs = lib.VirtualStep(_descs(lib, "fp32", 4), C=C, sigma=0.0)
    vs.zero()
    for lo, hi in ((0, 4), (4, 5), (5, 6)):
        vs.add([(a[lo:hi].contiguous(), None if g is None else g[lo:hi].contiguous()) for a, g in inputs], hi - lo)
    got = vs.finish(0).double().cpu().numpy()
    assert _rows_off(got, want) <= TOL["fp32"]
    with pytest.raises(ValueError, match="pipeline"):
        lib.ClipPipeline(_descs(lib, "fp32"), [((1,), (1,))] * 3, "fp32", C=1.0, sigma=1.0)


def test_many_blocks_of_noise(lib):
    """More than the 64 blocks that one noise launch takes."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n = 70
    inputs = [(torch.randn(3, 8, generator=g, device="cuda"), None) for _ in range(n)]
    steps = [lib.ClipStep([lib.kept_desc(B=3, p=8) for _ in range(n)], C=1.0, sigma=0.7, fuse_noise=f) for f in (True, False)]
    assert torch.equal(steps[0].run(inputs, seed=5), steps[1].run(inputs, seed=5))


class _Model(nn.Module):
    def __init__(self, emb, norm):
        super().__init__()
        self.embed, self.norm1 = emb(V, D, padding_idx=5), norm(D)
        self.up, self.norm2, self.head = nn.Linear(D, D), norm(D, bias=False), nn.Linear(D, V, bias=False)

    def forward(self, tokens):
        x = self.embed(tokens)
        x = x + torch.tanh(self.up(self.norm1(x)))
        return self.head(self.norm2(x))


def _loss(z, y):
    return nn.functional.cross_entropy(z.flatten(0, 1).float(), y.flatten(), reduction="none").view(y.shape).sum(1)


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 1e-4), (torch.bfloat16, 4e-2)], ids=["fp32", "bf16"])
@pytest.mark.parametrize("reduction", ["sum", "mean"])
def test_engine_equals_the_per_example_loop(lib, dtype, tol, reduction):
    # fp32: five layers and an embedding of 1e-5 each follow one another; bf16: both loops round every activation
    # to 2^-8, forward and back, so two of the framework's bf16 tolerances
    torch.backends.cuda.matmul.allow_tf32 = False
    torch.manual_seed(0)
    C = 0.8
    model = _Model(lib.Embedding, lib.LayerNorm).cuda().to(dtype)
    nn.init.normal_(model.norm1.weight, 1.0, 0.2)
    nn.init.normal_(model.norm1.bias, 0.0, 0.2)
    tokens = torch.randint(0, V, (B, T), device="cuda")
    tokens[:, ::5] = 5
    y = torch.randint(0, V, (B, T), device="cuda")
    engine = lib.PrivacyEngine(model, C=C, sigma=0.0, loss_reduction=reduction)
    l = _loss(model(tokens), y)
    (l.sum() if reduction == "sum" else l.mean()).backward()
    assert model.norm1.weight.grad is None   # the engine's to fill
    flat = engine.privatise(seed=0).double().cpu().numpy()
    names = [m for m in engine.layers]
    assert [type(m).__name__ for m in names] == ["Embedding", "LayerNorm", "Linear", "LayerNorm", "Linear"]
    assert model.norm1.weight.grad.shape == (D,) and model.embed.weight.grad.dtype == dtype
    engine.detach()

    plain = _Model(nn.Embedding, nn.LayerNorm).cuda().double()
    plain.load_state_dict({k: v.double() for k, v in model.state_dict().items()})
    layers = [plain.embed, plain.norm1, plain.up, plain.norm2, plain.head]
    want, shapes = 0.0, []
    for i in range(B):
        plain.zero_grad()
        z = plain(tokens[i:i + 1])
        nn.functional.cross_entropy(z[0], y[i], reduction="sum").backward()
        parts = []
        for m in layers:
            parts.append(m.weight.grad.flatten())
            if getattr(m, "bias", None) is not None:
                parts.append(m.bias.grad.flatten())
        shapes = [p.numel() for p in parts]
        g = torch.cat(parts).cpu().numpy()
        want = want + g * min(1.0, C / np.linalg.norm(g)) / B
    o = 0
    for n in shapes:   # each parameter against its own rms
        assert rel_rows(flat[o:o + n], want[o:o + n]) <= tol, n
        o += n
    # without the engine the module's gradients are autograd's
    model.zero_grad()
    _loss(model(tokens), y).sum().backward()
    plain.zero_grad()
    nn.functional.cross_entropy(plain(tokens).flatten(0, 1), y.flatten(), reduction="sum").backward()
    for m, q in ((model.norm1, plain.norm1), (model.norm2, plain.norm2), (model.embed, plain.embed)):
        assert rel_rows(m.weight.grad.double().cpu().numpy(), q.weight.grad.cpu().numpy()) <= tol


def test_engine_refuses_inputs_without_examples(lib):
    model = _Model(lib.Embedding, lib.LayerNorm).cuda()
    model.position = lib.Embedding(T, D).cuda()
    engine = lib.PrivacyEngine(model)
    tokens = torch.randint(0, V, (B, T), device="cuda")
    x = model(tokens) + model.position(torch.arange(T, device="cuda")).sum()   # one row of positions for the whole batch
    x.sum().backward()
    with pytest.raises(ValueError, match="examples"):
        engine.privatise(0)


def test_teacher_alternatives_feed_distillation(lib):
    """token_logprobs' alternatives are the teacher of distill_loss: with all of a small vocabulary's entries the
    loss is the divergence of the two distributions, and 0 where the student is the teacher."""
    g = torch.Generator(device="cuda").manual_seed(2)
    z, t = (torch.randn(3, 7, 100, generator=g, device="cuda") * 2 for _ in range(2))
    y = torch.randint(0, 100, (3, 7), generator=g, device="cuda")
    _, _, top, at = lib.token_logprobs(t, y, top=100)
    loss, dz = lib.distill_loss_and_grad(z, at, top)
    p, q = torch.log_softmax(t.double(), -1), torch.log_softmax(z.double(), -1)
    want = (p.exp() * (p - q)).sum((1, 2))
    # 7 rows of sums of 100 fp32 terms of size below 2^4
    assert (loss.double() - want).abs().max() <= 7 * 200 * 2.0 ** -24 * 16
    assert (dz.double() - (q.exp() - p.exp())).abs().max() <= 200 * 2.0 ** -24
    same, _ = lib.distill_loss_and_grad(t, at, top)
    assert same.abs().max() <= 7 * 200 * 2.0 ** -24 * 16


@pytest.fixture()
def example(lib):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import private_distillation
    return private_distillation


def test_example_with_trained_layers(lib, example):
    """The example's student with its embedding and layer norms trained: the privatised gradient is the per-example
    loop's, and its loop runs."""
    from test_sequence_example import _Plain
    torch.backends.cuda.matmul.allow_tf32 = False
    b, t, v, C = 4, 11, 30, 0.9
    torch.manual_seed(3)
    kw = dict(width=32, heads=4, kv_heads=2, head=8, context=32)
    student = example.Student(v, trained=lib, **kw).cuda()
    plain = example.Student(v, trained=nn, ops=_Plain, **kw).cuda().double()
    plain.load_state_dict({k: p.double() for k, p in student.state_dict().items()})
    tokens, lens, idx, teacher, labels, w = example.synthetic_batch(b, t, v, 6, seed=4)
    _, _, top, at = lib.token_logprobs(example.teacher_logits(idx, teacher, v), top=6)
    engine = lib.PrivacyEngine(student, C=C, sigma=0.0)
    loss, _ = lib.distill_loss(student(tokens, lens), at, top, labels=labels, weights=w, temperature=2.0, alpha=0.3)
    loss.sum().backward()
    flat = engine.privatise(seed=0).cpu().numpy()
    engine.detach()
    assert len(engine.layers) == 1 + 2 * 6 + 1
    find = dict(student.named_modules())
    names = {id(m): n for n, m in find.items()}
    mirror = [dict(plain.named_modules())[names[id(m)]] for m in engine.layers]
    want, sizes = 0.0, []
    for i in range(b):
        plain.zero_grad()
        z = plain(tokens[i:i + 1], lens[i:i + 1])[0]
        logq, logp = torch.log_softmax(z / 2.0, -1), torch.log_softmax(z, -1)
        p = torch.softmax(top[i].double() / 2.0, -1)
        kl = (p * (torch.log(p) - torch.gather(logq, 1, at[i].long()))).sum(-1)
        ((0.7 * 4.0 * kl - 0.3 * logp[torch.arange(t), labels[i]]) * w[i]).sum().backward()
        parts = [q.grad.flatten() for m in mirror for q in (m.weight, getattr(m, "bias", None)) if q is not None]
        sizes = [q.numel() for q in parts]
        g = torch.cat(parts).cpu().numpy()
        want = want + g * min(1.0, C / np.linalg.norm(g)) / b
    o = 0
    for n in sizes:   # fp32 layers and operators through two blocks: about fourteen of 1e-5 follow one another
        assert rel_rows(flat[o:o + n], want[o:o + n]) <= 2e-4, n
        o += n
    losses = example.main(["--steps", "2", "--trained", "--batch", "8", "--length", "16"])
    assert all(np.isfinite(losses)) and lib.dp_check_status() == lib.DP_OK


@pytest.mark.parametrize("which", ["embed", "norm1"])
def test_engine_refuses_a_layer_called_twice(lib, which):
    model = _Model(lib.Embedding, lib.LayerNorm).cuda()
    engine = lib.PrivacyEngine(model)
    tokens = torch.randint(0, V, (B, T), device="cuda")

    def twice():
        z = model(tokens)
        again = model.embed(tokens.flip(1)) if which == "embed" else model.norm1(model.embed.weight.detach()[tokens])
        return z.sum() + again.sum()
    with pytest.raises(RuntimeError, match="more than once"):
        twice().backward()
    for _ in range(2):   # passes that were not privatised do not count
        model(tokens).sum().backward()
    engine.privatise(0)
    with pytest.raises(RuntimeError, match="first"):
        engine.privatise(0)


def test_engine_that_is_refused_leaves_nothing_behind(lib):
    model = _Model(lib.Embedding, lib.LayerNorm).cuda()
    model.norm2._sink = lambda each: None   # another engine's
    with pytest.raises(ValueError, match="another engine"):
        lib.PrivacyEngine(model)
    assert model.norm1._sink is None and not model.embed._forward_hooks and not model.up._forward_hooks
    model.norm2._sink = None
    lib.PrivacyEngine(model).detach()
