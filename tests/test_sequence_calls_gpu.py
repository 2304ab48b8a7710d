"""What the binding of the sequence operators makes of a call's arguments, on the GPU."""
import pytest

pytestmark = pytest.mark.gpu


def _heads(*shape, dtype="bfloat16", seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(getattr(torch, dtype))


def _rows(B=2, T=3, V=500, K=4, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(B, T, V, generator=g, device="cuda")
    idx = torch.randint(0, V, (B, T, K), generator=g, device="cuda")
    top = torch.randn(B, T, K, generator=g, device="cuda") + 3
    y = torch.randint(0, V, (B, T), generator=g, device="cuda")
    return z, idx, top, y


@pytest.mark.parametrize("device", ["cpu", "cuda"])
def test_options_held_in_tensors(lib, device):
    """An option may be a 0-d tensor: each call goes by the value that it has then."""
    import torch

    def same(f, values, **kw):
        """f with the option `name` in one tensor that is changed in place, against plain numbers."""
        for name, (first, second) in values.items():
            held = torch.tensor(first, device=device)
            for x in (first, second, first):
                held.fill_(x)
                got, want = f(**{**kw, name: held}), f(**{**kw, name: x})
                assert all(torch.equal(a, b) for a, b in zip(got, want)), name
            assert not all(torch.equal(a, b) for a, b in zip(f(**{**kw, name: first}), f(**{**kw, name: second})))

    z, idx, top, y = _rows()
    option = dict(temperature=(4.0, 1.0), alpha=(0.25, 0.5))
    same(lambda **kw: lib.distill_loss(z, idx, top, labels=y, **kw), option, temperature=2.0, alpha=0.1)
    same(lambda **kw: lib.distill_loss_and_grad(z, idx, top, labels=y, **kw), option, temperature=2.0, alpha=0.1)
    q, k, v, do = (_heads(2, 70, 2, 64, seed=i) for i in range(4))
    option = dict(scale=(0.5, 0.05), window=(3, 9), causal=(True, False))
    for name, pair in option.items():
        kw = dict(causal=True) if name != "causal" else {}
        same(lambda **a: lib.attention_forward(q, k, v, **a), {name: pair}, **kw)
        o, lse = lib.attention_forward(q, k, v, **kw)
        same(lambda **a: lib.attention_backward(q, k, v, o, lse, do, **a), {name: pair}, **kw)
    table = lib.rotary_table(64, 70)
    same(lambda **a: lib.rotary(q, k, table, **a), dict(inverse=(True, False), interleaved=(False, True)))


def test_the_gradient_goes_by_the_forward_calls_options(lib):
    import torch
    z, idx, top, y = _rows()
    tau = torch.tensor(2.0)
    x = z.clone().requires_grad_()
    loss = lib.distill_loss(x, idx, top, labels=y, temperature=tau, alpha=0.5)[0]
    tau.fill_(7.0)
    loss.sum().backward()
    assert torch.equal(x.grad, lib.distill_loss_and_grad(z, idx, top, labels=y, temperature=2.0, alpha=0.5)[1])
    q, k, v, do = (_heads(2, 70, 2, 64, seed=i) for i in range(4))
    scale, causal = torch.tensor(0.25), torch.tensor(True)
    x = q.clone().requires_grad_()
    out = lib.attention(x, k, v, causal=causal, scale=scale)
    scale.fill_(1.0)
    causal.fill_(False)
    out.backward(do)
    o, lse = lib.attention_forward(q, k, v, causal=True, scale=0.25)
    assert torch.equal(out, o)
    assert torch.equal(x.grad, lib.attention_backward(q, k, v, o, lse, do, causal=True, scale=0.25)[0])
    table = lib.rotary_table(64, 70)
    inverse = torch.tensor(False)
    x = q.clone().requires_grad_()
    y1 = lib.rotary(x, None, table, inverse=inverse)[0]
    inverse.fill_(True)
    y1.backward(do)
    assert torch.equal(x.grad, lib.rotary(do, None, table, inverse=True)[0])
