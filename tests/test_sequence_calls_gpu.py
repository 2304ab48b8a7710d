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


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("V", [50, 40001])
@pytest.mark.parametrize("tau,alpha", [(1.0, 0.0), (2.0, 0.25), (3.0, 0.25)])
def test_distill_with_a_teacher_that_is_not_finite(lib, dtype, V, tau, alpha):
    """A softmax over NaN, +inf or nothing but -inf is NaN, and so is the row's loss and its gradient at the
    teacher's entries; one -inf among others is a probability of 0.  Other rows keep their bits."""
    import math

    import torch
    z, idx, top, y = _rows(2, 4, V, 5)
    idx = torch.arange(5, device="cuda").expand(2, 4, 5).contiguous() * 9
    z, top = z.to(getattr(torch, dtype)), top.to(getattr(torch, dtype))
    idx[1, 3, 4] = -1
    kw = dict(labels=y, temperature=tau, alpha=alpha)
    clean, clean_rows = lib.distill_loss(z, idx, top, **kw)
    clean_grad = lib.distill_loss_and_grad(z, idx, top, **kw)[1]
    bad = top.clone()
    bad[0, 1, 2], bad[0, 3, 0], bad[1, 3, :4] = math.nan, math.inf, -math.inf
    bad[1, 3, 4] = math.nan            # not an entry
    bad[1, 1, 1] = -math.inf
    off = torch.zeros(2, 4, dtype=torch.bool, device="cuda")
    off[0, 1] = off[0, 3] = off[1, 3] = True
    loss, rows = lib.distill_loss(z, idx, bad, **kw)
    both, grad = lib.distill_loss_and_grad(z, idx, bad, **kw)
    assert torch.equal(torch.isnan(rows), off)
    assert torch.isnan(loss).all() and torch.isnan(both).all()
    for t in range(4):
        for b in range(2):
            if off[b, t]:
                hit = torch.zeros(V, dtype=torch.bool, device="cuda")
                hit[idx[b, t][idx[b, t] >= 0]] = True
                assert torch.equal(torch.isnan(grad[b, t]), hit)
            elif (b, t) != (1, 1):
                assert torch.equal(rows[b, t], clean_rows[b, t]) and torch.equal(grad[b, t], clean_grad[b, t])
    assert torch.isfinite(grad[1, 1]).all() and torch.isfinite(clean).all()


def test_forward_mode_is_an_error(lib):
    """The operators have no forward-mode derivative: a tangent must not vanish without a word, with or
    without grad mode.  Inside a dual level without tangents they work as ever."""
    import torch
    import torch.autograd.forward_ad as fw
    z, idx, top, y = _rows()
    w = torch.ones(2, 3, device="cuda")
    q, k, v, do = (_heads(2, 40, 2, 64, dtype="float32", seed=i) for i in range(4))
    table = lib.rotary_table(64, 40)
    calls = [
        (lambda a, b, c: lib.attention(a, b, c), (q, k, v)),
        (lambda a, b, c: lib.attention_forward(a, b, c)[0], (q, k, v)),
        (lambda a, b, c: lib.rotary(a, b, c)[0], (q, k, table)),
        (lambda a, b, c: lib.distill_loss(a, idx, b, labels=y, weights=c, alpha=0.5)[0], (z, top, w)),
        (lambda a, b, c: lib.distill_loss_and_grad(a, idx, b, weights=w, upstream=c)[0], (z, top, torch.ones(2, device="cuda"))),
    ]
    o, lse = lib.attention_forward(q, k, v)
    calls.append((lambda a, b, c: lib.attention_backward(q, a, v, b, lse, c)[0], (k, o, do)))
    for f, xs in calls:
        want = f(*xs)
        with fw.dual_level():
            assert torch.equal(f(*xs), want)
            for i in range(3):
                dual = list(xs)
                dual[i] = fw.make_dual(xs[i], torch.ones_like(xs[i]))
                for mode in (torch.enable_grad, torch.no_grad):
                    with mode(), pytest.raises(NotImplementedError, match="forward"):
                        f(*dual)
        assert torch.equal(f(*xs), want)


def test_a_scale_of_zero_is_refused(lib):
    """The C entry points read 0 as 1/sqrt(D); a scale of 0 (or one that fp32 does not hold) asks for
    something else, and None is there for the default."""
    import torch
    q, k, v, do = (_heads(2, 40, 2, 64, dtype="float32", seed=i) for i in range(4))
    o, lse = lib.attention_forward(q, k, v, scale=None)
    assert torch.equal(o, lib.attention_forward(q, k, v, scale=0.125)[0])
    n = lib.dp_launch_count()
    x = q.clone().requires_grad_()
    for zero in (0.0, 0, -0.0, 1e-60, torch.tensor(0.0)):
        for f in (lambda: lib.attention_forward(q, k, v, scale=zero), lambda: lib.attention(q, k, v, scale=zero),
                  lambda: lib.attention(x, k, v, scale=zero),
                  lambda: lib.attention_backward(q, k, v, o, lse, do, scale=zero)):
            with pytest.raises(ValueError, match="scale"):
                f()
    assert lib.dp_launch_count() == n


def test_a_bad_position_is_reported_behind_the_norms_it_spoils(lib):
    import torch
    q = _heads(2, 8, 2, 64)
    table = lib.rotary_table(64, 16)
    pos = torch.arange(8, dtype=torch.int32, device="cuda").expand(2, 8).contiguous()
    pos[1, 3] = 16
    y = lib.rotary(q, None, table, positions=pos)[0]
    o = lib.attention_forward(y, y, q)[0]
    layer = lib.layer_desc(lib.DP_LINEAR, lib.DP_BF16, B=2, p=64, T=8, d=128)
    ws = torch.empty(lib.dp_workspace_size(layer), dtype=torch.uint8, device="cuda")
    sq, factors = torch.empty(1, 2, device="cuda"), torch.empty(1, 2, device="cuda")
    lib.dp_layer_sqnorms(layer, o, _heads(2, 8, 64, seed=1), sq[0], ws)
    lib.dp_clip_factors(sq, 2, 1, False, 1.0, factors)
    assert lib.dp_check_status() == lib.DP_ERR_INVALID_ARG
    assert torch.isfinite(sq[0, 0]) and torch.isnan(sq[0, 1])
    assert lib.dp_check_status() == lib.DP_OK


def test_a_window_wider_than_the_keys_hides_nothing(lib):
    """Up to the longest sequence and the widest window that are taken (their sum passes 32 bits): the
    gradient of the few last queries, which alone see a key, as with no window."""
    import torch
    T, S = 1 << 30, 200
    q, do = (torch.zeros(1, T, 1, 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q[:, -S:], do[:, -S:] = _heads(1, S, 1, 1), _heads(1, S, 1, 1, seed=1)
    k, v = _heads(1, S, 1, 1, seed=2), _heads(1, S, 1, 1, seed=3)
    o, lse = lib.attention_forward(q, k, v, causal=True)
    want = lib.attention_backward(q, k, v, o, lse, do, causal=True)
    assert want[1].any() and want[2].any()
    for window in (S, T // 2, T + S // 2, T + S - 1, T + S, 2 ** 31 - 1):
        got = lib.attention_backward(q, k, v, o, lse, do, causal=True, window=window)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), window
        del got
    last = lib.attention_forward(q[:, -S:].contiguous(), k, v, causal=True)
    assert torch.equal(last[0], o[:, -S:]) and torch.equal(last[1], lse[..., -S:])
    assert torch.isneginf(lse[..., :-S]).all()


def test_sizes_and_windows_past_32_bits(lib):
    """The descriptors hold 32-bit sizes: what does not fit is refused and not taken modulo 2^32, and a
    window that does not fit hides nothing."""
    import torch
    n, far = lib.dp_launch_count(), (1 << 32) + 8
    x = torch.zeros(1, 1, 1, 8, device="cuda")
    table = torch.zeros(1, 8, device="cuda")
    for shape in ((far, 1, 1, 8), (1, far, 1, 8), (1, 1, far, 8)):
        big = x.expand(shape)
        for f in (lambda: lib.rotary(big, None, table), lambda: lib.attention_forward(big, big, big),
                  lambda: lib.attention_forward(x, *(x.expand(1, far, 1, 8),) * 2)):
            with pytest.raises(ValueError, match="2147483647"):
                f()
    for f in (lambda: lib.rotary(x, None, torch.zeros(1, 8, device="cuda").expand(far, 8)),
              lambda: lib.rotary_table(2, far), lambda: lib.rotary_table(far, 2)):
        with pytest.raises(ValueError):
            f()
    z = torch.zeros(1, 1, 8, device="cuda").expand(far, 1, 8)
    empty = torch.zeros(far, 1, 0, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="2147483647"):
        lib.distill_loss(z, empty, empty.float())
    assert lib.dp_launch_count() == n
    q, k, v = (_heads(2, 40, 2, 64, seed=i) for i in range(3))
    want = lib.attention_forward(q, k, v, causal=True)
    for window in (1 << 31, far, 1 << 63, 1 << 70):
        assert all(torch.equal(a, b) for a, b in zip(lib.attention_forward(q, k, v, causal=True, window=window), want))
    for window in (-1, -far + 16, -(1 << 70)):
        with pytest.raises(lib.DPError, match="window"):
            lib.attention_forward(q, k, v, causal=True, window=window)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,T,V,K,tau,alpha", [
    (149, 11, 17884, 93, 2.0, 0.3), (43, 173, 24963, 119, 1.0, 0.0), (1033, 5, 7156, 49, 4.0, 1.0),
    (79, 50, 102670, 122, 1.0, 0.0), (538, 12, 12602, 59, 3.0, 0.5), (40, 128, 40000, 8, 1.0, 0.0),
])
def test_distill_many_rows_a_cta(lib, dtype, B, T, V, K, tau, alpha):
    """Each CTA streams row after row through the same slots: a chunk must not be copied over before every
    thread has read the one before it.  All entries against 64 bits, and the same bits in every call."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(V)
    z = (torch.randn(B, T, V, generator=g, device="cuda") * 2).to(getattr(torch, dtype))
    first = torch.randint(0, V, (B, T, 1), generator=g, device="cuda")
    idx = (first + torch.randint(1, V // K, (B, T, 1), generator=g, device="cuda") * torch.arange(K, device="cuda")) % V
    top = torch.randn(B, T, K, generator=g, device="cuda") * 2 + 5
    y = torch.randint(0, V, (B, T), generator=g, device="cuda")
    w = (torch.rand(B, T, generator=g, device="cuda") + 0.5) * (torch.rand(B, T, generator=g, device="cuda") < 0.8)
    kw = dict(labels=y, weights=w, temperature=tau, alpha=alpha)
    loss, grad = lib.distill_loss_and_grad(z, idx, top, **kw)
    alone, rows = lib.distill_loss(z, idx, top, **kw)
    assert torch.equal(loss, alone)
    # fp32 statistics and entries: within a few 1e-7 of an entry and of the row's largest; bf16: rounded once
    tol = 1e-5 if dtype == "float32" else 2 ** -8
    for b in range(0, B, 8):
        at = slice(b, b + 8)
        x = z[at].double()
        logq, p = torch.log_softmax(x / tau, -1), torch.softmax(top[at].double() / tau, -1)
        row = (1 - alpha) * tau ** 2 * (p * (torch.log(p) - torch.gather(logq, 2, idx[at]))).sum(-1)
        d = ((1 - alpha) * tau * torch.exp(logq)).scatter_add_(2, idx[at], p * (-(1 - alpha) * tau))
        if alpha:
            logp, hit = torch.log_softmax(x, -1), y[at].unsqueeze(-1)
            row = row - alpha * torch.gather(logp, 2, hit).squeeze(-1)
            d = (d + alpha * torch.exp(logp)).scatter_add_(2, hit, torch.full_like(logp[..., :1], -alpha))
        row, d = row * w[at], d * w[at].unsqueeze(-1)
        assert ((rows[at].double() - row).abs() <= 1e-5 * (1 + row.abs())).all()
        off = (grad[at].double() - d).abs()
        assert (off <= tol * d.abs() + 1e-6 * d.abs().amax(-1, keepdim=True) + 1e-38).all()
    for _ in range(10):
        again = lib.distill_loss_and_grad(z, idx, top, **kw)
        assert torch.equal(again[0], loss) and torch.equal(again[1], grad)
    assert lib.dp_check_status() == lib.DP_OK
