"""Embeddings, layer norms and log probabilities on the GPU against their definitions in 64 bits, inside the error
bounds that layers_reference derives beside its values."""
import math

import pytest

import layers_reference as ref

pytestmark = pytest.mark.gpu


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _r(name):
    return 2.0 ** -8 if name == "bf16" else 0.0   # half a step, relative


def _within(got, want, what=""):
    import torch
    val, err = want
    got = got.double()
    assert got.shape == val.shape
    off = (got - val).abs()
    assert torch.isfinite(got).all(), what
    assert (off <= err).all(), (what, float((off / err.clamp(min=1e-300)).max()))


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


# ------------------------------------------------------------------------------------- layer norm
NORM = [  # B, T, D: each layout of a row over threads, its edges, and more rows than CTAs
    (1, 1, 1), (2, 3, 7), (3, 5, 8), (2, 9, 31), (2, 4, 256), (2, 4, 257), (1, 33, 512), (3, 7, 520), (2, 40, 768),
    (2, 3, 776), (1, 5, 1001), (2, 2, 1024), (2, 3, 1032), (1, 3, 2048), (2, 2, 2056), (1, 2, 4096), (3, 1, 5003),
    (1, 2, 8192), (1, 2, 8200), (1, 3, 16384), (1, 2, 16383), (5, 700, 64), (1, 6000, 24), (300, 1, 40), (3, 500, 1500),
]


def _norm_inputs(B, T, D, dtype, wdtype, seed=0):
    import torch
    g = _gen(seed + B * 31 + T * 7 + D)
    x = (torch.randn(B, T, D, generator=g, device="cuda") * 2 + torch.randn(D, generator=g, device="cuda") * 3).to(_dt(dtype))
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(_dt(wdtype))
    b = torch.randn(D, generator=g, device="cuda").to(_dt(wdtype))
    dy = torch.randn(B, T, D, generator=g, device="cuda").to(_dt(dtype))
    return x, w, b, dy


@pytest.mark.parametrize("B,T,D", NORM)
@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("fp32", "fp32"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_layer_norm(lib, B, T, D, dtype, wdtype):
    x, w, b, dy = _norm_inputs(B, T, D, dtype, wdtype)
    y, mean, rstd = lib.layer_norm_forward(x, w, b)
    vy, vdx, vdw, vdb = ref.layer_norm(x, w, b, 1e-5, dy, _r(dtype), _r(wdtype))
    _within(y, vy, "y")
    dx, dw, db = lib.layer_norm_backward(dy, x, w, mean, rstd)
    assert dw.dtype == db.dtype == w.dtype
    _within(dx, vdx, "dx")
    _within(dw, vdw, "dw")
    _within(db, vdb, "db")
    _, _, vdw, vdb = ref.layer_norm(x, w, b, 1e-5, dy, _r(dtype), 0.0, per_example=True)
    dx2, each = lib.layer_norm_backward(dy, x, w, mean, rstd, per_example=True)
    assert each.shape == (B, 2 * D)
    _within(dx2, vdx, "dx")
    _within(each[:, :D], vdw, "each dw")
    _within(each[:, D:], vdb, "each db")
    # the weight alone, and parts left out
    dx3, dw3, none = lib.layer_norm_backward(dy, x, w, mean, rstd, bias=False, dx=False)
    assert dx3 is None and none is None
    _within(dw3, ref.layer_norm(x, w, b, 1e-5, dy, _r(dtype), _r(wdtype))[2], "dw alone")
    dx4, none, _ = lib.layer_norm_backward(dy, x, w, mean, rstd, params=False)
    _within(dx4, vdx, "dx alone")
    assert none is None


def test_layer_norm_without_parameters_large_means_and_eps(lib):
    import torch
    for dtype in ("fp32", "bf16"):
        x, _, _, dy = _norm_inputs(2, 5, 300, dtype, dtype)
        for shift, eps in ((0.0, 0.0), (500.0, 1e-5), (0.0, 3.0)):
            z = (x.double() + shift).to(x.dtype)
            y, mean, rstd = lib.layer_norm_forward(z, eps=eps)
            dx, dw, _ = lib.layer_norm_backward(dy, z, None, mean, rstd, bias=False)
            vy, vdx, vdw, _ = ref.layer_norm(z, eps=eps, dy=dy, r=_r(dtype))
            _within(y, vy)
            _within(dx, vdx)
            _within(dw, vdw)   # without a weight the gradient is fp32
            assert dw.dtype == torch.float32
    # a constant row is eps alone
    y, _, _ = lib.layer_norm_forward(torch.full((1, 2, 64), 3.0, device="cuda"))
    assert torch.equal(y, torch.zeros_like(y))


@pytest.mark.parametrize("B", [1, 8, 9, 64, 65, 700])
@pytest.mark.parametrize("n", [1, 33, 2002, 20000])
def test_example_sum(lib, B, n):
    """Every split of the rows; out (+)= sum_i f_i g_i, of B + 1 terms in one chain at most."""
    import torch
    rows, f, base = torch.randn(B, n, device="cuda"), torch.rand(B, device="cuda"), torch.randn(n, device="cuda")
    for accumulate in (False, True):
        out = base.clone()
        lib.dp_example_sum(rows, B, n, f, out, accumulate=accumulate)
        terms = rows.double() * f.double()[:, None]
        want = terms.sum(0) + (base.double() if accumulate else 0.0)
        size = terms.abs().sum(0) + (base.double().abs() if accumulate else 0.0)
        assert ((out.double() - want).abs() <= (B + 2) * 2.0 ** -24 * size).all()


def test_two_host_threads_on_their_streams(lib):
    import threading

    import torch
    x, w, b, dy = _norm_inputs(4, 300, 768, "bf16", "bf16")
    t = _tokens(4, 300, 5000, 1, "skewed").int()
    z = torch.randn(2, 320, 3000, device="cuda").bfloat16()
    y = torch.randint(0, 3000, (2, 320), device="cuda", dtype=torch.int32)

    def everything():
        n, m, r = lib.layer_norm_forward(x, w, b)
        out = [n, *lib.layer_norm_backward(dy, x, w, m, r), *lib.layer_norm_backward(dy, x, w, m, r, per_example=True)]
        out += [lib.embedding_backward(t, dy, 5000), lib.embedding_sqnorms(t, dy, 5000)]
        lp, h, st, best, at = lib.token_logprobs_forward(z, y, top=20)
        return out + [lp, h, best, at, lib.token_logprobs_backward(z, y, st, h, lp, h)]
    want = everything()
    torch.cuda.synchronize()
    wrong = []

    def run(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for i in range(15):
                got = everything()
                s.synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, want)):
                    wrong.append((k, i))
    threads = [threading.Thread(target=run, args=(k,)) for k in range(3)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong and lib.dp_check_status() == lib.DP_OK


@pytest.mark.parametrize("dtype,D", [("fp32", 1000), ("fp32", 1001), ("bf16", 1000), ("bf16", 250)])
def test_layer_norm_gradient_where_mean_times_rstd_overflows(lib, dtype, D):
    """Constant rows of 2^116 with rstd 2^20: h = 0, so dx = rs (u - mean u) and dw = 0 exactly."""
    import torch
    _, w, _, dy = _norm_inputs(2, 3, D, dtype, dtype)
    x = torch.full((2, 3, D), 2.0 ** 116, device="cuda").to(dy.dtype)
    mean = torch.full((2, 3), 2.0 ** 116, device="cuda")
    rstd = torch.full((2, 3), 2.0 ** 20, device="cuda")
    dx, dw, db = lib.layer_norm_backward(dy, x, w, mean, rstd)
    u = dy.double() * w.double()
    want = 2.0 ** 20 * (u - u.mean(-1, keepdim=True))
    # u and its mean: a product, a sum of D terms in chains of at most 64 with a tree of 10, 1 / D, two roundings
    # behind it; then the type's own
    err = 2.0 ** 20 * 80 * 2.0 ** -24 * u.abs().amax() + want.abs() * _r(dtype)
    assert ((dx.double() - want).abs() <= err).all()
    assert not dw.any()
    total = dy.double().sum((0, 1))
    assert ((db.double() - total).abs() <= 6 * 2.0 ** -24 * dy.double().abs().sum((0, 1)) + total.abs() * _r(dtype)).all()


@pytest.mark.parametrize("B,n", [(1, 1), (5, 3), (16, 2002), (3, 40001), (3, 200003), (304, 33000), (305, 33000)])
def test_example_sqnorms(lib, B, n):
    """Rows at any alignment, neighbours not read.  Positive terms: each thread's chain of at most n / 256 + 16
    roundings and the trees behind it bound the relative error."""
    import torch
    for off in (4, 5, 7):
        flat = torch.full((B * n + 16,), float("nan"), device="cuda")
        rows = flat[off:off + B * n].view(B, n)
        rows.copy_(torch.randn(B, n, device="cuda"))
        out = torch.empty(B, device="cuda")
        lib.dp_example_sqnorms(rows, B, n, out)
        want = rows.double().square().sum(1)
        assert ((out.double() - want).abs() <= want * (n / 256 + 48) * 2.0 ** -24).all()


def test_layer_norm_shapes_strides_and_bits(lib):
    import torch
    for dtype in ("fp32", "bf16"):
        for D in (64, 197, 3000):
            x, w, b, dy = _norm_inputs(3, 11, D, dtype, dtype)
            y, m, r = lib.layer_norm_forward(x, w, b)
            dx, dw, db = lib.layer_norm_backward(dy, x, w, m, r)
            # time first, every second row, rows off the 16-byte grid, an expanded gradient
            xt = x.transpose(0, 1).contiguous().transpose(0, 1)
            wide = torch.randn(3, 22, D + 9, device="cuda").to(x.dtype)
            wide[:, ::2, 1:D + 1] = x
            for z in (xt, wide[:, ::2, 1:D + 1]):
                y2, m2, r2 = lib.layer_norm_forward(z, w, b)
                dx2, dw2, db2 = lib.layer_norm_backward(dy, z, w, m2, r2)
                tol = (_r(dtype) or 2e-6) * 4
                assert (y2.double() - y.double()).abs().max() <= tol * y.abs().max()
                assert (dx2.double() - dx.double()).abs().max() <= tol * dx.abs().max()
                assert (dw2.double() - dw.double()).abs().max() <= tol * dw.abs().max()
                if z is xt:   # the same layout over threads
                    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
            row = torch.randn(D, device="cuda").to(x.dtype)
            e1 = lib.layer_norm_backward(row.expand(3, 11, D), x, w, m, r)
            e2 = lib.layer_norm_backward(row.expand(3, 11, D).contiguous(), x, w, m, r)
            assert all(torch.equal(p, q) for p, q in zip(e1, e2))
            # other ranks
            y4 = lib.layer_norm(x.view(3, 11, 1, D), w, b)
            assert y4.shape == (3, 11, 1, D) and torch.equal(y4.view_as(y), y)
            assert torch.equal(lib.layer_norm(x[:, 0], w, b), y[:, 0])
            # bit for bit, and no example's values in another's
            again = lib.layer_norm_backward(dy, x, w, m, r, per_example=True)
            bad = x.clone()
            bad[1] = float("nan")
            y5, m5, r5 = lib.layer_norm_forward(bad, w, b)
            other = lib.layer_norm_backward(dy, bad, w, m5, r5, per_example=True)
            for p, q in zip(again, other):
                assert torch.equal(p[[0, 2]], q[[0, 2]]) and torch.isnan(q[1]).any()
            assert torch.equal(y5[[0, 2]], y[[0, 2]]) and torch.isnan(y5[1]).all()


def test_layer_norm_gradient_against_differences(lib):
    import torch
    x, w, b, dy = _norm_inputs(2, 3, 50, "fp32", "fp32")
    leaves = [t.clone().requires_grad_() for t in (x, w, b)]
    (lib.layer_norm(*leaves) * dy).sum().backward()
    for leaf, at in zip(leaves, range(3)):
        direction = torch.randn_like(leaf)
        h = 1e-3
        ends = []
        for s in (h, -h):
            moved = [t.double() for t in (x, w, b)]
            moved[at] = moved[at] + s * direction.double()
            ends.append((ref.layer_norm(*moved)[0][0] * dy.double()).sum())
        slope = (ends[0] - ends[1]) / (2 * h)
        # the central difference is off by h^2 / 6 times a third derivative of the order of the values
        assert abs((leaf.grad.double() * direction).sum() - slope) <= 1e-4 * (1 + abs(slope)) + 1e-4 * direction.numel() ** 0.5


def test_layer_norm_offsets_past_32_bits(lib):
    import torch
    far = (1 << 31) + 16
    store = torch.empty(far + 64, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((2, 1, 64), (far, 64, 1))
    x.copy_(torch.randn(2, 1, 64, device="cuda"))
    y, m, r = lib.layer_norm_forward(x)
    z, m2, r2 = lib.layer_norm_forward(x.contiguous())
    assert torch.equal(y, z) and torch.equal(m, m2)
    dx, _, _ = lib.layer_norm_backward(x, x, None, m, r, bias=False)
    dx2, _, _ = lib.layer_norm_backward(x.contiguous(), x.contiguous(), None, m, r, bias=False)
    assert torch.equal(dx, dx2)


# ------------------------------------------------------------------------------------- embedding
EMBED = [  # B, T, V, D: one row, units of 32 sorted rows, runs over many units, every sort, odd widths, slabs
    (1, 1, 1, 1), (2, 3, 10, 8), (3, 50, 5, 40), (1, 100, 1, 16), (2, 32, 3, 24), (4, 300, 3, 197), (64, 1, 5000, 256),
    (1, 64, 2, 264), (3, 333, 70, 1000), (2, 2049, 600, 33), (2, 9000, 50, 72), (5, 6000, 400000, 16), (1, 20000, 2, 8),
    (7, 5003, 600, 17),
]


def _tokens(B, T, V, seed, kind):
    import torch
    g = _gen(seed)
    t = torch.randint(0, V, (B, T), generator=g, device="cuda")
    if kind == "skewed":   # half of them one token, so that its run covers units, and a sorted stretch
        t = torch.where(torch.rand(B, T, generator=g, device="cuda") < 0.5, torch.full_like(t, V // 2), t)
    return t


@pytest.mark.parametrize("B,T,V,D", EMBED)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["even", "skewed"])
def test_embedding(lib, B, T, V, D, dtype, kind):
    import torch
    if V * D * B > 1 << 26:
        D = 4
    g = _gen(B + T + V + D)
    t = _tokens(B, T, V, B + T + V, kind)
    w = torch.randn(V, D, generator=g, device="cuda").to(_dt(dtype))
    dy = torch.randn(B, T, D, generator=g, device="cuda").to(_dt(dtype))
    f = torch.rand(B, generator=g, device="cuda")
    f[0] = 0.0
    for tokens, scale, padding, factors in ((t, 1.0, None, None), (t.int(), 2.5, V - 1, f), (t.int(), -0.5, V // 2, None)):
        _within(lib.embedding(tokens, w, scale=scale, padding=padding), ref.embedding(tokens, w, scale, _r(dtype)), "y")
        out = _dt(dtype) if factors is None else torch.float32
        dw = lib.embedding_backward(tokens, dy, V, scale=scale, padding=padding, factors=factors, dtype=out)
        vdw, vsq = ref.embedding_grad(tokens, dy, V, scale, padding, factors, 0.0 if out == torch.float32 else _r("bf16"))
        _within(dw, vdw, "dw")
        sq = lib.embedding_sqnorms(tokens, dy, V, scale=scale, padding=padding)
        _within(sq, vsq, "sqnorms")
        # bit for bit
        assert torch.equal(dw, lib.embedding_backward(tokens, dy, V, scale=scale, padding=padding, factors=factors, dtype=out))
        assert torch.equal(sq, lib.embedding_sqnorms(tokens, dy, V, scale=scale, padding=padding))
    assert lib.dp_check_status() == lib.DP_OK


@pytest.mark.parametrize("B,T,V,D", [(3, 20000, 700, 520), (1, 45000, 2, 8), (2, 700, 40, 2104), (40, 1000, 3, 13), (5, 2500, 900, 768)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["even", "skewed"])
def test_embedding_of_many_rows(lib, B, T, V, D, dtype, kind):
    """Units of 16 and 32 rows, runs over hundreds of them, rows of more than one pass."""
    test_embedding(lib, B, T, V, D, dtype, kind)


@pytest.mark.parametrize("N", [1, 31, 32, 33, 1024, 1025, 4097, 16384, 16385, 40000, 300000])
@pytest.mark.parametrize("V", [1, 2, 511, 512, 70000, 1 << 20])
def test_embedding_order_is_a_stable_sort(lib, N, V):
    """The order buffer: the positions, then the sorted keys, of every sort's shape; padding last."""
    import torch
    t = torch.randint(0, V, (1, N), generator=_gen(N + V), device="cuda", dtype=torch.int32)
    d = lib.embedding_desc(lib.DP_FP32, B=1, T=N, V=V, D=1, padding=V // 3 if V > 2 else None)
    order = torch.empty(lib.dp_embedding_order_size(d), dtype=torch.uint8, device="cuda")
    ws = torch.empty(lib.dp_embedding_workspace(d), dtype=torch.uint8, device="cuda")
    lib.dp_embedding_order(d, t, order, ws)
    key = t[0].clone()
    if V > 2:
        key[key == V // 3] = V
    want_keys, want = torch.sort(key, stable=True)
    words = order.view(torch.int32)
    assert torch.equal(words[:N], want.int()) and torch.equal(words[words.numel() // 2:][:N], want_keys)


def test_embedding_bad_tokens(lib):
    import torch
    V, D = 12, 40
    t = torch.tensor([[0, 12, 3], [-1, 5, 5]], device="cuda")
    w, dy = torch.randn(V, D, device="cuda"), torch.randn(2, 3, D, device="cuda")
    for tokens in (t, t.int(), torch.where(t == 12, 2 ** 40, t)):
        y = lib.embedding(tokens, w)
        assert lib.dp_check_status() == lib.DP_ERR_INVALID_ARG and lib.dp_check_status() == lib.DP_OK
        bad = (tokens < 0) | (tokens >= V)
        assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], w[tokens[~bad].long()])
        dw = lib.embedding_backward(tokens, dy, V)
        assert lib.dp_check_status() == lib.DP_ERR_INVALID_ARG
        (want, err), _ = ref.embedding_grad(tokens, dy, V)
        _within(dw, (want, err))


def test_embedding_strides_accumulate_and_neighbours(lib):
    import torch
    B, T, V, D = 3, 70, 9, 128
    t = _tokens(B, T, V, 5, "skewed").int()
    big = torch.randn(V, 2 * D, device="cuda")
    for w in (big[:, :D], big[:, 3:D + 3]):
        assert torch.equal(lib.embedding(t, w, scale=2.0), 2.0 * w[t.long()])
    wide = torch.randn(B, T, 2 * D, device="cuda")
    for dy in (wide[:, :, :D], wide[:, :, 1:D + 1], wide[:, :, :D].transpose(0, 1).contiguous().transpose(0, 1),
               torch.randn(D, device="cuda").expand(B, T, D)):
        got, want = lib.embedding_backward(t, dy, V), lib.embedding_backward(t, dy.contiguous(), V)
        assert torch.equal(got, want)
        assert torch.allclose(lib.embedding_sqnorms(t, dy, V), lib.embedding_sqnorms(t, dy.contiguous(), V), rtol=1e-6)
    # accumulate: rows without a token stay as they are
    d = lib.embedding_desc(lib.DP_FP32, B=B, T=T, V=V, D=D, padding=0)
    order = torch.empty(lib.dp_embedding_order_size(d), dtype=torch.uint8, device="cuda")
    ws = torch.empty(lib.dp_embedding_workspace(d), dtype=torch.uint8, device="cuda")
    dy = wide[:, :, :D].contiguous()
    some = t.clamp(max=6)
    base = torch.randn(V, D, device="cuda")
    acc = base.clone()
    lib.dp_embedding_order(d, some, order, ws)
    lib.dp_embedding_grad(d, order, dy, None, acc, ws, accumulate=True)
    assert torch.equal(acc[[0, 7, 8]], base[[0, 7, 8]])
    (want, err), _ = ref.embedding_grad(some, dy, V, padding=0)
    _within(acc, (want + base.double(), err + 2 * ref.U * (want + base.double()).abs()))
    # an example's NaN stays with its norm
    sq = lib.embedding_sqnorms(t, dy, V)
    nan = dy.clone()
    nan[1] = float("nan")
    assert torch.equal(lib.embedding_sqnorms(t, nan, V)[[0, 2]], sq[[0, 2]])
    # an innermost stride other than 1 is refused
    with pytest.raises(ValueError, match="stride"):
        lib.embedding_backward(t, wide[:, :, ::2], V)


@pytest.mark.parametrize("N,V,D", [(1, 1, 1), (7, 50, 3), (1024, 3000, 33), (1500, 700, 128), (9000, 20011, 24), (20000, 4000, 40)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_embedding_sorted_and_summed_in_one_call(lib, N, V, D, dtype):
    """The bits of the two calls; dW at any alignment, its neighbours left, whatever it held before."""
    import torch
    out = lib.DP_BF16 if dtype == "bf16" else lib.DP_FP32
    d = lib.embedding_desc(lib.DP_FP32, B=1, T=N, V=V, D=D, scale=1.5, padding=V - 1 if V > 1 else None)
    d.out_dtype = out
    t = _tokens(1, N, V, N, "skewed").int()
    dy = torch.randn(1, N, D, device="cuda")
    f = torch.full((1,), 0.5, device="cuda")
    order, ws = (torch.empty(n, dtype=torch.uint8, device="cuda") for n in (lib.dp_embedding_order_size(d), lib.dp_embedding_workspace(d)))
    want = torch.empty(V, D, device="cuda", dtype=_dt(dtype))
    lib.dp_embedding_order(d, t, order, ws)
    lib.dp_embedding_grad(d, order, dy, f, want, ws)
    sorted_ = order.clone()
    for off in (8, 1, 3, 7):
        flat = torch.full((V * D + 24,), float("nan"), device="cuda", dtype=_dt(dtype))
        dw = flat[off:off + V * D].view(V, D)
        order.zero_()
        lib.dp_embedding_order_grad(d, t, order, dy, f, dw, ws)
        if off == 8:
            assert torch.equal(dw, want)
        else:   # narrower accesses add in the same order
            assert torch.allclose(dw.float(), want.float(), rtol=2.0 ** -7 if dtype == "bf16" else 1e-5, atol=1e-5)
        assert torch.equal(dw == 0, want == 0)
        assert flat[:off].isnan().all() and flat[off + V * D:].isnan().all()
        assert torch.equal(order.view(torch.int32)[:N], sorted_.view(torch.int32)[:N])
    if dtype == "fp32":
        base = torch.randn(V, D, device="cuda")
        one, two = base.clone(), base.clone()
        lib.dp_embedding_order_grad(d, t, order, dy, f, one, ws, accumulate=True)
        lib.dp_embedding_grad(d, order, dy, f, two, ws, accumulate=True)
        assert torch.equal(one, two)


def test_embedding_autograd(lib):
    import torch
    for dtype in ("bf16", "fp32"):
        w = torch.randn(50, 24, device="cuda").to(_dt(dtype)).requires_grad_()
        for shape in ((7,), (3, 9), (2, 3, 4)):
            t = torch.randint(0, 50, shape, device="cuda")
            w.grad = None
            y = lib.embedding(t, w, scale=3.0, padding=4)
            assert y.shape == (*shape, 24)
            up = torch.randn_like(y)
            (y * up).sum().backward()
            assert w.grad.dtype == w.dtype and not w.grad[4].any()
            (want, err), _ = ref.embedding_grad(t.view(shape[0], -1), up.view(shape[0], -1, 24), 50, 3.0, 4, r=_r(dtype))
            _within(w.grad, (want, err))


def test_embedding_offsets_past_32_bits(lib):
    import torch
    V, D = 2, 1 << 15
    T = (1 << 16) + 3   # T D is past 2^31
    t = torch.zeros(1, T, dtype=torch.int32, device="cuda")
    t[0, -2:] = 1
    dy = torch.zeros(1, T, D, dtype=torch.bfloat16, device="cuda")
    dy[0, -1] = 2.0
    dy[0, 5] = 1.0
    dw = lib.embedding_backward(t, dy, V)
    assert torch.equal(dw, torch.tensor([[1.0], [2.0]], device="cuda").expand(2, D))
    assert float(lib.embedding_sqnorms(t, dy, V)) == 5.0 * D
    y = lib.embedding(t, dw.bfloat16())
    assert (y[0, -1] == 2).all() and (y[0, -3] == 1).all()


# ------------------------------------------------------------------------------------- log probabilities
LOGP = [  # B, T, V, K: one logit, fewer vectors than threads, clusters, odd rows, every group size
    (1, 1, 1, 1), (1, 2, 7, 7), (2, 3, 33, 5), (4, 2, 300, 100), (4, 31, 1000, 16), (3, 5, 50257, 50), (1, 1, 131072, 20),
    (2, 2, 131071, 128), (2, 1, 250001, 1), (40, 10, 4097, 64), (1, 3, 600000, 7), (1, 1, 16000, 128), (200, 2, 128, 128),
]


@pytest.mark.parametrize("B,T,V,K", LOGP)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tau", [1.0, 0.7])
def test_token_logprobs(lib, B, T, V, K, dtype, tau):
    import torch
    g = _gen(B + T + V + K)
    z = (torch.randn(B, T, V, generator=g, device="cuda") * 3).to(_dt(dtype))
    y = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32 if tau == 1.0 else torch.int64)
    if B * T > 2:
        y[0, 0] = -1
    dl, dh = torch.randn(B, T, generator=g, device="cuda"), torch.randn(B, T, generator=g, device="cuda")
    vlp, vh, vall, vdz = ref.logprobs(z, y, tau, dl, dh, _r(dtype))
    for top in (K, 0):
        lp, h, stats, best, at = lib.token_logprobs_forward(z, y, top=top, temperature=tau)
        _within(lp, vlp, "logprob")
        _within(h, vh, "entropy")
        if top:
            want = ref.top(z, K)
            assert at.dtype == torch.int32 and torch.equal(at.long(), want)
            _within(best, (torch.gather(vall[0], 2, want), torch.gather(vall[1], 2, want)), "top")
        else:
            assert best is None and at is None
    _within(lib.token_logprobs_backward(z, y, stats, h, dl, dh, temperature=tau), vdz, "dz")
    for a, b in ((dl, None), (None, dh)):
        got = lib.token_logprobs_backward(z, y, stats, h, a, b, temperature=tau)
        _within(got, ref.logprobs(z, y, tau, a, b, _r(dtype))[3], "dz of one")
    assert not lib.token_logprobs_backward(z, y, stats, h, temperature=tau).any()
    assert lib.dp_check_status() == lib.DP_OK


@pytest.mark.parametrize("V", [1, 9, 500, 2049, 8195, 16390, 20001])
@pytest.mark.parametrize("K", [0, 1, 20, 32, 33, 64, 65])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_token_logprobs_of_many_rows(lib, V, K, dtype):
    """Enough rows that short ones are on 64 threads and ordinary ones on 128; rows on no 16-byte grid, one all
    masks, one with NaN, one of equal logits."""
    import torch
    K, N = min(K, V), 611
    g = _gen(V + K)
    z = (torch.randn(1, N, V, generator=g, device="cuda") * 2).to(_dt(dtype))
    z[0, 7] = -math.inf
    z[0, 8, V // 2] = math.nan
    z[0, 9] = 1.5
    z[0, 10, : V // 2] = torch.finfo(_dt(dtype)).min
    y = torch.randint(0, V, (1, N), generator=g, device="cuda")
    y[0, ::5] = -1
    good = torch.ones(N, dtype=torch.bool, device="cuda")
    good[7:9] = False
    lp, h, stats, best, at = lib.token_logprobs_forward(z, y, top=K)
    vlp, vh, vall = ref.logprobs(z[:, good], y[:, good], threads=64)
    _within(lp[:, good], vlp, "logprob")
    _within(h[:, good], vh, "entropy")
    assert torch.isnan(h[0, 7:9]).all()
    if K:
        want = ref.top(z, K)
        assert torch.equal(at[:, good].long(), want[:, good]) and torch.equal(at[0, 7].long(), want[0, 7])
        assert int(at[0, 8, 0]) == V // 2
        _within(best[:, good], (torch.gather(vall[0], 2, want[:, good]), torch.gather(vall[1], 2, want[:, good])), "top")
    assert lib.dp_check_status() == lib.DP_OK


@pytest.mark.parametrize("kind", ["zeros", "two values", "rising", "falling", "few above", "one stretch", "masked", "lowest",
                                  "all lowest", "strided"])
@pytest.mark.parametrize("V,K", [(1000, 20), (9000, 32), (9000, 64), (30001, 20), (30001, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_top_alternatives_of_equal_logits_in_many_rows(lib, kind, V, K, dtype):
    import torch
    row = _ties(kind, V, dtype)
    at = lib.token_logprobs(row.expand(1, 610, V).contiguous(), top=K)[3]
    assert torch.equal(at.long(), ref.top(row[None, None], K).expand(1, 610, K))


def _ties(kind, V, dtype):
    """Rows with more equal logits than there are places for."""
    import torch
    z = torch.zeros(V, device="cuda")
    i = torch.arange(V, device="cuda")
    if kind == "zeros":
        z[::2] = -0.0
    elif kind == "two values":
        z = (i % 3 == 0).float()
    elif kind == "rising":
        z = i.float() / 64
    elif kind == "falling":
        z = -i.float() / 64
    elif kind == "few above":   # ten above a plateau
        n = min(10, V)
        z[V - n:] = 1.0 + torch.arange(n, device="cuda") / 4
    elif kind == "one stretch":   # the largest all in a few threads' vectors
        z[: min(V, 4000)] = 5.0 + (i[: min(V, 4000)] % 7).float()
    elif kind == "masked":
        z[:] = -math.inf
        z[V // 2] = 1.0
        z[V // 3] = 0.5
    elif kind == "lowest":
        z[:] = torch.finfo(_dt(dtype)).min
        z[3 % V] = 0.0
    elif kind == "all lowest":
        z[:] = torch.finfo(_dt(dtype)).min
    elif kind == "strided":   # the largest all in the vectors of one thread
        z = ((i // 2048) % 2 == 0).float() * ((i % 2048) < 8).float() * 3.0 + (i % 5).float() / 8
    return z.to(_dt(dtype))


@pytest.mark.parametrize("kind", ["zeros", "two values", "rising", "falling", "few above", "one stretch", "masked", "lowest",
                                  "all lowest", "strided"])
@pytest.mark.parametrize("V", [5, 1000, 50257, 140000])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_top_alternatives_of_equal_logits(lib, kind, V, dtype):
    import torch
    row = _ties(kind, V, dtype)
    for B, K in ((1, min(V, 128)), (400, min(V, 20))):   # a cluster a row, and a CTA
        z = row.expand(B, 1, V).contiguous() if B * V < 1 << 26 else row.expand(160, 1, V).contiguous()
        lp, h, stats, best, at = lib.token_logprobs_forward(z, torch.zeros(z.shape[:2], dtype=torch.int32, device="cuda"), top=K)
        want = ref.top(row[None, None], K)
        assert torch.equal(at.long(), want.expand(z.shape[0], 1, K))
        lse = torch.log_softmax(row.double(), 0)
        n = torch.gather(lse, 0, want[0, 0])
        off = (best[0, 0].double() - n).abs()
        # 2^x, sums over V / 256 + 64 additions and the distance to the maximum, which fp32 holds to 2^-24
        tol = ref.EX2 + (V / 256 + 64) * ref.U + 8 * ref.U * torch.where(torch.isfinite(n), n.abs(), torch.zeros_like(n))
        assert ((off <= tol) | (best[0, 0].double() == n)).all()
        p = torch.exp(lse)
        want_h = -torch.where(p > 0, p * lse, torch.zeros_like(p)).sum()
        assert abs(h[0, 0].double() - want_h) <= (ref.EX2 + (V / 256 + 64) * ref.U) * (2 + 2 * want_h)


def test_token_logprobs_nan_inf_and_bad_tokens(lib):
    import torch
    V = 3000
    z = torch.randn(6, 1, V, device="cuda")
    z[1, 0, 17] = float("nan")
    z[2, 0, 5] = float("inf")
    z[3] = -float("inf")
    z[4, 0, 2000:] = -float("inf")
    y = torch.tensor([[5], [5], [6], [7], [2500], [V]], device="cuda")
    lp, h, stats, best, at = lib.token_logprobs_forward(z, y, top=3)
    assert lib.dp_check_status() == lib.DP_ERR_INVALID_ARG and lib.dp_check_status() == lib.DP_OK
    for i in (1, 2, 3):
        assert torch.isnan(lp[i]).all() and torch.isnan(h[i]).all() and torch.isnan(best[i]).all()
    assert int(at[1, 0, 0]) == 17 and int(at[2, 0, 0]) == 5 and at[3, 0].tolist() == [0, 1, 2]
    assert lp[4] == -float("inf") and torch.isfinite(h[4]).all() and torch.isfinite(best[4]).all()
    assert torch.isnan(lp[5]).all() and torch.isfinite(h[5]).all()
    one = torch.ones(6, 1, device="cuda")
    d = lib.token_logprobs_backward(z, y, stats, h, one, None)
    assert lib.dp_check_status() == lib.DP_ERR_INVALID_ARG
    assert torch.isnan(d[5]).all() and torch.isnan(d[1]).any() and torch.isfinite(d[[0, 4]]).all()
    assert float(d[4, 0, 2500]) == 1.0
    # rows without an upstream gradient are 0, whatever they hold
    zero = torch.zeros(6, 1, device="cuda")
    assert not lib.token_logprobs_backward(z, y.clamp(max=V - 1), stats, h, zero, zero).any()


def test_token_logprobs_strides_and_large_offsets(lib):
    import torch
    for dtype in ("bf16", "fp32"):
        V = 777
        wide = torch.randn(3, 5, V + 14, device="cuda").to(_dt(dtype))
        y = torch.randint(0, V, (3, 5), device="cuda")
        for z in (wide[:, :, :V], wide[:, :, 5:V + 5]):
            a, b = lib.token_logprobs_forward(z, y, top=9), lib.token_logprobs_forward(z.contiguous(), y, top=9)
            assert torch.equal(a[4], b[4])
            for p, q in zip(a[:4], b[:4]):   # another place on the vector grid: other orders of the sums
                assert (p - q).abs().max() <= (ref.EX2 + 80 * ref.U) * 20
            up = torch.randn(3, 5, device="cuda")
            d1, d2 = (lib.token_logprobs_backward(x, y, s[2], s[1], up, up) for x, s in ((z, b), (z.contiguous(), b)))
            assert torch.equal(d1, d2)
    far = (1 << 31) + 8
    store = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda")
    z = store.as_strided((1, 2, 4096), (far, far, 1))
    z.copy_(torch.randn(1, 2, 4096, device="cuda"))
    y = torch.tensor([[3, 4]], device="cuda")
    a, b = lib.token_logprobs_forward(z, y, top=4), lib.token_logprobs_forward(z.contiguous(), y, top=4)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_token_logprobs_autograd_and_differences(lib):
    import torch
    z = torch.randn(2, 3, 40, device="cuda")
    y = torch.randint(0, 40, (2, 3), device="cuda")
    dl, dh = torch.randn(2, 3, device="cuda"), torch.randn(2, 3, device="cuda")
    leaf = z.clone().requires_grad_()
    lp, h, best, at = lib.token_logprobs(leaf, y, top=5, temperature=1.3)
    assert not best.requires_grad and not at.requires_grad
    ((lp * dl).sum() + (h * dh).sum()).backward()
    vlp, vh, _, vdz = ref.logprobs(z, y, 1.3, dl, dh)
    _within(leaf.grad, vdz)
    direction, eps, ends = torch.randn(2, 3, 40, device="cuda").double(), 1e-4, []
    for s in (eps, -eps):
        a, b, _ = ref.logprobs(z.double() + s * direction, y, 1.3)
        ends.append((a[0] * dl.double()).sum() + (b[0] * dh.double()).sum())
    slope = (ends[0] - ends[1]) / (2 * eps)
    assert abs((leaf.grad.double() * direction).sum() - slope) <= 1e-5 * (1 + abs(slope)) + 1e-4
    # one of the two alone
    for pick, a, b in ((0, dl, None), (1, None, dh)):
        leaf = z.clone().requires_grad_()
        (lib.token_logprobs(leaf, y, temperature=1.3)[pick] * (dl if pick == 0 else dh)).sum().backward()
        _within(leaf.grad, ref.logprobs(z, y, 1.3, a, b)[3])
    # scores without tokens
    lp, h = lib.token_logprobs(z)
    assert not lp.any() and torch.allclose(h, torch.distributions.Categorical(logits=z).entropy(), atol=1e-5)


# ------------------------------------------------------------------------------------- calls
def test_streams_graphs_and_empty_calls(lib):
    import torch
    x, w, b, dy = _norm_inputs(4, 50, 256, "bf16", "bf16")
    t = _tokens(4, 50, 300, 1, "skewed")
    table = torch.randn(300, 256, device="cuda").bfloat16()
    z = torch.randn(4, 50, 2000, device="cuda").bfloat16()
    y = torch.randint(0, 2000, (4, 50), device="cuda")
    up = torch.randn(4, 50, device="cuda")

    def everything(**kw):
        n, m, r = lib.layer_norm_forward(x, w, b, **kw)
        out = [n, m, r, *lib.layer_norm_backward(dy, x, w, m, r, **kw)]
        out += lib.layer_norm_backward(dy, x, w, m, r, per_example=True, **kw)
        out += [lib.embedding(t, table, **kw), lib.embedding_backward(t, dy, 300, **kw), lib.embedding_sqnorms(t, dy, 300, **kw)]
        lp, h, st, best, at = lib.token_logprobs_forward(z, y, top=10, **kw)
        return out + [lp, h, best, at, lib.token_logprobs_backward(z, y, st, h, up, up, **kw)]

    want = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = everything(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graphs = []
    for _ in range(2):   # two graphs, replayed one inside the other's run
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = everything()
        graphs.append((g, out))
    for i in (0, 1, 1, 0):
        for o in graphs[i][1]:
            o.zero_()
        graphs[i][0].replay()
    assert all(torch.equal(p, q) for g, out in graphs for p, q in zip(out, want))
    x.copy_(torch.randn_like(x))   # a replay goes by the inputs that it finds
    t.copy_(t.flip(0))
    graphs[0][0].replay()
    assert all(torch.equal(p, q) for p, q in zip(graphs[0][1], everything()))
    # no rows
    e = torch.empty(0, 5, 8, device="cuda")
    n, m, r = lib.layer_norm_forward(e)
    assert n.shape == e.shape
    dx, dw, db = lib.layer_norm_backward(e, e, None, m, r)
    assert dx.shape == e.shape and not dw.any() and not db.any()
    none = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    assert lib.embedding(none, table).shape == (3, 0, 256)
    assert not lib.embedding_backward(none, torch.empty(3, 0, 8, device="cuda"), 10).any()
    assert not lib.embedding_sqnorms(none, torch.empty(3, 0, 8, device="cuda"), 10).any()
    lp, h, st, best, at = lib.token_logprobs_forward(torch.empty(2, 0, 9, device="cuda"), top=3)
    assert lp.shape == (2, 0) and best.shape == (2, 0, 3)


def test_options_held_in_tensors_and_forward_mode(lib):
    import torch
    import torch.autograd.forward_ad as fa
    z = torch.randn(1, 2, 50, device="cuda")
    tau = torch.tensor(2.0)
    first = lib.token_logprobs(z, temperature=tau)[1]
    tau.fill_(0.5)
    assert torch.equal(lib.token_logprobs(z, temperature=tau)[1], lib.token_logprobs(z, temperature=0.5)[1])
    assert torch.equal(first, lib.token_logprobs(z, temperature=2.0)[1])
    with fa.dual_level():
        with pytest.raises(NotImplementedError):
            lib.layer_norm_forward(fa.make_dual(z, z))
        with pytest.raises(NotImplementedError):
            lib.token_logprobs_forward(fa.make_dual(z, z))
        with pytest.raises(NotImplementedError):
            lib.embedding(torch.zeros(1, 2, dtype=torch.int32, device="cuda"), fa.make_dual(z[0], z[0]))
