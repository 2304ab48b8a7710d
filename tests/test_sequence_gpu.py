"""The sequence operators on the GPU against their definitions in 64 bits (seq_reference).

Attention is held to componentwise error bounds that seq_reference derives beside its values:
fp32 sums and statistics, and for bf16 the rounding (2^-8) of the probabilities and their
gradients in the second products, of the stored o and of the results.  The other operators'
tolerances are derived where they stand.
"""
import pytest

import seq_reference as ref
from helpers import TOL, rel_rows

pytestmark = pytest.mark.gpu


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _close(got, want, dtype):
    """The framework's tolerance, relative to |ref| + the rms of the reference."""
    import torch
    g, w = got.double().cpu(), want.double().cpu()
    assert torch.isfinite(g).all()
    assert rel_rows(g.numpy(), w.numpy()) <= TOL[dtype]


def _within(got, want):
    """got inside the error bound of want = (value, bound), -inf where the value is."""
    import torch
    val, err = want
    got = got.double()
    assert torch.equal(torch.isneginf(got), torch.isneginf(val))
    fine = torch.isfinite(val)
    off = (got - val)[fine].abs()
    assert torch.isfinite(off).all() and (off <= err[fine]).all(), float((off / err[fine].clamp(min=1e-300)).max())


def _r(dtype):
    return 2.0 ** -8 if dtype == "bf16" else 0.0   # 8 significant bits


# ---------------------------------------------------------------------------------------- rotary
@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "parts"])
@pytest.mark.parametrize("R,P", [(2, 5), (64, 300), (128, 131072)])
def test_rotary_table(lib, scaling, R, P):
    import torch
    kw = dict(theta=10000.0, scaling=scaling, factor=8.0, context=4096.0)
    got = lib.rotary_table(R, P, **kw).cpu().double()
    rows = torch.unique(torch.cat([torch.arange(min(P, 64)), torch.randint(0, P, (200,)), torch.tensor([P - 1])]))
    want = ref.table(R, P, **kw)[rows]
    # fp64 angles and functions (pow and the angle's rounding: ~1e-10 at 131072 rad), one rounding to fp32
    assert (got[rows] - want).abs().max() <= 1.3 * 2 ** -24 + 1e-8


ROTARY = [  # dtype, B, T, Hq, Hk, D, R
    ("bf16", 2, 33, 4, 2, 64, 64), ("bf16", 3, 1, 12, 12, 64, 64), ("bf16", 2, 5, 3, 1, 128, 64),
    ("bf16", 1, 7, 2, 2, 40, 40), ("bf16", 1, 9, 2, 0, 33, 10), ("bf16", 2, 3, 5, 5, 6, 2),
    ("fp32", 2, 33, 4, 2, 64, 32), ("fp32", 1, 2, 1, 1, 128, 128), ("fp32", 2, 4, 3, 3, 7, 6),
    ("fp32", 1, 300, 2, 2, 80, 80),
]


@pytest.mark.parametrize("dtype,B,T,Hq,Hk,D,R", ROTARY)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary(lib, dtype, B, T, Hq, Hk, D, R, interleaved, inverse):
    import torch
    g = torch.Generator(device="cuda").manual_seed(B * 100 + D)
    P = 5000
    table = lib.rotary_table(R, P, scaling="parts", factor=4.0)
    x = [torch.randn(B, T, h, D, generator=g, device="cuda").to(_dt(dtype)) if h else None for h in (Hq, Hk)]
    for pos in (None, torch.randint(0, P, (B, T), generator=g, device="cuda", dtype=torch.int64),
                torch.randint(0, P, (B, T), generator=g, device="cuda", dtype=torch.int32)):
        out = lib.rotary(x[0], x[1], table, positions=pos, interleaved=interleaved, inverse=inverse)
        at = pos if pos is not None else torch.arange(T, device="cuda").expand(B, T)
        for y, z in zip(out, x):
            if z is None:
                assert y is None
                continue
            want = ref.rotary(z, table, at, interleaved, inverse)
            # two products and a sum in fp32, one rounding to the type
            tol = (2 ** -8 if dtype == "bf16" else 2 ** -22) * (z.double().abs().max() * 2 + 1)
            assert (y.double() - want).abs().max() <= tol
            assert torch.equal(y[..., R:], z[..., R:])
    assert lib.dp_check_status() == lib.DP_OK


def test_rotary_strides_in_place_and_gradient(lib):
    import torch
    B, T, H, D, R = 2, 37, 3, 64, 32
    table = lib.rotary_table(R, 64)
    for dtype in (torch.bfloat16, torch.float32):
        qkv = torch.randn(B, T, 3, H, D, device="cuda").to(dtype)
        q, k = qkv[:, :, 0], qkv[:, :, 1]
        a, b = lib.rotary(q, k, table)
        c, d = lib.rotary(q.contiguous(), k.contiguous(), table)
        assert torch.equal(a, c) and torch.equal(b, d)
        # heads first in memory, and an odd offset into the storage
        hf = torch.randn(B, H, T, D, device="cuda").to(dtype).transpose(1, 2)
        odd = torch.randn(B * T * H * D + 1, device="cuda").to(dtype)[1:].view(B, T, H, D)
        a, b = lib.rotary(hf, odd, table)
        c, d = lib.rotary(hf.contiguous(), odd.clone(), table)
        assert torch.equal(a, c) and torch.equal(b, d)
        # in place through the C entry point
        st = lib.Strides(*q.stride()[:3])
        desc = lib.RotaryDesc(lib.DP_BF16 if dtype == torch.bfloat16 else lib.DP_FP32, B, T, H, H, D, R, 64, 0, 0, 0,
                              st, st, st, st)
        want = lib.rotary(q, k, table)
        v = qkv[:, :, 2].clone()
        lib.dp_rotary(desc, q, k, table, None, q, k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 2], v)
    # gradient: the transpose (<R x, y> = <x, R^T y>), through autograd and an expanded upstream
    q = torch.randn(B, T, H, D, device="cuda", requires_grad=True)
    k = torch.randn(B, T, 1, D, device="cuda", requires_grad=True)
    y, z = lib.rotary(q, k, table, interleaved=True)
    w = torch.randn_like(y)
    ((y * w).sum() + z.sum()).backward()
    back = ref.rotary(w, table, torch.arange(T, device="cuda").expand(B, T), True, True)
    _close(q.grad, back, "fp32")
    one = ref.rotary(torch.ones_like(k), table, torch.arange(T, device="cuda").expand(B, T), True, True)
    _close(k.grad, one, "fp32")


def test_rotary_position_out_of_table(lib):
    import torch
    table = lib.rotary_table(32, 16)
    q = torch.randn(2, 3, 2, 64, device="cuda")
    pos = torch.tensor([[0, 16, 1], [2, -1, 15]], device="cuda", dtype=torch.int32)
    y, _ = lib.rotary(q, None, table, positions=pos)
    assert lib.dp_check_status() == lib.DP_ERR_INVALID_ARG and lib.dp_check_status() == lib.DP_OK
    badrow = (pos < 0) | (pos >= 16)
    assert torch.isnan(y[..., :32][badrow]).all() and torch.isfinite(y[~badrow]).all()
    assert torch.equal(y[..., 32:], q[..., 32:])


def test_rotary_offsets_past_32_bits(lib):
    import torch
    far = (1 << 31) + 64
    base = torch.empty(far + 4 * 64, dtype=torch.bfloat16, device="cuda")
    q = base.as_strided((2, 2, 2, 64), (far, 128, 64, 1))
    q.copy_(torch.randn(2, 2, 2, 64, device="cuda"))
    table = lib.rotary_table(64, 8)
    a, _ = lib.rotary(q, None, table)
    b, _ = lib.rotary(q.contiguous(), None, table)
    assert torch.equal(a, b)


# ---------------------------------------------------------------------------------------- attention
ATTENTION = [  # B, T, S, Hq, Hk, D, causal, window, lengths
    (2, 1, 1, 2, 2, 64, False, 0, None),
    (2, 1, 300, 4, 2, 64, False, 0, None),
    (1, 300, 1, 2, 1, 128, False, 0, None),
    (2, 128, 128, 2, 2, 64, True, 0, None),
    (1, 129, 257, 2, 1, 128, True, 0, None),
    (1, 257, 129, 4, 2, 64, True, 0, None),            # queries before the first key: empty rows
    (3, 197, 197, 3, 3, 64, False, 0, None),
    (2, 400, 400, 4, 1, 128, True, 0, None),
    (2, 333, 333, 2, 2, 40, True, 50, None),
    (1, 600, 600, 1, 1, 128, True, 1, None),
    (1, 500, 700, 2, 2, 64, True, 200, None),
    (4, 150, 150, 2, 1, 64, True, 0, "ragged"),
    (4, 150, 270, 2, 2, 128, False, 0, "ragged"),
    (4, 300, 300, 2, 2, 80, True, 70, "ragged"),
    (5, 40, 260, 6, 2, 96, True, 0, "ragged"),
    (1, 65, 70, 2, 2, 8, False, 0, None),
    (1, 65, 70, 2, 2, 33, True, 0, None),
    (2, 70, 65, 2, 1, 1, False, 0, None),
    (2, 260, 260, 2, 2, 120, False, 0, None),
    # enough heads for two query tiles a CTA, one of them without a key or without a query
    (80, 257, 129, 1, 1, 128, True, 0, None),
    (80, 300, 300, 1, 1, 128, True, 0, "ragged"),
    # short sequences with a key head for every query head: a kernel of their own
    (5, 200, 256, 2, 2, 64, True, 0, "ragged"),
    (4, 256, 130, 3, 3, 48, True, 60, "ragged"),
    (5, 256, 256, 2, 2, 64, False, 0, "ragged"),
    (2, 256, 256, 2, 2, 64, True, 0, None),
    (2, 140, 120, 2, 2, 56, True, 0, None),
    (2, 120, 140, 2, 2, 64, True, 1, None),
    # few heads: the gradient's sums are split over CTAs and joined
    (1, 1500, 1500, 4, 1, 128, True, 0, None),
    (1, 900, 1300, 1, 1, 64, False, 0, None),
    (1, 130, 2000, 2, 1, 128, False, 0, None),
    (1, 1700, 300, 3, 1, 72, True, 200, None),
    (3, 1100, 1100, 2, 1, 64, True, 0, "ragged"),
]


def _attn_inputs(B, T, S, Hq, Hk, D, lengths, dtype, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + T * 7 + S * 3 + D)
    q, k, v, do = (torch.randn(B, n, h, D, generator=g, device="cuda").to(_dt(dtype))
                   for n, h in ((T, Hq), (S, Hk), (S, Hk), (T, Hq)))
    lq = lk = None
    if lengths:
        lq = torch.tensor(([T, 0, 1, T // 2 + 1, T - 1] * B)[:B], dtype=torch.int32, device="cuda")
        lk = torch.tensor(([S - 1, S, 0, S // 3 + 1, 1] * B)[:B], dtype=torch.int32, device="cuda")
    return q, k, v, do, lq, lk


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: "-".join(str(x) for x in c))
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention(lib, case, dtype):
    import torch
    B, T, S, Hq, Hk, D, causal, window, lengths = case
    q, k, v, do, lq, lk = _attn_inputs(B, T, S, Hq, Hk, D, lengths, dtype)
    kw = dict(causal=causal, window=window, q_lens=lq, k_lens=lk)
    o, lse = lib.attention_forward(q, k, v, **kw)
    grads = lib.attention_backward(q, k, v, o, lse, do, **kw)
    wants = ref.attention(q, k, v, do=do, r=_r(dtype), **kw)
    empty = torch.isneginf(wants[1][0])
    assert torch.equal(o.transpose(1, 2)[empty], torch.zeros_like(o.transpose(1, 2)[empty]))
    assert torch.equal(grads[0].transpose(1, 2)[empty], torch.zeros_like(o.transpose(1, 2)[empty]))
    for got, want in zip((o, lse) + grads, wants):
        _within(got, want)
    # the same bits again, and nothing raised on the device
    o2, lse2 = lib.attention_forward(q, k, v, **kw)
    again = lib.attention_backward(q, k, v, o, lse, do, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(a, b) for a, b in zip(grads, again))
    assert lib.dp_check_status() == lib.DP_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3.38e38])
@pytest.mark.parametrize("D,T,S,Hk", [(64, 150, 270, 1), (128, 150, 270, 1), (64, 150, 220, 2)])
def test_attention_padded_rows_may_hold_anything(lib, dtype, junk, D, T, S, Hk):
    import torch
    B, Hq = 5, 2
    q, k, v, do, lq, lk = _attn_inputs(B, T, S, Hq, Hk, D, "ragged", dtype)
    kw = dict(causal=True, q_lens=lq, k_lens=lk)
    clean_o, clean_l = lib.attention_forward(q, k, v, **kw)
    clean = lib.attention_backward(q, k, v, clean_o, clean_l, do, **kw)
    pq = torch.arange(T, device="cuda")[None] >= lq[:, None]
    pk = torch.arange(S, device="cuda")[None] >= lk[:, None]
    for x, m in ((q, pq), (do, pq), (k, pk), (v, pk)):
        x[m] = junk
    o, lse = lib.attention_forward(q, k, v, **kw)
    assert torch.equal(o, clean_o) and torch.equal(lse, clean_l)
    o[pq] = junk
    got = lib.attention_backward(q, k, v, o, lse, do, **kw)
    for a, b, m in zip(got, clean, (pq, pk, pk)):
        assert torch.equal(a, b) and not a[m].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_strides_alignment_and_lengths_out_of_range(lib, dtype):
    import torch
    B, T, H, D = 2, 150, 3, 64
    packed = torch.randn(B, T, 3, H, D, device="cuda").to(_dt(dtype))
    q, k, v = packed.unbind(2)
    want = lib.attention_forward(q.contiguous(), k.contiguous(), v.contiguous(), causal=True)
    got = lib.attention_forward(q, k, v, causal=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    hf = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
    got = lib.attention_forward(*hf, causal=True)
    assert torch.equal(got[0], want[0])
    # a base address off the 16-byte grid, and gradients of such inputs
    odd = [torch.cat([x.reshape(-1)[:1], x.reshape(-1)])[1:].view(B, T, H, D) for x in (q, k, v)]
    got = lib.attention_forward(*odd, causal=True)
    do = torch.randn(B, T, H, D, device="cuda").to(_dt(dtype))
    a = lib.attention_backward(q, k, v, want[0], want[1], do, causal=True)
    b = lib.attention_backward(*odd, want[0], want[1], do.transpose(1, 2).contiguous().transpose(1, 2), causal=True)
    wants = ref.attention(q, k, v, causal=True, do=do, r=_r(dtype))
    for x, w in zip(got + b, wants):
        _within(x, w)
    for x, w in zip(a, wants[2:]):
        _within(x, w)
    # one head expanded over all: strides of 0 on the inputs
    one = torch.randn(B, T, 1, D, device="cuda").to(_dt(dtype)).expand(B, T, H, D)
    got = lib.attention_forward(q, one, one, causal=True)
    _within(got[0], ref.attention(q, one, one, causal=True, r=_r(dtype))[0])
    # lengths outside the tensors are clamped
    low = torch.tensor([-5, T + 9], dtype=torch.int32, device="cuda")
    cut = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    x, y = (lib.attention_forward(q, k, v, q_lens=n, k_lens=n) for n in (low, cut))
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_large_scores_stay_finite(lib, dtype):
    """Scores of several hundred: the running maximum keeps exp in range, in both passes."""
    import torch
    B, T, H, D = 1, 300, 2, 64
    q, k, v, do, _, _ = _attn_inputs(B, T, T, H, H, D, None, dtype)
    q, k = (q * 16).contiguous(), (k * 4).contiguous()
    o, lse = lib.attention_forward(q, k, v, causal=True)
    grads = lib.attention_backward(q, k, v, o, lse, do, causal=True)
    wants = ref.attention(q, k, v, causal=True, do=do, r=_r(dtype))
    assert wants[1][0].max() > 100
    for got, want in zip((o, lse) + grads, wants):
        _within(got, want)


def test_attention_one_bad_example_stays_alone(lib):
    import torch
    q, k, v, do, _, _ = _attn_inputs(3, 200, 200, 2, 2, 64, None, "bf16")
    kw = dict(causal=True)
    o, lse = lib.attention_forward(q, k, v, **kw)
    g = lib.attention_backward(q, k, v, o, lse, do, **kw)
    q2, v2 = q.clone(), v.clone()
    q2[1], v2[1] = float("nan"), float("inf")
    o2, lse2 = lib.attention_forward(q2, k, v2, **kw)
    g2 = lib.attention_backward(q2, k, v2, o2, lse2, do, **kw)
    keep = [0, 2]
    assert not torch.isfinite(o2[1]).any()
    for a, b in zip((o, lse) + g, (o2, lse2) + g2):
        assert torch.equal(a[keep], b[keep])


def test_attention_gradient_against_differences(lib):
    """<grad, d> against the central difference of f = <o, w> along d, fp32: the truncation is
    h^2 |f'''| / 6 ~ 1e-5 |f| at h = 1e-2 and the rounding of f about 1e-6 |f| / h = 1e-4."""
    import torch
    B, T, S, Hq, Hk, D = 2, 70, 90, 4, 2, 32
    q, k, v, w, _, _ = _attn_inputs(B, T, S, Hq, Hk, D, None, "fp32")
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    (lib.attention(*leaves, causal=True, window=40) * w).sum().backward()
    g = torch.Generator(device="cuda").manual_seed(3)
    for i in range(3):
        d = torch.randn(leaves[i].shape, generator=g, device="cuda")
        f = []
        for h in (1e-2, -1e-2):
            x = [q, k, v]
            x[i] = x[i] + h * d
            f.append((lib.attention_forward(*x, causal=True, window=40)[0].double() * w.double()).sum().item())
        slope = (f[0] - f[1]) / 2e-2
        size = leaves[i].grad.double().norm().item()
        assert abs(slope - (leaves[i].grad.double() * d.double()).sum().item()) <= 2e-3 * size


def test_attention_stream_graph_and_empty(lib):
    import torch
    q, k, v, do, _, _ = _attn_inputs(2, 200, 200, 2, 2, 64, None, "bf16")
    o, lse = lib.attention_forward(q, k, v, causal=True)
    want = lib.attention_backward(q, k, v, o, lse, do, causal=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o2, lse2 = lib.attention_forward(q, k, v, causal=True)
        got = lib.attention_backward(q, k, v, o2, lse2, do, causal=True)
    side.synchronize()
    assert torch.equal(o, o2) and all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = lib.attention_forward(q, k, v, causal=True)
        got3 = lib.attention_backward(q, k, v, o3, lse3, do, causal=True)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    o4, lse4 = lib.attention_forward(q, k, v, causal=True)
    want4 = lib.attention_backward(q, k, v, o4, lse4, do, causal=True)
    assert torch.equal(o3, o4) and all(torch.equal(a, b) for a, b in zip(want4, got3))
    # no keys, no queries, no examples
    o, lse = lib.attention_forward(q, k[:, :0], v[:, :0])
    assert not o.any() and torch.isneginf(lse).all()
    dq, dk, dv = lib.attention_backward(q, k[:, :0], v[:, :0], o, lse, do)
    assert not dq.any() and dk.numel() == 0
    o, lse = lib.attention_forward(q[:, :0], k, v)
    assert lib.attention_backward(q[:, :0], k, v, o, lse, do[:, :0])[1].eq(0).all()
    assert lib.attention_forward(q[:0], k[:0], v[:0])[0].shape == (0, 200, 2, 64)


@pytest.mark.parametrize("D,T,H", [(64, 197, 24), (64, 500, 16), (128, 400, 16)])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_passes_back_to_back(lib, D, T, H, causal):
    """Many passes with nothing between them (a kernel's first CTAs start under the last of the
    one before): no wait gives up, and the last pass has the first one's bits."""
    import torch
    q, k, v, do, _, _ = _attn_inputs(16, T, T, H, H, D, None, "bf16")

    def one():
        o, lse = lib.attention_forward(q, k, v, causal=causal)
        return (o, lse) + lib.attention_backward(q, k, v, o, lse, do, causal=causal)

    want = one()
    torch.cuda.synchronize()
    assert lib.dp_check_status() == lib.DP_OK
    for _ in range(60):
        got = one()
    torch.cuda.synchronize()
    assert lib.dp_check_status() == lib.DP_OK
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_offsets_past_32_bits(lib, D):
    import torch
    T, far = 130, (1 << 31) + 64
    base = torch.empty(far + T * D, dtype=torch.bfloat16, device="cuda")
    far_view = base.as_strided((2, T, 1, D), (far, D, D, 1))
    far_view.copy_(torch.randn(2, T, 1, D, device="cuda"))
    near = far_view.contiguous()
    do = torch.randn_like(near)
    a, la = lib.attention_forward(far_view, far_view, far_view, causal=True)
    b, lb = lib.attention_forward(near, near, near, causal=True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    ga = lib.attention_backward(far_view, far_view, far_view, a, la, do, causal=True)
    gb = lib.attention_backward(near, near, near, a, la, do, causal=True)
    assert all(torch.equal(x, y) for x, y in zip(ga, gb))


# ---------------------------------------------------------------------------------------- distillation
DISTILL = [  # dtype, B, T, V, K, tau, alpha
    ("fp32", 2, 3, 17, 4, 1.0, 0.0), ("fp32", 2, 3, 1000, 16, 2.0, 0.5), ("bf16", 2, 5, 1001, 8, 1.0, 0.0),
    ("bf16", 1, 4, 50257, 32, 2.0, 0.3), ("bf16", 3, 1, 32000, 1, 4.0, 0.0), ("fp32", 1, 2, 70001, 100, 1.0, 1.0),
    ("bf16", 1, 2, 131072, 64, 0.5, 0.1), ("bf16", 1, 2, 300001, 128, 1.0, 0.0), ("fp32", 1, 2, 200000, 5, 1.0, 0.25),
    ("bf16", 2, 2, 1, 1, 1.0, 0.5), ("bf16", 1, 3, 7, 0, 1.0, 1.0), ("fp32", 1, 2, 5000, 1024, 3.0, 0.0),
    ("bf16", 1, 2, 8, 3, 1.0, 0.0), ("bf16", 1, 2, 700001, 9, 1.0, 0.4),
]


def _distill_inputs(dtype, B, T, V, K, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + V)
    z = (torch.randn(B, T, V, generator=g, device="cuda") * 3).to(_dt(dtype))
    idx = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(B * T)]).view(B, T, K) \
        if K <= V else torch.randint(0, V, (B, T, K), generator=g, device="cuda")
    t = (torch.randn(B, T, K, generator=g, device="cuda") * 2 + 5).to(_dt(dtype))
    y = torch.randint(0, V, (B, T), generator=g, device="cuda")
    return z, idx, t, y


# the loss: fp32 sums of up to 7e5 exponentials, 1e-6 relative, against a loss of order 1;
# the gradient in bf16 is rounded once (2^-9), in fp32 it is within a few 1e-7 of its entry.
L_TOL, G_TOL = 1e-5, {"fp32": 1e-5, "bf16": 2 ** -8}


def _distill_close(got, want, dtype, terms=0.0):
    """terms: the size of the gradient's terms where they may cancel to nothing (q - p with q = p)."""
    import torch
    loss, grad = got
    wl, _, wg = want
    assert ((loss.double() - wl).abs() <= L_TOL * (1 + wl.abs())).all()
    if grad is not None:
        big = wg.abs().amax(-1, keepdim=True).clamp(min=terms)
        assert torch.isfinite(grad).all()
        assert ((grad.double() - wg).abs() <= G_TOL[dtype] * wg.abs() + 1e-6 * big + 1e-38).all()


@pytest.mark.parametrize("dtype,B,T,V,K,tau,alpha", DISTILL)
def test_distill(lib, dtype, B, T, V, K, tau, alpha):
    import torch
    z, idx, t, y = _distill_inputs(dtype, B, T, V, K)
    up = torch.linspace(0.5, 2.0, B, device="cuda")
    w = torch.rand(B, T, device="cuda") + 0.5
    want = ref.distill(z, idx, t, y, w, up, tau, alpha)
    kw = dict(labels=y, weights=w, temperature=tau, alpha=alpha)
    for i in (idx, idx.to(torch.int32)):
        _distill_close(lib.distill_loss_and_grad(z, i, t, upstream=up, **kw), want, dtype)
    loss, rows = lib.distill_loss(z, idx, t, **kw)
    _distill_close((loss, None), want, dtype)
    assert ((rows.double() - want[1]).abs() <= L_TOL * (1 + want[1].abs())).all()
    leaf = z.clone().requires_grad_()
    loss, _ = lib.distill_loss(leaf, idx, t, **kw)
    (loss * up).sum().backward()
    _distill_close((loss.detach(), leaf.grad), want, dtype)
    assert lib.dp_check_status() == lib.DP_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [50, 4099, 140001])
def test_distill_missing_masked_and_repeated(lib, dtype, V):
    import torch
    B, T, K = 4, 2, 6
    z, idx, t, y = _distill_inputs(dtype, B, T, V, K)
    idx[0, 0, 2:] = -1                 # fewer entries
    idx[0, 1] = -1                     # no teacher: the label alone
    y[1, 0] = -100                     # no label: the teacher alone
    idx[1, 1], y[1, 1] = -1, -100      # neither
    idx[2, 0, 3] = idx[2, 0, 1]        # an entry twice
    y[2, 0] = idx[2, 0, 1]             # and it is the label
    t[2, 1, 4] = -float("inf")         # an entry of no probability ...
    z[2, 1, idx[2, 1, 4]] = -float("inf")   # ... that the student rules out
    y[2, 1] = idx[2, 1, 0]
    rest = torch.ones(V, dtype=torch.bool, device="cuda")
    rest[idx[3, 0]], rest[y[3, 0]] = False, False
    z[3, 0, rest] = torch.finfo(z.dtype).min   # the type's lowest value as a mask
    w = torch.ones(B, T, device="cuda")
    w[3, 1] = 0.0
    want = ref.distill(z, idx, t, y, w, None, 2.0, 0.25)
    z[3, 1] = float("nan")             # a row of weight 0 is not read
    got = lib.distill_loss_and_grad(z, idx, t, labels=y, weights=w, temperature=2.0, alpha=0.25)
    _distill_close(got, want, dtype)
    assert not got[1][1, 1].any() and not got[1][3, 1].any()
    again = lib.distill_loss_and_grad(z, idx, t, labels=y, weights=w, temperature=2.0, alpha=0.25)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    assert lib.dp_check_status() == lib.DP_OK


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0, 3.0])
def test_distill_rows_of_masks(lib, dtype, tau):
    """Nothing but the type's lowest value (a uniform softmax), all but one entry, and -inf
    instead of it; over a few chunks of a row, so that some threads see masks alone."""
    import torch
    V = 20011
    z, idx, t, y = _distill_inputs(dtype, 2, 3, V, 4)
    low = torch.finfo(z.dtype).min
    z[0, 0], z[0, 1], z[0, 2], z[1, 0] = low, low, -float("inf"), low
    z[0, 1, idx[0, 1, 0]] = z[0, 2, idx[0, 2, 0]] = 3.0
    z[1, 0, ::2] = -float("inf")
    t[0, 1, 1:] = t[0, 2, 1:] = -float("inf")
    idx[1, 0] = torch.tensor([1, 3, 5, 7], device="cuda")
    y[0, 1], y[0, 2], y[1, 0] = idx[0, 1, 0], idx[0, 2, 0], 9
    kw = dict(labels=y, temperature=tau, alpha=0.25)
    want = ref.distill(z, idx, t, y, None, None, tau, 0.25)
    # a softmax of one entry: q and p are both 1
    _distill_close(lib.distill_loss_and_grad(z, idx, t, **kw), want, dtype, terms=tau)
    want = ref.distill(z, idx, t, None, None, None, tau, 0.0)
    _distill_close(lib.distill_loss_and_grad(z, idx, t, temperature=tau), want, dtype, terms=tau)


def test_distill_index_out_of_vocabulary(lib):
    import torch
    z, idx, t, y = _distill_inputs("fp32", 3, 2, 100, 4)
    idx[0, 1, 2], y[2, 0] = 100, 1 << 20
    loss, rows = lib.distill_loss(z, idx, t, labels=y, alpha=0.5)
    assert lib.dp_check_status() == lib.DP_ERR_INVALID_ARG and lib.dp_check_status() == lib.DP_OK
    assert torch.equal(torch.isnan(rows), torch.tensor([[False, True], [False, False], [True, False]], device="cuda"))
    assert torch.isfinite(loss[1]) and not torch.isfinite(loss[[0, 2]]).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_distill_row_strides_and_offsets_past_32_bits(lib, dtype):
    import torch
    B, T, V, K = 2, 3, 1000, 5
    z, idx, t, y = _distill_inputs(dtype, B, T, V, K)
    want = lib.distill_loss_and_grad(z, idx, t, labels=y, alpha=0.5)
    for ld in (1001, 1016):            # rows off the 16-byte grid, and padded rows
        wide = torch.full((B, T, ld), 99.0, device="cuda").to(_dt(dtype))
        wide[..., :V] = z
        got = lib.distill_loss_and_grad(wide[..., :V], idx, t, labels=y, alpha=0.5)
        _close(got[0], want[0], "fp32")
        _close(got[1], want[1], "bf16" if dtype == "bf16" else "fp32")
    far = (1 << 31) + 8
    base = torch.empty(far + V, dtype=_dt(dtype), device="cuda")
    v = base.as_strided((2, 1, V), (far, far, 1))
    v.copy_(z[:, :1])
    a = lib.distill_loss_and_grad(v, idx[:, :1].contiguous(), t[:, :1].contiguous())
    b = lib.distill_loss_and_grad(z[:, :1].contiguous(), idx[:, :1].contiguous(), t[:, :1].contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_distill_gradient_against_differences(lib):
    """Central differences of the fp32 loss along a direction: truncation h^2/6 and rounding
    1e-6/h relative to the slope's scale, both below 1e-3 at h = 1e-2."""
    import torch
    z, idx, t, y = _distill_inputs("fp32", 3, 4, 300, 8)
    kw = dict(labels=y, temperature=2.0, alpha=0.3)
    _, grad = lib.distill_loss_and_grad(z, idx, t, **kw)
    d = torch.randn_like(z)
    f = [lib.distill_loss(z + h * d, idx, t, **kw)[0].double().sum().item() for h in (1e-2, -1e-2)]
    assert abs((f[0] - f[1]) / 2e-2 - (grad.double() * d.double()).sum().item()) <= 3e-3 * grad.double().norm().item()


@pytest.mark.parametrize("D", [64, 128])
def test_another_stream_owns_what_a_call_allocates(lib, D):
    """stream=: while the side stream's work still waits, the caller's stream reuses freed memory.
    The gradient's workspace must not be among it: the late kernels would write over new tensors."""
    import torch
    q, k, v, do, _, _ = _attn_inputs(2, 300, 300, 2, 2, D, None, "bf16")
    z, idx, t, y = _distill_inputs("bf16", 2, 5, 1001, 8)
    table = lib.rotary_table(D, 300)
    want = (lib.attention_forward(q, k, v, causal=True) + lib.rotary(q, k, table) +
            lib.distill_loss_and_grad(z, idx, t, labels=y, alpha=0.5))
    want += lib.attention_backward(q, k, v, *want[:2], do, causal=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for s in (side, side.cuda_stream):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)   # some 10 ms ahead of the calls
        got = (lib.attention_forward(q, k, v, causal=True, stream=s) + lib.rotary(q, k, table, stream=s) +
               lib.distill_loss_and_grad(z, idx, t, labels=y, alpha=0.5, stream=s))
        got += lib.attention_backward(q, k, v, *got[:2], do, causal=True, stream=s)
        new = [torch.full((n,), 7.0, device="cuda") for n in (600, 1200, 2400, 5000, 20000, 1 << 20) for _ in range(8)]
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(x.eq(7).all() for x in new)
    own = lib.rotary_table(D, 300, stream=side)
    side.synchronize()
    assert torch.equal(own, table)


@pytest.mark.parametrize("mode", ["GHOST", "INSTANTIATE"])
def test_clipped_path_right_behind_an_operator(lib, mode):
    """What an operator has just written is the A or G of the next call: the kernels that may load
    their inputs early must not load these, nor may the ones behind them.  Every operator's output
    lies where zeros lay before, and the norms must be those of a run that waits in between.  (312
    rows: a few CTAs write a second one while the others' SMs are free for the next kernel.)"""
    import torch
    B, T, V, d, H, D = 3, 104, 65536, 64, 8, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(B, T, V, generator=g, device="cuda").bfloat16()
    idx = torch.randint(0, V, (B, T, 16), generator=g, device="cuda", dtype=torch.int32)
    top = torch.randn(B, T, 16, generator=g, device="cuda").bfloat16()
    q, k, v = (torch.randn(B, T, H, D, generator=g, device="cuda").bfloat16() for _ in range(3))
    A = torch.randn(B, T, d, generator=g, device="cuda").bfloat16()
    small = torch.randn(B, T, 64, generator=g, device="cuda").bfloat16()
    mode = getattr(lib, "DP_NORM_" + mode)
    head = lib.layer_desc(lib.DP_LINEAR, lib.DP_BF16, B=B, p=V, T=T, d=d)
    other = lib.layer_desc(lib.DP_LINEAR, lib.DP_BF16, B=B, p=64, T=T, d=H * D)
    ws = [torch.empty(lib.dp_workspace_size(x, mode), dtype=torch.uint8, device="cuda") for x in (head, other)]
    sq = torch.empty(3, B, device="cuda")

    def zeros_then(f, *shapes):
        old = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in shapes]
        torch.cuda.synchronize()
        del old   # the operator's outputs take this memory
        torch.cuda._sleep(2_000_000)   # about 1 ms: everything is queued before any of it runs
        return f()

    def run(wait, between):
        sq.zero_()
        o = zeros_then(lambda: lib.attention_forward(q, k, v)[0], q.shape)
        if wait:
            torch.cuda.synchronize()
        lib.dp_layer_sqnorms(other, o, small, sq[0], ws[1], mode=mode)
        torch.cuda.synchronize()
        dz = zeros_then(lambda: lib.distill_loss_and_grad(z, idx, top)[1], z.shape)
        if wait:
            torch.cuda.synchronize()
        if between:
            lib.dp_layer_sqnorms(other, o, small, sq[1], ws[1], mode=mode)   # lets the next one start
        lib.dp_layer_sqnorms(head, A, dz, sq[2], ws[0], mode=mode)
        torch.cuda.synchronize()
        return sq.clone()

    for between in (False, True):
        want = run(True, between)
        assert (want[[0, 1, 2] if between else [0, 2]] > 0).all()
        for _ in range(5):
            assert torch.equal(run(False, between), want)


def test_no_second_derivative(lib):
    """The gradients are not differentiable themselves: asking for it is an error, not a zero."""
    import torch
    q, k, v, _, _, _ = _attn_inputs(1, 8, 8, 1, 1, 64, None, "fp32")
    z, idx, t, _ = _distill_inputs("fp32", 1, 3, 17, 4)
    leaves = [x.requires_grad_() for x in (q, k, v, z)]
    table = lib.rotary_table(64, 8)
    for out, x in ((lib.attention(*leaves[:3]), q), (lib.rotary(q, k, table)[0], q), (lib.distill_loss(z, idx, t)[0], z)):
        (g,) = torch.autograd.grad(out.square().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.sum(), x)


def test_operators_refuse_on_the_host(lib):
    """What the binding refuses: nothing is launched."""
    import torch
    n = lib.dp_launch_count()
    q = torch.randn(2, 8, 4, 64, device="cuda")
    k = torch.randn(2, 8, 2, 64, device="cuda")
    bad = [
        lambda: lib.attention_forward(q, k, k.bfloat16()), lambda: lib.attention_forward(q.half(), k.half(), k.half()),
        lambda: lib.attention_forward(q[0], k, k), lambda: lib.attention_forward(q, k[:1], k[:1]),
        lambda: lib.attention_forward(q.transpose(2, 3), k, k), lambda: lib.attention_forward(q, k, k[:, :4]),
        lambda: lib.attention_forward(q, k, k, q_lens=torch.zeros(2, device="cuda")),
        lambda: lib.attention_forward(q, k, k, q_lens=torch.zeros(3, dtype=torch.int32, device="cuda")),
        lambda: lib.rotary(q, k, torch.zeros(8, 64)), lambda: lib.rotary(q, k[:, :4], torch.zeros(8, 64, device="cuda")),
        lambda: lib.rotary_table(64, 8, scaling="other"), lambda: lib.rotary_table(64, 0),
        lambda: lib.distill_loss(q, q, q), lambda: lib.distill_loss(q[:, 0].half(), q[:, 0].int(), q[:, 0]),
        lambda: lib.distill_loss(q[:, 0], q[:, 0].float(), q[:, 0]),
        lambda: lib.distill_loss(q[:, 0].transpose(1, 2), q[:, 0].int(), q[:, 0]),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    three = torch.randn(2, 8, 3, 64, device="cuda")
    refused = [
        lambda: lib.attention_forward(q, three, three),                                    # 4 heads over 3
        lambda: lib.attention_forward(q, k, k, window=3),                                  # a window without causal
        lambda: lib.attention_forward(q, k, k, scale=float("inf")),
        lambda: lib.attention_forward(*(torch.randn(1, 4, 1, 136, device="cuda"),) * 3),   # too wide
        lambda: lib.rotary_table(63, 8), lambda: lib.rotary_table(64, 8, scaling="linear", factor=0.5),
        lambda: lib.rotary(q, k, torch.zeros(8, 66, device="cuda")),
        lambda: lib.rotary(q, k, torch.zeros(4, 64, device="cuda")),                       # T > P without positions
        lambda: lib.distill_loss(q[:, 0].contiguous(), k[:, :4, 0, :2].int().contiguous(),
                                 k[:, :4, 0, :2].contiguous(), temperature=0.0),
        lambda: lib.distill_loss(q[:, 0].contiguous(), k[:, :4, 0, :2].int().contiguous(),
                                 k[:, :4, 0, :2].contiguous(), alpha=1.5),
    ]
    for f in refused:
        with pytest.raises(lib.DPError):
            f()
    assert lib.dp_launch_count() == n
