"""Clipped sums and norms of linear layers whose rows do not lie on 128-byte lines (d = 1000): many examples
a CTA, several column tiles with a narrow last one.  All of dW and db against 64 bits, the same bits in
every call, and no wait that gave up."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,p,d", [(64, 64, 1536, 1000), (64, 128, 1536, 1000), (64, 197, 768, 1000),
                                     (300, 197, 768, 1000), (200, 64, 1536, 712), (300, 100, 1000, 1288)])
@pytest.mark.parametrize("bias", [True, False])
def test_rows_off_the_lines(lib, B, T, p, d, bias):
    import torch
    g = torch.Generator(device="cuda").manual_seed(B + T + d)
    A = torch.randn(B, T, d, generator=g, device="cuda").bfloat16()
    G = (torch.randn(B, T, p, generator=g, device="cuda") * 0.1).bfloat16()
    f = torch.rand(B, generator=g, device="cuda")
    layer = lib.layer_desc(lib.DP_LINEAR, lib.DP_BF16, B=B, p=p, T=T, d=d, has_bias=bias)
    want, wb, norms = torch.zeros(p, d, dtype=torch.float64, device="cuda"), torch.zeros(p, device="cuda").double(), []
    size, sb = want.clone(), wb.clone()    # sums of the terms' sizes
    for i in range(B):
        P, b = G[i].double().T @ A[i].double(), G[i].double().sum(0)
        want, wb = want + f[i].double() * P, wb + f[i].double() * b
        size += f[i].double() * (G[i].double().abs().T @ A[i].double().abs())
        sb += f[i].double() * G[i].double().abs().sum(0)
        norms.append((P.square().sum() + (b.square().sum() if bias else 0)).item())
    norms = torch.tensor(norms, dtype=torch.float64, device="cuda")
    for mode in (lib.DP_NORM_GHOST, lib.DP_NORM_INSTANTIATE):
        ws = torch.empty(lib.dp_workspace_size(layer, mode), dtype=torch.uint8, device="cuda")
        first = None
        for _ in range(6):
            sq, dW = torch.full((B,), float("nan"), device="cuda"), torch.full((p, d), float("nan"), device="cuda")
            db = torch.full((p,), float("nan"), device="cuda") if bias else None
            lib.dp_layer_sqnorms(layer, A, G, sq, ws, mode=mode)
            lib.dp_clipped_sum(layer, A, G, f, dW, db, ws)
            got = [sq, dW] + ([db] if bias else [])
            assert lib.dp_check_status() == lib.DP_OK
            if first is None:
                first = got
                # products of bf16 are exact in fp32; sums of B T of them, any order, are off by at most
                # B T 2^-24 of their sizes, typically by its root
                tol = (B * T) ** 0.5 * 4 * 2.0 ** -24
                assert ((dW.double() - want).abs() <= tol * size).all()
                assert not bias or ((db.double() - wb).abs() <= tol * sb).all()
                assert ((sq.double() - norms).abs() <= 2e-3 * norms).all()
            assert all(torch.equal(a, b) for a, b in zip(first, got))
