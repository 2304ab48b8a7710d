"""Output gradients and statistics of other shapes than their tensors, whose sizes would fit, are refused."""
import pytest
import torch


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request):   # on the CPU the shape is what is refused first
    if request.param == "cuda":
        request.getfixturevalue("lib")
    return request.param


def _lists(device, *shapes):
    return [torch.zeros(s, device=device) for s in shapes]


@pytest.mark.parametrize("dy,mean,rstd,what", [
    ((2, 4, 3, 8), (2, 3, 4), (2, 3, 4), "dy"), ((2, 2, 6, 8), (2, 3, 4), (2, 3, 4), "dy"), ((4, 3, 2, 8), (2, 3, 4), (2, 3, 4), "dy"),
    ((2, 3, 4, 8), (2, 4, 3), (2, 3, 4), "mean"), ((2, 3, 4, 8), (2, 3, 4), (4, 3, 2), "rstd"),
    ((2, 3, 4, 8), (2, 3, 4, 1), (2, 3, 4), "mean"), ((2, 3, 4, 8), (25,), (2, 3, 4), "mean"),
    ((2, 3, 4, 8), (2, 3, 4), (), "rstd")])
def test_layer_norm(monkeypatch, device, dy, mean, rstd, what):
    import example_gradient_clipping_gb300 as dp
    import example_gradient_clipping_gb300.layers as layers
    if device == "cpu":
        monkeypatch.setattr(layers, "_rows3", lambda x, name: x.flatten(1, -2))
    x, g, m, r = _lists(device, (2, 3, 4, 8), dy, mean, rstd)
    with pytest.raises(ValueError, match=what):
        dp.layer_norm_backward(g, x, None, m, r)


@pytest.mark.parametrize("tokens,dy", [((2, 3, 4), (2, 4, 3, 8)), ((2, 3, 4), (2, 12, 1, 8)), ((2, 3, 4), (4, 3, 2, 8)),
                                       ((6,), (5, 8)), ((2, 6, 1, 2), (2, 1, 6, 2, 8))])
def test_embedding(monkeypatch, device, tokens, dy):
    import example_gradient_clipping_gb300 as dp
    import example_gradient_clipping_gb300.layers as layers
    if device == "cpu":
        monkeypatch.setattr(layers, "_rows3", lambda x, name: pytest.fail("taken"))
    t, g = torch.zeros(tokens, dtype=torch.int32, device=device), torch.zeros(dy, device=device)
    for f in (dp.embedding_backward, dp.embedding_sqnorms):
        with pytest.raises(ValueError, match="does not fit"):
            f(t, g, 10)


@pytest.mark.gpu
def test_the_shapes_that_fit(lib):
    g = torch.Generator(device="cuda").manual_seed(0)
    x, dy = (torch.randn(2, 3, 4, 8, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd = lib.layer_norm_forward(x)
    assert mean.shape == rstd.shape == (2, 3, 4)
    want = lib.layer_norm_backward(dy, x, None, mean, rstd)
    flat = lib.layer_norm_backward(dy.view(2, 12, 8), x.view(2, 12, 8), None, mean.view(2, 12), rstd.view(24))
    for m, r in ((mean.view(2, 12), rstd), (mean.view(24), rstd.view(2, 12))):
        got = lib.layer_norm_backward(dy, x, None, m, r)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a.view(b.shape), b) for a, b in zip(flat, want))
    got = lib.layer_norm_backward(dy.view(2, 12, 8), x, None, mean, rstd)   # one row after another, as x
    assert got[0].shape == x.shape and all(torch.equal(a, b) for a, b in zip(got, want))
    one = lib.layer_norm_backward(dy[:, 0, 0], x[:, 0, 0], None, mean[:, 0, 0].contiguous(), rstd[:, 0, 0].contiguous())
    assert torch.equal(one[0], want[0][:, 0, 0])
    t = torch.randint(0, 10, (2, 3, 4), generator=g, device="cuda")
    assert torch.equal(lib.embedding_backward(t, dy, 10), lib.embedding_backward(t, dy.view(2, 12, 8), 10))
    assert lib.embedding_backward(t[:, 0, 0].contiguous(), dy[:, 0, 0], 10).shape == (10, 8)
