"""A step whose grad, sqnorms or factors a caller has replaced by buffers of its own works in those."""
import numpy as np
import pytest
import torch

from host_library import STREAM, Host

NAMES = {  # C entry of the step: where its calls here say which buffers they use (positional arguments)
    "dp_example_sqnorms": {"sqnorms": 3}, "dp_embedding_sqnorms": {"sqnorms": 3}, "dp_layer_sqnorms": {"sqnorms": 3},
    "dp_clip_factors": {"sqnorms": 0, "factors": 5}, "dp_example_sum": {"factors": 3, "grad": 4},
    "dp_embedding_grad": {"factors": 3, "grad": 4}, "dp_clipped_sum": {"factors": 3, "grad": 4},
    "dp_clipped_sum_noised": {"factors": 3, "grad": 4}, "dp_add_noise": {"grad": 0}, "dp_add_noise_blocks": {"grad": 0},
}


@pytest.fixture(scope="module")
def host():
    return Host()


def _descs(dp):
    return [dp.embedding_desc(dp.DP_FP32, B=4, T=3, V=10, D=8), dp.kept_desc(B=4, p=8, has_bias=True),
            dp.layer_desc(dp.DP_LINEAR, dp.DP_FP32, B=4, p=6, T=3, d=8)]


@pytest.mark.parametrize("per_layer", [False, True])
@pytest.mark.parametrize("fuse", [False, True])
def test_replaced_buffers_are_the_ones_used(host, monkeypatch, per_layer, fuse):
    import example_gradient_clipping_gb300.step as module
    used = {"grad": [], "sqnorms": [], "factors": []}

    def recorded(name, where):
        real = getattr(module, name)

        def call(*a, **kw):
            for what, i in where.items():
                used[what].append(a[i] if isinstance(a[i], int) else a[i].data_ptr())
            return real(*a, **kw)
        return call
    for name, where in NAMES.items():
        monkeypatch.setattr(module, name, recorded(name, where))
    with host.installed():
        step = host.dp.ClipStep(_descs(host.dp), C=1.0, sigma=0.5, per_layer=per_layer, device="cpu", fuse_noise=fuse)
        step.grad, step.sqnorms, step.factors = (torch.empty_like(x) for x in (step.grad, step.sqnorms, step.factors))
        x = torch.zeros(4, 3, 8)
        inputs = [(torch.zeros(4, 3, dtype=torch.int32), x), (torch.zeros(4, 16), None), (x, torch.zeros(4, 3, 6))]
        assert step.run(inputs, seed=1, stream=STREAM) is step.grad
        # all of a layer's, one after another
        L = [0, 1, 2]
        assert used["sqnorms"][:3] == [step.sqnorms[l].data_ptr() for l in L]
        assert used["factors"][1:] == [step.factors[l if per_layer else 0].data_ptr() for l in L]
        assert used["grad"][:3] == [step.layer_views(l)[0].data_ptr() for l in L]
    for what, at in used.items():
        t = getattr(step, what)
        ends = t.data_ptr(), t.data_ptr() + t.numel() * 4
        assert at and all(ends[0] <= p < ends[1] for p in at), what
    assert step.layer_views(1)[1].data_ptr() == step.grad.data_ptr() + (80 + 8) * 4


@pytest.mark.gpu
@pytest.mark.parametrize("per_layer", [False, True])
def test_a_step_on_a_buffer_of_the_callers(lib, per_layer):
    g = torch.Generator(device="cuda").manual_seed(0)
    x, dy = torch.randn(4, 3, 8, generator=g, device="cuda"), torch.randn(4, 3, 8, generator=g, device="cuda")
    tokens = torch.randint(0, 10, (4, 3), generator=g, device="cuda", dtype=torch.int32)
    inputs = [(tokens, dy), (torch.randn(4, 16, generator=g, device="cuda"), None),
              (x, torch.randn(4, 3, 6, generator=g, device="cuda"))]
    want, step = (lib.ClipStep(_descs(lib), C=0.7, sigma=0.5, per_layer=per_layer) for _ in range(2))
    flat = torch.full((step.n_params + 8,), 7.0, device="cuda")   # a slice of a larger one
    step.grad, step.factors, step.sqnorms = flat[4:-4], torch.empty_like(step.factors), torch.empty_like(step.sqnorms)
    got = step.run(inputs, seed=3)
    assert got.data_ptr() == flat.data_ptr() + 16
    assert torch.equal(got, want.run(inputs, seed=3)) and torch.equal(step.factors, want.factors)
    assert (flat[:4] == 7).all() and (flat[-4:] == 7).all()
    np.testing.assert_array_equal(step.sqnorms.cpu().numpy(), want.sqnorms.cpu().numpy())
