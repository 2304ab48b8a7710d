"""A step's embeddings and kept gradients refuse tensors that are not of their descriptor's type or size, which the
kernels would read past; on a stand-in for the CUDA runtime."""
import pytest
import torch

from host_library import PTR, STREAM, Host

B, T, V, D = 4, 3, 10, 8


@pytest.fixture()
def fake():
    host = Host()
    with host.installed():
        yield host


def _inputs(**kw):
    x = dict(tokens=torch.zeros(B, T, dtype=torch.int32), dy=torch.zeros(B, T, D), each=torch.zeros(B, 2 * D))
    x.update(kw)
    return [(x["tokens"], x["dy"]), (x["each"], None)]


def _descs(dp, i64=False, dtype=1):
    return [dp.embedding_desc(dtype, B=B, T=T, V=V, D=D, index_i64=i64), dp.kept_desc(B=B, p=D, has_bias=True)]


WRONG = [(dict(tokens=torch.zeros(B, T, dtype=torch.int64)), "tokens"), (dict(tokens=torch.zeros(B, T - 1, dtype=torch.int32)), "tokens"),
         (dict(tokens=torch.zeros(T, B, dtype=torch.int32).t()), "tokens"), (dict(dy=torch.zeros(B, T, D).bfloat16()), "output gradient"),
         (dict(dy=torch.zeros(B, T, D - 1)), "output gradient"), (dict(dy=torch.zeros(B, D, T).transpose(1, 2)), "output gradient"),
         (dict(each=torch.zeros(B, D)), "gradients"), (dict(each=torch.zeros(B, 2 * D).double()), "gradients")]


@pytest.mark.parametrize("kw,what", WRONG)
def test_inputs_that_do_not_fit(fake, kw, what):
    dp = fake.dp
    step, virtual = dp.ClipStep(_descs(dp), C=1.0, sigma=1.0, device="cpu"), dp.VirtualStep(_descs(dp), C=1.0, sigma=1.0, device="cpu")
    for call in (lambda: step.norms(_inputs(**kw), STREAM), lambda: virtual.add(_inputs(**kw), B, STREAM)):
        with pytest.raises(ValueError, match=what):
            call()


def test_inputs_that_fit(fake):
    dp = fake.dp
    step = dp.ClipStep(_descs(dp), C=1.0, sigma=1.0, device="cpu")
    step.norms(_inputs(), STREAM)
    step.norms(_inputs(tokens=torch.zeros(B + 1, T, dtype=torch.int32)), STREAM)   # a larger buffer
    step.norms([(PTR, PTR), (PTR, None)], STREAM)                                  # addresses are the caller's
    dp.ClipStep(_descs(dp, True, 0), C=1.0, sigma=1.0, device="cpu").norms(
        _inputs(tokens=torch.zeros(B, T, dtype=torch.int64), dy=torch.zeros(B, T, D).bfloat16()), STREAM)
    strided = _descs(dp)                                                           # a descriptor of other strides
    strided[0].dy = dp.RowStrides(D, B * D)
    dp.ClipStep(strided, C=1.0, sigma=1.0, device="cpu").norms(_inputs(dy=torch.zeros(T, B, D).transpose(0, 1)), STREAM)
    virtual = dp.VirtualStep(_descs(dp), C=1.0, sigma=1.0, device="cpu")
    for b in (B, 1, 2):
        virtual.add([(a[:b], None if g is None else g[:b]) for a, g in _inputs()], b, STREAM)
    with pytest.raises(ValueError):
        virtual.add([(a[:1], None if g is None else g[:1]) for a, g in _inputs()], 2, STREAM)
