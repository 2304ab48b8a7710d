"""What the entry points of embeddings, layer norms and log probabilities refuse, by status and message, with
nothing launched; on a stand-in for the CUDA runtime (host_library), so that nothing reaches a GPU."""
import ctypes

import pytest

from host_library import PTR, STREAM, Host

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def host():
    return Host()


@pytest.fixture()
def fake(host):
    with host.installed():
        yield host


def _refused(fake, call, status, text):
    with pytest.raises(fake.dp.DPError) as e:
        call()
    assert e.value.status == status and text in str(e.value), str(e.value)
    assert fake.launches() == []


def _norm(fake, **kw):
    dp = fake.dp
    d = dict(dtype=0, w_dtype=0, B=2, T=3, D=64, has_bias=1, per_example=0, eps=1e-5)
    d.update({n: v for n, v in kw.items() if n in d})
    desc = dp.LayerNormDesc(**d)
    desc.x, desc.dy = dp.RowStrides(*kw.get("x", (192, 64))), dp.RowStrides(*kw.get("dy", (192, 64)))
    return desc


def _embed(fake, **kw):
    dp = fake.dp
    d = dict(dtype=0, out_dtype=1, B=2, T=3, V=50, D=64, index_i64=0, padding=-1, scale=1.0, ld=64)
    d.update({n: v for n, v in kw.items() if n in d})
    desc = dp.EmbeddingDesc(**d)
    desc.dy = dp.RowStrides(*kw.get("dy", (192, 64)))
    return desc


def _logp(fake, **kw):
    d = dict(dtype=0, B=2, T=3, V=100, K=4, token_i64=0, ld=100, ld_grad=100, tau=1.0)
    d.update(kw)
    return fake.dp.LogprobsDesc(**d)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=7), INVALID, "dtype"), (dict(w_dtype=-1), INVALID, "dtype"), (dict(B=0), INVALID, "> 0"),
    (dict(T=-3), INVALID, "> 0"), (dict(D=0), INVALID, "> 0"), (dict(D=16385), UNSUPPORTED, "16384"),
    (dict(eps=-1.0), INVALID, "eps"), (dict(eps=float("nan")), INVALID, "eps"), (dict(x=(-1, 64)), INVALID, "strides"),
    (dict(B=1 << 20, T=1 << 20), UNSUPPORTED, "2^30"),
])
def test_layer_norm_refuses(fake, kw, status, text):
    dp = fake.dp
    d = _norm(fake, **kw)
    _refused(fake, lambda: dp.dp_layer_norm(d, PTR, PTR, PTR, PTR, PTR, PTR, stream=STREAM), status, text)
    _refused(fake, lambda: dp.dp_layer_norm_grad(d, PTR, PTR, PTR, PTR, PTR, PTR, PTR, PTR, 1 << 40, stream=STREAM), status, text)
    assert dp.dp_layer_norm_grad_workspace(d) == 0


def test_layer_norm_pointers_and_workspace(fake):
    dp, d = fake.dp, _norm(fake)
    for a in ((None, PTR, PTR, PTR, PTR, PTR), (PTR, PTR, PTR, None, PTR, PTR), (PTR, PTR, PTR, PTR, None, PTR),
              (PTR, PTR, PTR, PTR, PTR, None)):
        _refused(fake, lambda: dp.dp_layer_norm(d, *a, stream=STREAM), INVALID, "non-NULL")
    need = dp.dp_layer_norm_grad_workspace(d)
    assert need >= 2 * 64 * 4
    full = [PTR] * 7
    for i in (0, 1, 3, 4):
        a = list(full)
        a[i] = None
        _refused(fake, lambda: dp.dp_layer_norm_grad(d, *a, PTR, need, stream=STREAM), INVALID, "non-NULL")
    _refused(fake, lambda: dp.dp_layer_norm_grad(d, PTR, PTR, PTR, PTR, PTR, None, None, PTR, need, stream=STREAM), INVALID,
             "asked for")
    for ws, n, text in ((None, need, "workspace"), (PTR, need - 1, "workspace"), (PTR + 4, need, "aligned")):
        _refused(fake, lambda: dp.dp_layer_norm_grad(d, *full, ws, n, stream=STREAM), INVALID, text)
    _refused(fake, lambda: dp.dp_layer_norm_grad(_norm(fake, dy=(-1, 64)), *full, PTR, need, stream=STREAM), INVALID, "strides")
    # nothing needed: dx alone, or examples of one slice
    dp.dp_layer_norm_grad(d, PTR, PTR, None, PTR, PTR, PTR, None, stream=STREAM)
    one = _norm(fake, per_example=1, T=1, x=(64, 64), dy=(64, 64))
    assert dp.dp_layer_norm_grad_workspace(one) == 0
    dp.dp_layer_norm_grad(one, *full, stream=STREAM)
    dp.dp_layer_norm(d, PTR, None, None, PTR, stream=STREAM)
    assert len(fake.launches()) == 3


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=2), INVALID, "dtype"), (dict(out_dtype=2), INVALID, "dtype"), (dict(B=0), INVALID, "> 0"),
    (dict(V=0), INVALID, "> 0"), (dict(D=-1), INVALID, "> 0"), (dict(ld=63), INVALID, "ld"),
    (dict(scale=float("inf")), INVALID, "scale"), (dict(padding=50), INVALID, "padding"), (dict(dy=(192, -64)), INVALID, "strides"),
    (dict(B=1 << 16, T=1 << 16), UNSUPPORTED, "2^30"), (dict(V=(1 << 30) + 1), UNSUPPORTED, "2^30"),
])
def test_embedding_refuses(fake, kw, status, text):
    dp, d = fake.dp, _embed(fake, **kw)
    big = 1 << 40
    for call in (lambda: dp.dp_embedding(d, PTR, PTR, PTR, stream=STREAM),
                 lambda: dp.dp_embedding_order(d, PTR, PTR, PTR, big, stream=STREAM),
                 lambda: dp.dp_embedding_sqnorms(d, PTR, PTR, PTR, PTR, big, stream=STREAM),
                 lambda: dp.dp_embedding_grad(d, PTR, PTR, PTR, PTR, PTR, big, stream=STREAM)):
        _refused(fake, call, status, text)
    assert dp.dp_embedding_order_size(d) == 0 and dp.dp_embedding_workspace(d) == 0


def test_embedding_pointers_and_workspace(fake):
    dp, d = fake.dp, _embed(fake, T=30000, dy=(30000 * 64, 64))
    need = dp.dp_embedding_workspace(d)
    assert dp.dp_embedding_order_size(d) >= 2 * 60000 * 4 and need >= 60000 * 4
    for a in ((None, PTR, PTR), (PTR, None, PTR), (PTR, PTR, None)):
        _refused(fake, lambda: dp.dp_embedding(d, *a, stream=STREAM), INVALID, "non-NULL")
        _refused(fake, lambda: dp.dp_embedding_sqnorms(d, *a, PTR, need, stream=STREAM), INVALID, "non-NULL")
        _refused(fake, lambda: dp.dp_embedding_grad(d, a[0], a[1], PTR, a[2], PTR, need, stream=STREAM), INVALID, "non-NULL")
    for a in ((None, PTR), (PTR, None)):
        _refused(fake, lambda: dp.dp_embedding_order(d, *a, PTR, need, stream=STREAM), INVALID, "non-NULL")
    for ws, n, text in ((None, need, "workspace"), (PTR, need - 1, "workspace"), (PTR + 4, need, "aligned")):
        _refused(fake, lambda: dp.dp_embedding_order(d, PTR, PTR, ws, n, stream=STREAM), INVALID, text)
        _refused(fake, lambda: dp.dp_embedding_sqnorms(d, PTR, PTR, PTR, ws, n, stream=STREAM), INVALID, text)
        _refused(fake, lambda: dp.dp_embedding_grad(d, PTR, PTR, PTR, PTR, ws, n, stream=STREAM), INVALID, text)
    _refused(fake, lambda: dp.dp_embedding_order(d, PTR, PTR + 8, PTR, need, stream=STREAM), INVALID, "aligned")
    half = _embed(fake, out_dtype=0)
    _refused(fake, lambda: dp.dp_embedding_grad(half, PTR, PTR, PTR, PTR, PTR, 1 << 40, accumulate=True, stream=STREAM), INVALID,
             "fp32")


def test_embedding_order_grad_refuses(fake):
    dp, d = fake.dp, _embed(fake, T=30000, dy=(30000 * 64, 64))
    need = dp.dp_embedding_workspace(d)
    for i in (0, 1, 2, 4):   # tokens, order, dY, dW
        a = [PTR] * 5
        a[i] = None
        _refused(fake, lambda: dp.dp_embedding_order_grad(d, *a, PTR, need, stream=STREAM), INVALID, "non-NULL")
    a = [PTR] * 5
    for ws, n, text in ((None, need, "workspace"), (PTR, need - 1, "workspace"), (PTR + 4, need, "aligned")):
        _refused(fake, lambda: dp.dp_embedding_order_grad(d, *a, ws, n, stream=STREAM), INVALID, text)
    _refused(fake, lambda: dp.dp_embedding_order_grad(d, PTR, PTR + 8, PTR, PTR, PTR, PTR, need, stream=STREAM), INVALID, "aligned")
    _refused(fake, lambda: dp.dp_embedding_order_grad(_embed(fake, V=0), *a, PTR, need, stream=STREAM), INVALID, "> 0")
    half = _embed(fake, out_dtype=0)
    _refused(fake, lambda: dp.dp_embedding_order_grad(half, *a, PTR, 1 << 40, accumulate=True, stream=STREAM), INVALID, "fp32")
    assert ctypes.CDLL(dp.LIB_PATH)["dp_embedding_order_grad"](*[None] * 10) == INVALID


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=3), INVALID, "dtype"), (dict(B=0), INVALID, "> 0"), (dict(V=0), INVALID, "> 0"), (dict(K=-1), INVALID, ">= 0"),
    (dict(K=101), INVALID, "alternatives"), (dict(V=500, ld=500, ld_grad=500, K=129), UNSUPPORTED, "128"),
    (dict(ld=99), INVALID, "ld"), (dict(tau=0.0), INVALID, "tau"), (dict(tau=-1.0), INVALID, "tau"),
    (dict(tau=float("nan")), INVALID, "tau"), (dict(tau=1e-39), INVALID, "tau"), (dict(tau=float("inf")), INVALID, "tau"),
    (dict(B=1 << 20, T=1 << 20), UNSUPPORTED, "rows"),
])
def test_token_logprobs_refuse(fake, kw, status, text):
    dp, d = fake.dp, _logp(fake, **kw)
    _refused(fake, lambda: dp.dp_token_logprobs(d, *[PTR] * 7, stream=STREAM), status, text)
    _refused(fake, lambda: dp.dp_token_logprobs_grad(d, *[PTR] * 7, stream=STREAM), status, text)


def test_token_logprobs_pointers_and_limits(fake):
    dp, d = fake.dp, _logp(fake)
    for i in (0, 2, 3, 4, 5, 6):
        a = [PTR] * 7
        a[i] = None
        _refused(fake, lambda: dp.dp_token_logprobs(d, *a, stream=STREAM), INVALID, "non-NULL")
    for i in (0, 2, 3, 6):
        a = [PTR] * 7
        a[i] = None
        _refused(fake, lambda: dp.dp_token_logprobs_grad(d, *a, stream=STREAM), INVALID, "non-NULL")
    _refused(fake, lambda: dp.dp_token_logprobs_grad(_logp(fake, ld_grad=99), *[PTR] * 7, stream=STREAM), INVALID, "ld_grad")
    far = dict(V=(1 << 22) + 1, ld=1 << 23, ld_grad=1 << 23)
    _refused(fake, lambda: dp.dp_token_logprobs(_logp(fake, **far), *[PTR] * 7, stream=STREAM), UNSUPPORTED, "2^22")
    dp.dp_token_logprobs(_logp(fake, **{**far, "K": 0}), *[PTR] * 5, stream=STREAM)
    for V in (1, 7, 4096, 131072, 1 << 22):
        for dtype in (0, 1):
            dp.dp_token_logprobs(_logp(fake, dtype=dtype, V=V, K=min(V, 128), ld=V), PTR, None, *[PTR] * 5, stream=STREAM)
    launches = fake.launches()
    assert len(launches) == 11 and all(x[4] == 0 for x in launches)   # none was refused for its shared memory


def test_examples_refuse(fake):
    dp = fake.dp
    for a in ((None, 2, 5, PTR), (PTR, 2, 5, None)):
        _refused(fake, lambda: dp.dp_example_sqnorms(*a, stream=STREAM), INVALID, "non-NULL")
    for B, n in ((0, 5), (-1, 5), (2, 0)):
        _refused(fake, lambda: dp.dp_example_sqnorms(PTR, B, n, PTR, stream=STREAM), INVALID, "> 0")
        _refused(fake, lambda: dp.dp_example_sum(PTR, B, n, PTR, PTR, stream=STREAM), INVALID, "> 0")
    for a in ((None, 2, 5, PTR, PTR), (PTR, 2, 5, None, PTR), (PTR, 2, 5, PTR, None)):
        _refused(fake, lambda: dp.dp_example_sum(*a, stream=STREAM), INVALID, "non-NULL")


def test_null_everything(fake):
    for name, n in (("dp_token_logprobs", 9), ("dp_token_logprobs_grad", 9), ("dp_layer_norm", 8), ("dp_layer_norm_grad", 11),
                    ("dp_embedding", 5), ("dp_embedding_order", 6), ("dp_embedding_sqnorms", 7), ("dp_embedding_grad", 9)):
        f = ctypes.CDLL(fake.dp.LIB_PATH)[name]
        assert f(*[None] * n) == INVALID, name


def test_every_device_takes_its_shared_memory(fake):
    """Kernels above 48 KB of shared memory are allowed it on each device."""
    dp = fake.dp
    for dev in (0, 3, 0):
        fake.so.fake_device(dev)
        for N in (500, 3000, 16000, 50000):
            d = _embed(fake, B=1, T=N, dy=(N * 64, 64))
            dp.dp_embedding_order(d, PTR, PTR, PTR, 1 << 40, stream=STREAM)
        dp.dp_token_logprobs(_logp(fake, V=1 << 22, ld=1 << 22), *[PTR] * 7, stream=STREAM)
        launches = fake.launches()
        assert launches and all(x[2] == dev and x[4] == 0 for x in launches)
    fake.so.fake_device(0)


def test_python_side_refuses():
    import torch
    import example_gradient_clipping_gb300 as dp
    x, t = torch.zeros(2, 3, 8), torch.zeros(2, 3, dtype=torch.int32)
    for f in (lambda: dp.layer_norm(x), lambda: dp.embedding(t, x[0]), lambda: dp.embedding_backward(t, x, 5),
              lambda: dp.token_logprobs(x), lambda: dp.embedding_sqnorms(t, x, 5), lambda: dp.layer_norm(x[0, 0])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: dp.LayerNorm((3, 4)), lambda: dp.Embedding(4, 4, max_norm=1.0), lambda: dp.Embedding(4, 4, sparse=True),
              lambda: dp.Embedding(4, 4, scale_grad_by_freq=True), lambda: dp.kept_desc(0, 3)):
        with pytest.raises(ValueError):
            f()


def test_engine_takes_the_packages_layers_alone():
    import torch.nn as nn
    import example_gradient_clipping_gb300 as dp
    model = nn.Sequential(dp.Embedding(10, 4), dp.LayerNorm(4), nn.Linear(4, 10))
    engine = dp.PrivacyEngine(model)
    assert len(engine.layers) == 3 and model[1]._sink is not None
    with pytest.raises(RuntimeError, match="backward"):
        engine.privatise(0)
    with pytest.raises(ValueError, match="another engine"):
        dp.PrivacyEngine(model)
    engine.detach()
    assert model[1]._sink is None
    dp.PrivacyEngine(nn.Sequential(nn.Linear(4, 4), dp.LayerNorm(4, elementwise_affine=False))).detach()
    model[2].weight = model[0].weight   # a tied head
    for m in (model, nn.Sequential(model[2], model[0]), nn.Sequential(nn.Linear(4, 4), nn.Embedding(3, 4)),
              nn.Sequential(nn.Linear(4, 4), nn.LayerNorm(4))):
        with pytest.raises(ValueError):
            dp.PrivacyEngine(m)
    half = dp.LayerNorm(4)
    half.bias.requires_grad_(False)
    with pytest.raises(ValueError, match="bias"):
        dp.PrivacyEngine(nn.Sequential(nn.Linear(4, 4), half))
