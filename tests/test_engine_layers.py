"""What PrivacyEngine takes from embeddings and layer norms: of the calls that are differentiated, and of those alone.

On the CPU the two operators are replaced by torch's, so that autograd's side runs without a GPU."""
import pytest
import torch
import torch.nn as nn

from host_library import STREAM, Host

pytestmark = pytest.mark.filterwarnings("ignore:Full backward hook is firing")

B, T, V, D = 4, 6, 11, 8


def _on_the_cpu(monkeypatch):
    import example_gradient_clipping_gb300.layers as layers

    def forward(x, w, b, eps):
        mean, var = x.mean(-1), x.var(-1, unbiased=False)
        rstd = 1 / torch.sqrt(var + eps)
        return nn.functional.layer_norm(x, x.shape[-1:], w, b, eps), mean, rstd

    def backward(dy, x, w, mean, rstd, bias=True, per_example=False, dx=True, params=True):
        h = (x - mean[..., None]) * rstd[..., None]
        u = dy * w
        gx = rstd[..., None] * (u - u.mean(-1, keepdim=True) - h * (u * h).mean(-1, keepdim=True))
        each = torch.cat([(dy * h).flatten(1, -2).sum(1)] + ([dy.flatten(1, -2).sum(1)] if bias else []), 1)
        if per_example:
            return gx, each
        return gx, each[:, :x.shape[-1]].sum(0), each[:, x.shape[-1]:].sum(0) if bias else None

    def grad(tokens, dy, V, scale=1.0, padding=None, factors=None, dtype=torch.float32, stream=None):
        w = torch.zeros(V, dy.shape[-1]).index_add_(0, tokens.flatten().long(), scale * dy.flatten(0, -2))
        if padding is not None:
            w[padding] = 0
        return w.to(dtype)
    monkeypatch.setattr(layers, "_lookup", lambda tokens, w, scale, padding: scale * w.detach()[tokens.long()])
    monkeypatch.setattr(layers, "embedding_backward", grad)
    monkeypatch.setattr(layers, "layer_norm_forward", forward)
    monkeypatch.setattr(layers, "layer_norm_backward", backward)
    monkeypatch.setattr(layers, "_norm", lambda x, w, b, eps, stats: forward(x, w, b, eps))


@pytest.fixture(params=["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def device(request, monkeypatch):
    if request.param == "cpu":
        _on_the_cpu(monkeypatch)
    else:
        request.getfixturevalue("lib")
    return request.param


class _Model(nn.Module):
    def __init__(self, device, **kw):
        super().__init__()
        import example_gradient_clipping_gb300 as dp
        torch.manual_seed(0)
        self.embed, self.norm, self.head = dp.Embedding(V, D, **kw), dp.LayerNorm(D), nn.Linear(D, V)
        self.to(device)

    def forward(self, tokens):
        return self.head(self.norm(self.embed(tokens)))


def _tokens(device, seed=0, b=B, t=T, dtype=torch.int64):
    return torch.randint(0, V, (b, t), generator=torch.Generator().manual_seed(seed)).to(device, dtype)


def _engine(model, **kw):
    import example_gradient_clipping_gb300 as dp
    return dp.PrivacyEngine(model, C=0.1, sigma=0.0, **kw)


def _privatised(model, tokens, between=lambda model: None):
    """The flat gradient on a GPU; on the CPU what the engine would take it from."""
    engine = _engine(model)
    loss = model(tokens).square().sum()
    between(model)
    loss.backward()
    if tokens.is_cuda:
        out = [engine.privatise(0).clone()]
    else:
        out = [x.clone() for pair in zip(engine._acts[:2], engine._grads[:2]) for x in pair if x is not None]
    engine.detach()
    return out


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("t", [T, T + 3, 1])
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_a_call_between_forward_and_backward(device, grad, t, dtype):
    """The embedding called with other tokens (to log something) while a backward pass is still to come."""
    model, tokens = _Model(device), _tokens(device)
    want = _privatised(model, tokens)

    def log(model):
        with torch.set_grad_enabled(grad):
            model.embed(_tokens(device, 1, t=t, dtype=dtype))
    got = _privatised(model, tokens, log)
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_parameters_under_an_engine_have_no_gradient_but_the_engines(device):
    model, tokens = _Model(device), _tokens(device)
    model(tokens).square().sum().backward()
    plain = model.embed.weight.grad.clone()
    model.zero_grad()
    engine = _engine(model)
    model(tokens).square().sum().backward()
    assert all(p.grad is None for p in (model.embed.weight, model.norm.weight, model.norm.bias))
    engine.detach()
    model.zero_grad()
    model(tokens).square().sum().backward()
    assert torch.equal(model.embed.weight.grad, plain)


def test_two_engines_take_the_same_embedding(device):
    """As they take the same linear layer: each has its own copy, and one's end leaves the other's."""
    model, tokens = _Model(device), _tokens(device)
    model.norm.requires_grad_(False)   # (a layer norm is one engine's)
    first, second = _engine(model), _engine(model)
    loss = model(tokens).square().sum()
    loss.backward(retain_graph=True)
    for e in (first, second):
        assert torch.equal(e._acts[0], tokens) and e._grads[0].shape == (B, T, D)
        e._acts, e._grads = [None, None], [None, None]
    first.detach()
    assert len(model.embed._sinks) == 1
    model(tokens).square().sum().backward()
    assert first._acts[0] is None and second._acts[0] is not None
    second.detach()
    assert model.embed._sinks == ()


def test_descriptors_of_the_differentiated_call(monkeypatch):
    """The step's sizes come from the tokens and output gradient that belong together."""
    host = Host()
    _on_the_cpu(monkeypatch)
    model = _Model("cpu", padding_idx=2)
    engine = _engine(model)
    loss = model(_tokens("cpu")).sum()
    with torch.no_grad():
        model.embed(_tokens("cpu", 1, t=50, dtype=torch.int32))
    loss.backward()
    with host.installed():
        engine.privatise(0, stream=STREAM)
    d = engine._step.descs[0]
    assert (d.B, d.T, d.V, d.D, d.index_i64, d.padding) == (B, T, V, D, 1, 2)


@pytest.mark.parametrize("use", ["tied head", "of the tokens' rows", "a penalty", "norm weight", "norm bias"])
def test_parameters_used_beside_their_layer(device, use):
    """Gradients that reach a parameter around its layer are in no example's, so that pass is an error."""
    model, tokens = _Model(device), _tokens(device)
    engine = _engine(model)
    x = model.norm(model.embed(tokens))
    loss = model.head(x).sum()
    if use == "tied head":
        loss = loss + nn.functional.linear(x, model.embed.weight).sum()
    elif use == "of the tokens' rows":
        loss = loss + model.embed.weight[tokens[0]].sum()
    elif use == "a penalty":
        loss = loss + model.embed.weight.square().sum()
    else:
        loss = loss + (model.norm.weight if use == "norm weight" else model.norm.bias).sum()
    with pytest.raises(RuntimeError, match="beside the layer's own call"):
        loss.backward()
    model.zero_grad()
    for _ in range(2):   # the engine's gradients are no such use, whether or not they are cleared between steps
        model(tokens).sum().backward()
        if tokens.is_cuda:
            engine.privatise(0)
            assert all(p.grad is not None for p in model.parameters())
    # detached values are numbers like others, and without an engine every use is autograd's
    (model(tokens).sum() + (model.embed.weight.detach() * 2).sum()).backward()
    engine.detach()
    (model(tokens).sum() + model.embed.weight.sum() + model.norm.bias.sum()).backward()


@pytest.mark.gpu
def test_an_embedding_whose_options_change_between_steps(lib):
    """Scale and padding token are the differentiated call's: each step's gradient is a new engine's."""
    model, tokens = _Model("cuda"), _tokens("cuda")
    engine = _engine(model)
    for scale, padding in ((1.0, None), (3.0, None), (3.0, 2), (0.5, 7), (1.0, None)):
        model.embed.scale, model.embed.padding_idx = scale, padding
        loss = model(tokens).square().sum()
        model.embed.scale = 17.0   # after the forward call
        loss.backward()
        got = engine.privatise(0).clone()
        model.embed.scale = scale
        assert torch.equal(got, _privatised_beside(engine, model, tokens)), (scale, padding)


def _privatised_beside(engine, model, tokens):
    """A new engine's gradient, with `engine` away meanwhile."""
    sink, model.norm._sink = model.norm._sink, None
    sinks, model.embed._sinks = model.embed._sinks, ()
    try:
        return _privatised(model, tokens)[0]
    finally:
        model.norm._sink, model.embed._sinks = sink, sinks


@pytest.mark.parametrize("change", ["scale", "padding", "device"])
def test_the_step_is_built_anew_for_other_options(monkeypatch, change):
    host = Host()
    _on_the_cpu(monkeypatch)
    model = _Model("cpu", padding_idx=2)
    engine = _engine(model)

    def step():
        model(_tokens("cpu")).sum().backward()
        with host.installed():
            engine.privatise(0, stream=STREAM)
        return engine._step
    first = step()
    assert step() is first and (first.descs[0].scale, first.descs[0].padding) == (1.0, 2)
    if change == "scale":
        model.embed.scale = 0.25
        assert step().descs[0].scale == 0.25
    elif change == "padding":
        model.embed.padding_idx = None
        assert step().descs[0].padding == -1
    else:   # (as if the model had moved)
        engine._key = tuple("cuda:1" if isinstance(k, torch.device) else k for k in engine._key)
        assert step() is not first


@pytest.mark.parametrize("reentrant", [True, False])
@pytest.mark.parametrize("which", ["embed", "norm"])
def test_a_layer_in_two_checkpointed_segments(device, which, reentrant):
    """Segments that a backward pass runs again: a layer of two of them is reached twice by one step."""
    from torch.utils.checkpoint import checkpoint
    model, tokens = _Model(device), _tokens(device)
    want = _privatised(model, tokens)
    engine = _engine(model)
    on = torch.ones((), device=device, requires_grad=True)   # what a segment needs to be run again
    first = lambda on: model.embed(tokens) * on              # noqa: E731
    second = model.norm

    def segments(again):
        x = checkpoint(first, on, use_reentrant=reentrant)
        x = checkpoint(second, x, use_reentrant=reentrant)
        if again:
            x = checkpoint((lambda x: x + first(on)) if which == "embed" else second, x, use_reentrant=reentrant)
        return model.head(x).square().sum()
    with pytest.raises(RuntimeError, match="more than once"):
        segments(True).backward()
    with pytest.raises(RuntimeError, match="more than once"):   # one of them in a segment, the other not
        y = segments(False)
        x = model.norm(model.embed(tokens)) if which == "embed" else model.norm(torch.zeros(B, T, D, device=device))
        (y + x.sum()).backward()
    for _ in range(2):   # once in each pass, the passes not privatised
        segments(False).backward()
    if tokens.is_cuda:
        assert torch.equal(engine.privatise(0), want[0])
    else:
        got = [x for pair in zip(engine._acts[:2], engine._grads[:2]) for x in pair if x is not None]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("how", ["deepcopy", "layers"])
def test_a_copy_of_a_model_under_an_engine(device, how):
    """A copy trains as a model without an engine, and its passes are none of the engine's."""
    import copy
    import pickle
    model, tokens = _Model(device), _tokens(device)
    plain = copy.deepcopy(model)
    want = _privatised(model, tokens)
    engine = _engine(model)
    if how == "deepcopy":
        other = copy.deepcopy(model)
    else:   # (a linear layer's hook cannot be pickled)
        other = copy.deepcopy(plain)
        other.embed, other.norm = pickle.loads(pickle.dumps(model.embed)), copy.deepcopy(model.norm)
    loss = model(tokens).square().sum()
    for m in (plain, other):
        m(_tokens(device, 1)).square().sum().backward()
    for (name, p), q in zip(plain.named_parameters(), other.parameters()):
        assert q.grad is not None and torch.equal(p.grad, q.grad), name
    assert all(x is None for x in engine._acts + engine._grads)
    loss.backward()
    other(_tokens(device, 2)).sum().backward()
    if tokens.is_cuda:
        assert torch.equal(engine.privatise(0), want[0])
    else:
        got = [x for pair in zip(engine._acts[:2], engine._grads[:2]) for x in pair if x is not None]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    _engine(other).detach()   # and may have an engine of its own
