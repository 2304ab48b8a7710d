"""What the sequence operators' C entry points refuse, by status and message, and that nothing was
launched; and what they must go on taking.  On a stand-in for the CUDA runtime (host_library), so that a
descriptor that slips through reaches no GPU."""
import pytest

import test_sequence_abi as abi
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
    assert e.value.status == status and text in str(e.value)
    assert fake.launches() == []


def _attention(fake, grad=False, ws_bytes=1 << 40, **kw):
    d = abi._attn(fake.dp, **kw)
    if grad:
        fake.dp.dp_attention_grad(d, *[PTR] * 9, PTR, ws_bytes=ws_bytes, stream=STREAM)
    else:
        fake.dp.dp_attention(d, PTR, PTR, PTR, PTR, None, stream=STREAM)


def _rotary(fake, **kw):
    dp = fake.dp
    d = dict(dtype=dp.DP_FP32, B=2, T=4, Hq=2, Hk=2, D=64, R=64, P=8, interleaved=0, inverse=0, pos_i64=0)
    d.update({n: v for n, v in kw.items() if n in d})
    desc = dp.RotaryDesc(**d)
    for n in ("q", "k", "q_out", "k_out"):
        setattr(desc, n, dp.Strides(*kw.get(n, (512, 128, 64))))
    dp.dp_rotary(desc, PTR, PTR, PTR, None, PTR, PTR, stream=STREAM)


# rows on one another: (b, t, h) strides of a [2, 4, 2, 64] tensor
OVERLAP = [(64, 64, 64), (512, 64, 64), (128, 128, 64), (512, 128, 63), (512, 100, 64), (256, 128, 64),
           (0, 128, 64), (512, 0, 64), (512, 128, 0), (1024, 64, 128)]
# heads first, packed projections, examples innermost, padded rows
APART = [(512, 128, 64), (512, 64, 256), (1536, 384, 64), (64, 256, 128), (64, 128, 512), (128, 512, 64),
         (1 << 40, 130, 65),
         (1 << 62, 1 << 40, 64)]


@pytest.mark.parametrize("st", OVERLAP)
def test_overlapping_rows_are_refused(fake, st):
    for out in ("q_out", "k_out"):
        _refused(fake, lambda: _rotary(fake, **{out: st}), INVALID, "overlap")
    shape = dict(B=2, T=4, S=4, Hq=2, Hk=2, D=64)
    _refused(fake, lambda: _attention(fake, o=st, **shape), INVALID, "overlap")
    for out in ("dq", "dk", "dv"):
        _refused(fake, lambda: _attention(fake, True, **{out: st}, **shape), INVALID, "overlap")


@pytest.mark.parametrize("st", APART)
def test_rows_apart_are_taken(fake, st):
    shape = dict(B=2, T=4, S=4, Hq=2, Hk=2, D=64)
    _rotary(fake, q_out=st, k_out=st)
    _attention(fake, o=st, **shape)
    _attention(fake, True, dq=st, dk=st, dv=st, **shape)
    assert len(fake.launches()) >= 3


def test_extents_of_one_have_any_stride(fake):
    for B, T, H, st in ((1, 4, 2, (0, 128, 64)), (2, 1, 2, (128, 7, 64)), (2, 4, 1, (256, 64, 0)), (1, 1, 1, (0, 0, 0))):
        _rotary(fake, B=B, T=T, Hq=H, Hk=H, q_out=st, k_out=st)
        _attention(fake, o=st, B=B, T=T, S=4, Hq=H, Hk=H)
    assert len(fake.launches()) == 8


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=7), INVALID, "dtype"), (dict(B=0), INVALID, "> 0"), (dict(T=0), INVALID, "> 0"),
    (dict(S=-1), INVALID, "> 0"), (dict(Hq=3), INVALID, "multiple"), (dict(D=0), INVALID, "> 0"),
    (dict(D=129), UNSUPPORTED, "128"), (dict(window=-1), INVALID, "window"),
    (dict(window=4, causal=0), INVALID, "window"), (dict(scale=-1.0), INVALID, "scale"),
    (dict(scale=float("nan")), INVALID, "scale"), (dict(q=(-1, 64, 64)), INVALID, "strides"),
    (dict(T=(1 << 30) + 1), UNSUPPORTED, "2^30"), (dict(B=1 << 20, T=1 << 16), UNSUPPORTED, "too large"),
])
def test_attention_and_gradient_refuse(fake, kw, status, text):
    _refused(fake, lambda: _attention(fake, **kw), status, text)
    _refused(fake, lambda: _attention(fake, True, **kw), status, text)


def test_attention_gradient_refuses(fake):
    _refused(fake, lambda: _attention(fake, True, d_o=(-2, 1, 1)), INVALID, "negative")
    need = fake.dp.dp_attention_grad_workspace(abi._attn(fake.dp))
    _refused(fake, lambda: _attention(fake, True, need - 1), INVALID, "workspace")
    d = abi._attn(fake.dp)
    for i in range(9):
        a = [PTR] * 9
        a[i] = None
        _refused(fake, lambda: fake.dp.dp_attention_grad(d, *a, PTR, ws_bytes=need, stream=STREAM), INVALID, "non-NULL")
    for ws, n, text in ((None, need, "workspace"), (PTR + 4, need, "aligned")):
        _refused(fake, lambda: fake.dp.dp_attention_grad(d, *[PTR] * 9, ws, ws_bytes=n, stream=STREAM), INVALID, text)
    for i in range(4):
        a = [PTR] * 4
        a[i] = None
        _refused(fake, lambda: fake.dp.dp_attention(d, *a, None, stream=STREAM), INVALID, "non-NULL")


@pytest.mark.parametrize("kw,text", [
    (dict(R=3), "even"), (dict(R=0), "even"), (dict(P=0), "> 0"), (dict(scaling=9), "scaling"),
    (dict(theta=0.0), "theta"), (dict(theta=float("inf")), "theta"), (dict(scaling=1, factor=0.5), "factor"),
    (dict(scaling=3, factor=2.0, context=0.0), "context"), (dict(scaling=3, factor=2.0, slow=5.0, fast=5.0), "slow"),
])
def test_rotary_table_refuses(fake, kw, text):
    d = dict(P=8, R=4, scaling=0, theta=1e4, factor=1.0, context=64.0, slow=1.0, fast=32.0)
    d.update(kw)
    _refused(fake, lambda: fake.dp.dp_rotary_table(fake.dp.RotaryTableDesc(**d), PTR, stream=STREAM), INVALID, text)


@pytest.mark.parametrize("kw,text", [
    (dict(dtype=2), "dtype"), (dict(B=0), "> 0"), (dict(Hq=0), "> 0"), (dict(Hk=-1), ">= 0"), (dict(R=5), "even"),
    (dict(R=66), "even"), (dict(P=0), "> 0"), (dict(P=3), "positions"), (dict(q=(-1, 1, 1)), "strides"),
])
def test_rotary_refuses(fake, kw, text):
    _refused(fake, lambda: _rotary(fake, **kw), INVALID, text)


@pytest.mark.parametrize("kw,status,text", [
    (dict(dtype=3), INVALID, "dtype"), (dict(teacher_dtype=-1), INVALID, "dtype"), (dict(B=0), INVALID, "> 0"),
    (dict(V=0), INVALID, "> 0"), (dict(K=-1), INVALID, ">= 0"), (dict(K=1025), UNSUPPORTED, "1024"),
    (dict(ld=99), INVALID, "ld"), (dict(ld_grad=99), INVALID, "ld_grad"), (dict(tau=0.0), INVALID, "tau"),
    (dict(tau=float("nan")), INVALID, "tau"), (dict(alpha=-0.1), INVALID, "alpha"),
    (dict(alpha=float("nan")), INVALID, "alpha"),
])
def test_distill_refuses(fake, kw, status, text):
    d = dict(dtype=0, teacher_dtype=0, B=2, T=3, V=100, K=4, index_i64=0, label_i64=0, ld=100, ld_grad=100, tau=1.0,
             alpha=0.0)
    dp = fake.dp

    def call(desc, **a):
        dp.dp_distill(dp.DistillDesc(**desc), PTR, PTR, PTR, stream=STREAM, **a)
    _refused(fake, lambda: call({**d, **kw}, row_loss=PTR, loss=PTR, dlogits=PTR), status, text)
    _refused(fake, lambda: call(d), INVALID, "asked for")
    _refused(fake, lambda: call(d, loss=PTR), INVALID, "row_loss")
    call(d, row_loss=PTR, loss=PTR, dlogits=PTR)
    assert len(fake.launches()) == 2


@pytest.mark.parametrize("device", ["cpu", "meta"])
@pytest.mark.parametrize("stream", [None, STREAM])
def test_rotary_table_on_the_host_is_refused(fake, device, stream):
    """The table is written by a kernel: memory that is not the GPU's must not get that far."""
    import torch
    for d in (device, torch.device(device)) + ((None,) if device == "cpu" else ()):   # None: torch's default device
        with pytest.raises(ValueError, match="CUDA device"):
            fake.dp.rotary_table(8, 4, device=d, stream=stream)
    assert fake.launches() == []
