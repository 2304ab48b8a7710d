"""CPU checks of the sequence operators' C entry points: descriptors and pointers that do not
fit are refused on the host, with a message, before anything is launched."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dp():
    import __graft_entry__
    __graft_entry__.build()
    import example_gradient_clipping_gb300 as m
    return m


def _attn(dp, **kw):
    d = dict(dtype=dp.DP_BF16, B=2, T=5, S=6, Hq=4, Hk=2, D=64, causal=1, window=0, scale=0.0)
    d.update(kw)
    q, k = (d["T"] * d["Hq"] * d["D"], d["Hq"] * d["D"], d["D"]), (d["S"] * d["Hk"] * d["D"], d["Hk"] * d["D"], d["D"])
    st = {n: q if n in ("q", "o", "d_o", "dq") else k for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")}
    st.update({n: kw[n] for n in st if n in kw})
    desc = dp.AttnDesc(*[d[n] for n in ("dtype", "B", "T", "S", "Hq", "Hk", "D", "causal", "window", "scale")])
    for n, s in st.items():
        setattr(desc, n, dp.Strides(*s))
    return desc


ONE = 256   # a pointer that is never followed: the calls below are refused before any launch


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), 1), (dict(B=0), 1), (dict(T=0), 1), (dict(S=-1), 1), (dict(Hq=3), 1), (dict(Hk=0), 1),
    (dict(D=0), 1), (dict(D=129), 2), (dict(window=-1), 1), (dict(window=4, causal=0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(q=(-1, 64, 64)), 1), (dict(o=(0, 256, 64)), 1),
    (dict(T=(1 << 30) + 1), 2), (dict(B=1 << 20, T=1 << 16), 2),
])
def test_attention_refuses(dp, kw, status):
    with pytest.raises(dp.DPError) as e:
        dp.dp_attention(_attn(dp, **kw), ONE, ONE, ONE, ONE, None, stream=1)
    assert e.value.status == status and len(str(e.value)) > 20
    assert dp.dp_launch_count() == 0


@pytest.mark.parametrize("kw", [dict(dq=(0, 256, 64)), dict(dk=(768, 0, 64)), dict(dv=(768, 128, 8)), dict(d_o=(-2, 1, 1))])
def test_attention_grad_refuses(dp, kw):
    with pytest.raises(dp.DPError):
        dp.dp_attention_grad(_attn(dp, **kw), *[ONE] * 9, ONE, ws_bytes=1 << 20, stream=1)
    assert dp.dp_attention_grad_workspace(_attn(dp, **kw)) == 0


def test_null_pointers_and_workspace(dp):
    d = _attn(dp)
    for i in range(4):
        a = [ONE] * 4
        a[i] = None
        with pytest.raises(dp.DPError):
            dp.dp_attention(d, *a, None, stream=1)
    need = dp.dp_attention_grad_workspace(d)
    assert need >= 2 * 4 * 5 * 4
    for i in range(9):
        a = [ONE] * 9
        a[i] = None
        with pytest.raises(dp.DPError):
            dp.dp_attention_grad(d, *a, ONE, ws_bytes=need, stream=1)
    for ws, n in ((None, need), (ONE, need - 1), (ONE + 4, need)):
        with pytest.raises(dp.DPError):
            dp.dp_attention_grad(d, *[ONE] * 9, ws, ws_bytes=n, stream=1)
    lib = ctypes.CDLL(dp.LIB_PATH)
    for name, n in (("dp_attention", 9), ("dp_attention_grad", 15), ("dp_rotary", 8), ("dp_rotary_table", 3),
                    ("dp_distill", 11)):
        assert getattr(lib, name)(*[None] * n) == dp.DP_ERR_INVALID_ARG, name


@pytest.mark.parametrize("kw", [dict(R=3), dict(R=0), dict(P=0), dict(scaling=9), dict(theta=0.0), dict(theta=float("inf")),
                                dict(scaling=1, factor=0.5), dict(scaling=3, factor=2.0, context=0.0),
                                dict(scaling=3, factor=2.0, slow=5.0, fast=5.0)])
def test_rotary_table_refuses(dp, kw):
    d = dict(P=8, R=4, scaling=0, theta=1e4, factor=1.0, context=64.0, slow=1.0, fast=32.0)
    d.update(kw)
    with pytest.raises(dp.DPError):
        dp.dp_rotary_table(dp.RotaryTableDesc(**d), ONE, stream=1)


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(B=0), dict(Hq=0), dict(Hk=-1), dict(R=5), dict(R=66), dict(P=0),
                                dict(P=3), dict(q=(-1, 1, 1)), dict(q_out=(64, 64, 64)), dict(k_out=(0, 0, 0))])
def test_rotary_refuses(dp, kw):
    d = dict(dtype=dp.DP_FP32, B=2, T=4, Hq=2, Hk=2, D=64, R=64, P=8, interleaved=0, inverse=0, pos_i64=0)
    d.update({n: v for n, v in kw.items() if n in d})
    desc = dp.RotaryDesc(**d)
    for n in ("q", "k", "q_out", "k_out"):
        setattr(desc, n, dp.Strides(*kw.get(n, (512, 128, 64))))
    with pytest.raises(dp.DPError):
        dp.dp_rotary(desc, ONE, ONE, ONE, None, ONE, ONE, stream=1)


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(teacher_dtype=-1), dict(B=0), dict(V=0), dict(K=-1), dict(K=1025),
                                dict(ld=99), dict(ld_grad=99), dict(tau=0.0), dict(tau=float("nan")), dict(alpha=-0.1),
                                dict(alpha=float("nan"))])
def test_distill_refuses(dp, kw):
    d = dict(dtype=0, teacher_dtype=0, B=2, T=3, V=100, K=4, index_i64=0, label_i64=0, ld=100, ld_grad=100, tau=1.0,
             alpha=0.0)
    d.update(kw)
    with pytest.raises(dp.DPError):
        dp.dp_distill(dp.DistillDesc(**d), ONE, ONE, ONE, row_loss=ONE, loss=ONE, dlogits=ONE, stream=1)
    good = dp.DistillDesc(0, 0, 2, 3, 100, 4, 0, 0, 100, 100, 1.0, 0.0)
    for a in (dict(), dict(loss=ONE), ):
        with pytest.raises(dp.DPError):
            dp.dp_distill(good, ONE, ONE, ONE, stream=1, **a)


def test_tensors_on_the_host_are_refused(dp):
    import torch
    q = torch.zeros(1, 2, 2, 8)
    for f in (lambda: dp.attention(q, q, q), lambda: dp.rotary(q, q, torch.zeros(4, 8)),
              lambda: dp.distill_loss(q[0], q[0].int(), q[0])):
        with pytest.raises(ValueError):
            f()
