"""The sequence operators on several devices of one process: a kernel's shared-memory attribute belongs to
the device that is current when it is set, and a failure to set it is not kept.  On a stand-in for the CUDA
runtime (host_library) that refuses a launch above 48 KB on a device where the kernel has no leave."""
import pytest

import test_sequence_abi as abi
from host_library import HERE, PTR, ROOT, STREAM, Host


@pytest.fixture(scope="module")
def host():
    return Host()


@pytest.fixture()
def fake(host):
    with host.installed():
        yield host
        host.so.fake_fail_attributes(0)


def _attn(dp, dtype, B, T, Hq, Hk, D, causal=0):
    q, k = (T * Hq * D, Hq * D, D), (T * Hk * D, Hk * D, D)
    return abi._attn(dp, dtype=dtype, B=B, T=T, S=T, Hq=Hq, Hk=Hk, D=D, causal=causal,
                     **{n: q for n in ("q", "o", "d_o", "dq")}, **{n: k for n in ("k", "v", "dk", "dv")})


def _attention(dp, *shape):
    dp.dp_attention(_attn(dp, *shape), PTR, PTR, PTR, PTR, None, stream=STREAM)


def _gradient(dp, *shape):
    dp.dp_attention_grad(_attn(dp, *shape), *[PTR] * 9, PTR, ws_bytes=1 << 40, stream=STREAM)


def _distill(dp, dtype, tau, labels):
    d = dp.DistillDesc(dtype, dtype, 2, 3, 1000, 16, 0, 0, 1000, 1000, tau, 0.5 if labels else 0.0)
    dp.dp_distill(d, PTR, PTR, PTR, labels=PTR if labels else None, row_loss=PTR, loss=PTR, dlogits=PTR, stream=STREAM)


BF16, FP32 = 0, 1
CALLS = {
    "forward 64": lambda dp: _attention(dp, BF16, 2, 300, 2, 2, 64),
    "forward 128": lambda dp: _attention(dp, BF16, 1, 300, 2, 2, 128),
    "forward 128, pairs": lambda dp: _attention(dp, BF16, 16, 1024, 16, 16, 128),
    "gradient 64": lambda dp: _gradient(dp, BF16, 2, 300, 4, 2, 64),
    "gradient 128": lambda dp: _gradient(dp, BF16, 2, 300, 4, 2, 128),
    "gradient, short": lambda dp: _gradient(dp, BF16, 2, 100, 2, 2, 64),
    **{f"fp32 forward {D}": lambda dp, D=D: _attention(dp, FP32, 2, 100, 2, 2, D) for D in (32, 33, 64, 128)},
    **{f"fp32 gradient {D}": lambda dp, D=D: _gradient(dp, FP32, 2, 100, 2, 2, D) for D in (32, 33, 64, 128)},
    **{f"bf16 odd {D}": lambda dp, D=D: (_attention(dp, BF16, 2, 100, 2, 2, D), _gradient(dp, BF16, 2, 100, 2, 2, D))
       for D in (31, 63, 127)},
    **{f"distill {t} {y} {tau}": lambda dp, t=t, y=y, tau=tau: _distill(dp, t, tau, y)
       for t in (BF16, FP32) for y, tau in ((False, 1.0), (True, 1.0), (True, 2.0), (True, 3.0), (True, 4.0))},
}


@pytest.mark.parametrize("name", CALLS)
def test_every_device_and_once_on_each(fake, name):
    for dev in (0, 1, 5, 1, 0):
        fake.so.fake_device(dev)
        CALLS[name](fake.dp)
        assert {(d, status) for _, _, d, _, status in fake.launches()} == {(dev, 0)}
    n = fake.so.fake_attribute_calls()
    for dev in (0, 1, 5):
        fake.so.fake_device(dev)
        CALLS[name](fake.dp)
    assert fake.so.fake_attribute_calls() == n


def test_a_failure_is_not_kept():
    """In a process of its own, where no kernel has been asked for yet."""
    import subprocess
    import sys
    code = """
import sys
sys.path[:0] = [%r, %r]
import test_operator_devices as t
h = t.Host()
with h.installed():
    for name, call in t.CALLS.items():
        n = h.so.fake_attribute_calls()
        h.so.fake_fail_attributes(1)
        try:
            call(h.dp)
        except h.dp.DPError as e:
            assert e.status == h.dp.DP_ERR_CUDA, name
        else:
            assert h.so.fake_attribute_calls() == n, name    # the kernel had been asked for before
        h.so.fake_fail_attributes(0)
        call(h.dp)
        assert all(s == 0 for *_, s in h.launches()[-1:]), name
""" % (ROOT, HERE)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
