"""The stream order of the clipped path behind sequence operators.  Its norm and sum kernels may load
A and G before the launch in front of them has finished, and an operator writes what can be an A or G:
the first launch behind an operator must not start under it, whoever makes it and whatever other host
threads do on the stream.  On a stand-in for the CUDA runtime (host_library), whose log says which
launches may start under the one before."""
import subprocess
import sys

import pytest

from host_library import HERE, PTR, ROOT, STREAM, Host


@pytest.fixture(scope="module")
def host():
    return Host()


@pytest.fixture()
def fake(host):
    with host.installed():
        yield host
        host.so.fake_hook(None)
        host.so.fake_fail_launches(0)


_streams = iter(range(1 << 16, 1 << 24, 1 << 8))   # handles that no other test has used


def _operator(h, stream):
    dp = h.dp
    dp.dp_rotary(dp.RotaryDesc(0, 2, 4, 2, 0, 64, 64, 8, 0, 0, 0, *[dp.Strides(512, 128, 64)] * 4), PTR, None, PTR, None,
                 PTR, None, stream=stream)


def _norm(h, stream, mode="GHOST", T=104):
    dp = h.dp
    d = dp.layer_desc(dp.DP_LINEAR, dp.DP_BF16, B=3, p=64, T=T, d=512)
    dp.dp_layer_sqnorms(d, PTR, PTR, PTR, PTR, mode=getattr(dp, "DP_NORM_" + mode), ws_bytes=1 << 40, stream=stream)


def _sum(h, stream):
    dp = h.dp
    d = dp.layer_desc(dp.DP_LINEAR, dp.DP_BF16, B=3, p=64, T=104, d=512)
    dp.dp_clipped_sum(d, PTR, PTR, PTR, PTR, PTR, PTR, ws_bytes=1 << 40, stream=stream)


def _noise(h, stream):
    h.dp.dp_add_noise(PTR, 1.0, 1.0, 2, 3, n=64, stream=stream)


CALLS = [lambda h, s: _norm(h, s), lambda h, s: _norm(h, s, "INSTANTIATE"), lambda h, s: _norm(h, s, T=700), _sum, _noise]


def _early(h):
    """Of the launches since the last look, which may start under the one before (the operators' left out)."""
    return [early for kernel, _, _, early, _ in h.launches() if "rotary" not in kernel]


def _at_once(h, f):
    """f is called inside the next launch and before it, as by another host thread."""
    keep = h.hook_type(f)
    h.so.fake_hook(keep)
    return keep


@pytest.mark.parametrize("call", CALLS, ids=["ghost", "instantiate", "ghost-split", "sum", "noise"])
def test_the_first_launch_behind_an_operator_waits(fake, call):
    s = next(_streams)
    call(fake, s)
    assert all(_early(fake))
    for _ in range(2):
        _operator(fake, s)
        _operator(fake, s)
        call(fake, s)
        first, *rest = _early(fake)
        assert not first and all(rest)
        call(fake, s)
        assert all(_early(fake))


def test_streams_are_told_apart(fake):
    a, b = next(_streams), next(_streams)
    _operator(fake, a)
    _noise(fake, b)
    _noise(fake, a)
    assert _early(fake) == [True, False]
    fake.so.fake_device(1)   # the same handle on another device
    _operator(fake, a)
    fake.so.fake_device(0)
    _noise(fake, a)
    fake.so.fake_device(1)
    _noise(fake, a)
    assert _early(fake) == [True, False]


def test_another_threads_launch_before_the_operators(fake):
    """It comes between the operator's look at the stream and its launch: what follows still waits."""
    s = next(_streams)
    keep = _at_once(fake, lambda: _noise(fake, s))
    _operator(fake, s)
    log = [("rotary" in kernel, early) for kernel, _, _, early, _ in fake.launches()]
    assert [op for op, _ in log] == [False, True]
    _norm(fake, s)
    assert _early(fake)[0] is False
    del keep


@pytest.mark.parametrize("call", CALLS, ids=["ghost", "instantiate", "ghost-split", "sum", "noise"])
def test_another_threads_launch_before_the_one_that_waits(fake, call):
    """Two threads behind one operator: the one that looked second is launched first, and must wait too."""
    s = next(_streams)
    _operator(fake, s)
    keep = _at_once(fake, lambda: _noise(fake, s))
    call(fake, s)
    assert _early(fake)[:2] == [False, False]
    call(fake, s)
    assert all(_early(fake))
    del keep


def test_an_operator_between_the_look_and_the_launch(fake):
    """The ordinary launch came to stand behind it or before it: the next one waits in any case."""
    s = next(_streams)
    _operator(fake, s)
    keep = _at_once(fake, lambda: _operator(fake, s))
    _noise(fake, s)
    _noise(fake, s)
    _noise(fake, s)
    assert _early(fake) == [False, False, True]
    del keep


def test_both_handles_of_the_default_stream(fake):
    for op, other in ((0, 1), (1, 0)):   # 1: cudaStreamLegacy
        _operator(fake, op)
        _noise(fake, other)
        _noise(fake, op)
        assert _early(fake) == [False, True]


def test_a_launch_that_failed_covers_nothing(fake):
    s = next(_streams)
    _operator(fake, s)
    fake.so.fake_fail_launches(1)
    with pytest.raises(fake.dp.DPError):
        _noise(fake, s)
    _noise(fake, s)
    _noise(fake, s)
    assert _early(fake) == [False, False, True]
    # nor does an operator that was not launched ask for anything
    fake.so.fake_fail_launches(1)
    with pytest.raises(fake.dp.DPError):
        _operator(fake, s)
    _noise(fake, s)
    assert _early(fake) == [True]


_captures = iter(range(1, 1 << 20))


def test_a_captured_launch_covers_no_operator_on_the_stream(fake):
    """Nothing is put on the stream: what is launched after the capture still waits."""
    s = next(_streams)
    _operator(fake, s)
    fake.so.fake_capture(s, next(_captures))
    _noise(fake, s)
    fake.so.fake_capture(s, 0)
    fake.launches()
    _noise(fake, s)
    _noise(fake, s)
    assert _early(fake) == [False, True]


@pytest.mark.parametrize("call", CALLS, ids=["ghost", "instantiate", "ghost-split", "sum", "noise"])
def test_captured_behind_an_operator(fake, call):
    s = next(_streams)
    for _ in range(2):   # a stream is captured again
        fake.so.fake_capture(s, next(_captures))
        _noise(fake, s)
        fake.launches()
        _noise(fake, s)
        assert _early(fake) == [True]
        _operator(fake, s)
        call(fake, s)
        first, *rest = _early(fake)
        assert not first and all(rest)
        call(fake, s)
        assert all(_early(fake))
        fake.so.fake_capture(s, 0)


def test_captured_behind_an_operator_of_another_stream(fake):
    """An event's wait makes the operator one of the kernels that the launch would start under."""
    a, b = next(_streams), next(_streams)
    fake.so.fake_capture(a, next(_captures))
    _operator(fake, a)
    fake.so.fake_join(b, a)
    _norm(fake, b)
    assert _early(fake)[0] is False
    _norm(fake, b)
    assert all(_early(fake))
    _operator(fake, a)
    fake.so.fake_join(b, a)      # now behind its own last launch and the operator
    _norm(fake, b)
    assert _early(fake)[0] is False
    _norm(fake, b)
    assert all(_early(fake))
    _operator(fake, a)
    fake.so.fake_join(a, a)      # another library's kernel behind the operator
    fake.so.fake_join(b, a)
    _norm(fake, b)
    assert _early(fake)[0] is False
    for x in (a, b):
        fake.so.fake_capture(x, 0)


def test_the_per_thread_stream_and_more_streams_than_slots():
    """A process of its own: from then on every launch waits."""
    code = """
import sys
sys.path[:0] = [%r, %r]
import test_operator_order as t
h = t.Host()
with h.installed():
    t._noise(h, 2)
    t._operator(h, 1 << 16)
    t._noise(h, 2)
    assert t._early(h) == [True, False]
    for i in range(2000):
        t._operator(h, (i + 2) << 16)
    h.launches()
    for i in (3, 1500, 1990, 3):
        t._noise(h, i << 16)
    assert t._early(h) == [False] * 4
""" % (ROOT, HERE)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
