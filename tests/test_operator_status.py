"""dp_check_status with several conditions raised: the cause is reported before its effect, and the message
names each.  On a stand-in for the CUDA runtime (host_library)."""
import pytest

from host_library import STREAM, Host

NONFINITE, TIMEOUT, INDEX = 1, 2, 4   # the device word's bits


@pytest.fixture(scope="module")
def host():
    return Host()


@pytest.mark.parametrize("bits,name", [
    (0, "DP_OK"), (NONFINITE, "DP_ERR_NONFINITE"), (INDEX, "DP_ERR_INVALID_ARG"), (TIMEOUT, "DP_ERR_TIMEOUT"),
    (INDEX | NONFINITE, "DP_ERR_INVALID_ARG"),      # an index out of range makes NaN rows, and these such norms
    (TIMEOUT | INDEX | NONFINITE, "DP_ERR_TIMEOUT"),  # a kernel that gave up leaves its outputs unwritten
    (TIMEOUT | NONFINITE, "DP_ERR_TIMEOUT"),
])
def test_the_cause_before_the_effect(host, bits, name):
    words = {NONFINITE: "not finite", TIMEOUT: "wait gave up", INDEX: "out of range"}
    with host.installed():
        host.so.fake_status(bits)
        assert host.dp.dp_check_status(STREAM) == getattr(host.dp, name)
        text = host.so.dp_last_error().decode() if bits else ""
        assert all((w in text) == bool(bits & b) for b, w in words.items())
        assert host.dp.dp_check_status(STREAM) == host.dp.DP_OK
