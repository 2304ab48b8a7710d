"""The sizes that the sums and norms of given per-example gradients take; on a stand-in for the CUDA runtime."""
import pytest

from host_library import PTR, STREAM, Host

UNSUPPORTED = 2


@pytest.fixture(scope="module")
def host():
    return Host()


@pytest.mark.parametrize("B,n,text", [((1 << 30) + 1, 1, "2^30"), (2 ** 31 - 1, 1, "2^30"), (1, (1 << 35) + 1, "2^35")])
def test_sums_refuse(host, B, n, text):
    with host.installed():
        with pytest.raises(host.dp.DPError) as e:
            host.dp.dp_example_sum(PTR, B, n, PTR, PTR, stream=STREAM)
        assert e.value.status == UNSUPPORTED and text in str(e.value) and host.launches() == []


def test_the_largest_sizes_are_taken(host):
    with host.installed():
        host.dp.dp_example_sum(PTR, 1 << 30, 1, PTR, PTR, stream=STREAM)
        host.dp.dp_example_sum(PTR, 1, 1 << 35, PTR, PTR, stream=STREAM)
        host.dp.dp_example_sqnorms(PTR, 2 ** 31 - 1, 1, PTR, stream=STREAM)
        host.dp.dp_example_sqnorms(PTR, 1, 1 << 36, PTR, stream=STREAM)
        with pytest.raises(host.dp.DPError):
            host.dp.dp_example_sqnorms(PTR, 1, (1 << 36) + 1, PTR, stream=STREAM)
        assert len(host.launches()) == 4
