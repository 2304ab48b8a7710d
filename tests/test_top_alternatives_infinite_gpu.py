"""The largest alternatives of rows with more infinities than there are places for and some NaN above them, index
by index: a NaN ranks above every number, +inf above every other, equal ones by their index."""
import math

import pytest

import layers_reference as ref

pytestmark = pytest.mark.gpu

KINDS = ["one NaN", "NaN apart", "fewer NaN than places", "more NaN than places", "all NaN", "a stretch of NaN", "all inf",
         "inf above numbers", "NaN and numbers", "NaN above masks", "inf and masks"]


def _row(kind, V, K, dtype):
    import torch
    i = torch.arange(V, device="cuda")
    z = torch.full((V,), math.inf, device="cuda")
    if kind == "one NaN":
        z[V // 2] = math.nan
    elif kind == "NaN apart":
        z[:: max(1, V // 17)] = math.nan
    elif kind == "fewer NaN than places":
        z[(torch.arange(max(0, K - 1), device="cuda") * 37 + 5) % V] = math.nan
    elif kind == "more NaN than places":
        z[1::3] = math.nan
    elif kind == "all NaN":
        z[:] = math.nan
    elif kind == "a stretch of NaN":
        z[V // 3: V // 3 + max(1, K // 2)] = math.nan
    elif kind == "inf above numbers":
        z[::2] = (i[::2] % 5).float()
    elif kind == "NaN and numbers":
        z[:] = 2.0
        z[3 % V] = math.nan
    elif kind == "NaN above masks":
        z[:] = -math.inf
        z[V - 1] = math.nan
    elif kind == "inf and masks":
        z[1::2] = -math.inf
    return z.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", KINDS)
def test_alternatives_of_rows_with_infinities_and_nan(lib, kind, dtype):
    import torch
    # 256 threads a row, a row a cluster, and (many rows) 64 and 128 threads
    for N, V, K in ((1, 5, 3), (3, 3000, 20), (3, 50257, 128), (1, 140000, 50), (400, 9001, 128), (610, 3000, 20), (610, 9001, 32),
                    (610, 30001, 64)):
        row = _row(kind, V, K, dtype)
        lp, h, _, best, at = lib.token_logprobs_forward(row.expand(1, N, V).contiguous(), top=K)
        assert torch.equal(at.long(), ref.top(row[None, None], K).expand(1, N, K)), (N, V, K)
        assert torch.isnan(h).all() and torch.isnan(best).all(), (N, V, K)   # a NaN or +inf spoils the row's values
        assert not lp.any()
    assert lib.dp_check_status() == lib.DP_OK
