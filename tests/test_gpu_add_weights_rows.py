"""kv_add_weights: a row whose lse is -inf adds nothing, whatever its query and
the keys hold (a padded row, or one that the caller leaves out of the count)."""
import math

import pytest
import torch

from test_gpu_add_weights import check, given_lse, run, start
from tree_cases import BF16, F32, Batch

pytestmark = pytest.mark.gpu


def left_out(x, seed):
    """About a third of the (row, head)s, and every head of each fifth row."""
    out = torch.rand((x.rows, x.hq), generator=torch.Generator().manual_seed(seed)) < 0.3
    out[::5] = True
    return out


@pytest.mark.parametrize("dtype,hq,hkv", [(BF16, 8, 2), (BF16, 16, 1), (BF16, 32, 8), (F32, 8, 2), (F32, 8, 1)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_rows_left_out_add_nothing(dtype, hq, hkv, bad):
    """NaN or infinite scores of such rows, in tiles of the context (all rows see
    every key) and in those of the drafted tokens; up to 1,024 rows a KV head."""
    x = Batch([700, 40, 129, 1100, 17], [9, 3, 2, 64, 17], hq, hkv, dtype=dtype, seed=hq)
    lse, w = given_lse(x), start(x)
    out = left_out(x, hq)
    lse[out] = -math.inf
    x.q[out] = 0
    clean = run(x, w, lse)
    check(x, w, clean, lse)
    x.q[out] = bad
    assert torch.equal(run(x, w, lse), clean)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_key_that_is_infinite_for_rows_left_out_only(dtype):
    """Context tokens with NaN and infinite keys: a sequence without a counted row keeps its sums."""
    x = Batch([300, 200], [5, 40], 8, 2, dtype=dtype, seed=3)
    lse, w = given_lse(x), start(x)
    clean = run(x, w, lse)
    lse[:5] = -math.inf
    for t, bad in ((0, math.nan), (17, math.inf), (140, -math.inf), (296, math.nan)):
        x.k[int(x.table[0, t // 16]), :, t % 16] = bad
    after = run(x, w, lse)
    assert torch.equal(after[0], w[0]) and torch.equal(after[1], clean[1])
