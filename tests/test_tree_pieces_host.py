"""The batches of more than 32 pieces: each tile's loss would show, and the late
keys leave nothing to the first 33 pieces (no GPU)."""
import pytest

from oracle import tree as T
from tree_cases import Batch
from tree_tiles import late_maximum, mark_tiles, tile_shares


@pytest.mark.parametrize("n,hq,hkv,drafted", [(5100, 4, 1, 9), (20000, 4, 2, 5), (90100, 8, 1, 3)])
def test_every_tile_counts(n, hq, hkv, drafted):
    x = mark_tiles(Batch([n], [drafted], hq, hkv, seed=n + hkv))
    ref, _ = T.tree_attention(*x.args())
    tol, _ = x.bounds(ref)
    part, _ = tile_shares(x, 0)
    assert float((part.abs() / (tol + 1e-300)[:, :, None]).amax((0, 1, 3)).min()) > 5


@pytest.mark.parametrize("n", [5100, 20000])
def test_late_keys_take_all_the_weight(n):
    x = late_maximum(mark_tiles(Batch([n], [9], 4, 1, seed=n)), 0.85, n)
    part, weight = tile_shares(x, 0)
    early = int(0.85 * n) // 128
    assert early > 32                                    # the tiles of 33 pieces and more
    assert float(weight[:, :, :early].sum(2).max()) < 2.0 ** -128   # a maximum among them would overflow fp32
    ref, _ = T.tree_attention(*x.args())
    tol, _ = x.bounds(ref)
    shown = (part.abs() / (tol + 1e-300)[:, :, None]).amax((0, 1, 3))
    assert float(shown[early + 1:].min()) > 4
