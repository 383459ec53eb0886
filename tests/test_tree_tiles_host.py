"""The bound of the long tree batches rejects a tile that is lost, counted
twice or in another's place (no GPU)."""
import pytest
import torch

from oracle import tree as T
from tree_cases import Batch
from tree_tiles import mark_tiles, tile_shares


@pytest.mark.parametrize("lens,drafted,hq,hkv", [([20011, 5000], [3, 1], 8, 8), ([20000], [9], 8, 2)])
def test_every_tile_counts(lens, drafted, hq, hkv):
    x = mark_tiles(Batch(lens, drafted, hq, hkv, seed=hq))
    ref, _ = T.tree_attention(*x.args())
    tol, _ = x.bounds(ref)
    for b in range(len(lens)):
        rows = slice(int(x.offsets[b]), int(x.offsets[b + 1]))
        part, weight = tile_shares(x, b)
        assert float((part.sum(2) - ref[rows]).abs().max()) < 1e-12
        room = tol[rows] + 1e-300                # channels without a tile: 0, exactly
        lost = (part.abs() / room[:, :, None]).amax((0, 1, 3))              # by this many times the bound, per tile
        assert float(lost.min()) > 10
        # values of the next tile in a tile's place (and the other way round)
        value = part / weight[..., None]
        step = (value[:, :, 1:] - value[:, :, :-1]) * (weight[:, :, :-1] - weight[:, :, 1:])[..., None]
        swapped = (step.abs() / room[:, :, None]).amax((0, 1, 3))
        assert float(swapped.min()) > 3


def test_random_values_would_hide_a_tile():
    """Why the values are marked: the same bound with random ones."""
    x = Batch([20011], [3], 8, 8, seed=8)
    ref, _ = T.tree_attention(*x.args())
    tol, _ = x.bounds(ref)
    part, _ = tile_shares(x, 0)
    assert float((part.abs() / tol[:, :, None]).amax((0, 1, 3)).min()) < 1
