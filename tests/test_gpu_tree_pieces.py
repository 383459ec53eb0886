"""paged_tree_attention: one sequence cut into more than 32 pieces, up to one for
each CTA, which the second kernel joins (it holds the first 32 in a warp's lanes)."""
import pytest
import torch

from oracle import tree as T
from test_gpu_tree import check, run
from tree_cases import Batch
from tree_tiles import late_maximum, mark_tiles

pytestmark = pytest.mark.gpu

# 40 tiles a KV head (a piece each), 157 (a piece for almost each CTA; few tiles a
# CTA) and 704 (several tiles a piece); one KV head and two, up to 512 rows
LONG = [(5100, 4, 1, 9), (5100, 8, 2, 64), (20000, 8, 1, 5), (20000, 4, 2, 40), (90100, 8, 1, 3), (90100, 4, 2, 17)]


@pytest.mark.parametrize("n,hq,hkv,drafted", LONG)
def test_every_tile_of_every_piece(n, hq, hkv, drafted):
    x = mark_tiles(Batch([n], [drafted], hq, hkv, seed=n + hkv))
    out, lse = run(x)
    check(x, out, lse)
    again = run(x)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("n,hq,hkv,drafted", LONG)
def test_the_maximum_comes_from_a_late_piece(n, hq, hkv, drafted):
    x = late_maximum(mark_tiles(Batch([n], [drafted], hq, hkv, seed=n)), 0.85, n)
    out, lse = run(x)
    ref, ref_lse = T.tree_attention(*x.args())
    tol, tol_lse = x.bounds(ref)
    # the early keys' weights lie below fp32's range: one of less than 2^-126 of
    # the largest is 0, which takes at most n 2^-126 max |v| off a result whose
    # sum of weights is at least 1
    tol = tol + n * 2.0 ** -126 * float(torch.nan_to_num(x.v).abs().max())
    assert bool(((out.double() - ref).abs() <= tol).all())
    assert bool(((lse.double() - ref_lse).abs() <= tol_lse).all())


def test_pieces_that_a_row_sees_nothing_of():
    """No context: a row sees only some of the drafted tokens of the one tile, next to a long sequence."""
    x = mark_tiles(Batch([5100, 64, 9], [5, 64, 9], 4, 1, seed=7, mask="random"))
    check(x, *run(x))
