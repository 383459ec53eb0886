"""paged_tree_attention over long sequences whose values tell their tiles apart."""
import pytest

from test_gpu_tree import check, run
from tree_cases import BF16, F32, Batch
from tree_tiles import mark_tiles

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,hq,drafted", [(BF16, 8, 3), (BF16, 32, 20), (BF16, 64, 64), (F32, 8, 3)])
def test_every_tile_in_its_place(dtype, hq, drafted):
    """Few rows, more than 128 and more than 256 of a KV head; many tiles a CTA."""
    x = mark_tiles(Batch([20011, 5000], [drafted, 1], hq, 8, dtype=dtype, seed=hq))
    check(x, *run(x))
