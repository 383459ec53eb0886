"""What paged_tree_attention rounds in bf16: the weights (to bf16, as they
multiply the values) and the result; not their sum, nor lse."""
import torch

import pytest

from oracle import tree as T
from test_gpu_tree import run
from tree_cases import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("drafted,hq", [(1, 1), (5, 8), (33, 8)])
def test_a_late_key_between_1_and_256_times_the_earlier_maximum(drafted, hq):
    """Sequence b's last context key scores up to nine powers of two above a key
    of the first tile: up to eight the running maximum stays where it was, and
    the late key's weight is a number that bf16 does not hold."""
    steps = torch.linspace(0, 9, 40).tolist()
    x = Batch([300 + drafted] * 40, [drafted] * 40, hq, 1, seed=drafted, mask="chain")
    g = torch.Generator().manual_seed(1)
    common = torch.randn(128, generator=g)
    x.q = (common + 0.02 * torch.randn(x.q.shape, generator=g)).to(x.q.dtype)
    unit = common / float(common.norm() ** 2) / x.scale / 1.4426950408889634   # scores one power of two more
    for b, s in enumerate(steps):
        for t, power in ((3, 20.0), (299, 20.0 + s)):
            x.k[int(x.table[b, t // 16]), 0, t % 16] = (power * unit).to(x.k.dtype)
    out, lse = run(x)
    ref, ref_lse = T.tree_attention(*x.args())
    tol, tol_lse = x.bounds(ref)            # 2^-8 of each weight's part and of the result
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert bool(((lse.double() - ref_lse).abs() <= tol_lse).all())
    assert float(tol_lse.max()) < 2.0 ** -9    # a sum of rounded weights would be off by up to 2^-8
    # the late key holds up to 512 times the early one's weight, and more than all others together
    late = torch.tensor([float(ref_lse[(b + 1) * drafted - 1, 0]) for b in range(40)])
    assert float(late[-1] - late[0]) > 5.0
