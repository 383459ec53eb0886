"""paged_decode_attention_fp8_block with queries of wide range and at the ends of
bf16, against the fp64 oracle."""
import pytest
import torch

import block_cases as C
from test_gpu_fp8_block_extremes import _decode_case

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.mark.parametrize("hkv,group", [(4, 4), (1, 8), (2, 16)])
@pytest.mark.parametrize("n", [40, 900])
@pytest.mark.parametrize("down", [12, 20, 28])
def test_decode_queries_of_wide_range(down, n, hkv, group, monkeypatch):
    """One element 2^down times the others, at a dimension where the keys are
    zero: the scores are those of the small elements.  The largest, 2, becomes
    2^14, so f16 keeps a bf16 number's bits down to 2^-17 / 2^13 = 2^-30, and a
    smaller one is off by at most half an f16 subnormal, 2^-25 / 2^13 = 2^-38.  A
    key's score is so off by at most delta = scale * 2^-38 * the sum of its |k| at
    those elements, and a weight by the factor e^(2 delta)."""
    pools, q, table = _decode_case([n], hkv, group, seed=n + down)
    q[:, :, 77] = 2.0
    q = (q.float() * 2.0 ** -down).to(torch.bfloat16)
    q[:, :, 77] = 2.0
    pools.codes[0][..., 77] = 0
    pools.scale[0] = (pools.scale[0].int() + down).to(torch.uint8)
    small = (q[0].double().abs() < 2.0 ** -30).double()                              # [heads, 128]
    keys = pools.values(0)[table[0].long()].abs().transpose(0, 1).flatten(1, 2)      # [KV heads, keys, 128]
    delta = SCALE * 2.0 ** -38 * torch.einsum("hgd,hnd->hgn", small.view(hkv, group, 128), keys).amax(-1)
    weights = torch.expm1(2.0 * delta).reshape(1, hkv * group, 1)
    bound = C.bound
    monkeypatch.setattr(C, "bound", lambda ref, ref_abs, rel: bound(ref, ref_abs, rel + weights))
    got = C.decode(pools, q, table, [n], SCALE)
    C.check_decode(pools, q, table, [n], SCALE, got)
    if down < 28:
        assert float(weights.max()) < 2.0 ** -11         # nothing beside the bound's own terms


def test_decode_queries_at_the_ends_of_bf16():
    """Heads of subnormals, of zeros and of the largest numbers, in one batch."""
    lens = [60, 600, 33]
    pools, q, table = _decode_case(lens, 4, 4, seed=3, k_spread=0)
    pools.scale[0][:] = 127
    q = q.float() * 2.0 ** -7
    q[0] *= 2.0 ** -130
    q[1, 3] = 0.0
    q = q.to(torch.bfloat16)
    C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, table, lens, SCALE))
    pools.scale[0][:] = 5
    q = (q.float().clamp(-1.0, 1.0) * 2.0 ** 127).to(torch.bfloat16)
    q[2, 5, 9] = torch.finfo(torch.bfloat16).max
    C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, table, lens, SCALE))
