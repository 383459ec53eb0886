"""paged_decode_attention_fp8 where the softmax scale and the K scales are far
apart: their product is taken first, so that neither is rounded as a subnormal."""
import pytest
import torch

import block_cases as C
import oracle
from oracle import fp8 as F
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hkv,group", [(4, 4), (3, 2), (4, 16)])
@pytest.mark.parametrize("lens", [[40, 7], [900]])
def test_a_subnormal_softmax_scale(lens, hkv, group):
    """scale 2^-145 and K scales of 2^127: with log2(e) the scale alone would be
    rounded to 5 bits.  Queries of 2^13 leave scores of a few units."""
    table, nb = C.tables(lens, hkv)
    g = torch.Generator().manual_seed(hkv)
    kc, vc = ((torch.randn(nb, hkv, 16, 128, generator=g) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
              .view(torch.uint8) for _ in "kv")
    q = (torch.randn(len(lens), hkv * group, 128, generator=g) * 2.0 ** 13).to(torch.bfloat16)
    scale, k_scale, v_scale = 2.0 ** -145, torch.full((hkv,), 2.0 ** 127), torch.full((hkv,), 2.0 ** -7)
    k, v = (torch.from_numpy(F.decode(x.numpy())) * s.double()[:, None, None] for x, s in ((kc, k_scale), (vc, v_scale)))
    sl = torch.tensor(lens, dtype=torch.int32)
    out = torch.zeros(len(lens), hkv * group, 128, dtype=torch.bfloat16, device="cuda")
    B.paged_decode_attention_fp8(out, q.cuda(), kc.cuda(), vc.cuda(), k_scale.cuda(), v_scale.cuda(), table.cuda(),
                                 sl.cuda(), max(lens), scale,
                                 B.decode_workspace(len(lens), hkv * group, 128, max(lens)))
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    ref = oracle.paged_decode(q.double(), k, v, table, sl, scale)
    ref_abs = oracle.paged_decode(q.double(), k, v.abs(), table, sl, scale)
    # half a step of bf16; weights and partials rounded to f16 (2^-11 each, and
    # 2^-25 of a weight's codes of at most 448 below its range); scores below 2^-13
    flush = sl.double()[:, None, None] * 2.0 ** -25 * 448.0 * 2.0 ** -7
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -10 + 2.0 ** -13) * ref_abs + flush
    assert bool(((out.cpu().double() - ref).abs() <= bound).all())
