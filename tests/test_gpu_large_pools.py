"""Blocks that lie beyond 2^32 elements of their pool: every call of the
block-scaled cache and the rotating append gives there, bit for bit, what it
gives over a small pool."""
import pytest
import torch

import block_cases as C
import rope_cases as R
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu

HKV, D, SCALE = 8, 128, 128 ** -0.5
NB = 2 ** 32 // (HKV * 16 * D) + 64          # the last 64 blocks lie beyond


def _rope():
    return B.Rope(R.table(128, D).cuda())


def test_block_scaled_append_decode_and_prefill():
    t = 40
    q, k, v, pos = (x.cuda() for x in R.draw(t, 16, HKV, D, torch.bfloat16, 3, num_positions=128))
    table, nb = C.tables([t], 3)
    p = torch.arange(t)
    outs = []
    for blocks, base in ((nb, 0), (NB, NB - nb)):
        codes = [torch.empty(blocks, HKV, 16, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
        scale = [torch.zeros(blocks, HKV, dtype=torch.uint8, device="cuda") for _ in "kv"]
        for c in codes:
            c[base:] = 0
        row = (table[0] + base).cuda()
        slots = (table[0, p // 16].long() + base).cuda() * 16 + (p % 16).cuda()
        qo = torch.empty_like(q)
        for part in (slice(0, 21), slice(21, t)):            # the second continues a block
            B.kv_append_fp8_block(k[part], v[part], *codes, *scale, slots[part], q_out=qo[part], q=q[part],
                                  positions=pos[:, part].contiguous(), rope=_rope())
        pre, dec = torch.empty_like(qo), torch.empty_like(qo[:1])
        B.chunked_prefill_attention_fp8_block(pre, qo, *codes, *scale, row, 0, SCALE)
        B.paged_decode_attention_fp8_block(dec, qo[-1:], *codes, *scale, row[None],
                                           torch.tensor([t], dtype=torch.int32, device="cuda"), t, SCALE)
        torch.cuda.synchronize()
        assert B.get_device_error() == 0
        outs.append([x.cpu() for x in (qo, pre, dec, codes[0][base:], codes[1][base:], scale[0][base:],
                                       scale[1][base:])])
        del codes
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert bool(outs[0][1].float().abs().sum() > 0)


@pytest.mark.parametrize("d,rot", [(128, 128), (128, 20)])    # whole chunks, single pairs
def test_rotating_append(d, rot):
    t = 5
    q, k, v, pos = (x.cuda() for x in R.draw(t, 4, HKV, d, torch.bfloat16, 4, num_positions=128))
    rope = B.Rope(R.table(128, rot).cuda())
    outs = []
    for blocks in (4, NB):
        pools = [torch.empty(blocks, HKV, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        for x in pools:
            x[-4:] = 0
        slots = (blocks * 16 - 1 - 7 * torch.arange(t)).cuda()
        qo = torch.empty_like(q)
        B.kv_append_rope(qo, q, k, v, *pools, slots, pos, rope)
        torch.cuda.synchronize()
        assert B.get_device_error() == 0
        outs.append([x.cpu() for x in (qo, pools[0][-4:], pools[1][-4:])])
        del pools
    assert all(torch.equal(a, b) for a, b in zip(*outs))
