"""paged_decode_attention_fp8_block on the GPU against the fp64 oracle over
the dequantised pools, within the bound derived in ``block_cases``."""
import math

import numpy as np
import pytest
import torch

import block_cases as C
from oracle import fp8_block as FB
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


def _q(b, hq, seed, size=1.0):
    g = torch.Generator().manual_seed(700 + seed)
    return (torch.randn(b, hq, 128, generator=g) * size).to(torch.bfloat16)


def _case(lens, hkv, group, seed=1, poison=True, **kw):
    table, nb = C.tables(lens, seed)
    pools = C.Pools(nb, hkv, seed, **kw)
    if poison:
        C.poison(pools, table, lens)
    return pools, _q(len(lens), hkv * group, seed), table


@pytest.mark.parametrize("hkv,group", [(8, 4), (4, 1), (4, 16), (8, 8), (2, 4), (1, 8), (1, 1), (3, 2), (1, 16), (5, 1)])
@pytest.mark.parametrize("lens", [[1], [16, 1, 17, 15], [777], [64, 65, 63, 128, 1000, 512, 513, 2]])
def test_against_the_oracle(lens, hkv, group):
    pools, q, table = _case(lens, hkv, group, seed=hkv * group + len(lens))
    C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, table, lens, SCALE))


@pytest.mark.parametrize("b,longest,hkv,group", [(1, 20000, 8, 4), (2, 9000, 1, 8), (40, 1500, 8, 4), (200, 300, 4, 2),
                                                 (30, 3000, 2, 4), (1, 5000, 2, 16)])
def test_batches_cut_into_shares(b, longest, hkv, group):
    g = torch.Generator().manual_seed(b)
    lens = [max(1, int(longest * float(torch.rand(1, generator=g)))) for _ in range(b)]
    lens[0] = longest
    pools, q, table = _case(lens, hkv, group, seed=b)
    got = C.decode(pools, q, table, lens, SCALE)
    rows = sorted({0, b - 1, int(np.argmin(lens)), b // 2})
    C.check_decode(pools, q, table, lens, SCALE, got, rows=rows)
    assert torch.equal(got, C.decode(pools, q, table, lens, SCALE))     # and the same again, bit for bit


def test_large_max_seq_len_changes_only_the_cut():
    lens = [100, 1, 700]
    pools, q, table = _case(lens, 4, 4)
    wide = torch.zeros(3, 4096, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    for msl in (700, 5000, 65536):
        C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, wide, lens, SCALE, max_seq_len=msl))


@pytest.mark.parametrize("hkv", [4, 2])
def test_block_scales_far_apart(hkv):
    """Scales spread over 2^+-20 from block to block, K and V."""
    lens = [300, 33]
    pools, q, table = _case(lens, hkv, 4, k_spread=3, v_spread=20)
    C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, table, lens, SCALE))


@pytest.mark.parametrize("hkv", [4, 1])
@pytest.mark.parametrize("byte", [1, 90])
def test_a_block_that_takes_the_weight_and_holds_small_values(hkv, byte):
    """The first block draws almost all of the softmax while its V scale is
    far below the others': its weight still counts in the sum."""
    lens = [200]
    pools, q, table = _case(lens, hkv, 2, poison=False)
    q = torch.ones_like(q)
    first = int(table[0, 0])
    pools.codes[0][first] = 0x70                             # 128 * 2^-7 = 1 in every element: score 11.3
    pools.scale[0][first] = 120
    pools.scale[1][first] = byte
    got = C.decode(pools, q, table, lens, SCALE)
    C.check_decode(pools, q, table, lens, SCALE, got)


@pytest.mark.parametrize("hkv,group", [(4, 4), (4, 16), (4, 1), (3, 8)])
@pytest.mark.parametrize("spread", [20, 45, 60])
def test_v_scales_far_apart(spread, hkv, group):
    """Beyond a spread of 40 binades the softmax sum is taken on its own."""
    lens = [700, 90, 33, 2000]
    pools, q, table = _case(lens, hkv, group, seed=spread, v_spread=spread)
    C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, table, lens, SCALE))


@pytest.mark.parametrize("hkv", [4, 3])
@pytest.mark.parametrize("at", [0, 5, 31, 32, 36])
@pytest.mark.parametrize("byte", [1, 60, 86, 87, 88, 200])
def test_one_block_far_from_the_others(at, byte, hkv):
    """A block that holds most of the weight and whose V scale is far below or
    above the others' (40 binades from one of them on), first, later and last."""
    lens = [590, 20]
    pools, q, table = _case(lens, hkv, 2, poison=False)
    q = torch.ones_like(q)
    blk = int(table[0, at])
    pools.codes[0][blk] = 0x70                               # 128 * 2^-7 = 1 in every element: score 11.3
    pools.scale[0][blk] = 120
    pools.scale[1][blk] = byte
    C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, table, lens, SCALE))


@pytest.mark.parametrize("hkv", [4, 1])
@pytest.mark.parametrize("n", [200, 3000])
def test_rare_keys_with_large_values(n, hkv):
    """A quarter of the keys weighs 2^-33 of the others and holds values 2^33
    as large: both count alike, in whichever piece they fall."""
    pools, q, table = _case([n], hkv, 2, poison=False, k_spread=0, v_spread=0)
    q = torch.ones_like(q)
    far = table[0, : n // 64].long()
    pools.codes[0][far] = 0xF0                               # -128 * 2^-6 = -2 in every element: score -22.6
    pools.scale[0][far] = 121
    pools.scale[1][far] += 33
    C.check_decode(pools, q, table, [n], SCALE, C.decode(pools, q, table, [n], SCALE))


def test_large_and_small_queries_and_scales():
    lens = [90, 700]
    for size, k_exp in ((2.0 ** 70, -80), (2.0 ** -70, 60), (2.0 ** 17, -20)):
        pools, q, table = _case(lens, 4, 4)
        q = (q.float() * size).to(torch.bfloat16)
        pools.scale[0] = (pools.scale[0].int() + k_exp).to(torch.uint8)
        got = C.decode(pools, q, table, lens, SCALE)
        C.check_decode(pools, q, table, lens, SCALE, got)


def test_extreme_v_scales():
    lens = [600]
    for byte in (1, 20, 220, 230):
        pools, q, table = _case(lens, 4, 4, v_spread=0)
        pools.scale[1][:] = byte
        got = C.decode(pools, q, table, lens, SCALE)
        if byte > 1:
            C.check_decode(pools, q, table, lens, SCALE, got)
        else:                                                # values of at most 448 * 2^-126: subnormal results may flush
            assert bool((got.double().abs() <= 448.0 * 2.0 ** -126).all())


def test_padded_rows_are_left_alone():
    lens = [40, 0, 700, 0]
    pools, q, table = _case(lens, 4, 4)
    for msl in (None, 40000):
        wide = torch.zeros(4, 2500, dtype=torch.int32)
        wide[:, :table.shape[1]] = table
        out = torch.full((4, 16, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        got = C.decode(pools, q, wide, lens, SCALE, max_seq_len=msl, out=out)
        C.check_decode(pools, q, table, lens, SCALE, got)
        assert bool((got[1] == 3).all()) and bool((got[3] == 3).all())
    none = C.decode(pools, q, table, [0, 0, 0, 0], SCALE, max_seq_len=40)
    assert not bool(none.any())


def test_bad_lengths_and_blocks_are_reported():
    lens = [40, 50, 60]
    pools, q, table = _case(lens, 4, 4, poison=False)
    good = C.decode(pools, q, table, lens, SCALE)
    for bad in (61, -1, 1 << 30):
        got = C.decode(pools, q, table, [40, bad, 60], SCALE, max_seq_len=60, expect=3)
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])
    for bad in (-1, pools.codes[0].shape[0], 1 << 30):
        t2 = table.clone()
        t2[1, 1] = bad
        got = C.decode(pools, q, t2, lens, SCALE, expect=2)
        assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])


def test_nan_code_makes_its_sequence_nan():
    lens = [40, 50]
    pools, q, table = _case(lens, 4, 1, poison=False)
    good = C.decode(pools, q, table, lens, SCALE)
    pools.codes[0][int(table[1, 2]), 1, 3, 7] = C.NAN_CODE
    got = C.decode(pools, q, table, lens, SCALE)
    assert torch.equal(got[0], good[0]) and torch.equal(got[1, [0, 2, 3]], good[1, [0, 2, 3]])
    assert bool(got[1, 1].isnan().all())


def test_empty_batch_and_graphs_that_share_a_workspace():
    lens = [700, 1500]
    pools, q, table = _case(lens, 4, 4)
    C.decode(pools, q[:0], table[:0], [], SCALE, max_seq_len=16)
    ref = C.decode(pools, q, table, lens, SCALE)
    dev = pools.cuda()
    ws = B.decode_workspace_fp8_block(2, 16, 4, 128, 1500)
    qs = [q.cuda(), q.flip(0).contiguous().cuda()]
    ts = [table.cuda(), table.flip(0).contiguous().cuda()]
    ls = [torch.tensor(x, dtype=torch.int32).cuda() for x in (lens, lens[::-1])]
    outs = [torch.zeros(2, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            B.paged_decode_attention_fp8_block(outs[i], qs[i], *dev, ts[i], ls[i], 1500, SCALE, ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    assert torch.equal(outs[0].cpu(), ref) and torch.equal(outs[1].cpu(), ref.flip(0))


def test_workspace_of_a_larger_batch_serves_smaller_ones():
    """A small batch has shorter splits and so more partials a row than a large
    one; a workspace too small for them makes the splits longer."""
    n = B.decode_fp8_block_workspace_bytes
    lens = [4000, 33, 2100]
    pools, q, table = _case(lens, 4, 4)
    least = B.decode_workspace_bytes(3, 16, 128, 4000)
    full = n(3, 16, 4, 128, 4000)
    assert least < full
    for size in (least, least + 512, (least + full) // 2 // 256 * 256, full):
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, table, lens, SCALE, workspace=ws))
    with pytest.raises(B.PagedKVError, match="status 3"):
        C.decode(pools, q, table, lens, SCALE, workspace=torch.empty(least - 256, dtype=torch.uint8, device="cuda"))


def test_up_to_512_tokens_need_no_workspace():
    lens = [500, 3]
    pools, q, table = _case(lens, 4, 4)
    out = torch.zeros(2, 16, 128, dtype=torch.bfloat16, device="cuda")
    B.paged_decode_attention_fp8_block(out, q.cuda(), *pools.cuda(), table.cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda(), 500, SCALE)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    C.check_decode(pools, q, table, lens, SCALE, out.cpu())


def test_other_stream():
    lens = [300, 20]
    pools, q, table = _case(lens, 4, 4)
    ref = C.decode(pools, q, table, lens, SCALE)
    s = torch.cuda.Stream()
    assert torch.equal(C.decode(pools, q, table, lens, SCALE, stream=s), ref)


def test_one_scale_everywhere_matches_the_per_head_cache():
    """With one power of two for all blocks of a head the two caches hold the
    same values."""
    lens = [130, 900]
    pools, q, table = _case(lens, 4, 4, k_spread=0, v_spread=0)
    got = C.decode(pools, q, table, lens, SCALE)
    kc, vc, _, _ = pools.cuda()
    out = torch.zeros_like(got).cuda()
    one = torch.full((4,), 2.0 ** -7, device="cuda")
    B.paged_decode_attention_fp8(out, q.cuda(), kc, vc, one, one, table.cuda(),
                                 torch.tensor(lens, dtype=torch.int32).cuda(), 900, SCALE,
                                 B.decode_workspace(2, 16, 128, 900))
    C.check_decode(pools, q, table, lens, SCALE, out.cpu())
    C.check_decode(pools, q, table, lens, SCALE, got)
