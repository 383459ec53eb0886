"""chunked_prefill_attention_fp8_block on the GPU against the fp64 oracle over
the dequantised pools, within the bound derived in ``block_cases``: the kernel
rounds each weight to f16 and the result to bf16."""
import pytest
import torch

import block_cases as C
import oracle
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


def _case(prior, chunk, hkv, group, seed=1, poison=True, **kw):
    table, nb = C.tables([prior + chunk], seed)
    pools = C.Pools(nb, hkv, seed, **kw)
    if poison:
        C.poison(pools, table, [prior + chunk])
    g = torch.Generator().manual_seed(800 + seed)
    return pools, torch.randn(chunk, hkv * group, 128, generator=g).to(torch.bfloat16), table[0]


def _run(pools, q, row, prior, expect=0, stream=None):
    kc, vc, ks, vs = pools.cuda()
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    B.chunked_prefill_attention_fp8_block(out, q.cuda(), kc, vc, ks, vs, row.cuda(), prior, SCALE, stream)
    torch.cuda.synchronize()
    assert B.get_device_error() == expect
    return out.cpu()


def _check(pools, q, row, prior, got, rows=None):
    """As block_cases.check_decode: weights rounded to f16 (2^-11, or 2^-25 of
    the largest weight times V scale), scores and sums below 2^-13."""
    chunk = q.shape[0]
    rows = sorted({0, chunk // 2, chunk - 1}) if rows is None else rows
    pairs = [(r, (7 * i) % q.shape[1]) for i, r in enumerate(rows)]
    pairs += [(rows[-1], h) for h in range(q.shape[1])]
    used = row[:-(-(prior + chunk) // 16)].long()                # unused blocks may hold NaN
    k, v = (torch.nan_to_num(pools.values(i)[used], 0.0) for i in (0, 1))
    ids = torch.arange(len(used), dtype=torch.int32)
    unit = torch.exp2(pools.scale[1][used].double() - 127)[:, :, None, None].expand_as(v).contiguous()
    ref, ref_abs, top = (oracle.chunked_prefill(q.double(), k, x, ids, prior, SCALE, rows=pairs)
                         for x in (v, v.abs(), unit))
    keys = torch.tensor([prior + r + 1.0 for r, _ in pairs]).double()[:, None]
    got = torch.stack([got[r, h] for r, h in pairs]).double()
    over = (got - ref).abs() - C.bound(ref, ref_abs, 2.0 ** -11 + 2.0 ** -13) - keys * 2.0 ** -25 * 448.0 * top
    assert bool((over <= 0).all()), float(over.max())


@pytest.mark.parametrize("hkv,group", [(8, 4), (2, 1), (4, 8), (1, 16), (3, 2), (1, 1)])
@pytest.mark.parametrize("prior,chunk", [(0, 1), (0, 16), (5, 1), (127, 1), (128, 1), (500, 77), (0, 129), (300, 260),
                                         (1023, 2)])
def test_against_the_oracle(prior, chunk, hkv, group):
    pools, q, row = _case(prior, chunk, hkv, group, seed=prior + chunk + hkv)
    _check(pools, q, row, prior, _run(pools, q, row, prior))


@pytest.mark.parametrize("prior,chunk", [(2000, 600), (4096, 2048), (777, 1111)])
def test_large_chunks(prior, chunk):
    pools, q, row = _case(prior, chunk, 8, 4, seed=chunk)
    got = _run(pools, q, row, prior)
    _check(pools, q, row, prior, got, rows=[0, 127, 128, chunk // 2, chunk - 1])


def test_every_code_and_many_scales():
    """All finite codes, subnormals among them, K scales from 2^-20 to 2^20 and
    V scales from 2^-39 to 2^39."""
    pools, q, row = _case(300, 40, 2, 2, poison=False)
    n = pools.codes[0].shape[0]
    codes = torch.arange(256, dtype=torch.uint8).repeat(16 * 128 // 256).reshape(16, 128)
    codes[(codes & 0x7F) == 0x7F] = 0
    for i, step in ((0, 5), (1, 10)):
        pools.codes[i][:] = codes
        pools.scale[i][:] = (127 - 4 * step + step * (torch.arange(n) % 9))[:, None].to(torch.uint8)
    q = (q.float() * 2.0 ** -20).to(torch.bfloat16)
    _check(pools, q, row, 300, _run(pools, q, row, 300))


@pytest.mark.parametrize("spread", [20, 45, 60])
@pytest.mark.parametrize("prior,chunk", [(0, 60), (400, 200)])
def test_v_scales_far_apart(spread, prior, chunk):
    """Beyond a spread of 40 binades the softmax sum is taken on its own."""
    pools, q, row = _case(prior, chunk, 2, 4, seed=spread, v_spread=spread)
    _check(pools, q, row, prior, _run(pools, q, row, prior))


@pytest.mark.parametrize("at", [0, 5, 9, 30, 37])
@pytest.mark.parametrize("byte", [1, 60, 200])
def test_one_block_far_from_the_others(at, byte):
    """A block that holds most of the weight and whose V scale is far below
    or above the others', in the first tile, a later one and the chunk's own."""
    prior, chunk = 480, 128
    pools, q, row = _case(prior, chunk, 2, 2, poison=False)
    q = torch.ones_like(q)
    blk = int(row[at])
    pools.codes[0][blk] = 0x70                               # 128 * 2^-7 = 1 in every element: score 11.3
    pools.scale[0][blk] = 120
    pools.scale[1][blk] = byte
    _check(pools, q, row, prior, _run(pools, q, row, prior), rows=[0, 1, 15, 16, 100, 112, 113, 127])


@pytest.mark.parametrize("prior,chunk,hkv", [(480, 32, 1), (900, 130, 8), (3000, 1, 2)])
def test_rare_keys_with_large_values(prior, chunk, hkv):
    """A quarter of the keys weighs 2^-33 of the others and holds values 2^33
    as large: both count alike, in whichever CTA they fall."""
    pools, q, row = _case(prior, chunk, hkv, 2, poison=False, k_spread=0, v_spread=0)
    q = torch.ones_like(q)
    far = row[: prior // 64].long()
    pools.codes[0][far] = 0xF0                               # -128 * 2^-6 = -2 in every element: score -22.6
    pools.scale[0][far] = 121
    pools.scale[1][far] += 33
    _check(pools, q, row, prior, _run(pools, q, row, prior))


def test_zero_values_still_take_their_weight():
    pools, q, row = _case(300, 30, 2, 2, poison=False)
    for b in row[2:9].tolist():
        pools.codes[1][b] = 0
        pools.scale[1][b] = 1                                # as an append of zeros leaves it
    _check(pools, q, row, 300, _run(pools, q, row, 300))


@pytest.mark.parametrize("byte", [0, 1, 7, 8, 134, 135, 240])
def test_extreme_v_scales(byte):
    pools, q, row = _case(100, 30, 2, 2, poison=False)
    pools.scale[1][:] = byte
    got = _run(pools, q, row, 100)
    if byte > 1:
        _check(pools, q, row, 100, got)
    else:                                                    # subnormal results may flush
        assert bool((got.double().abs() <= 448.0 * 2.0 ** (byte - 127)).all())


@pytest.mark.parametrize("size,k_exp", [(2.0 ** 70, -80), (2.0 ** -70, 60), (2.0 ** 17, -20), (2.0 ** -100, -90)])
def test_large_and_small_queries_and_scales(size, k_exp):
    pools, q, row = _case(200, 50, 2, 2)
    q = (q.float() * size).to(torch.bfloat16)
    pools.scale[0] = (pools.scale[0].int() + k_exp).to(torch.uint8)
    _check(pools, q, row, 200, _run(pools, q, row, 200))


def test_agrees_with_the_bf16_call_on_the_same_values():
    """A code times its scale is a bf16 number, so both calls attend over the
    same values; the bf16 call also rounds its weights to bf16 (2^-8)."""
    pools, q, row = _case(300, 200, 8, 4, poison=False)
    got = _run(pools, q, row, 300)
    kc, vc = (pools.values(i).to(torch.bfloat16).cuda() for i in (0, 1))
    assert torch.equal(kc.cpu().double(), pools.values(0))
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    B.chunked_prefill_attention(out, q.cuda(), kc, vc, row.cuda(), 300, SCALE)
    mean_abs = float(pools.values(1).abs().max())
    assert float((got.double() - out.cpu().double()).abs().max()) <= (2.0 ** -8 + 2.0 ** -7) * mean_abs


def test_nan_codes_reach_the_rows_that_see_them():
    for which in (0, 1):
        pools, q, row = _case(100, 60, 2, 2, poison=False)
        good = _run(pools, q, row, 100)
        pools.codes[which][int(row[130 // 16]), 1, 130 % 16, 9] = 0xFF
        got = _run(pools, q, row, 100)
        assert torch.equal(got[:, :2], good[:, :2])          # the other KV head's queries
        assert torch.equal(got[:30], good[:30])              # rows before the key
        assert bool(got[30:, 2:, 9].isnan().all())
        assert which == 1 or bool(got[30:, 2:].isnan().all())
    pools, q, row = _case(300, 20, 2, 2, poison=False)       # and a key that every row sees
    pools.codes[1][int(row[1]), 0, 3, 9] = 0x7F
    assert bool(_run(pools, q, row, 300)[:, :2, 9].isnan().all())


def test_bad_block_is_reported_and_skipped():
    pools, q, row = _case(100, 60, 2, 2, poison=False)
    for bad in (-1, pools.codes[0].shape[0], 1 << 30):
        r2 = row.clone()
        r2[3] = bad
        _run(pools, q, r2, 100, expect=2)
        assert B.get_device_error() == 0
    assert bool(_run(pools, q, row, 100).isfinite().all())


def test_chunks_add_up_and_empty_chunk():
    pools, q, row = _case(0, 400, 4, 4)
    whole = _run(pools, q, row, 0)
    _check(pools, q, row, 0, whole, rows=[0, 1, 15, 16, 128, 399])
    # a chunk that begins on a tile's border reads the same tiles
    parts = [_run(pools, q[:256], row, 0), _run(pools, q[256:], row, 256)]
    assert torch.equal(torch.cat(parts), whole)
    assert _run(pools, q[:0], row, 0).shape[0] == 0


def test_graph_and_other_stream():
    pools, q, row = _case(200, 100, 4, 4)
    ref = _run(pools, q, row, 200)
    assert torch.equal(_run(pools, q, row, 200, stream=torch.cuda.Stream()), ref)
    kc, vc, ks, vs = pools.cuda()
    qd, rd, out = q.cuda(), row.cuda(), torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.chunked_prefill_attention_fp8_block(out, qd, kc, vc, ks, vs, rd, 200, SCALE)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), ref)


@pytest.mark.parametrize("hkv,group,prior,chunk", [
    (8, 4, 1000, 500),      # 64 items: clusters of 2
    (4, 2, 1200, 1270),     # 40 items: 3
    (1, 2, 960, 50),        # one item of 8 tiles: 4
    (1, 2, 590, 40),        # of 5: 5
    (1, 2, 730, 30),        # of 6: 6
    (1, 2, 850, 40),        # of 7: 7
    (1, 2, 3100, 60),       # of 25: 8
    (1, 1, 3100, 200), (3, 1, 1500, 300), (16, 16, 300, 140)])
def test_every_cluster_size(hkv, group, prior, chunk):
    pools, q, row = _case(prior, chunk, hkv, group, seed=9)
    _check(pools, q, row, prior, _run(pools, q, row, prior))
