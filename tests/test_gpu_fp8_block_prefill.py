"""chunked_prefill_attention_fp8_block on the GPU.

A code times its scale is a bf16 number, so the call is held to two things:
the bf16 prefill over pools that hold the same values gives the same result
bit for bit, and the fp64 oracle over the dequantised pools agrees.  The
second bound counts the kernel's roundings: the weights to bf16 (2^-8 each,
numerator only), the bf16 result, and fp32 scores and sums below 2^-13."""
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


def _bf16(pools, q, row, prior):
    kc, vc = (torch.nan_to_num(pools.values(i), 0.0).to(torch.bfloat16).cuda() for i in (0, 1))
    out = torch.zeros(q.shape, dtype=torch.bfloat16, device="cuda")
    B.chunked_prefill_attention(out, q.cuda(), kc, vc, row.cuda(), prior, SCALE)
    torch.cuda.synchronize()
    return out.cpu()


def _check(pools, q, row, prior, got, rows=None):
    k, v = (torch.nan_to_num(pools.values(i), 0.0) for i in (0, 1))
    pairs = None
    if rows is not None:
        pairs = [(r, (7 * i) % q.shape[1]) for i, r in enumerate(rows)]
        got = torch.stack([got[r, h] for r, h in pairs])
    ref = oracle.chunked_prefill(q.double(), k, v, row, prior, SCALE, rows=pairs)
    ref_abs = oracle.chunked_prefill(q.double(), k, v.abs(), row, prior, SCALE, rows=pairs)
    over = (got.double() - ref).abs() - C.bound(ref, ref_abs, 2.0 ** -8 + 2.0 ** -13)
    assert bool((over <= 0).all()), float(over.max())


@pytest.mark.parametrize("hkv,group", [(8, 4), (2, 1), (4, 8), (1, 16), (3, 2), (1, 1)])
@pytest.mark.parametrize("prior,chunk", [(0, 1), (0, 16), (5, 1), (127, 1), (128, 1), (500, 77), (0, 129), (300, 260),
                                         (1023, 2)])
def test_against_the_bf16_call_and_the_oracle(prior, chunk, hkv, group):
    pools, q, row = _case(prior, chunk, hkv, group, seed=prior + chunk + hkv)
    got = _run(pools, q, row, prior)
    assert torch.equal(got, _bf16(pools, q, row, prior))
    _check(pools, q, row, prior, got, rows=sorted({0, chunk // 2, chunk - 1}))


@pytest.mark.parametrize("prior,chunk", [(2000, 600), (4096, 2048), (777, 1111)])
def test_large_chunks(prior, chunk):
    pools, q, row = _case(prior, chunk, 8, 4, seed=chunk)
    got = _run(pools, q, row, prior)
    assert torch.equal(got, _bf16(pools, q, row, prior))
    _check(pools, q, row, prior, got, rows=[0, 127, 128, chunk // 2, chunk - 1])


def test_every_code_and_many_scales():
    """All finite codes, subnormals among them, under scales from 2^-60 to 2^60."""
    pools, q, row = _case(300, 40, 2, 2, poison=False)
    n = pools.codes[0].shape[0]
    codes = torch.arange(256, dtype=torch.uint8).repeat(16 * 128 // 256).reshape(16, 128)
    codes[(codes & 0x7F) == 0x7F] = 0
    for i in (0, 1):
        pools.codes[i][:] = codes
        pools.scale[i][:] = torch.tensor([67, 100, 120, 127, 134, 135, 150, 187])[torch.arange(n) % 8][:, None]
    q = (q.float() * 2.0 ** -60).to(torch.bfloat16)
    got = _run(pools, q, row, 300)
    assert torch.equal(got, _bf16(pools, q, row, 300))


@pytest.mark.parametrize("byte", [0, 1, 7, 8, 134, 135, 246])
def test_extreme_v_scales(byte):
    pools, q, row = _case(100, 30, 2, 2, poison=False)
    pools.scale[1][:] = byte
    pools.codes[1][:] &= 0xF7                        # below 448 / 2 in size: 2^119 * 448 sums to no infinity
    got = _run(pools, q, row, 100)
    assert torch.equal(got, _bf16(pools, q, row, 100))


def test_nan_codes_reach_the_rows_that_see_them():
    for which in (0, 1):
        pools, q, row = _case(100, 60, 2, 2, poison=False)
        good = _run(pools, q, row, 100)
        pools.codes[which][int(row[130 // 16]), 1, 130 % 16, 9] = 0xFF
        got = _run(pools, q, row, 100)
        assert torch.equal(got[:, :2], good[:, :2])          # the other KV head's queries
        assert torch.equal(got[:30], good[:30])              # rows before the key
        assert bool(got[30:, 2:].isnan().all())


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
