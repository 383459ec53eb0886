"""The attention over the block-scaled fp8 cache at the ends of its number
ranges, against the fp64 oracle within the bounds of ``block_cases``."""
import pytest
import torch

import block_cases as C
import test_gpu_fp8_block_prefill as P

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(autouse=True)
def subnormal_results(monkeypatch):
    """The shared bound counts half a step of bf16 relative to the value.  The
    subnormal numbers, below 2^-126, are 2^-133 apart: a result rounded to one is
    off by up to 2^-134 (and by 2^-150 for each of the few fp32 subnormals it
    may be made of, together below 2^-143)."""
    bound = C.bound
    monkeypatch.setattr(C, "bound", lambda *a: bound(*a) + 2.0 ** -134 + 2.0 ** -143)


def _decode_case(lens, hkv, group, seed, **kw):
    table, nb = C.tables(lens, seed)
    pools = C.Pools(nb, hkv, seed, **kw)
    g = torch.Generator().manual_seed(900 + seed)
    return pools, torch.randn(len(lens), hkv * group, 128, generator=g).to(torch.bfloat16), table


@pytest.mark.parametrize("hkv,group", [(4, 4), (1, 8), (3, 2), (4, 16)])
@pytest.mark.parametrize("lens", [[20], [300, 5], [600], [3000]])   # one piece, and several
@pytest.mark.parametrize("byte", [0, 1, 2, 240, 246])
def test_decode_v_scales(byte, lens, hkv, group):
    """Every V scale the same: the smallest, and up to values of 448 * 2^119."""
    pools, q, table = _decode_case(lens, hkv, group, seed=byte + lens[0], v_spread=0)
    pools.scale[1][:] = byte
    got = C.decode(pools, q, table, lens, SCALE)
    assert bool(got.isfinite().all()) and bool(got.any())
    C.check_decode(pools, q, table, lens, SCALE, got)


@pytest.mark.parametrize("hkv", [4, 1])
@pytest.mark.parametrize("n", [16, 500, 4000])
@pytest.mark.parametrize("code,byte", [(32, 246), (0x7E, 246), (0xFE, 246), (1, 0), (0x7E, 0), (0x81, 1)])
def test_decode_of_equal_values_is_that_value(n, code, byte, hkv):
    """The mean of equal values, the largest and the smallest of the cache: the
    value itself, to the f16 rounding of its weights and the bf16 one's half step."""
    pools, q, table = _decode_case([n], hkv, 2, seed=n, v_spread=0)
    pools.codes[1][:] = code
    pools.scale[1][:] = byte
    got = C.decode(pools, q, table, [n], SCALE).double()
    value = float(torch.tensor([code], dtype=torch.uint8).view(torch.float8_e4m3fn).double()) * 2.0 ** (byte - 127)
    assert float((got - value).abs().max()) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13) * abs(value) + 2.0 ** -134


@pytest.mark.parametrize("hkv", [4, 1])
@pytest.mark.parametrize("n", [100, 700, 3000])
@pytest.mark.parametrize("low,high", [(1, 246), (0, 200), (60, 246), (1, 60)])
def test_decode_small_and_large_v_scales_together(low, high, n, hkv):
    """Far apart, in turn: the small blocks' weights count beside the large blocks' values."""
    pools, q, table = _decode_case([n], hkv, 4, seed=n, v_spread=0)
    pools.scale[1][table[0, ::2].long()] = low
    pools.scale[1][table[0, 1::2].long()] = high
    C.check_decode(pools, q, table, [n], SCALE, C.decode(pools, q, table, [n], SCALE))


# a query's size against its keys' scale: scores of ordinary size, and 2^-4 of that
SIZES = [(2.0 ** 120, 0), (2.0 ** 116, 0), (2.0 ** 120, 1), (2.0 ** -110, 230)]


@pytest.mark.parametrize("hkv", [4, 3])
@pytest.mark.parametrize("size,byte", SIZES + [(2.0 ** -126, 246)])
def test_decode_k_scales(size, byte, hkv):
    lens = [90, 700]
    pools, q, table = _decode_case(lens, hkv, 4, seed=hkv, k_spread=0)
    q = (q.float() * size).to(torch.bfloat16)
    pools.scale[0][:] = byte
    C.check_decode(pools, q, table, lens, SCALE, C.decode(pools, q, table, lens, SCALE))


@pytest.mark.parametrize("size,byte", SIZES)
def test_prefill_k_scales(size, byte):
    pools, q, row = P._case(200, 50, 2, 2, k_spread=0)
    q = (q.float() * size).to(torch.bfloat16)
    pools.scale[0][:] = byte
    P._check(pools, q, row, 200, P._run(pools, q, row, 200))


@pytest.mark.parametrize("prior,chunk", [(100, 30), (3000, 60)])         # one CTA to an item, and a cluster
@pytest.mark.parametrize("byte", [0, 1, 2, 246])
def test_prefill_v_scales(byte, prior, chunk):
    pools, q, row = P._case(prior, chunk, 2, 2, v_spread=0)
    pools.scale[1][:] = byte
    got = P._run(pools, q, row, prior)
    assert bool(got.isfinite().all()) and bool(got.any())
    P._check(pools, q, row, prior, got)


def _far_block_that_counts_for_nothing(pools, ids, bigger, far):
    """V scales of the smallest block but for one of scale 2^-67, whose keys (from
    -8 in every element, score -90) weigh nothing: the results are of the size of the
    smallest scale, and the softmax sum is taken on its own.  Another block's keys
    beat the first ones by a little (score 5.7)."""
    pools.scale[1][:] = 1
    pools.scale[1][int(ids[far])] = 60
    pools.codes[0][int(ids[bigger])] = 0x68                  # 64 * 2^-7 = 0.5
    pools.scale[0][int(ids[bigger])] = 120
    pools.codes[0][int(ids[far])] = 0xF0                     # -128 * 2^-4 = -8
    pools.scale[0][int(ids[far])] = 123


@pytest.mark.parametrize("hkv", [4, 3])
@pytest.mark.parametrize("bigger", [12, 24])
def test_decode_small_results_beside_a_large_scale(bigger, hkv):
    pools, q, table = _decode_case([500], hkv, 2, seed=5, k_spread=0)
    _far_block_that_counts_for_nothing(pools, table[0], bigger, 20)
    got = C.decode(pools, torch.ones_like(q), table, [500], SCALE)
    assert bool(got.any())
    C.check_decode(pools, torch.ones_like(q), table, [500], SCALE, got)


@pytest.mark.parametrize("hkv,prior,chunk", [(2, 500, 77), (1, 3100, 60), (8, 1000, 500), (1, 850, 40)])
def test_prefill_small_elements_beside_large_ones(hkv, prior, chunk):
    """Queries of zero give every key the same weight, a power of two, so P is
    exact and a result is the mean of the codes rounded to bf16: elements of 448
    and ones of 2^-13 in one row, whichever CTAs of a cluster they come from."""
    pools, q, row = P._case(prior, chunk, hkv, 2, poison=False, k_spread=0, v_spread=0)
    codes = torch.zeros(16, 128, dtype=torch.uint8)
    codes[:, :64] = 0x7E
    codes[torch.arange(128) % 16, torch.arange(128)] = 1     # 2^-9 in every 16th key
    codes[:, :64] = 0x7E
    pools.codes[1][:] = codes
    pools.scale[1][:] = 127
    got = P._run(pools, torch.zeros_like(q), row, prior).double()
    seen = prior + torch.arange(chunk)[:, None] + 1          # keys of each row; those of its 16th: d, d + 16, ...
    mean = ((seen - 1 - torch.arange(128) % 16) // 16 + 1) * 2.0 ** -9 / seen
    mean[:, :64] = 448.0
    # half a step of bf16, and 2^-20 for the fp32 sums of a few thousand exact terms
    assert bool(((got - mean[:, None]).abs() <= (2.0 ** -8 + 2.0 ** -20) * mean[:, None]).all())


@pytest.mark.parametrize("prior,chunk", [(0, 600), (420, 80)])
@pytest.mark.parametrize("bigger", [9, 17, 25])              # before, in and behind the tile of the far block
def test_prefill_small_results_beside_a_large_scale(bigger, prior, chunk):
    pools, q, row = P._case(prior, chunk, 2, 2, poison=False, k_spread=0)
    _far_block_that_counts_for_nothing(pools, row, bigger, 20)
    got = P._run(pools, torch.ones_like(q), row, prior)
    P._check(pools, torch.ones_like(q), row, prior, got, rows=[0, 1, chunk // 2, chunk - 1])
