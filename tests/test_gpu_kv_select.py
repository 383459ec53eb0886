"""kv_select against the oracle: whole numbers, equal."""
import math

import pytest
import torch

from oracle import tree as T
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu
D = "cuda"


def run(w, lens, budget, sinks, recent, max_len=None):
    b, hkv, m = w.shape
    kept = torch.full((b, hkv, budget), -7, dtype=torch.int32, device=D)
    n = torch.full((b,), -7, dtype=torch.int32, device=D)
    B.kv_select(kept, n, w.to(D), torch.tensor(lens, dtype=torch.int32, device=D), max_len or m, sinks, recent)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    return kept.cpu(), n.cpu()


def check(w, lens, budget, sinks, recent, **kw):
    kept, n = run(w, lens, budget, sinks, recent, **kw)
    ref = T.select(w, lens, budget, sinks, recent)
    for b, length in enumerate(lens):
        m = min(length, budget)
        assert int(n[b]) == m
        for h in range(w.shape[1]):
            assert kept[b, h, :m].tolist() == ref[b][h]
        assert bool((kept[b, :, m:] == -7).all())


def tailed(b, hkv, m, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(2 * torch.randn((b, hkv, m), generator=g) - 4)
    return w * (torch.rand((b, hkv, m), generator=g) > 0.1)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 255, 1000, 1023, 1024, 1025, 2301, 4097, 9000])
@pytest.mark.parametrize("part", [0.0, 0.1, 0.5, 1.0])
def test_lengths(n, part):
    budget = max(1, int(n * part))
    sinks = min(4, budget // 3)
    check(tailed(2, 3, n + 5, n), [n, max(1, n - 1)], budget, sinks, budget // 4)


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (8, 8, 0), (8, 0, 8), (8, 3, 5),
                                                 (9, 3, 5), (300, 0, 0), (301, 0, 0), (299, 298, 1)])
def test_budgets(budget, sinks, recent):
    check(tailed(3, 2, 300, 5), [300, 0, 299], budget, sinks, recent)


@pytest.mark.parametrize("values", [[0.0], [0.0, -0.0], [1.0, 0.0], [1.0, math.inf, -math.inf], [0.0, math.nan],
                                    [math.nan], [1e-45, 0.0, -1e-45], [-math.inf], [3.4e38, 3.3e38, math.inf]])
@pytest.mark.parametrize("n", [50, 1500, 5000])
def test_ties_and_odd_numbers(values, n):
    g = torch.Generator().manual_seed(n)
    w = torch.tensor(values)[torch.randint(0, len(values), (1, 2, n), generator=g)]
    for budget in (1, n // 3, n - 1):
        check(w, [n], budget, 0, 0)


def test_equal_in_the_leading_bits():
    """Weights that differ in their last bits only."""
    base = torch.tensor(1.5).view(torch.int32)
    g = torch.Generator().manual_seed(1)
    for span in (2, 200, 70000):
        w = (base + torch.randint(0, span, (2, 2, 6000), generator=g, dtype=torch.int32)).view(torch.float32)
        check(w, [6000, 5000], 1700, 2, 30)


@pytest.mark.parametrize("n", [700, 3500, 8000, 20000])
def test_many_share_the_leading_digits(n):
    """More and fewer than 256 tokens with the threshold's first 11 or 22 bits."""
    base = torch.tensor(1.5).view(torch.int32)
    g = torch.Generator().manual_seed(n)
    for bits in (3, 9, 12, 20, 23):
        w = (base + torch.randint(0, 1 << bits, (1, 2, n), generator=g, dtype=torch.int32)).view(torch.float32)
        w = w * (torch.rand((1, 2, n), generator=g) > 0.9 if bits == 23 else 1)
        for budget in (5, n // 16, n // 2):
            check(w, [n], budget, 0, 3)


@pytest.mark.parametrize("same", [255, 256, 257, 300])
def test_ties_around_the_rankings_bound(same):
    w = torch.zeros(1, 1, 5000)
    w[0, 0, 7::16][:same] = 2.0
    w[0, 0, 3::50] = 3.0
    for budget in (99, 101, 200, 100 + same, 101 + same):
        check(w, [5000], budget, 0, 0)


def test_ragged_batch_and_width():
    lens = [1, 4000, 0, 17, 2048, 1024, 3999, 333]
    check(tailed(8, 4, 4100, 9), lens, 1024, 4, 64, max_len=4000)


def test_long():
    check(tailed(1, 2, 40000, 2), [39999], 4096, 4, 512)
    check(tailed(1, 1, 150001, 3), [150001], 70000, 0, 1)


def test_what_lies_past_the_end_does_not_count():
    w = tailed(2, 2, 700, 4)
    a = run(w, [600, 333], 100, 2, 10, max_len=700)
    w[0, :, 600:], w[1, :, 333:] = math.inf, math.nan
    b = run(w, [600, 333], 100, 2, 10, max_len=700)
    assert torch.equal(a[0], b[0])


def test_length_out_of_range():
    w = tailed(3, 2, 100, 4).to(D)
    kept = torch.full((3, 2, 10), -7, dtype=torch.int32, device=D)
    n = torch.full((3,), -7, dtype=torch.int32, device=D)
    B.kv_select(kept, n, w, torch.tensor([101, 50, -1], dtype=torch.int32, device=D), 100, 1, 1)
    assert B.get_device_error() == 3
    assert n.tolist() == [0, 10, 0] and bool((kept[0] == -7).all()) and bool((kept[1] >= 0).all())


def test_captured_and_replayed():
    w = tailed(2, 2, 3000, 6).to(D)
    lens = torch.tensor([3000, 700], dtype=torch.int32, device=D)
    kept, n = torch.zeros((2, 2, 500), dtype=torch.int32, device=D), torch.zeros(2, dtype=torch.int32, device=D)
    B.kv_select(kept, n, w, lens, 3000, 4, 50)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.kv_select(kept, n, w, lens, 3000, 4, 50)
    w.copy_(tailed(2, 2, 3000, 7))
    kept.zero_()
    graph.replay()
    torch.cuda.synchronize()
    ref = T.select(w.cpu(), [3000, 700], 500, 4, 50)
    assert kept.cpu().tolist() == ref


# a bound over 65,536 takes the kernel for any length, whatever the lengths are
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (7, 3, 4), (64, 0, 30), (1000, 4, 100)])
def test_any_length(budget, sinks, recent):
    lens = [65537, 0, 1, 8, 9, 63, 64, 65, 1001, 8191, 8193, 66000]
    check(tailed(len(lens), 2, 66001, 8), lens, budget, sinks, recent, max_len=66001)


@pytest.mark.parametrize("values", [[0.0], [0.0, -0.0], [1.0, math.inf, -math.inf], [0.0, math.nan], [math.nan],
                                    [1e-45, 0.0, -1e-45], [3.4e38, 3.3e38, math.inf]])
def test_any_length_ties_and_odd_numbers(values):
    g = torch.Generator().manual_seed(11)
    w = torch.tensor(values)[torch.randint(0, len(values), (2, 2, 70003), generator=g)]
    for budget in (1, 20000, 70002):
        check(w, [70003, 20001], budget, 0, 0)


def test_any_length_equal_in_the_leading_bits():
    base = torch.tensor(1.5).view(torch.int32)
    g = torch.Generator().manual_seed(12)
    for span in (2, 200, 70000, 1 << 22):
        w = (base + torch.randint(0, span, (2, 1, 131071), generator=g, dtype=torch.int32)).view(torch.float32)
        check(w, [131071, 100000], 30001, 2, 30)


def test_a_million_tokens():
    check(tailed(1, 1, 1048577, 13), [1048577], 5000, 4, 64)
