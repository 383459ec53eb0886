"""kv_add_weights against the fp64 oracle."""
import math
import random

import pytest
import torch

from oracle import tree as T
from paged_kv_cache_104_gb300 import binding as B
from tree_cases import BF16, F32, Batch

pytestmark = pytest.mark.gpu
D = "cuda"


def given_lse(x):
    _, lse = T.tree_attention(*x.args())
    return torch.nan_to_num(lse, nan=0.0, neginf=-math.inf).float()


def run(x, weights, lse, max_len=None, max_draft=None):
    w = weights.to(D)
    B.kv_add_weights(w, x.q.to(D), x.k.to(D), x.table.to(D), x.lens.to(D), x.offsets.to(D),
                     None if x.mask is None else x.mask.to(D), lse.to(D), max_len or x.max_len,
                     max_draft or x.max_draft, x.scale)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    return w.cpu()


def start(x, extra=3, seed=1):
    return torch.rand((len(x.lens), x.hkv, x.max_len + extra), generator=torch.Generator().manual_seed(seed))


def check(x, before, after, lse):
    ref = T.add_weights(before, x.q, x.k, x.table, x.lens, x.offsets, x.mask, lse, x.scale)
    # a weight is off by its score's error, by that of lse * log2 e and of the
    # exponent's own rounding, and by ex2's 2^-21; the sum by half a step a term
    live = lse[torch.isfinite(lse)]
    most = float(live.abs().max()) if live.numel() else 0.0
    rel = 2 * x.score_error() + (most + 30) * 2.0 ** -21 + 2.0 ** -20
    terms = x.max_draft * x.hq // x.hkv
    tol = (ref - before.double()) * (rel + terms * 2.0 ** -24) + ref.abs() * 2.0 ** -23 + 1e-12
    err = (after.double() - ref).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    untouched = ref == before.double()
    assert torch.equal(after[untouched], before[untouched])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (8, 2), (16, 2), (16, 1), (3, 3), (32, 8)])
@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
def test_head_layouts(hq, hkv, mask):
    x = Batch([300, 40, 1, 129], [9, 3, 1, 2], hq, hkv, seed=hq, mask=mask, spare_rows=2)
    lse, w = given_lse(x), start(x)
    check(x, w, run(x, w, lse), lse)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 127, 128, 129, 256, 257, 1100])
@pytest.mark.parametrize("drafted", [1, 7])
def test_lengths(n, drafted):
    x = Batch([n], [min(drafted, n)], 8, 2, seed=n)
    lse, w = given_lse(x), start(x)
    check(x, w, run(x, w, lse), lse)


@pytest.mark.parametrize("drafted", [1, 2, 16, 31, 33, 63, 64])
@pytest.mark.parametrize("hq", [1, 4, 8, 16])
def test_drafted(drafted, hq):
    x = Batch([190 + drafted], [drafted], hq, 1, seed=drafted, mask="tree")
    lse, w = given_lse(x), start(x)
    check(x, w, run(x, w, lse), lse)


@pytest.mark.parametrize("hq,most", [(32, 16), (64, 64), (8, 64), (128, 40)])
def test_many_items_per_cta(hq, most):
    """More key tiles than SMs, sequences beyond the first 32, up to 640 rows
    of a KV head: every CTA walks several streams, some of them twice."""
    pick = random.Random(hq)
    lens = [pick.choice([pick.randint(64, 300), pick.randint(64, 1300)]) for _ in range(40)]
    drafted = [pick.choice([0, 1, 1, pick.randint(1, most)]) for _ in lens]
    drafted[7] = drafted[39] = most
    x = Batch(lens, drafted, hq, 8, seed=hq, mask="random" if hq == 8 else "tree")
    lse, w = given_lse(x), start(x)
    after = run(x, w, lse)
    check(x, w, after, lse)
    assert torch.equal(after, run(x, w, lse))


@pytest.mark.parametrize("hq,drafted", [(8, 1), (64, 20)])
def test_long_sequences(hq, drafted):
    x = Batch([20011, 5000], [drafted, 1], hq, 8, seed=hq)
    lse, w = given_lse(x), start(x)
    check(x, w, run(x, w, lse), lse)


def test_a_row_adds_up_to_one():
    x = Batch([500, 90], [8, 5], 8, 2, seed=3)
    w = run(x, torch.zeros(2, 2, 510), given_lse(x)).double()
    assert bool((w[0].sum(1) / (8 * 4) - 1).abs().max() < 1e-5) and bool((w[1].sum(1) / (5 * 4) - 1).abs().max() < 1e-5)


@pytest.mark.parametrize("dim,hq,hkv", [(16, 4, 2), (128, 8, 1)])
def test_fp32(dim, hq, hkv):
    x = Batch([300, 17, 1, 190], [9, 17, 1, 33], hq, hkv, dim, F32, seed=dim + hq)
    lse, w = given_lse(x), start(x)
    check(x, w, run(x, w, lse), lse)


def test_empty_sequences_and_rows():
    x = Batch([700, 0, 33, 2049, 5], [4, 0, 0, 64, 5], 8, 2, seed=6, spare_rows=5)
    x.mask[-10:-5] = 0                      # the last sequence is all drafted: these rows see nothing
    lse, w = given_lse(x), start(x)
    assert bool(torch.isinf(lse[68:73]).all())
    lse[73:] = float("nan")                 # rows of no sequence are not read
    x.q[73:] = float("nan")
    after = run(x, w, lse)
    lse = torch.nan_to_num(lse, nan=0.0, neginf=-math.inf)
    check(x, w, after, lse)
    assert torch.equal(after[[1, 2, 4]], w[[1, 2, 4]])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_keys_that_a_row_does_not_see(dtype):
    x = Batch([140, 77], [12, 8], 8, 2, dtype=dtype, seed=8)
    lse, w = given_lse(x), start(x)
    clean = run(x, w, lse)
    t = 140 - 12 + 7
    x.mask[:12] &= ~(1 << 7)                # nobody sees drafted token 7
    lse = given_lse(x)
    clean = run(x, w, lse)
    assert torch.equal(clean[0, :, t], w[0, :, t])
    for bad in (float("nan"), float("inf")):
        x.k[int(x.table[0, t // 16]), :, t % 16] = bad
        assert torch.equal(run(x, w, lse), clean)


def test_same_bits_and_larger_bounds():
    x = Batch([2100, 40, 777], [9, 3, 20], 16, 4, seed=13)
    lse, w = given_lse(x), start(x, 40)
    first = run(x, w, lse)
    for _ in range(3):
        assert torch.equal(first, run(x, w, lse))
    assert torch.equal(first, run(x, w, lse, max_len=2120, max_draft=20))
    check(x, w, run(x, w, lse, max_draft=64), lse)


def test_captured_and_replayed_twice():
    x = Batch([600, 33], [5, 2], 8, 2, seed=15)
    lse, w = given_lse(x), start(x)
    t = [v.to(D) for v in (w, x.q, x.k, x.table, x.lens, x.offsets, x.mask, lse)]

    def call():
        B.kv_add_weights(*t, x.max_len, x.max_draft, x.scale)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    t[0].copy_(w)
    graph.replay()
    once = t[0].cpu()
    check(x, w, once, lse)
    graph.replay()
    check(x, once, t[0].cpu(), lse)


def test_device_errors():
    x = Batch([100, 40], [3, 2], 8, 2, seed=18)
    lse, w = given_lse(x), start(x)

    def code(lens, off):
        t = w.to(D)
        B.kv_add_weights(t, x.q.to(D), x.k.to(D), x.table.to(D), torch.tensor(lens, dtype=torch.int32, device=D),
                         torch.tensor(off, dtype=torch.int32, device=D), x.mask.to(D), lse.to(D), 100, 3, x.scale)
        return B.get_device_error(), t.cpu()

    assert code([100, 40], [0, 3, 5])[0] == 0
    got, after = code([101, 40], [0, 3, 5])
    assert got == 3 and torch.equal(after[0], w[0]) and not torch.equal(after[1], w[1])
    assert code([100, 40], [0, 4, 5])[0] == 8
