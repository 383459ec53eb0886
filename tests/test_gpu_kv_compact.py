"""kv_compact against the oracle: byte for byte."""
import random

import pytest
import torch

from oracle import tree as T
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu
D = "cuda"


def pools(lens, hkv, dim, dtype, seed):
    g, pick = torch.Generator().manual_seed(seed), random.Random(seed)
    per = [-(-n // 16) for n in lens]
    nb = sum(per) + 3
    order = list(range(nb))
    pick.shuffle(order)
    table = torch.zeros((len(lens), max(per + [1]) + 1), dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    k, v = (torch.randint(0, 256, (nb, hkv, 16, dim * dtype.itemsize), generator=g, dtype=torch.uint8).view(dtype)
            for _ in "kv")
    w = torch.rand((len(lens), hkv, max(lens + [1]) + 6), generator=g)
    return k, v, w, table


def ascending(lens, heads, counts, first, seed):
    pick = random.Random(seed)
    kept = torch.full((len(lens), heads, max(counts + [1])), 1 << 30, dtype=torch.int32)
    for b, (n, m, at) in enumerate(zip(lens, counts, first)):
        for h in range(heads):
            kept[b, h, :m] = torch.tensor(sorted(pick.sample(range(at, n), m)), dtype=torch.int32)
    return kept


def same(x, y):
    return torch.equal(x.cpu().view(torch.uint8), y.view(torch.uint8))


def check(lens, counts, first, hkv=2, heads=None, dim=128, dtype=torch.bfloat16, weights=True, seed=1, kept=None):
    k, v, w, table = pools(lens, hkv, dim, dtype, seed)
    kept = ascending(lens, heads or hkv, counts, first or [0] * len(lens), seed) if kept is None else kept
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    ref = T.compact(k.view(torch.uint8), v.view(torch.uint8), w, table, lens, kept, counts, first)
    gk, gv, gw = k.to(D), v.to(D), w.to(D)
    B.kv_compact(gk, gv, table.to(D), i32(lens).to(D), kept.to(D), i32(counts).to(D),
                 None if first is None else i32(first).to(D), gw if weights else None)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    assert same(gk, ref[0]) and same(gv, ref[1])
    assert same(gw, ref[2] if weights else w)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 129, 600, 2301])
@pytest.mark.parametrize("part", [0.0, 0.04, 0.5, 0.97, 1.0])
def test_lengths(n, part):
    m = int(n * part)
    check([n, n // 2], [m, m // 3], None, seed=n)


@pytest.mark.parametrize("dtype,dim", [(torch.bfloat16, 8), (torch.bfloat16, 64), (torch.bfloat16, 128), (torch.uint8, 16),
                                       (torch.uint8, 128), (torch.uint8, 80), (torch.float32, 16), (torch.float32, 256),
                                       (torch.bfloat16, 512), (torch.uint8, 1008)])
def test_rows(dtype, dim):
    check([700, 33, 200], [350, 20, 1], None, dim=dim, dtype=dtype, hkv=3)


@pytest.mark.parametrize("hkv", [1, 2, 5, 8])
@pytest.mark.parametrize("shared", [True, False])
def test_heads(hkv, shared):
    check([300, 0, 47], [130, 0, 47], None, hkv=hkv, heads=1 if shared else hkv)


@pytest.mark.parametrize("weights", [True, False])
def test_accepted_paths(weights):
    lens = [100, 64, 3, 2301, 17]
    drafted = [16, 64, 3, 9, 1]
    first = [n - d for n, d in zip(lens, drafted)]
    check(lens, [5, 64, 0, 9, 1], first, hkv=4, heads=1, weights=weights)
    check(lens, [0, 1, 1, 3, 0], first, hkv=4, heads=1, weights=weights)
    check(lens, [16, 20, 3, 0, 0], first, hkv=4, heads=4, weights=weights)


@pytest.mark.parametrize("dtype,dim,most", [(torch.bfloat16, 128, 16), (torch.bfloat16, 128, 17), (torch.uint8, 128, 32),
                                            (torch.uint8, 16, 32), (torch.float32, 256, 4), (torch.uint8, 80, 5),
                                            (torch.uint8, 128, 33)])
def test_few_rows(dtype, dim, most):
    """Around the bounds of the kernel for a few rows, heads together and apart."""
    lens, counts = [90, most, 0, 33, 47], [most, most, 0, 1, most // 2]
    check(lens, counts, [90 - 2 * most if most < 40 else 0, 0, 0, 31, 3], hkv=3, heads=1, dim=dim, dtype=dtype)
    check(lens, counts, None, hkv=3, dim=dim, dtype=dtype)


def test_many_sequences():
    pick = random.Random(3)
    lens = [pick.randrange(0, 400) for _ in range(150)]
    check(lens, [pick.randrange(0, n + 1) for n in lens], None, hkv=4)


def test_long():
    check([33000, 9000], [16000, 8999], None, hkv=2, seed=4)
    check([12345], [12345 // 8], None, hkv=8, dtype=torch.uint8, seed=5)


def test_every_row_from_one_place():
    """A position may occur twice; the list need not ascend."""
    n = 500
    kept = torch.full((1, 2, n), n - 1, dtype=torch.int32)
    check([n], [n], None, kept=kept)
    pick = random.Random(1)
    kept = torch.tensor([[[pick.randrange(i, n) for i in range(n)] for _ in range(2)]], dtype=torch.int32)
    check([n], [n], None, kept=kept)
    kept = torch.arange(n, dtype=torch.int32).clamp(max=n - 2) + 1      # every row moves up by one
    check([n], [n], None, kept=kept.expand(1, 2, n).contiguous())


def test_errors_are_reported_and_skipped():
    lens, n = [100, 40], torch.tensor([100, 40], dtype=torch.int32)
    k, v, w, table = pools(lens, 2, 128, torch.bfloat16, 2)
    kept = ascending(lens, 2, [10, 10], [0, 0], 2)

    def code(kept, counts=(10, 10), lens=n, first=None, table=table):
        g = [k.to(D), v.to(D), w.to(D)]
        B.kv_compact(g[0], g[1], table.to(D), lens.to(D), kept.to(D), torch.tensor(counts, dtype=torch.int32, device=D),
                     None if first is None else torch.tensor(first, dtype=torch.int32, device=D), g[2])
        return B.get_device_error(), [x.cpu() for x in g]

    for i, value in ((3, 2), (3, 100), (9, -1), (0, 1 << 30)):
        bad = kept.clone()
        bad[0, 1, i] = value
        fine = kept.clone()
        fine[0, 1, i] = i                       # the row in its own place: nothing moves
        got, after = code(bad)
        assert got == 9
        assert all(same(x, y) for x, y in zip(after, code(fine)[1]))
    for counts in ((11, 10), (-1, 10)):
        got, after = code(kept, counts)
        assert got == 9
        ref = T.compact(k, v, w, table, lens, kept, [0, 10], [100, 0])   # sequence 0 is left alone
        assert all(same(x, y) for x, y in zip(after, ref))
    assert code(kept, first=[95, 0])[0] == 9
    assert code(kept, first=[-1, 0])[0] == 9
    assert code(kept, lens=torch.tensor([100, 107], dtype=torch.int32))[0] == 3
    for block in (-1, 10 ** 6):
        t = table.clone()
        t[0, 0] = block
        assert code(kept, table=t)[0] == 2


def test_captured_and_replayed():
    lens = [900, 300]
    k, v, w, table = pools(lens, 2, 128, torch.bfloat16, 7)
    kept = ascending(lens, 2, [400, 100], [0, 0], 7)
    g = [x.to(D) for x in (k, v, w)]
    t = [table.to(D), torch.tensor(lens, dtype=torch.int32, device=D), kept.to(D),
         torch.tensor([400, 100], dtype=torch.int32, device=D)]
    B.kv_compact(g[0], g[1], *t, None, g[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.kv_compact(g[0], g[1], *t, None, g[2])
    for x, y in zip(g, (k, v, w)):
        x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    ref = T.compact(k, v, w, table, lens, kept, [400, 100], None)
    assert all(same(x, y) for x, y in zip(g, ref))
