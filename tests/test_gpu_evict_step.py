"""The operators for drafted tokens and eviction as a serving loop runs them:
append the drafts, attend, count the attention, accept a path, move it up,
and when the sequences have grown, keep the tokens that got most attention."""
import random

import pytest
import torch

import oracle
from oracle import tree as T
from paged_kv_cache_104_gb300 import binding as B
from tree_cases import BF16, F32, Batch, signed, tree_words

pytestmark = pytest.mark.gpu
D = "cuda"


def slots_of(table, b, positions):
    return [int(table[b, p // 16]) * 16 + p % 16 for p in positions]


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("dtype,hq,hkv,dim", [(BF16, 8, 2, 128), (F32, 4, 2, 16)])
def test_speculate_accept_evict(dtype, hq, hkv, dim):
    """Three verified drafts, then an eviction, then a decode over what is left:
    every step against the oracle on the same inputs."""
    pick, gen = random.Random(1), torch.Generator().manual_seed(1)
    lens, room = [200, 37, 90], 96
    x = Batch([n + room for n in lens], [1, 1, 1], hq, hkv, dim, dtype, seed=2)
    table, scale = x.table, x.scale
    k, v = torch.nan_to_num(x.k).to(D), torch.nan_to_num(x.v).to(D)
    w = torch.zeros((3, hkv, max(lens) + room), device=D)
    table_d = table.to(D)
    ws = B.tree_workspace(hq, hkv, dim, 16, max(lens) + room)

    for step in range(3):
        drafted = [pick.randint(1, 16) for _ in lens]
        words = signed([t for n in drafted for t in tree_words(n, pick)])
        off, rows = [0], sum(drafted)
        for n in drafted:
            off.append(off[-1] + n)
        kn, vn = (torch.randn((rows, hkv, dim), generator=gen).to(dtype) for _ in "kv")
        q = torch.randn((rows, hq, dim), generator=gen).to(dtype)
        slots = [s for b, n in enumerate(drafted) for s in slots_of(table, b, range(lens[b], lens[b] + n))]
        B.kv_append(kn.to(D), vn.to(D), k, v, torch.tensor(slots, device=D))
        total = i32([n + d for n, d in zip(lens, drafted)])
        ml = int(total.max())
        out, lse = torch.zeros_like(q, device=D), torch.zeros((rows, hq), device=D)
        before = w.cpu()
        B.paged_tree_attention(out, q.to(D), k, v, table_d, total.to(D), i32(off).to(D), words.to(D), ml, 16, scale, ws,
                               lse)
        B.kv_add_weights(w, q.to(D), k, table_d, total.to(D), i32(off).to(D), words.to(D), lse, ml, 16, scale)
        kc, vc = k.cpu(), v.cpu()
        ref, ref_lse = T.tree_attention(q, kc, vc, table, total, off, words, scale)
        assert float((out.cpu().double() - ref).abs().max()) <= (2e-2 if dtype is BF16 else 1e-5)
        assert float((lse.cpu().double() - ref_lse).abs().max()) <= 1e-5
        ref_w = T.add_weights(before, q, kc, table, total, off, words, lse.cpu(), scale)
        assert float((w.cpu().double() - ref_w).abs().max()) <= 1e-5
        # accept a random path: some ancestors of a drafted token, itself the last
        path = []
        for b, n in enumerate(drafted):
            word = int(words[off[b] + pick.randrange(n)])
            path.append([lens[b] + j for j in range(n) if (word >> j) & 1])
        kept = torch.zeros((3, 1, 16), dtype=torch.int32)
        for b, p in enumerate(path):
            kept[b, 0, :len(p)] = i32(p)
        counts = [len(p) for p in path]
        exp = T.compact(kc, vc, w.cpu(), table, total, kept, counts, lens)
        B.kv_compact(k, v, table_d, total.to(D), kept.to(D), i32(counts).to(D), i32(lens).to(D), w)
        assert all(torch.equal(a.cpu(), e) for a, e in zip((k, v, w), exp))
        lens = [n + c for n, c in zip(lens, counts)]

    budget = 64
    kept, n = torch.zeros((3, hkv, budget), dtype=torch.int32, device=D), torch.zeros(3, dtype=torch.int32, device=D)
    lens_d = i32(lens).to(D)
    B.kv_select(kept, n, w, lens_d, max(lens), 4, 16)
    ref = T.select(w.cpu(), lens, budget, 4, 16)
    assert all(kept[b, h, :len(ref[b][h])].tolist() == ref[b][h] for b in range(3) for h in range(hkv))
    exp = T.compact(k.cpu(), v.cpu(), w.cpu(), table, lens, kept.cpu(), n.cpu(), None)
    B.kv_compact(k, v, table_d, lens_d, kept, n, None, w)
    assert all(torch.equal(a.cpu(), e) for a, e in zip((k, v, w), exp))
    # the next decode reads the shorter sequences
    q = torch.randn((3, hq, dim), generator=gen).to(dtype)
    out = torch.zeros_like(q, device=D)
    B.paged_decode_attention(out, q.to(D), k, v, table_d, n, budget, scale, B.decode_workspace(3, hq, dim, budget))
    ref = oracle.paged_decode(q, exp[0], exp[1], table, n.cpu(), scale)
    assert float((out.cpu().double() - ref.double()).abs().max()) <= (2e-2 if dtype is BF16 else 1e-5)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0


def test_one_graph_of_the_whole_step():
    """Attention, weights, selection and compaction in one captured graph,
    replayed for other inputs, against the same calls one by one."""
    def inputs(seed):
        x = Batch([700, 260, 65], [5, 9, 1], 8, 2, seed=seed)
        return x, [t.to(D) for t in (x.q, torch.nan_to_num(x.k), torch.nan_to_num(x.v), x.table, x.lens, x.offsets,
                                     x.mask)]

    x, t = inputs(3)
    out, lse = torch.zeros_like(t[0]), torch.zeros((x.rows, 8), device=D)
    w = torch.zeros((3, 2, 720), device=D)
    kept, n = torch.zeros((3, 2, 128), dtype=torch.int32, device=D), torch.zeros(3, dtype=torch.int32, device=D)
    ws = B.tree_workspace(8, 2, 128, 9, 700)

    def step():
        q, k, v, table, lens, off, mask = t
        B.paged_tree_attention(out, q, k, v, table, lens, off, mask, 700, 9, x.scale, ws, lse)
        B.kv_add_weights(w, q, k, table, lens, off, mask, lse, 700, 9, x.scale)
        B.kv_select(kept, n, w, lens, 700, 2, 10)
        B.kv_compact(k, v, table, lens, kept, n, None, w)

    results = []
    for seed in (3, 4):
        for a, s in zip(t, inputs(seed)[1]):
            a.copy_(s)
        w.zero_()
        kept.zero_()
        step()
        results.append([a.clone() for a in (out, lse, w, kept, n, t[1], t[2])])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, want in zip((3, 4), results):
        for a, s in zip(t, inputs(seed)[1]):
            a.copy_(s)
        w.zero_()
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, e) for a, e in zip((out, lse, w, kept, n, t[1], t[2]), want))
    assert B.get_device_error() == 0
