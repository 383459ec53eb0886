"""The operators for drafted tokens and eviction at the edges of what their
callers may do: pools and sums beyond 2^32 elements, results at any 16 bytes,
calls side by side, batches of hundreds of sequences, nothing to do."""
import random
import threading

import pytest
import torch

from oracle import tree as T
from paged_kv_cache_104_gb300 import binding as B
from tree_cases import BF16, F32, Batch

pytestmark = pytest.mark.gpu
D = "cuda"
BEYOND = 2 ** 32 // (8 * 16 * 128) + 64          # blocks of a pool whose last 64 lie beyond 2^32 elements


def on(x):
    return [t.to(D) for t in (x.q, torch.nan_to_num(x.k), torch.nan_to_num(x.v), x.table, x.lens, x.offsets)] + [
        None if x.mask is None else x.mask.to(D)]


def attend(x, t, out=None, lse=None, ws=None, stream=None):
    out = torch.zeros_like(t[0]) if out is None else out
    lse = torch.zeros((x.rows, x.hq), device=D) if lse is None else lse
    ws = B.tree_workspace(x.hq, x.hkv, x.dim, x.max_draft, x.max_len) if ws is None else ws
    B.paged_tree_attention(out, *t, x.max_len, x.max_draft, x.scale, ws, lse, stream)
    return out, lse


def check(x, out, lse):
    ref, ref_lse = T.tree_attention(*x.args())
    tol, tol_lse = x.bounds(ref)
    used, live = int(x.offsets[-1]), torch.isfinite(ref_lse)
    assert bool(((out.cpu().double() - ref).abs() <= tol)[:used].all())
    assert bool(((lse.cpu().double() - ref_lse).abs() <= tol_lse)[live].all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_blocks_beyond_2_to_32_elements(dtype):
    x = Batch([300, 45], [7, 3], 16, 8, dtype=dtype, seed=1)
    t = on(x)
    kept = torch.stack([torch.randperm(250, generator=torch.Generator().manual_seed(h))[:40].sort().values
                        for h in range(16)]).reshape(2, 8, 40).to(torch.int32)
    kept[1] = kept[1] % 45
    kept[1] = torch.maximum(kept[1].sort(1).values, torch.arange(40))
    results = []
    for blocks, base in ((x.num_blocks, 0), (BEYOND, BEYOND - x.num_blocks)):
        k, v = (torch.empty((blocks, 8, 16, 128), dtype=dtype, device=D) for _ in "kv")
        k[base:], v[base:] = t[1], t[2]
        u = [t[0], k, v, t[3] + base, *t[4:]]
        out, lse = attend(x, u)
        w = torch.zeros((2, 8, 300), device=D)
        B.kv_add_weights(w, u[0], k, u[3], u[4], u[5], u[6], lse, 300, 7, x.scale)
        B.kv_compact(k, v, u[3], u[4], kept.to(D), torch.tensor([40, 40], dtype=torch.int32, device=D), None, w)
        torch.cuda.synchronize()
        assert B.get_device_error() == 0
        results.append([a.cpu() for a in (out, lse, w, k[base:], v[base:])])
        del k, v, u
    assert all(torch.equal(a, b) for a, b in zip(*results))
    check(x, *results[0][:2])


def test_sums_beyond_2_to_32_elements():
    """weights [2, 8, 2^28 + 7]: the last sequence's rows start beyond 2^31 and 2^32."""
    x = Batch([300, 280], [7, 3], 16, 8, seed=2)
    t = on(x)
    _, lse = attend(x, t)
    results = []
    for width in (300, 2 ** 28 + 7):
        w = torch.empty((2, 8, width), device=D)
        w[:, :, :300] = 0.5
        k, v = t[1].clone(), t[2].clone()
        B.kv_add_weights(w, t[0], k, *t[3:6], t[6], lse, 300, 7, x.scale)
        kept = torch.zeros((2, 8, 64), dtype=torch.int32, device=D)
        n = torch.zeros(2, dtype=torch.int32, device=D)
        B.kv_select(kept, n, w, t[4], 300, 4, 8)
        before = w[:, :, :300].clone()
        B.kv_compact(k, v, t[3], t[4], kept, n, None, w)
        torch.cuda.synchronize()
        assert B.get_device_error() == 0
        results.append([a.cpu() for a in (before, w[:, :, :300], kept, n, k, v)])
        del w
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert results[0][2].tolist() == T.select(results[0][0], [300, 280], 64, 4, 8)


@pytest.mark.parametrize("draft", [3, 40])
def test_results_at_any_16_bytes(draft):
    """q and out that start 16 bytes behind a 32-byte boundary."""
    x = Batch([400, 90], [draft, 2], 8, 2, seed=3)
    t = on(x)
    ref = attend(x, t)
    q = torch.empty(x.q.numel() + 8, dtype=BF16, device=D)[8:].view(x.q.shape)
    out = torch.zeros(x.q.numel() + 8, dtype=BF16, device=D)[8:].view(x.q.shape)
    q.copy_(t[0])
    assert q.data_ptr() % 32 == 16 and out.data_ptr() % 32 == 16
    got = attend(x, [q, *t[1:]], out=out)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_two_streams_at_once():
    """Two batches on streams of their own, each with its workspace, many times."""
    xs = [Batch([2100, 40, 777], [9, 3, 20], 16, 4, seed=s) for s in (4, 5)]
    ts = [on(x) for x in xs]
    want = [attend(x, t) for x, t in zip(xs, ts)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    ws = [B.tree_workspace(16, 4, 128, 20, 2100) for _ in xs]
    got = [[torch.zeros_like(a) for a in w] for w in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, t, g, w, s in zip(xs, ts, got, ws, streams):
            attend(x, t, g[0], g[1], w, s)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_two_host_threads():
    xs = [Batch([700, 40], [9, 3], 16, 4, seed=6), Batch([90, 1300], [2, 33], 8, 1, seed=7)]
    ts = [on(x) for x in xs]
    want = [attend(x, t) for x, t in zip(xs, ts)]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                got = attend(xs[i], ts[i])
                w = torch.zeros((2, xs[i].hkv, xs[i].max_len), device=D)
                t = ts[i]
                B.kv_add_weights(w, t[0], t[1], *t[3:6], t[6], got[1], xs[i].max_len, xs[i].max_draft, xs[i].scale)
            s.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad and B.get_device_error() == 0


@pytest.mark.parametrize("dtype,hq,hkv", [(BF16, 4, 2), (BF16, 1, 1), (F32, 2, 1)])
def test_hundreds_of_sequences(dtype, hq, hkv):
    """Many windows of 32 sequences, a good part of them without drafted tokens."""
    pick = random.Random(8)
    lens = [pick.choice([0, pick.randint(1, 40), pick.randint(1, 200)]) for _ in range(701)]
    drafted = [min(n, pick.choice([0, 0, 1, 2, pick.randint(1, 9)])) for n in lens]
    lens[133:260], drafted[133:260] = [0] * 127, [0] * 127       # windows with nothing to do
    lens[-1], drafted[-1] = 150, 9
    x = Batch(lens, drafted, hq, hkv, dtype=dtype, seed=8, spare_rows=1)
    t = on(x)
    out, lse = attend(x, t)
    assert B.get_device_error() == 0
    check(x, out, lse)
    w = torch.zeros((701, hkv, x.max_len), device=D)
    B.kv_add_weights(w, t[0], t[1], *t[3:6], t[6], lse, x.max_len, x.max_draft, x.scale)
    rows = torch.tensor([float(n * hq // hkv) for n in drafted])
    assert float((w.cpu().sum(2) - rows[:, None]).abs().max()) < 1e-4
    kept = torch.zeros((701, hkv, 16), dtype=torch.int32, device=D)
    n = torch.zeros(701, dtype=torch.int32, device=D)
    B.kv_select(kept, n, w, t[4], x.max_len, 1, 3)
    ref = T.select(w.cpu(), lens, 16, 1, 3)
    assert all(kept[b, h, :len(ref[b][h])].tolist() == ref[b][h] for b in range(0, 701, 7) for h in range(hkv))
    exp = T.compact(t[1].cpu(), t[2].cpu(), w.cpu(), x.table, lens, kept.cpu(), n.tolist(), None)
    B.kv_compact(t[1], t[2], t[3], t[4], kept, n, None, w)
    assert B.get_device_error() == 0
    assert all(torch.equal(a.cpu(), e) for a, e in zip((t[1], t[2], w), exp))


def test_nothing_to_do():
    x = Batch([40, 30], [0, 0], 8, 2, seed=9, spare_rows=3)
    t = on(x)
    out, lse = attend(x, t, out=torch.full_like(t[0], 7.0), lse=torch.full((3, 8), 7.0, device=D))
    w = torch.full((2, 2, 40), 7.0, device=D)
    B.kv_add_weights(w, t[0], t[1], *t[3:6], t[6], lse, 40, 1, x.scale)
    empty = t[0][:0]
    B.paged_tree_attention(empty.clone(), empty, *t[1:6], None, 40, 1, x.scale, None, None)
    none = [a[:0] for a in t[3:5]]
    B.paged_tree_attention(out, t[0], t[1], t[2], *none, t[5][:1], t[6], 40, 1, x.scale, None, lse)
    kept, n = torch.full((2, 2, 0), 7, dtype=torch.int32, device=D), torch.zeros(2, dtype=torch.int32, device=D)
    k = t[1].clone()
    B.kv_compact(k, t[2].clone(), t[3], t[4], kept, n, t[4], w)      # all before `first` stays
    B.kv_select(torch.zeros((0, 2, 5), dtype=torch.int32, device=D), n[:0], w[:0], t[4][:0], 40, 1, 1)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    assert bool((out == 7).all()) and bool((lse == 7).all()) and bool((w == 7).all()) and torch.equal(k, t[1])


def test_a_selection_that_leaves_nothing_to_choose():
    """sinks + recent = budget: no weight matters, NaN included."""
    w = torch.full((2, 2, 9000), float("nan"), device=D)
    lens = torch.tensor([9000, 50], dtype=torch.int32, device=D)
    kept, n = torch.zeros((2, 2, 60), dtype=torch.int32, device=D), torch.zeros(2, dtype=torch.int32, device=D)
    B.kv_select(kept, n, w, lens, 9000, 20, 40)
    assert n.tolist() == [60, 50]
    assert kept[0, 1].tolist() == list(range(20)) + list(range(8960, 9000)) and kept[1, 0, :50].tolist() == list(range(50))


def test_debug_mode_lets_good_calls_pass():
    x = Batch([100, 0, 40], [3, 0, 2], 8, 2, seed=10)
    t = on(x)
    B.set_debug(True)
    try:
        out, lse = attend(x, t)
        w = torch.zeros((3, 2, 100), device=D)
        B.kv_add_weights(w, t[0], t[1], *t[3:6], t[6], lse, 100, 3, x.scale)
        kept, n = torch.zeros((3, 2, 20), dtype=torch.int32, device=D), torch.zeros(3, dtype=torch.int32, device=D)
        B.kv_select(kept, n, w, t[4], 100, 2, 5)
        B.kv_compact(t[1], t[2], t[3], t[4], kept, n, None, w)
    finally:
        B.set_debug(False)
    check(x, out, lse)


def test_rows_before_the_first_sequence():
    """draft_offsets that do not start at 0: q's rows before them are nobody's."""
    x = Batch([200, 33, 90], [5, 0, 17], 8, 2, seed=11)
    t = on(x)
    want = attend(x, t)
    pad = torch.zeros((3, 8, 128), dtype=BF16, device=D)
    out, lse = torch.full((x.rows + 3, 8, 128), 7.0, dtype=BF16, device=D), torch.full((x.rows + 3, 8), 7.0, device=D)
    B.paged_tree_attention(out, torch.cat([pad, t[0]]), *t[1:5], t[5] + 3, torch.cat([t[6][:3], t[6]]), x.max_len,
                           x.max_draft, x.scale, B.tree_workspace(8, 2, 128, x.max_draft, x.max_len), lse)
    assert B.get_device_error() == 0
    assert bool((out[:3] == 7).all()) and bool((lse[:3] == 7).all())
    assert torch.equal(out[3:], want[0]) and torch.equal(lse[3:], want[1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_bounds_above_the_batch(dtype):
    """max_seq_len and max_draft are bounds: larger ones change nothing but rounding."""
    x = Batch([700, 2, 90], [5, 2, 1], 8, 2, dtype=dtype, seed=12)
    x.table = torch.cat([x.table, torch.full((3, 500), -1, dtype=torch.int32)], 1)
    x.max_len, x.max_draft = x.table.shape[1] * 16, 64
    t = on(x)
    out, lse = attend(x, t)
    assert B.get_device_error() == 0
    check(x, out, lse)
    w = torch.zeros((3, 2, x.max_len), device=D)
    B.kv_add_weights(w, t[0], t[1], *t[3:6], t[6], lse, x.max_len, 64, x.scale)
    assert B.get_device_error() == 0
    rows = torch.tensor([20.0, 8.0, 4.0])
    assert float((w.cpu().sum(2) - rows[:, None]).abs().max()) < 1e-4
    assert bool((w[1, :, 2:] == 0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_replayed_graph_follows_what_its_tensors_hold(dtype):
    """One capture; then other lengths, other numbers of drafted tokens, other
    trees and blocks in the same tensors."""
    first = Batch([900, 40, 64, 0], [12, 3, 64, 0], 8, 2, dtype=dtype, seed=13)
    t = on(first)
    ws = B.tree_workspace(8, 2, 128, 64, 900)
    width = t[3].shape[1]
    out, lse, w = torch.zeros_like(t[0]), torch.zeros((first.rows, 8), device=D), torch.zeros((4, 2, 900), device=D)

    def both():
        B.paged_tree_attention(out, *t, 900, 64, first.scale, ws, lse)
        B.kv_add_weights(w, t[0], t[1], *t[3:6], t[6], lse, 900, 64, first.scale)

    both()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed, lens, drafted in ((14, [33, 700, 1, 200], [2, 40, 1, 11]), (15, [0, 0, 0, 1], [0, 0, 0, 1]),
                                (16, [64, 64, 64, 64], [0, 0, 64, 15])):
        x = Batch(lens, drafted, 8, 2, dtype=dtype, seed=seed)
        assert x.num_blocks <= first.num_blocks and x.rows <= first.rows
        t[0][:x.rows] = x.q.to(D)
        t[1][:x.num_blocks], t[2][:x.num_blocks] = torch.nan_to_num(x.k).to(D), torch.nan_to_num(x.v).to(D)
        t[3].zero_()
        t[3][:, :min(width, x.table.shape[1])] = x.table[:, :width].to(D)
        t[4].copy_(x.lens)
        t[5].copy_(x.offsets)
        t[6][:x.rows] = x.mask.to(D)
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert B.get_device_error() == 0
        check(x, out[:x.rows], lse[:x.rows])
        rows = torch.tensor([4.0 * n for n in drafted])
        assert float((w.cpu().sum(2) - rows[:, None]).abs().max()) < 1e-4


def test_compaction_by_a_replayed_graph_whose_lists_change():
    g = torch.Generator().manual_seed(17)
    k, v = (torch.randn((80, 2, 16, 128), generator=g).bfloat16() for _ in "kv")
    table = torch.randperm(80, generator=g).to(torch.int32).view(2, 40)
    w = torch.rand((2, 2, 640), generator=g)
    dk, dv, dw, dt = k.to(D), v.to(D), w.to(D), table.to(D)
    lens = torch.tensor([640, 500], dtype=torch.int32, device=D)
    kept, n = torch.zeros((2, 2, 200), dtype=torch.int32, device=D), torch.zeros(2, dtype=torch.int32, device=D)

    def both():
        B.kv_select(kept, n, dw, lens, 640, 4, 30)
        B.kv_compact(dk, dv, dt, lens, kept, n, None, dw)

    lens.zero_()
    both()                                                 # nothing stored: nothing moves
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for now in ([640, 500], [201, 199], [0, 300]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        k, v, w = dk.cpu(), dv.cpu(), dw.cpu()
        graph.replay()
        torch.cuda.synchronize()
        assert B.get_device_error() == 0
        ref = T.select(w, now, 200, 4, 30)
        assert n.tolist() == [min(x, 200) for x in now]
        assert all(kept[b, h, :len(ref[b][h])].tolist() == ref[b][h] for b in range(2) for h in range(2))
        exp = T.compact(k, v, w, table, now, kept.cpu(), n.tolist(), None)
        assert all(torch.equal(a.cpu(), e) for a, e in zip((dk, dv, dw), exp))


@pytest.mark.parametrize("hq,hkv,most", [(32, 8, 1000), (4, 4, 260), (32, 2, 700), (6, 6, 3000)])
def test_many_short_sequences(hq, hkv, most):
    """KV heads that go in pairs, whole and cut between CTAs, next to sequences
    of more rows or tiles that do not; drafted values of one head that are
    infinite or NaN reach only the rows of that head that see them."""
    pick = random.Random(most)
    lens = [pick.randint(1, most) for _ in range(160)]
    drafted = [min(n, pick.choice([1, 2, 5, 8, pick.randint(0, 64)])) for n in lens]
    x = Batch(lens, drafted, hq, hkv, seed=most)
    for b in range(0, 160, 3):
        if drafted[b] == 0:
            continue
        t, h = lens[b] - 1 - pick.randrange(drafted[b]), pick.randrange(hkv)
        x.v[int(x.table[b, t // 16]), h, t % 16, pick.randrange(128)] = pick.choice([float("inf"), float("nan"), 1e30])
    d = [a.to(D) for a in (x.q, x.k, x.v, x.table, x.lens, x.offsets, x.mask)]
    out, lse = attend(x, d)
    assert B.get_device_error() == 0
    ref, ref_lse = T.tree_attention(*x.args())
    tol, tol_lse = x.bounds(ref)
    out, lse = out.cpu().double(), lse.cpu().double()
    plain = torch.isfinite(ref) & (ref.abs() < 1e20)
    assert bool(((out - ref).abs() <= tol)[plain].all())
    assert bool((torch.isnan(out) == torch.isnan(ref)).all()) and bool((out[torch.isinf(ref)] == ref[torch.isinf(ref)]).all())
    assert bool(((lse - ref_lse).abs() <= tol_lse).all())
    again = attend(x, d)
    assert torch.equal(again[0].cpu().double().nan_to_num(), out.nan_to_num())
