"""paged_tree_attention against the fp64 oracle."""
import math
import random

import pytest
import torch

from oracle import tree as T
from paged_kv_cache_104_gb300 import binding as B
from tree_cases import BF16, F32, Batch

pytestmark = pytest.mark.gpu


def run(x, out=None, lse=True, workspace=None, stream=None, max_len=None, max_draft=None):
    d = "cuda"
    out = torch.full_like(x.q, 7.0, device=d) if out is None else out
    e = torch.full((x.rows, x.hq), 7.0, device=d) if lse else None
    ml, md = max_len or x.max_len, max_draft or x.max_draft
    ws = B.tree_workspace(x.hq, x.hkv, x.dim, md, ml) if workspace is None else workspace
    B.paged_tree_attention(out, x.q.to(d), x.k.to(d), x.v.to(d), x.table.to(d), x.lens.to(d), x.offsets.to(d),
                           None if x.mask is None else x.mask.to(d), ml, md, x.scale, ws, e, stream)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    return out.cpu(), None if e is None else e.cpu()


def check(x, out, lse=None):
    ref, ref_lse = T.tree_attention(*x.args())
    used = int(x.offsets[-1])
    tol, tol_lse = x.bounds(ref)
    err = (out.double() - ref).abs()
    assert bool((err[:used] <= tol[:used]).all()), float((err - tol)[:used].max())
    empty = torch.isinf(ref_lse)
    assert bool((out.double()[empty] == 0).all())
    if lse is not None:
        assert torch.equal(torch.isinf(lse.double()[:used]), empty[:used])
        live = ~empty
        live[used:] = False
        assert bool(((lse.double() - ref_lse).abs()[live] <= tol_lse[live]).all())
        assert bool((lse[used:] == 7).all())
    assert bool((out[used:] == 7).all())           # rows behind the last sequence


HEADS = [(1, 1), (2, 1), (8, 2), (16, 2), (16, 1), (3, 3), (12, 3)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
def test_head_layouts(hq, hkv, mask):
    x = Batch([300, 40, 1, 129], [9, 3, 1, 2], hq, hkv, seed=hq, mask=mask, spare_rows=2)
    check(x, *run(x))


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 255, 256, 257, 500, 1100, 3000])
@pytest.mark.parametrize("drafted", [1, 5])
def test_lengths(n, drafted):
    x = Batch([n], [min(drafted, n)], 8, 2, seed=n, mask="tree")
    check(x, *run(x))


@pytest.mark.parametrize("drafted", [1, 2, 7, 16, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("hq", [1, 4, 8, 16])
def test_drafted(drafted, hq):
    """Up to 1,024 rows of one KV head; the drafted tokens straddle tiles."""
    x = Batch([190 + drafted], [drafted], hq, 1, seed=drafted, mask="tree")
    check(x, *run(x))


def test_nothing_but_drafted_tokens():
    for mask in ("tree", "chain", "random"):
        x = Batch([64, 20, 1], [64, 20, 1], 8, 2, seed=4, mask=mask)
        check(x, *run(x))


def test_rows_that_see_nothing():
    x = Batch([5, 130], [5, 3], 4, 2, seed=5)
    x.mask[:5] = 0
    out, lse = run(x)
    assert bool((out[:5] == 0).all()) and bool((lse[:5] == -math.inf).all())
    check(x, out, lse)


def test_ragged_batch_with_empty_sequences():
    lens, drafted = [700, 0, 33, 2049, 16, 5, 260, 1], [4, 0, 0, 64, 16, 2, 33, 0]
    x = Batch(lens, drafted, 8, 2, seed=6, spare_rows=5)
    check(x, *run(x))
    x.lens[1], x.lens[2] = -5, 1 << 30        # lengths of sequences without rows are not used
    x2 = Batch(lens, drafted, 8, 2, seed=6, spare_rows=5)
    out, _ = run(x)
    assert torch.equal(out, run(x2)[0])


@pytest.mark.parametrize("hq,most", [(32, 16), (64, 64), (8, 64), (128, 5)])
def test_many_items_per_cta(hq, most):
    """More key tiles than SMs, sequences beyond the first 32: every CTA walks
    several streams, whole and cut, of few rows and of many."""
    pick = random.Random(hq)
    lens = [pick.choice([pick.randint(64, 300), pick.randint(64, 1500)]) for _ in range(45)]
    drafted = [pick.choice([0, 1, pick.randint(1, most), most]) for _ in lens]
    x = Batch(lens, drafted, hq, 8, seed=hq, mask="random" if hq == 8 else "tree")
    out = run(x)
    check(x, *out)
    again = run(x)
    assert torch.equal(out[0], again[0]) and torch.equal(out[1], again[1])


@pytest.mark.parametrize("hq,drafted", [(8, 3), (32, 20), (64, 64)])
def test_long_sequences(hq, drafted):
    x = Batch([20011, 5000], [drafted, 1], hq, 8, seed=hq)
    check(x, *run(x))


@pytest.mark.parametrize("dim,hq,hkv", [(16, 4, 2), (128, 8, 1), (128, 2, 2), (16, 8, 1)])
@pytest.mark.parametrize("mask", ["tree", "chain", "random"])
def test_fp32(dim, hq, hkv, mask):
    x = Batch([300, 17, 1, 90], [9, 17, 1, 33], hq, hkv, dim, F32, seed=dim + hq, mask=mask)
    check(x, *run(x))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_that_a_row_does_not_see_never_reach_it(dtype):
    """NaN and infinities in a drafted token's key and value: the rows that do
    not see it are those of a batch where it is harmless."""
    x = Batch([140, 77], [12, 8], 8, 2, dtype=dtype, seed=8)
    clean = run(x)
    hidden = 7                                 # drafted token 7 of sequence 0, a leaf or not
    t = 140 - 12 + hidden
    for bad in (float("nan"), float("inf"), -float("inf"), 3e38):
        y = Batch([140, 77], [12, 8], 8, 2, dtype=dtype, seed=8)
        y.k[int(y.table[0, t // 16]), :, t % 16] = bad
        y.v[int(y.table[0, t // 16]), :, t % 16] = bad
        out, lse = run(y)
        blind = [i for i in range(12) if not (int(x.mask[i]) >> hidden) & 1] + list(range(12, 20))
        assert len(blind) > 8
        assert torch.equal(out[blind], clean[0][blind]) and torch.equal(lse[blind], clean[1][blind])
        if bad != bad:
            assert bool(torch.isnan(out[hidden]).all())


def test_visible_infinities():
    """A value of +inf that a row sees gives +inf where its weight is not zero."""
    x = Batch([140], [12], 4, 1, seed=9)
    t = 140 - 12 + 3
    x.v[int(x.table[0, t // 16]), :, t % 16, :5] = float("inf")
    out, _ = run(x)
    for i in range(12):
        see = (int(x.mask[i]) >> 3) & 1
        assert bool(torch.isinf(out[i, :, :5]).all()) == bool(see)
        assert bool(torch.isfinite(out[i, :, 5:]).all())


@pytest.mark.parametrize("gain", [30.0, 1e-3])
def test_sharp_and_flat_softmax(gain):
    x = Batch([400, 90], [6, 4], 8, 2, seed=10, q_gain=gain)
    check(x, *run(x))


def test_scores_beyond_the_first_tiles_maximum():
    """Keys that grow along the sequence: the running maximum moves at every tile."""
    x = Batch([900], [4], 4, 1, seed=11)
    for t in range(900):
        x.k[int(x.table[0, t // 16]), :, t % 16] *= 0.2 + t / 150
    check(x, *run(x))


def test_without_lse_and_with_larger_bounds():
    x = Batch([300, 40], [9, 3], 8, 2, seed=12)
    base, _ = run(x)
    out, none = run(x, lse=False, max_len=304, max_draft=64)
    assert none is None
    check(x, out)


def test_same_bits_every_time_and_on_a_stream_of_its_own():
    x = Batch([2100, 40, 777, 1300], [9, 3, 20, 1], 16, 4, seed=13)
    first = run(x)
    s = torch.cuda.Stream()
    for k in range(3):
        with torch.cuda.stream(s):
            again = run(x, stream=s if k == 2 else None)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_workspace_of_garbage():
    x = Batch([2100, 40, 777], [9, 3, 20], 8, 2, seed=14)
    ws = B.tree_workspace(8, 2, 128, 20, 2100).fill_(0xff)
    check(x, *run(x, workspace=ws))


def test_captured_and_replayed():
    d = "cuda"
    x = Batch([2100, 40, 777], [9, 3, 20], 8, 2, seed=15)
    y = Batch([2100, 40, 777], [9, 3, 20], 8, 2, seed=16)
    ws = B.tree_workspace(8, 2, 128, 20, 2100)
    t = [v.to(d) for v in (x.q, x.k, x.v, x.table, x.lens, x.offsets, x.mask)]
    out, lse = torch.zeros_like(t[0]), torch.zeros((x.rows, 8), device=d)

    def call():
        B.paged_tree_attention(out, *t[:6], t[6], 2100, 20, x.scale, ws, lse)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for src in (y, x):
        for a, v in zip(t, (src.q, src.k, src.v, src.table, src.lens, src.offsets, src.mask)):
            a.copy_(v)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(src, out.cpu(), lse.cpu())


def test_agrees_with_decode():
    """One drafted token: the decode of the same sequence."""
    x = Batch([2301, 100, 33], [1, 1, 1], 32, 8, seed=17, mask="chain")
    out, _ = run(x)
    d = "cuda"
    ref = torch.empty_like(x.q, device=d)
    B.paged_decode_attention(ref, x.q.to(d), x.k.to(d), x.v.to(d), x.table.to(d), x.lens.to(d), 2301, x.scale,
                             B.decode_workspace(3, 32, 128, 2301))
    tol, _ = x.bounds(out.double())
    assert bool(((out.double() - ref.cpu().double()).abs() <= 2 * tol).all())


def test_device_errors():
    d = "cuda"

    def code(**kw):
        x = Batch([100, 40], [3, 2], 8, 2, seed=18)
        for k, v in kw.items():
            getattr(x, k).copy_(torch.tensor(v, dtype=getattr(x, k).dtype)) if k != "block" else None
        if "block" in kw:
            x.table[0, 2] = kw["block"]
        out = torch.full_like(x.q, 7.0, device=d)
        B.paged_tree_attention(out, x.q.to(d), x.k.to(d), x.v.to(d), x.table.to(d), x.lens.to(d), x.offsets.to(d),
                               x.mask.to(d), 100, 3, x.scale, B.tree_workspace(8, 2, 128, 3, 100))
        torch.cuda.synchronize()
        return B.get_device_error(), out.cpu()

    assert code()[0] == 0
    for kw, want in ((dict(offsets=[0, 4, 5]), 8), (dict(offsets=[-1, 2, 5]), 8), (dict(offsets=[0, 3, 6]), 8),
                     (dict(offsets=[3, 0, 2]), 8), (dict(lens=[2, 40]), 3), (dict(lens=[101, 40]), 3),
                     (dict(lens=[-1, 40]), 3), (dict(block=-1), 2), (dict(block=10 ** 6), 2)):
        got, out = code(**kw)
        assert got == want, kw
        if want == 3:
            assert bool((out[:3] == 7).all()) and bool((out[3:] != 7).any())


@pytest.mark.parametrize("dim", [16, 128])
@pytest.mark.parametrize("hq,hkv,drafted", [(1, 1, 1), (2, 1, 4), (4, 2, 4), (8, 1, 1), (3, 3, 9), (8, 2, 4), (2, 1, 8),
                                            (4, 1, 5), (8, 1, 64)])
@pytest.mark.parametrize("mask", [None, "tree", "random"])
def test_fp32_rows_and_parts(dim, hq, hkv, drafted, mask):
    """Up to 8, 16 and more rows a KV head: keys split between four, two and no warps."""
    x = Batch([700, drafted, drafted + 1, 33 + drafted, 0, 300], [drafted, drafted, max(1, drafted - 1), drafted, 0, 1],
              hq, hkv, dim=dim, dtype=F32, mask=mask, seed=hq + drafted, spare_rows=2)
    check(x, *run(x))


@pytest.mark.parametrize("most", [1, 128, 129, 256, 257, 384, 385, 512, 513])
@pytest.mark.parametrize("count,hq,hkv,drafted", [(1, 8, 2, 5), (3, 16, 1, 40), (70, 4, 4, 3), (60, 3, 3, 9), (40, 8, 1, 20)])
def test_short_sequences_around_where_they_are_cut(most, count, hq, hkv, drafted):
    """One to five tiles: whole streams or parts, one KV head or two to an item."""
    pick = random.Random(most)
    lens = [most] + [pick.randint(0, most) for _ in range(count - 1)]
    x = Batch(lens, [min(n, pick.randint(0, drafted)) if i else min(n, drafted) for i, n in enumerate(lens)], hq, hkv,
              seed=most + count, spare_rows=1)
    check(x, *run(x))
