"""The operators for drafted tokens and eviction without a GPU: the oracle's
own checks, host refusals of the library and of the binding, debug mode."""
import ctypes
import math

import pytest
import torch

from oracle import tree as T
from paged_kv_cache_104_gb300 import binding as B
from paged_kv_cache_104_gb300 import validate as V
from tree_cases import F32, Batch, signed, tree_words

P = 0x1000


def _tree(fn, **kw):
    a = dict(out=P, lse=P, q=P, k_cache=P, v_cache=P, block_table=P, seq_lens=P, draft_offsets=P, tree_mask=P,
             weights=P, workspace=P, workspace_bytes=1 << 40, weights_len=1000, num_blocks=32, num_seqs=4, num_rows=20,
             max_blocks_per_seq=64, max_seq_len=1000, max_draft=8, num_q_heads=16, num_kv_heads=4, head_dim=128,
             block_size=16, dtype=1, scale=0.1)
    a.update(kw)
    return getattr(B.load(), fn)(ctypes.byref(B.TreeArgs(**a)), None)


SHARED = [
    (dict(num_q_heads=0), 1), (dict(num_q_heads=18), 1), (dict(num_kv_heads=0), 1), (dict(head_dim=0), 1),
    (dict(block_size=0), 1), (dict(block_size=32), 5), (dict(head_dim=64), 5), (dict(num_q_heads=12), 5),
    (dict(num_q_heads=128), 5), (dict(dtype=7), 2), (dict(dtype=0, num_q_heads=64), 5), (dict(num_seqs=-1), 1),
    (dict(num_rows=-1), 1), (dict(max_blocks_per_seq=0), 1), (dict(max_seq_len=0), 1), (dict(num_blocks=0), 1),
    (dict(max_draft=0), 1), (dict(max_draft=65), 5), (dict(num_seqs=8193), 3), (dict(max_seq_len=1025), 1),
    (dict(scale=math.inf), 1), (dict(scale=0.0), 1), (dict(scale=-0.1), 1), (dict(scale=math.nan), 1),
    (dict(q=0), 1), (dict(k_cache=0), 1), (dict(block_table=0), 1), (dict(seq_lens=0), 1), (dict(draft_offsets=0), 1),
    (dict(q=0x1008), 1), (dict(k_cache=0x1008), 1), (dict(block_table=0x1002), 1), (dict(seq_lens=0x1001), 1),
    (dict(draft_offsets=0x1002), 1), (dict(tree_mask=0x1004), 1), (dict(lse=0x1002), 1),
    (dict(num_seqs=8192, max_blocks_per_seq=1 << 20, max_seq_len=1 << 24, weights_len=1 << 24), 3),
    (dict(num_seqs=1, max_blocks_per_seq=1 << 27, max_seq_len=2 ** 31 - 1, weights_len=1 << 31), 3),
    (dict(num_rows=2 ** 31 - 1), 3), (dict(num_seqs=0), 0), (dict(num_rows=0), 0)]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(out=0), 1), (dict(v_cache=0), 1), (dict(out=0x1008), 1), (dict(v_cache=0x1008), 1),
    (dict(workspace_bytes=100), 3), (dict(workspace=0), 1), (dict(workspace=0x1010), 1)])
def test_attention_refuses(kw, status):
    assert _tree("pkv_paged_tree_attention", **kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(weights=0), 1), (dict(lse=0), 1), (dict(weights=0x1002), 1), (dict(weights_len=999), 1)])
def test_add_weights_refuses(kw, status):
    assert _tree("pkv_kv_add_weights", **kw) == status


@pytest.mark.parametrize("fn", ["pkv_paged_tree_attention", "pkv_kv_add_weights", "pkv_kv_compact"])
def test_null_arguments(fn):
    assert getattr(B.load(), fn)(None, None) == 1


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), 1), (dict(hkv=0), 1), (dict(max_seq_len=0), 1), (dict(budget=0), 1), (dict(sinks=-1), 1),
    (dict(recent=-1), 1), (dict(sinks=60, recent=41), 1), (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), 1),
    (dict(weights_len=999), 1), (dict(num_seqs=8193), 3), (dict(max_seq_len=2 ** 31 - 1, weights_len=2 ** 31), 3),
    (dict(kept=0), 1), (dict(kept_lens=0), 1), (dict(weights=0), 1), (dict(seq_lens=0), 1), (dict(kept=0x1002), 1),
    (dict(kept_lens=0x1002), 1), (dict(weights=0x1002), 1), (dict(seq_lens=0x1002), 1), (dict(num_seqs=0), 0)])
def test_select_refuses(kw, status):
    a = dict(kept=P, kept_lens=P, weights=P, weights_len=1000, seq_lens=P, num_seqs=4, hkv=4, max_seq_len=1000,
             budget=100, sinks=4, recent=10)
    a.update(kw)
    assert B.load().pkv_kv_select(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(num_seqs=-1), 1), (dict(max_blocks_per_seq=0), 1), (dict(num_blocks=0), 1), (dict(num_kv_heads=0), 1),
    (dict(kept_len=-1), 1), (dict(row_bytes=0), 1), (dict(block_size=0), 1), (dict(kept_heads=2), 1),
    (dict(kept_heads=0), 1), (dict(block_size=32), 5), (dict(row_bytes=24), 5), (dict(row_bytes=1040), 5),
    (dict(num_seqs=8193), 3), (dict(max_blocks_per_seq=1 << 27), 3), (dict(k_cache=0), 1), (dict(v_cache=0), 1),
    (dict(block_table=0), 1), (dict(seq_lens=0), 1), (dict(kept=0), 1), (dict(kept_lens=0), 1),
    (dict(v_cache=P), 1), (dict(weights_len=0), 1), (dict(k_cache=0x3008), 1), (dict(v_cache=0x1008), 1),
    (dict(block_table=0x1002), 1), (dict(seq_lens=0x1002), 1), (dict(kept=0x1002), 1), (dict(kept_lens=0x1002), 1),
    (dict(first=0x1002), 1), (dict(weights=0x1002), 1), (dict(num_seqs=0), 0)])
def test_compact_refuses(kw, status):
    a = dict(k_cache=P, v_cache=2 * P, weights=P, block_table=P, seq_lens=P, kept=P, kept_lens=P, first=P,
             weights_len=1000, num_blocks=32, num_seqs=4, max_blocks_per_seq=64, num_kv_heads=4, kept_heads=4,
             kept_len=100, row_bytes=256, block_size=16)
    a.update(kw)
    assert B.load().pkv_kv_compact(ctypes.byref(B.CompactArgs(**a)), None) == status


def test_packed_arguments_are_the_structures():
    assert B._TREE.size == ctypes.sizeof(B.TreeArgs) - 4 and B._COMPACT.size == ctypes.sizeof(B.CompactArgs) - 4
    a = B.TreeArgs.from_buffer_copy(B._TREE.pack(*range(1, 25), 0.5) + bytes(4))
    assert [getattr(a, n) for n, _ in B.TreeArgs._fields_] == list(range(1, 25)) + [0.5]
    c = B.CompactArgs.from_buffer_copy(B._COMPACT.pack(*range(1, 18)) + bytes(4))
    assert [getattr(c, n) for n, _ in B.CompactArgs._fields_] == list(range(1, 18))


def test_workspace_depends_on_the_rows():
    n = B.tree_workspace_bytes
    assert n(32, 8, 128, 64, 32768) == n(32, 8, 128, 64, 100000) >= 2 * 152 * 256 * 130 * 4
    assert 0 < n(32, 8, 128, 1, 32768) < n(32, 8, 128, 16, 32768)
    assert n(0, 8, 128, 1, 100) == n(32, 5, 128, 1, 100) == n(32, 8, 128, 0, 100) == 0


def _tensors():
    x = Batch([100, 40], [3, 2], 8, 2, seed=1)
    return dict(out=x.q.clone(), q=x.q, k=x.k, v=x.v, bt=x.table, sl=x.lens, off=x.offsets, mask=x.mask), x


@pytest.mark.parametrize("key,change,name", [
    ("k", lambda t: t.float(), "q is|v_cache"), ("v", lambda t: t.float(), "v_cache"), ("v", lambda t: t[:4], "v_cache"),
    ("q", lambda t: t.float(), "q is"), ("q", lambda t: t[0], "q is not"), ("q", lambda t: t[..., :64], "q is"),
    ("out", lambda t: t.half(), "out"), ("out", lambda t: t[:1], "out"), ("bt", lambda t: t.long(), "block_table"),
    ("bt", lambda t: t.T.contiguous().T, "block_table"), ("sl", lambda t: t.long(), "seq_lens"),
    ("sl", lambda t: t[:1], "seq_lens"), ("off", lambda t: t[:2], "draft_offsets"), ("off", lambda t: t.long(), "draft_offsets"),
    ("mask", lambda t: t.int(), "tree_mask"), ("mask", lambda t: t[:4], "tree_mask")])
def test_binding_names_the_tensor(key, change, name, monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    a, x = _tensors()
    a[key] = change(a[key])
    with pytest.raises(B.PagedKVError, match=name):
        B.paged_tree_attention(*a.values(), 100, 3, 0.1)


def test_binding_refuses_other_tensors(monkeypatch):
    a, x = _tensors()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(B.PagedKVError, match="current CUDA device"):
        B.paged_tree_attention(*a.values(), 100, 3, 0.1)
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    lse, w = torch.zeros(5, 8), torch.zeros(2, 2, 100)
    weights = lambda lse, w: B.kv_add_weights(w, a["q"], a["k"], a["bt"], a["sl"], a["off"], a["mask"], lse, 100, 3, 0.1)  # noqa: E731
    for bad, bad_w, name in ((None, w, "no lse"), (lse[:4], w, "lse"), (lse.double(), w, "lse"), (lse, w[0], "weights"),
                             (lse, w.double(), "weights"), (lse, w[:, :1], "weights"), (lse, None, "no weights")):
        with pytest.raises(B.PagedKVError, match=name):
            weights(bad, bad_w)
    kept, n = torch.zeros(2, 2, 5, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for args, name in (((kept[0], n, w, a["sl"]), "kept"), ((kept.long(), n, w, a["sl"]), "kept"),
                       ((kept, n[:1], w, a["sl"]), "kept_lens"), ((kept, n, w.half(), a["sl"]), "weights"),
                       ((kept[:, :1], n, w, a["sl"]), "kept"), ((kept, n, w, a["sl"].long()), "seq_lens")):
        with pytest.raises(B.PagedKVError, match=name):
            B.kv_select(*args, 100, 1, 1)
    compact = lambda **kw: B.kv_compact(**{**dict(k_cache=a["k"], v_cache=a["v"], block_table=a["bt"], seq_lens=a["sl"],  # noqa: E731
                                                  kept=kept, kept_lens=n, first=None, weights=w), **kw})
    for kw, name in ((dict(v_cache=a["v"][:3]), "v_cache"), (dict(kept=kept[0]), "kept"), (dict(kept=kept.long()), "kept"),
                     (dict(kept_lens=n[:1]), "kept_lens"), (dict(first=n.long()), "first"),
                     (dict(weights=w[:, :1]), "weights"), (dict(block_table=a["bt"][:1]), "seq_lens")):
        with pytest.raises(B.PagedKVError, match=name):
            compact(**kw)
    with pytest.raises(TypeError, match="dtype"):
        compact(k_cache=a["k"].half(), v_cache=a["v"].half())


def test_debug_checks():
    bt = torch.arange(8, dtype=torch.int32).reshape(2, 4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    V.check_tree(bt, i32(40, 64), i32(0, 3, 3), 3, 64, 4, 8, 16)
    V.check_tree(bt, i32(40, -9), i32(0, 3, 3), 3, 64, 4, 8, 16)
    for lens, off, nb, name in ((i32(40, 64), i32(0, 5, 5), 8, "draft_offsets"), (i32(40, 64), i32(0, 3, 2), 8, "draft_offsets"),
                                (i32(40, 64), i32(0, 3, 4), 8, "draft_offsets"), (i32(2, 64), i32(0, 3, 3), 8, "seq_lens"),
                                (i32(65, 64), i32(0, 3, 3), 8, "seq_lens"), (i32(40, 64), i32(0, 3, 3), 2, "block 2")):
        with pytest.raises(V.ValidationError, match=name):
            V.check_tree(bt, lens, off, 3, 64, 4, nb, 16)
    V.check_lengths(i32(0, 5), 5)
    with pytest.raises(V.ValidationError, match=r"seq_lens\[1\]"):
        V.check_lengths(i32(0, 6), 5)
    kept = torch.tensor([[[1, 5]], [[20, 30]]], dtype=torch.int32)
    V.check_compact(bt, i32(40, 64), kept, i32(2, 2), i32(0, 20), 64, 8, 16)
    V.check_compact(bt, i32(40, 64), kept, i32(2, 2), None, None, 8, 16)
    for kw, name in ((dict(seq_lens=i32(65, 64)), "seq_lens"), (dict(weights_len=39), "seq_lens"),
                     (dict(kept_lens=i32(3, 0)), "kept_lens"), (dict(first=i32(39, 0)), "kept_lens"),
                     (dict(first=i32(0, 21)), r"kept\[1\]\[0\]\[0\]"), (dict(seq_lens=i32(5, 64)), r"kept\[0\]\[0\]\[1\]"),
                     (dict(num_blocks=5), "block 5")):
        with pytest.raises(V.ValidationError, match=name):
            V.check_compact(**{**dict(block_table=bt, seq_lens=i32(40, 64), kept=kept, kept_lens=i32(2, 2), first=None,
                                      weights_len=64, num_blocks=8, block_size=16), **kw})


def test_debug_mode_runs_the_checks(monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    a, x = _tensors()
    kept, n = torch.full((2, 2, 5), 200, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    w = torch.zeros(2, 2, 100)
    B.set_debug(True)
    try:
        with pytest.raises(B.PagedKVError, match=r"seq_lens\[0\]"):
            B.paged_tree_attention(*a.values(), 99, 3, 0.1)
        with pytest.raises(B.PagedKVError, match="draft_offsets"):
            B.kv_add_weights(w, a["q"], a["k"], a["bt"], a["sl"], a["off"], a["mask"], torch.zeros(5, 8), 100, 2, 0.1)
        with pytest.raises(B.PagedKVError, match=r"seq_lens\[0\]"):
            B.kv_select(kept, n, w, a["sl"], 50, 1, 1)
        with pytest.raises(B.PagedKVError, match=r"kept\[0\]\[0\]\[0\]"):
            B.kv_compact(a["k"], a["v"], a["bt"], a["sl"], kept, n)
    finally:
        B.set_debug(False)


# --------------------------------------------------------------- the oracle
def test_oracle_chain_is_the_causal_oracle(oracle_mod):
    """A chain of drafts is the last rows of full causal attention."""
    x = Batch([20], [6], 4, 2, 16, F32, seed=3, mask="chain")
    out, lse = T.tree_attention(*x.args())
    k, v = (T.rows_of(p, x.table, 0, h, 20) for p, h in ((x.k, 1), (x.v, 1)))
    for i in range(6):
        s = x.q[i, 3].double() @ k[:15 + i].T * x.scale
        assert torch.allclose(out[i, 3], torch.softmax(s, 0) @ v[:15 + i], atol=1e-12)
        assert abs(float(lse[i, 3] - torch.logsumexp(s, 0))) < 1e-12
        one = oracle_mod.paged_decode(x.q[i:i + 1], x.k, x.v, x.table,
                                      torch.tensor([15 + i], dtype=torch.int32), x.scale)
        assert torch.allclose(out[i], one[0].double(), atol=1e-6)


def test_oracle_mask_words():
    import random
    words = tree_words(64, random.Random(1))
    assert int(signed(words)[63]) < 0                       # bit 63 is the sign
    assert T.sees(signed(words), 64, 70, 63)[-1] and T.sees(signed(words), 64, 70, 0).sum() == 7
    assert T.sees(None, 3, 5, 1).tolist() == [True, True, True, True, False]
    assert T.sees(torch.tensor([4, 0, 1]), 3, 4, 0).tolist() == [True, False, False, True]


def test_oracle_weights_add_up():
    x = Batch([30, 9], [4, 9], 4, 2, 16, F32, seed=4)
    _, lse = T.tree_attention(*x.args())
    w = T.add_weights(torch.zeros(2, 2, 31), x.q, x.k, x.table, x.lens, x.offsets, x.mask, lse, x.scale)
    assert torch.allclose(w.sum(2), torch.tensor([[8.0, 8.0], [18.0, 18.0]], dtype=torch.float64))


def test_oracle_select_and_compact():
    w = torch.tensor([[[5.0, 1.0, 3.0, 3.0, 9.0, math.nan, 0.0]]])
    assert T.select(w, [7], 4, 1, 1) == [[[0, 2, 4, 6]]]
    assert T.select(w, [7], 6, 0, 0) == [[[0, 1, 2, 3, 4, 6]]] and T.select(w, [3], 4, 1, 1) == [[[0, 1, 2]]]
    k = torch.arange(32.0).reshape(2, 1, 16, 1)
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    kept = torch.tensor([[[3, 17]]], dtype=torch.int32)
    a, b, c = T.compact(k, -k, torch.arange(1.0, 21).reshape(1, 1, 20), table, [18], kept, [2], [2])
    assert a[1, 0, :4, 0].tolist() == [16, 17, 19, 1] and b[1, 0, 3, 0] == -1 and a[0, 0, 1, 0] == 1
    assert c[0, 0].tolist() == [1, 2, 4, 18] + [0] * 14 + [19, 20]
