"""The attention over the block-scaled fp8 cache without a GPU: host refusals
of the library and of the binding, the workspace's size, the debug mode."""
import ctypes

import pytest
import torch

from paged_kv_cache_104_gb300 import binding as B
from paged_kv_cache_104_gb300 import validate as V


def _decode(**kw):
    P = 0x1000
    a = dict(out=P, q=P, k=P, v=P, ks=0x1001, vs=0x1003, bt=P, sl=P, B=4, mb=64, msl=1000, nb=32, hq=16, hkv=4,
             d=128, bs=16, scale=0.1, ws=0x1000, wsb=1 << 30)
    a.update(kw)
    return B.load().pkv_paged_decode_attention_fp8_block(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), 1), (dict(hq=18), 1), (dict(hkv=0), 1), (dict(d=0), 1), (dict(bs=0), 1), (dict(bs=32), 5),
    (dict(d=64), 5), (dict(hq=12), 5), (dict(hq=128), 5), (dict(B=-1), 1), (dict(mb=0), 1), (dict(msl=0), 1),
    (dict(nb=0), 1), (dict(B=8193), 3), (dict(msl=1025), 1), (dict(scale=float("inf")), 1),
    (dict(out=0), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(ks=0), 1), (dict(vs=0), 1),
    (dict(bt=0), 1), (dict(sl=0), 1), (dict(q=0x1008), 1), (dict(bt=0x1002), 1), (dict(sl=0x1001), 1),
    (dict(wsb=100), 3), (dict(ws=0, wsb=0), 3), (dict(ws=0), 1), (dict(ws=0x1010), 1), (dict(msl=2 ** 31 - 1, mb=2 ** 28), 3),
    (dict(B=0), 0)])
def test_decode_refuses(kw, status):
    assert _decode(**kw) == status


def test_workspace_follows_the_batch():
    n = B.decode_fp8_block_workspace_bytes
    assert n(1, 32, 8, 128, 64) == 0                       # one split of 64 tokens
    assert n(0, 32, 8, 128, 64) == 0
    rows = 1 * 32 * (13 + 1)                               # 777 tokens: 13 splits of 64, one more piece
    assert 0 <= n(1, 32, 8, 128, 777) - (rows * 130 * 4 + 32 * 4) < 768
    # a large batch has the splits of 512 of the other decodes
    assert n(128, 32, 8, 128, 32768) == B.decode_workspace_bytes(128, 32, 128, 32768)
    for b, hkv, msl in ((1, 8, 5000), (4, 2, 900), (64, 8, 2301), (16, 1, 20000)):
        assert n(b, 32, hkv, 128, msl) >= B.decode_workspace_bytes(b, 32, 128, msl)


def _tensors():
    k = torch.zeros(8, 4, 16, 128, dtype=torch.uint8)
    sc = torch.zeros(8, 4, dtype=torch.uint8)
    q = torch.zeros(2, 16, 128, dtype=torch.bfloat16)
    return dict(out=q.clone(), q=q, k=k, v=k.clone(), ks=sc, vs=sc.clone(), bt=torch.zeros(2, 4, dtype=torch.int32),
                sl=torch.tensor([1, 40], dtype=torch.int32))


@pytest.mark.parametrize("key,change,name", [
    ("k", lambda t: t.to(torch.bfloat16), "pools"), ("v", lambda t: t.float(), "v_cache"), ("v", lambda t: t[:4], "v_cache"),
    ("ks", lambda t: t.float(), "k_scale"), ("vs", lambda t: t[:, :2], "v_scale"), ("q", lambda t: t.float(), "q is"),
    ("q", lambda t: t[0], "q is not"), ("q", lambda t: t[..., :64], "q is"), ("out", lambda t: t.half(), "out"),
    ("out", lambda t: t[:1], "out"), ("bt", lambda t: t.long(), "block_table"), ("bt", lambda t: t[:1], "block_table"),
    ("bt", lambda t: t.T.contiguous().T, "block_table"), ("sl", lambda t: t.long(), "seq_lens")])
def test_binding_names_the_tensor(key, change, name, monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    a = _tensors()
    a[key] = change(a[key])
    with pytest.raises(B.PagedKVError, match=name):
        B.paged_decode_attention_fp8_block(*a.values(), 40, 0.1)


def test_binding_refuses_tensors_off_the_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(B.PagedKVError, match="current CUDA device"):
        B.paged_decode_attention_fp8_block(*_tensors().values(), 40, 0.1)


def test_debug_mode_allows_padded_rows_only_here(monkeypatch):
    bt, sl = torch.zeros(2, 4, dtype=torch.int32), torch.tensor([0, 40], dtype=torch.int32)
    V.check_decode(bt, sl, 64, 8, 16, empty_ok=True)
    with pytest.raises(V.ValidationError, match="seq_lens"):
        V.check_decode(bt, sl, 64, 8, 16)
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    B.set_debug(True)
    try:
        a = _tensors()
        a["sl"] = torch.tensor([0, 65], dtype=torch.int32)
        with pytest.raises(B.PagedKVError, match="seq_lens"):
            B.paged_decode_attention_fp8_block(*a.values(), 64, 0.1)
    finally:
        B.set_debug(False)


def _prefill(**kw):
    P = 0x1000
    a = dict(out=P, q=P, k=P, v=P, ks=0x1001, vs=0x1003, bt=P, mb=64, prior=100, C=50, nb=32, hq=16, hkv=4, d=128,
             bs=16, scale=0.1)
    a.update(kw)
    return B.load().pkv_chunked_prefill_attention_fp8_block(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(hq=0), 1), (dict(hq=18), 1), (dict(hkv=0), 1), (dict(bs=32), 5), (dict(d=64), 5), (dict(hq=12), 5),
    (dict(mb=0), 1), (dict(prior=-1), 1), (dict(C=-1), 1), (dict(nb=0), 1), (dict(C=1000), 1),
    (dict(scale=float("nan")), 1), (dict(scale=0.0), 1), (dict(scale=-0.1), 1),
    (dict(out=0), 1), (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(ks=0), 1), (dict(vs=0), 1), (dict(bt=0), 1), (dict(k=0x1008), 1), (dict(bt=0x1001), 1), (dict(C=0, out=0, q=0), 0),
    (dict(prior=2 ** 31 - 60, mb=2 ** 28), 3)])
def test_prefill_refuses(kw, status):
    assert _prefill(**kw) == status


@pytest.mark.parametrize("key,change,name", [
    ("k", lambda t: t.float(), "pools"), ("v", lambda t: t[:4], "v_cache"), ("ks", lambda t: t.int(), "k_scale"),
    ("vs", lambda t: t[:4], "v_scale"), ("q", lambda t: t.float(), "q is"), ("q", lambda t: t[:, 0], "q is not"),
    ("out", lambda t: t[:1], "out"), ("bt", lambda t: t.long(), "block_table_row"), ("bt", lambda t: t[None], "q is not"),
    ("bt", lambda t: t[::2], "block_table_row")])
def test_prefill_binding_names_the_tensor(key, change, name, monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    a = _tensors()
    a["bt"] = torch.zeros(8, dtype=torch.int32)
    del a["sl"]
    a[key] = change(a[key])
    with pytest.raises(B.PagedKVError, match=name):
        B.chunked_prefill_attention_fp8_block(*a.values(), 0, 0.1)


def test_prefill_debug_mode_names_the_block(monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    a = _tensors()
    a["bt"] = torch.tensor([0, 8], dtype=torch.int32)
    del a["sl"]
    B.set_debug(True)
    try:
        with pytest.raises(B.PagedKVError, match="block 8"):
            B.chunked_prefill_attention_fp8_block(*a.values(), 20, 0.1)
    finally:
        B.set_debug(False)
