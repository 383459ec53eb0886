"""Pools that the tree attention and the counts do not take are refused (no GPU)."""
import pytest
import torch

from paged_kv_cache_104_gb300 import binding as B
from tree_cases import Batch


@pytest.mark.parametrize("dtype", [torch.uint8, torch.float16, torch.float8_e4m3fn, torch.float64])
@pytest.mark.parametrize("queries", ["as the pools", "bf16"])
def test_other_pools(dtype, queries, monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    x = Batch([100, 40], [3, 2], 8, 2, seed=1)
    k = torch.zeros(x.k.shape).to(dtype)
    q = torch.zeros(x.q.shape).to(dtype if queries == "as the pools" else torch.bfloat16)
    lse, w = torch.zeros(5, 8), torch.zeros(2, 2, 100)
    with pytest.raises((TypeError, B.PagedKVError), match="dtype|q is"):
        B.paged_tree_attention(q.clone(), q, k, k.clone(), x.table, x.lens, x.offsets, x.mask, 100, 3, 0.1)
    with pytest.raises((TypeError, B.PagedKVError), match="dtype|q is"):
        B.kv_add_weights(w, q, k, x.table, x.lens, x.offsets, x.mask, lse, 100, 3, 0.1)
