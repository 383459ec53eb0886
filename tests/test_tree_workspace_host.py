"""pkv_tree_workspace_bytes gives 0 on exactly the sizes that the attention refuses (no GPU)."""
import ctypes

import pytest

from paged_kv_cache_104_gb300 import binding as B

P, MOST = 0x1000, 2 ** 31 - 1 - 65536


def refused(hq, hkv, dim, draft, length):
    """Does the attention refuse these sizes for what they are?  (Its workspace is too small here, which it says last
    of all sizes, with another status for every other reason.)"""
    a = B.TreeArgs(out=P, lse=P, q=P, k_cache=P, v_cache=P, block_table=P, seq_lens=P, draft_offsets=P, tree_mask=None,
                   weights=None, workspace=P, workspace_bytes=0, weights_len=0, num_blocks=32, num_seqs=1, num_rows=1,
                   max_blocks_per_seq=1 << 27, max_seq_len=length, max_draft=draft, num_q_heads=hq, num_kv_heads=hkv,
                   head_dim=dim, block_size=16, dtype=B.PKV_BF16, scale=0.1)
    status = B.load().pkv_paged_tree_attention(ctypes.byref(a), None)
    assert status in (1, 3, 5)
    return status != 3 or length > MOST


@pytest.mark.parametrize("hq,hkv,dim,draft,length", [
    (12, 4, 128, 8, 1000), (128, 4, 128, 8, 1000), (24, 4, 128, 8, 1000), (96, 2, 128, 8, 1000), (32, 8, 128, 65, 1000),
    (32, 8, 128, 2 ** 31 - 1, 1000), (2 ** 31 - 1, 1, 128, 64, 1000), (32, 8, 64, 8, 1000), (32, 8, 16, 8, 1000),
    (32, 8, 256, 8, 1000), (-32, -8, 128, 8, 1000), (32, -8, 128, 8, 1000), (32, 8, 128, -1, 1000),
    (32, 8, 128, 8, 0), (32, 8, 128, 8, MOST + 1), (32, 8, 128, 8, 2 ** 31 - 1)])
def test_sizes_that_no_call_takes(hq, hkv, dim, draft, length):
    assert refused(hq, hkv, dim, draft, length)
    assert B.tree_workspace_bytes(hq, hkv, dim, draft, length) == 0


@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("draft,length", [(1, 1), (64, 1000), (64, MOST)])
def test_sizes_that_a_call_takes(group, hkv, draft, length):
    assert not refused(group * hkv, hkv, 128, draft, length)
    assert B.tree_workspace_bytes(group * hkv, hkv, 128, draft, length) > 0
