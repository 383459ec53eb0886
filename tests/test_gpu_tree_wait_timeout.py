"""The give-up paths of the tree attention and the counts: waits that run out
are reported, the calls return and the GPU stays usable.

As in the test of the decode's waits, a test-only build (``build.build_wait_test``)
has its wait limits cut to about 2 ms and its key and value producers withhold
every copy: the issuer, the guard and the softmax or summing warps run into
their limits with none of those copies in flight, the first one raises the
CTA's abort flag, and every other wait ends by that or by its own limit.  Then
the shipped library, on the same GPU and inputs, gives the results it gave before."""
import ctypes

import pytest
import torch

from paged_kv_cache_104_gb300 import binding as B
from paged_kv_cache_104_gb300 import build as BL
from test_gpu_tree_edges import attend, on
from tree_cases import Batch

pytestmark = pytest.mark.gpu
D = "cuda"
PKV_DEVERR_TIMEOUT = 4

BATCHES = {
    "cut, both sides in turn": ([700, 33, 1500, 64], [5, 2, 30, 1], 8, 2),
    "up to 512 rows": ([900, 5000], [64, 40], 16, 2),
    "whole sequences": ([200, 90, 17], [9, 3, 17], 8, 2),
    "KV heads in pairs": ([100 + 3 * i for i in range(60)], [1 + i % 16 for i in range(60)], 16, 8),
}


def error_of(lib):
    code = ctypes.c_int(-1)
    assert lib.pkv_get_device_error(ctypes.byref(code), 1) == 0
    return code.value


@pytest.mark.parametrize("name", BATCHES)
def test_waits_that_run_out(name):
    lib = B.open_library(BL.build_wait_test())
    lens, drafted, hq, hkv = BATCHES[name]
    x = Batch(lens, drafted, hq, hkv, seed=len(lens))
    t = on(x)
    out, lse = attend(x, t)
    w = torch.zeros((len(lens), hkv, x.max_len), device=D)
    B.kv_add_weights(w, t[0], t[1], *t[3:6], t[6], lse, x.max_len, x.max_draft, x.scale)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0

    ws = B.tree_workspace(hq, hkv, 128, x.max_draft, x.max_len)
    scrap = torch.zeros_like(out), lse.clone(), torch.zeros_like(w)
    a = B.TreeArgs(out=scrap[0].data_ptr(), lse=scrap[1].data_ptr(), q=t[0].data_ptr(), k_cache=t[1].data_ptr(),
                   v_cache=t[2].data_ptr(), block_table=t[3].data_ptr(), seq_lens=t[4].data_ptr(),
                   draft_offsets=t[5].data_ptr(), tree_mask=t[6].data_ptr(), weights=scrap[2].data_ptr(),
                   workspace=ws.data_ptr(), workspace_bytes=ws.numel(), weights_len=x.max_len,
                   num_blocks=x.num_blocks, num_seqs=len(lens), num_rows=x.rows, max_blocks_per_seq=x.table.shape[1],
                   max_seq_len=x.max_len, max_draft=x.max_draft, num_q_heads=hq, num_kv_heads=hkv, head_dim=128,
                   block_size=16, dtype=B.PKV_BF16, scale=x.scale)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert error_of(lib) == 0
    for call in (lib.pkv_paged_tree_attention, lib.pkv_kv_add_weights):
        assert call(ctypes.byref(a), stream) == 0
        torch.cuda.synchronize()
        assert error_of(lib) == PKV_DEVERR_TIMEOUT

    again = attend(x, t, ws=ws)
    w2 = torch.zeros_like(w)
    B.kv_add_weights(w2, t[0], t[1], *t[3:6], t[6], again[1], x.max_len, x.max_draft, x.scale)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip((*again, w2), (out, lse, w)))
