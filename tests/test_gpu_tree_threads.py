"""Host threads with streams of their own: attention and counts at once, every result compared."""
import threading

import pytest
import torch

from paged_kv_cache_104_gb300 import binding as B
from test_gpu_tree_edges import attend, check, on
from tree_cases import BF16, F32, Batch

pytestmark = pytest.mark.gpu
D = "cuda"


def counts(x, t, lse, w):
    B.kv_add_weights(w, t[0], t[1], *t[3:6], t[6], lse, x.max_len, x.max_draft, x.scale)
    return w


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_two_host_threads_count_alike(dtype):
    xs = [Batch([700, 40], [9, 3], 16, 4, dtype=dtype, seed=6), Batch([90, 1300], [2, 33], 8, 1, dtype=dtype, seed=7)]
    ts = [on(x) for x in xs]
    start = [torch.rand((2, x.hkv, x.max_len), generator=torch.Generator().manual_seed(i)).to(D)
             for i, x in enumerate(xs)]
    want = []
    for x, t, w in zip(xs, ts, start):
        out, lse = attend(x, t)
        check(x, out, lse)
        want.append((out, lse, counts(x, t, lse, w.clone())))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for n in range(30):
                out, lse = attend(xs[i], ts[i])
                got = (out, lse, counts(xs[i], ts[i], lse, start[i].clone()))
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append((i, n))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad and B.get_device_error() == 0
