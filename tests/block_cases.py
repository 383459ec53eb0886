"""Inputs and references shared by the tests of the attention over the
block-scaled fp8 cache."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from oracle import fp8_block as FB
from paged_kv_cache_104_gb300 import binding as B

NAN_CODE = 0x7F


class Pools:
    """Filled pools, their scale bytes, and fp64 values (CPU)."""

    def __init__(self, nb, hkv, seed, k_spread=2, v_spread=2):
        g = torch.Generator().manual_seed(seed)
        self.codes, self.scale = [], []
        for spread in (k_spread, v_spread):
            x = torch.randn(nb, hkv, 16, 128, generator=g)
            e = torch.randint(-spread, spread + 1, (nb, hkv), generator=g) if spread else torch.zeros(nb, hkv)
            # N(0, 1) at exponent -7 covers the code range; the block's size varies by 2^e
            self.codes.append((x * 2.0 ** 7).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            self.scale.append((127 - 7 + e).to(torch.uint8))

    def values(self, which):
        return torch.from_numpy(FB.dequantize(self.codes[which].numpy(), self.scale[which].numpy()))

    def cuda(self):
        return self.codes[0].cuda(), self.codes[1].cuda(), self.scale[0].cuda(), self.scale[1].cuda()


def tables(lens, seed, spare=2):
    """(block tables int32 with unrelated ids in the tails, pool size)."""
    g = torch.Generator().manual_seed(500 + seed)
    need = [-(-n // 16) for n in lens]
    nb = sum(need) + spare
    ids = torch.randperm(nb, generator=g).to(torch.int32)
    table = torch.randint(0, nb, (len(lens), max(max(need), 1)), generator=g).to(torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, nb


def used_rows(table, lens, nb):
    m = torch.zeros(nb, 16, dtype=torch.bool)
    for r, n in enumerate(lens):
        for j in range(-(-n // 16)):
            m[int(table[r, j]), :min(16, n - 16 * j)] = True
    return m


def poison(pools, table, lens):
    """NaN codes in every row no sequence uses."""
    bad = ~used_rows(table, lens, pools.codes[0].shape[0])
    for c in pools.codes:
        c.permute(0, 2, 1, 3)[bad] = NAN_CODE


def bound(ref, ref_abs, rel):
    """Half a step of the bf16 result, plus `rel` of the weighted mean of |v|
    for the rounding of the weights and of the scores."""
    return 2.0 ** -8 * ref.abs() + rel * ref_abs


def decode(pools, q, table, lens, scale, max_seq_len=None, out=None, workspace=None, stream=None, expect=0):
    kc, vc, ks, vs = pools.cuda() if isinstance(pools, Pools) else pools
    b, hq, _ = q.shape
    msl = max(max(lens), 1) if max_seq_len is None else max_seq_len
    out = torch.zeros(b, hq, 128, dtype=torch.bfloat16, device="cuda") if out is None else out
    ws = B.decode_workspace_fp8_block(b, hq, kc.shape[1], 128, msl) if workspace is None else workspace
    ws.fill_(0xFF)                                   # NaN to whoever reads what this call did not write
    B.paged_decode_attention_fp8_block(out, q.cuda(), kc, vc, ks, vs, table.cuda(),
                                       torch.tensor(lens, dtype=torch.int32).cuda(), msl, scale, ws, stream)
    torch.cuda.synchronize()
    assert B.get_device_error() == expect
    return out.cpu()


def check_decode(pools, q, table, lens, scale, got, rows=None):
    """got against the fp64 oracle.  The kernel rounds each weight to f16
    (2^-11 relative, or 2^-25 of the largest weight times V scale, below its
    normal range, times a code of at most 448); its scores and sums are fp32
    and its exponentials good to 2^-22, together well below 2^-13."""
    k, v = pools.values(0), pools.values(1)
    rows = [i for i in range(len(lens)) if lens[i] > 0] if rows is None else rows
    qd, bt, sl = q[rows].double(), table[rows], torch.tensor([lens[i] for i in rows], dtype=torch.int32)
    used = sorted({int(x) for i, r in enumerate(rows) for x in table[r, :-(-lens[r] // 16)]})
    remap = torch.zeros(k.shape[0], dtype=torch.int32)
    remap[used] = torch.arange(len(used), dtype=torch.int32)
    bt, k, v = remap[bt.long()], k[used], v[used]    # unused blocks may hold NaN
    k, v = torch.nan_to_num(k, 0.0), torch.nan_to_num(v, 0.0)
    ref = oracle.paged_decode(qd, k, v, bt, sl, scale)
    ref_abs = oracle.paged_decode(qd, k, v.abs(), bt, sl, scale)
    unit = torch.exp2(pools.scale[1][used].double() - 127)
    ones = unit[:, :, None, None].expand_as(v).contiguous()
    # a row's largest weight times V scale is at most the sum of them
    top = oracle.paged_decode(qd, k, ones, bt, sl, scale)
    flush = sl.double()[:, None, None] * 2.0 ** -25 * 448.0 * top
    err = (got[rows].double() - ref).abs()
    over = err - bound(ref, ref_abs, 2.0 ** -11 + 2.0 ** -13) - flush
    assert bool((over <= 0).all()), f"off by {float(err.max())}, {float(over.max())} over its bound"
