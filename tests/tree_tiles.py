"""Long batches whose values say which tile of 128 tokens they come from.

With random values the result of n tokens shrinks as 1 / sqrt(n) while its
bound does not, so that a lost tile of a long sequence would pass.  Here a
tile's values lie in one channel only: a channel holds a few tiles' weights,
all of one sign, and its bound is a small part of each."""
from __future__ import annotations

import torch

from oracle import tree as T
from tree_cases import Batch

TILE = 128


def mark_tiles(x: Batch) -> Batch:
    """Token t's value: 1, 1.25, 1.5, .. in the channel of its tile (the size tells
    the tiles of one channel apart), 0 in the others."""
    for b, n in enumerate(x.lens.tolist()):
        t = torch.arange(n)
        tile, channels = t // TILE, x.dim
        rows = torch.zeros((n, x.dim))
        rows[t, tile % channels] = 1 + 0.25 * (tile // channels).float()
        at = x.table[b, t // 16].long()
        for h in range(x.hkv):
            x.v[at, h, t % 16] = rows.to(x.v.dtype)
    return x


def late_maximum(x: Batch, start: float, seed: int) -> Batch:
    """All queries share a direction, and in the tokens behind the part `start`
    of each sequence every fifth key points there: scores some 200 powers of
    two above all others, so that an earlier maximum would overflow."""
    g = torch.Generator().manual_seed(seed)
    common = torch.randn(x.dim, generator=g)
    x.q = (common + 0.05 * torch.randn(x.q.shape, generator=g)).to(x.q.dtype)
    for b, n in enumerate(x.lens.tolist()):
        t = torch.arange(int(n * start), n - int(x.offsets[b + 1] - x.offsets[b]), 5)
        at = x.table[b, t // 16].long()
        for h in range(x.hkv):
            keys = 150 * common / common.norm() + 0.3 * torch.randn((len(t), x.dim), generator=g)
            x.k[at, h, t % 16] = keys.to(x.k.dtype)
    return x


def tile_shares(x: Batch, b: int):
    """What each tile of sequence b gives to `out`, fp64 [rows, query heads,
    tiles, dim], and the tiles' sums of weights [rows, query heads, tiles]."""
    n, lo, hi = int(x.lens[b]), int(x.offsets[b]), int(x.offsets[b + 1])
    pad, g = -n % TILE, x.hq // x.hkv
    parts, sums = [], []
    for h in range(x.hkv):
        k, v = (T.rows_of(p, x.table, b, h, n) for p in (x.k, x.v))
        words = None if x.mask is None else x.mask[lo:hi]
        seen = torch.tensor([T.sees(words, hi - lo, n, i).tolist() for i in range(hi - lo)])[:, None]
        s = x.q[lo:hi, h * g:(h + 1) * g].double() @ k.T * x.scale
        p = torch.softmax(torch.where(seen, s, -float("inf")), 2)
        p = torch.nn.functional.pad(p, (0, pad)).unflatten(2, (-1, TILE))
        v = torch.nn.functional.pad(v, (0, 0, 0, pad)).unflatten(0, (-1, TILE))
        parts.append(torch.einsum("mgtn,tnd->mgtd", p, v))
        sums.append(p.sum(3))
    return torch.cat(parts, 1), torch.cat(sums, 1)
