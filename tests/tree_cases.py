"""Batches for the operators of drafted tokens and eviction: paged pools with
NaN in every row that no sequence stores, drafted tokens, trees; and the error
bounds of their results."""
from __future__ import annotations

import random

import torch

from oracle import tree as T

BF16, F32 = torch.bfloat16, torch.float32


def tree_words(drafted: int, pick: random.Random):
    """A random forest: each drafted token sees itself and its ancestors."""
    seen = []
    for i in range(drafted):
        parent = pick.randint(-1, i - 1)
        seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
    return seen


def signed(words):
    return torch.tensor([w - (1 << 64) if w >> 63 else w for w in words], dtype=torch.int64)


class Batch:
    """lens: stored tokens (drafted ones among them); drafted: their numbers.
    All tensors are on the CPU; ``on`` copies them."""

    def __init__(self, lens, drafted, hq, hkv, dim=128, dtype=BF16, seed=0, mask="tree", spare_rows=0, scale=None,
                 q_gain=1.0):
        gen, pick = torch.Generator().manual_seed(seed), random.Random(seed)
        self.hq, self.hkv, self.dim, self.dtype = hq, hkv, dim, dtype
        self.scale = dim ** -0.5 if scale is None else scale
        per = [-(-n // 16) for n in lens]
        self.num_blocks = sum(per) + 3
        order = list(range(self.num_blocks))
        pick.shuffle(order)
        width = max(per + [1]) + 2
        self.table = torch.tensor([[pick.randrange(self.num_blocks) for _ in range(width)] for _ in lens],
                                  dtype=torch.int32)
        shape = (self.num_blocks, hkv, 16, dim)
        self.k = torch.full(shape, float("nan")).to(dtype)
        self.v = torch.full(shape, float("nan")).to(dtype)
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :per[b]] = torch.tensor(order[at:at + per[b]], dtype=torch.int32)
            at += per[b]
            for j in range(per[b]):
                rows = min(16, n - 16 * j)
                blk = int(self.table[b, j])
                self.k[blk, :, :rows] = torch.randn((hkv, rows, dim), generator=gen).to(dtype)
                self.v[blk, :, :rows] = torch.randn((hkv, rows, dim), generator=gen).to(dtype)
        self.lens = torch.tensor(lens, dtype=torch.int32)
        off = [0]
        for n in drafted:
            off.append(off[-1] + n)
        self.rows = off[-1] + spare_rows
        self.offsets = torch.tensor(off, dtype=torch.int32)
        self.max_len, self.max_draft = max(max(lens), 1), max(max(drafted), 1)
        self.q = (torch.randn((self.rows, hq, dim), generator=gen) * q_gain).to(dtype)
        self.mask = None
        if mask == "tree":
            words = [w for n in drafted for w in tree_words(n, pick)] + [1] * spare_rows
            self.mask = signed(words)
        elif mask == "random":   # any bits: rows that see nothing, bits past the drafted tokens
            self.mask = signed([pick.choice([0, 0, pick.getrandbits(64), 1 << 63]) for _ in range(self.rows)])

    def args(self):
        return self.q, self.k, self.v, self.table, self.lens, self.offsets, self.mask, self.scale

    def score_error(self):
        """Bound on the error of one scaled score in fp32: D steps of half a
        unit of the sum of absolute products, which the norms bound; twice, as
        a tensor core's sum may truncate."""
        top = [float(torch.nan_to_num(x.double()).pow(2).sum(-1).max().sqrt()) if x.numel() else 0.0
               for x in (self.q, self.k)]
        return 2 * self.dim * 2.0 ** -24 * top[0] * top[1] * self.scale

    def bounds(self, ref_out):
        """Bounds on out and lse: a score's error moves a weight by its own
        size (and the sum by as much), bf16 weights are off by 2^-8 of
        themselves and so are bf16 results, ex2 and the sums by 2^-20 and
        2^-23 a term."""
        mag, lse = T.tree_attention(self.q, self.k, torch.nan_to_num(self.v).abs(), *self.args()[3:])
        half = 2.0 ** -8 if self.dtype is BF16 else 2.0 ** -24
        rel = 4 * self.score_error() + 2.0 ** -20 + self.max_len * 2.0 ** -23
        out = mag * (rel + half) + ref_out.abs() * half
        return out, rel + lse.abs() * 2.0 ** -22
