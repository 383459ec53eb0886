"""Inputs shared by the tests of the rotating and block-scaled appends."""
from __future__ import annotations

import torch

BS = 16


def table(positions: int, rot_dim: int) -> torch.Tensor:
    """cos and sin of position times frequency, float32 [positions, rot_dim]."""
    half = rot_dim // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def sections(rot_dim: int, axes: int, in_turn: bool = False):
    """Each pair's axis: equal sections of the pairs, or the axes in turn."""
    half = rot_dim // 2
    return [i % axes if in_turn else i * axes // half for i in range(half)]


def draw(t, hq, hkv, d, dtype, seed, axes=1, num_positions=997):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(t, hq, d, generator=g).to(dtype)
    k = torch.randn(t, hkv, d, generator=g).to(dtype)
    v = torch.randn(t, hkv, d, generator=g).to(dtype)
    pos = torch.randint(0, num_positions, (axes, t), generator=g).to(torch.int32)
    return q, k, v, pos


def scattered_slots(t, num_blocks, seed):
    g = torch.Generator().manual_seed(100 + seed)
    return torch.randperm(num_blocks * BS, generator=g)[:t].to(torch.int64)


def run_slots(pieces, num_blocks, seed):
    """Slots of sequences' new tokens: pieces = [(first row, tokens)], each in
    blocks of its own, dealt from a shuffled pool."""
    g = torch.Generator().manual_seed(200 + seed)
    ids = torch.randperm(num_blocks, generator=g).tolist()
    out, at = [], 0
    for first, n in pieces:
        out += [ids[at + (first + i) // BS] * BS + (first + i) % BS for i in range(n)]
        at += (first + n - 1) // BS + 1
    assert at <= num_blocks
    return torch.tensor(out, dtype=torch.int64)
