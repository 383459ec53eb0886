"""kv_append_fp8_block where a run's largest rotated key lies beside a border of
the scale, 448 * 2^e, or beyond fp32: codes and scale bytes are the oracle's for
the fp64 rotation, bit for bit."""
import numpy as np
import pytest
import torch

import rope_cases as R
from oracle import rope as O
from test_gpu_fp8_block_append import _pools, _rotated_exactly

pytestmark = pytest.mark.gpu

D = 128


def _slots(tokens, first_row):
    """Each token in a block of its own (a decode step), or one run."""
    if first_row is None:
        return R.run_slots([((7 * i) % 16, 1) for i in range(tokens)], tokens, tokens)
    return R.run_slots([(first_row, tokens)], tokens // 16 + 3, tokens)


def _check(k, cs, pos, interleaved, slots, seed):
    nb = int(slots.max()) // 16 + 1
    codes, scale = _pools(nb, k.shape[1], k.shape[2], seed)
    _rotated_exactly(k.bfloat16(), cs, pos, interleaved, codes, scale, slots)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("first_row", [0, 9])
@pytest.mark.parametrize("hkv", [2, 80])                 # a head to a CTA, and four
def test_a_low_frequency_pair_at_a_small_position(hkv, first_row, interleaved):
    """An ordinary table: position 1 of the slowest pair leaves 3.5 + 2.5e-8,
    which fp32 rounds to 3.5 = 448 * 2^-7."""
    half = D // 2
    angle = torch.arange(4).double()[:, None] * 500000.0 ** (-torch.arange(half).double() / half)
    cs = torch.cat([angle.cos(), angle.sin()], 1).float()
    first, second = O.pair_columns(D, interleaved)
    g = torch.Generator().manual_seed(hkv)
    k = torch.randn(3, hkv, D, generator=g) * 0.3
    k[1, :, first[half - 1]], k[1, :, second[half - 1]] = 3.5, -0.01001
    pos = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    turned = O.rotate(k[1:2].bfloat16().double().numpy(), cs.numpy(), pos[:, 1:2].numpy(), interleaved)
    assert (np.abs(turned).max((0, 2)) > 3.5).all() and (np.abs(turned).max((0, 2)).astype(np.float32) == 3.5).all()
    _check(k, cs, pos, interleaved, torch.arange(3) + 16 + first_row, hkv)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hkv,first_row", [(1, 1, None), (40, 4, None), (300, 8, None), (2000, 1, None),
                                                  (13, 3, 2), (40, 80, 9), (600, 8, 0)])
def test_maxima_within_fp32_rounding_of_a_border(tokens, hkv, first_row, interleaved):
    """Each token's table turns one pair to within 2 ulps of 448 * 2^n on either
    side, exactly onto it among them; all else is smaller."""
    rng = np.random.default_rng(tokens + hkv)
    half = D // 2
    first, second = O.pair_columns(D, interleaved)
    cs = np.zeros((tokens, D), np.float32)
    cs[:, :half] = 1.0
    k = torch.from_numpy(rng.uniform(-100, 100, (tokens, hkv, D))).bfloat16().double().numpy()
    n = 2.0 ** rng.integers(-20, 20, tokens) if first_row is None else np.full(tokens, 0.25)
    k *= n[:, None, None]
    at = rng.integers(0, half, tokens)
    for t in range(tokens):
        a, b = 448.0 * n[t], n[t] * float(torch.tensor(rng.uniform(0.1, 100.0)).bfloat16())
        if t % 3:
            a = n[t] * float(torch.tensor(rng.uniform(300.0, 600.0)).bfloat16())
        s = np.float32(rng.uniform(-0.9, 0.9)) * np.float32(2.0 ** -18 if t % 3 == 0 else 1.0)
        c = np.float32((448.0 * n[t] + b * float(s)) / a)
        c = np.nextafter(c, np.float32(4.0 if t % 2 else -4.0)) if t % 5 == 0 else c
        cs[t, at[t]], cs[t, half + at[t]] = c, s
        k[t, :, first[at[t]]], k[t, :, second[at[t]]] = a * (1 if t % 4 else -1), b * (1 if t % 4 else -1)
        if abs(b * float(c) + a * float(s)) > 440.0 * n[t]:   # the pair's other element must be the smaller one
            cs[t, half + at[t]] = s * np.float32(2.0 ** -10)
            cs[t, at[t]] = np.float32((448.0 * n[t] + b * float(cs[t, half + at[t]])) / a)
    pos = torch.arange(tokens, dtype=torch.int32)[None]
    _check(torch.from_numpy(k), torch.from_numpy(cs), pos, interleaved, _slots(tokens, first_row), tokens)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hkv", [(1, 1), (20, 2), (70, 72)])
@pytest.mark.parametrize("gain", [1.0, 4.0, -2.0 ** 20])
def test_rotations_beyond_fp32(tokens, hkv, gain, interleaved):
    """Finite keys whose rotation overflows fp32, alone in their run and beside
    others, and ones whose products overflow while their difference does not."""
    half = D // 2
    first, second = O.pair_columns(D, interleaved)
    cs = torch.zeros(3, D)
    cs[:, :half], cs[:, half:] = 0.75 * gain, 0.625 * gain
    cs[2, half:] = 0.75 * gain
    k = torch.zeros(tokens, hkv, D)
    k[:, :, first[3]], k[:, :, second[3]] = 3.3e38, -3.2e38
    k[1::3, :, first[5]] = 1.5
    k[2::3, :, first[3]] = k[2::3, :, second[3]] = 3.3e38         # a' = 0 at position 2
    k[2::3, :, second[7]] = 7.0
    pos = (torch.arange(tokens) % 3).to(torch.int32)[None]
    for slots in (_slots(tokens, None), _slots(tokens, 4)):
        _check(k, cs, pos, interleaved, slots, tokens)
