"""Block-scaled FP8 storage for the KV-cache oracle.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

One power-of-two scale 2^(byte - 127) per block of 16 tokens and KV head; an
element is E4M3(x / scale).  New rows of a block arrive as a run of
consecutive slots.  A run at row 0 starts the block anew; a later one keeps
the rows before it, and where the scale grows, by 2^d, their codes become
E4M3(decode(code) / 2^d).  The exponent is the smallest e in [-126, 119] with
every finite |x| of the run at most 448 * 2^e, and at least the kept rows' e.
fp64 numpy; the E4M3 rounding is that of ``oracle.fp8``.
"""
from __future__ import annotations

import numpy as np

from . import fp8

E_MIN, E_MAX, BIAS = -126, 119, 127
BLOCK = 16


def exponent(amax: float) -> int:
    """Smallest e in [E_MIN, E_MAX] with amax <= 448 * 2^e (or E_MAX)."""
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def encode(y) -> np.ndarray:
    """E4M3 codes of y (already divided by the scale); NaN stays NaN and
    infinities saturate."""
    y = np.asarray(y, dtype=np.float64)
    codes = fp8.encode(np.where(np.isnan(y), 0.0, y))
    return np.where(np.isnan(y), np.uint8(0x7F), codes).astype(np.uint8)


def runs(slots):
    """[(first entry, length)] of the runs of consecutive slots in one block."""
    out, prev = [], None
    for t, s in enumerate(slots):
        s = int(s)
        if s >= 0:
            if prev == s - 1 and s % BLOCK:
                out[-1][1] += 1
            else:
                out.append([t, 1])
        prev = s
    return out


def append_pool(new, pool, scale, slots) -> None:
    """new fp64 [T, H, D] into pool uint8 [NB, H, 16, D], scale uint8 [NB, H]
    (both in place)."""
    new = np.asarray(new, dtype=np.float64)
    for t, n in runs(slots):
        blk, row = int(slots[t]) // BLOCK, int(slots[t]) % BLOCK
        for h in range(pool.shape[1]):
            x = new[t:t + n, h]
            a = np.abs(x[np.isfinite(x)])
            e = exponent(float(a.max()) if a.size else 0.0)
            if row > 0:
                byte = int(scale[blk, h])
                if 1 <= byte <= 253:
                    old = byte - BIAS
                    if e > old:
                        pool[blk, h, :row] = encode(fp8.decode(pool[blk, h, :row]) * 2.0 ** (old - e))
                    e = max(e, old)
                else:
                    pool[blk, h, :row] = 0
            pool[blk, h, row:row + n] = encode(x * 2.0 ** -e)
            scale[blk, h] = e + BIAS


def dequantize(pool, scale) -> np.ndarray:
    """fp64 values of a pool [NB, H, 16, D] with scale bytes [NB, H]."""
    return fp8.decode(pool) * np.exp2(scale.astype(np.float64) - BIAS)[:, :, None, None]
