"""fp64 oracle of the operators for drafted tokens and eviction: attention of
drafted tokens over a paged cache, the sums of its weights, the selection of
the tokens that stay and their move.  Plain loops over sequences and heads; no
code shared with the CUDA side."""
from __future__ import annotations

import numpy as np
import torch


def rows_of(pool, table, b: int, h: int, n: int, bs: int = 16):
    """The n rows that sequence b stores in head h, fp64 [n, D]."""
    ids = [int(x) for x in table[b, :-(-n // bs)]]
    if not n:
        return torch.zeros(0, pool.shape[3], dtype=torch.float64)
    return torch.cat([pool[i, h].double() for i in ids])[:n]


def sees(mask_words, drafted: int, n: int, i: int):
    """Which of a sequence's n tokens drafted token i sees (numpy bool [n])."""
    s = np.ones(n, dtype=bool)
    for j in range(drafted):
        s[n - drafted + j] = (j <= i) if mask_words is None else bool((int(mask_words[i]) >> j) & 1)
    return s


def _per_row(q, k_cache, table, seq_lens, offsets, mask, scale):
    """For every sequence, KV head and row: (b, g, query heads, row of q, scores [G, n], seen [n])."""
    hkv = k_cache.shape[1]
    g = q.shape[1] // hkv
    for b in range(len(seq_lens)):
        lo, hi, n = int(offsets[b]), int(offsets[b + 1]), int(seq_lens[b])
        if hi == lo:
            continue
        words = None if mask is None else mask[lo:hi]
        for h in range(hkv):
            k = rows_of(k_cache, table, b, h, n)
            heads = slice(h * g, (h + 1) * g)
            for i in range(hi - lo):
                yield b, h, heads, lo + i, q[lo + i, heads].double() @ k.T * scale, sees(words, hi - lo, n, i)


def tree_attention(q, k_cache, v_cache, table, seq_lens, offsets, mask, scale):
    """out [N, Hq, D] and lse [N, Hq] in fp64; rows of no sequence are NaN."""
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float64)
    values = {}
    for b, h, heads, row, s, seen in _per_row(q, k_cache, table, seq_lens, offsets, mask, scale):
        if (b, h) not in values:
            values = {(b, h): rows_of(v_cache, table, b, h, int(seq_lens[b]))}
        at = np.flatnonzero(seen)
        if not len(at):
            out[row, heads], lse[row, heads] = 0, -float("inf")
            continue
        s = s[:, at]
        top = s.amax(1, keepdim=True)
        p = torch.exp(s - top)
        total = p.sum(1, keepdim=True)
        out[row, heads] = (p / total) @ values[b, h][at]
        lse[row, heads] = (top + torch.log(total))[:, 0]
    return out, lse


def add_weights(weights, q, k_cache, table, seq_lens, offsets, mask, lse, scale):
    """weights (fp64, a copy) with the softmax weights of the rows added."""
    w = weights.double().clone()
    for b, h, heads, row, s, seen in _per_row(q, k_cache, table, seq_lens, offsets, mask, scale):
        at = np.flatnonzero(seen)
        for j in range(s.shape[0]):
            given = float(lse[row, heads][j])
            if given != -float("inf"):
                w[b, h, at] += torch.exp(s[j, at] - given)
    return w


def select(weights, seq_lens, budget: int, sinks: int, recent: int):
    """Positions that stay: a list per sequence of a list per KV head."""
    kept = []
    for b, n in enumerate(int(x) for x in seq_lens):
        heads = []
        for h in range(weights.shape[1]):
            w = [float(x) for x in weights[b, h, :n]]
            if n <= budget:
                heads.append(list(range(n)))
                continue
            always = list(range(sinks)) + list(range(n - recent, n))
            rest = sorted(range(sinks, n - recent),
                          key=lambda t: (1, 0.0, t) if w[t] != w[t] else (0, -w[t], t))
            heads.append(sorted(always + rest[:budget - sinks - recent]))
        kept.append(heads)
    return kept


def compact(k_cache, v_cache, weights, table, seq_lens, kept, kept_lens, first, bs: int = 16):
    """Copies of the pools and weights with the kept rows moved up."""
    k, v = k_cache.clone(), v_cache.clone()
    w = None if weights is None else weights.clone()
    for b in range(len(seq_lens)):
        n, m = int(seq_lens[b]), int(kept_lens[b])
        at = 0 if first is None else int(first[b])
        for h in range(k.shape[1]):
            rows = kept[b, h if kept.shape[1] > 1 else 0, :m].tolist()
            for i, r in enumerate(rows):
                src, dst = int(table[b, r // bs]), int(table[b, (at + i) // bs])
                k[dst, h, (at + i) % bs] = k_cache[src, h, r % bs]
                v[dst, h, (at + i) % bs] = v_cache[src, h, r % bs]
            if w is not None:
                w[b, h, at:n] = 0
                for i, r in enumerate(rows):
                    w[b, h, at + i] = weights[b, h, r]
    return k, v, w
