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


def _per_head(q, k_cache, table, seq_lens, offsets, mask, scale):
    """For every sequence with drafted tokens and KV head: (b, h, rows of q,
    query heads, scores [m, G, n], seen [m, 1, n])."""
    hkv = k_cache.shape[1]
    g = q.shape[1] // hkv
    for b in range(len(seq_lens)):
        lo, hi, n = int(offsets[b]), int(offsets[b + 1]), int(seq_lens[b])
        if hi == lo:
            continue
        words = None if mask is None else mask[lo:hi]
        seen = torch.tensor(np.stack([sees(words, hi - lo, n, i) for i in range(hi - lo)]))[:, None]
        for h in range(hkv):
            heads = slice(h * g, (h + 1) * g)
            s = q[lo:hi, heads].double() @ rows_of(k_cache, table, b, h, n).T * scale
            yield b, h, slice(lo, hi), heads, s, seen


def tree_attention(q, k_cache, v_cache, table, seq_lens, offsets, mask, scale):
    """out [N, Hq, D] and lse [N, Hq] in fp64; rows of no sequence are NaN.
    The value of a key that a row does not see is not touched: 0 x inf never
    arises."""
    out = torch.full(q.shape, float("nan"), dtype=torch.float64)
    lse = torch.full(q.shape[:2], float("nan"), dtype=torch.float64)
    for b, h, rows, heads, s, seen in _per_head(q, k_cache, table, seq_lens, offsets, mask, scale):
        s = torch.where(seen, s, -float("inf"))
        top = s.amax(2, keepdim=True)
        p = torch.exp(s - torch.where(torch.isinf(top) & (top < 0), 0.0, top))
        total = p.sum(2, keepdim=True)
        v = rows_of(v_cache, table, b, h, s.shape[2])
        odd = ~torch.isfinite(v).all(1)                       # values that need the care
        acc = p[:, :, ~odd] @ v[~odd]
        for n in odd.nonzero()[:, 0].tolist():
            acc = acc + torch.where(seen[:, :, n:n + 1], p[:, :, n:n + 1] * v[n], 0.0)
        out[rows, heads] = torch.where(total == 0, 0.0, acc / total)
        lse[rows, heads] = torch.where(total == 0, -float("inf"), top + torch.log(total))[..., 0]
    return out, lse


def add_weights(weights, q, k_cache, table, seq_lens, offsets, mask, lse, scale):
    """weights (fp64, a copy) with the softmax weights of the rows added."""
    w = weights.double().clone()
    for b, h, rows, heads, s, seen in _per_head(q, k_cache, table, seq_lens, offsets, mask, scale):
        given = lse[rows, heads].double()[..., None]
        p = torch.where(seen & (given != -float("inf")), torch.exp(s - given), 0.0)
        w[b, h, :s.shape[2]] += p.sum((0, 1))
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
