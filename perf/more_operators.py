"""Cases of the operators for drafted tokens and for eviction over the paged
cache.

  tree       paged_tree_attention: each sequence's drafted tokens attend to its
             cached context and to the drafted tokens that their mask names
  weights    kv_add_weights: what those rows' softmax gave each key, added to a
             running sum per sequence, KV head and token
  select     kv_select: which tokens stay, by that sum
  compact    kv_compact: the rows that stay move up in place

``own`` False: the plain forms, elementary torch operations in fp32.  ``own``
True: the library's calls.  Pools are [blocks, KV heads, 16, head_dim], read
through block_table [sequences, blocks]; sequence b's drafted tokens are rows
draft_offsets[b] .. draft_offsets[b + 1] - 1 of q and the last tokens stored.
"""
import math
import random

import torch

own = False

BS = 16   # tokens per cache block


# ------------------------------------------------------------------ the cases
def _tree(name, sequences, shortest, longest, least, draft, q_heads=32, kv_heads=8, op="tree", mask=True, fp32=False,
          dim=128):
    return {"name": name, "op": op, "sequences": sequences, "shortest": shortest, "longest": longest, "least": least,
            "draft": draft, "q_heads": q_heads, "kv_heads": kv_heads, "mask": mask, "fp32": fp32, "dim": dim}


def listed():
    return [
        # one short conversation, a small draft: latency
        _tree("tree, 8 drafted over 777", 1, 777, 777, 8, 8),
        # the even batch of the llama8b_decode workload, each sequence with a tree of 16
        _tree("tree, 64 sequences of 2301, 16 drafted", 64, 2301, 2301, 16, 16),
        # long documents with the largest trees
        _tree("tree, 8 sequences of 32001, 64 drafted", 8, 32001, 32001, 64, 64),
        # a ragged batch with trees of any size, eight query heads to a KV head
        _tree("tree, 32 ragged, group 8", 32, 128, 16384, 1, 64, 64, 8),
        # a chain of drafts in fp32
        _tree("tree, fp32, 4 chains of 5", 4, 500, 1500, 5, 5, 8, 4, mask=False, fp32=True),
        # a decode step that keeps count of the attention each token gets
        _tree("weights, 64 sequences of 2301, one token", 64, 2301, 2301, 1, 1, op="weights", mask=False),
        # the last tokens of long prompts observe what came before
        _tree("weights, 8 sequences of 32001, window of 32", 8, 32001, 32001, 32, 32, op="weights", mask=False),
        # the even batch, down to less than half
        {"name": "select, 64 sequences of 2301 to 1024", "op": "select", "sequences": 64, "shortest": 2301,
         "longest": 2301, "budget": 1024, "sinks": 4, "recent": 128, "kv_heads": 8},
        # long documents, down to an eighth
        {"name": "select, 8 sequences of 32001 to 4096", "op": "select", "sequences": 8, "shortest": 32001,
         "longest": 32001, "budget": 4096, "sinks": 4, "recent": 512, "kv_heads": 8},
        # the accepted paths of 64 verified trees: a few rows each
        {"name": "compact, 64 accepted paths", "op": "compact", "sequences": 64, "shortest": 2301, "longest": 2301,
         "budget": 6, "draft": 16, "kv_heads": 8, "dim": 128, "type": "bf16"},
        # what stays of long documents, another set in every head
        {"name": "compact, 8 sequences of 32001 to 4096", "op": "compact", "sequences": 8, "shortest": 32001,
         "longest": 32001, "budget": 4096, "draft": 0, "kv_heads": 8, "dim": 128, "type": "bf16"},
        # a ragged batch of E4M3 codes
        {"name": "compact, 48 ragged, codes", "op": "compact", "sequences": 48, "shortest": 128, "longest": 16384,
         "budget": 2048, "draft": 0, "kv_heads": 8, "dim": 128, "type": "fp8"},
    ]


def _log_int(rng, low, high):
    """An integer in [low, high], spread evenly over its logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "weights", "weights", "select", "compact", "compact"])
    longest = _log_int(rng, 1, 32768)
    shortest = longest if rng.random() < 0.3 else _log_int(rng, 1, longest)
    kv = rng.choice([1, 2, 4, 8])
    if op in ("tree", "weights"):
        fp32 = rng.random() < 0.2
        heads = kv * rng.choice([1, 2, 4, 8] if fp32 else [1, 2, 4, 4, 8, 16])
        dim = rng.choice([16, 128]) if fp32 else 128
        most = min(64, shortest)
        draft = _log_int(rng, 1, most)
        # within the largest listed batch: stored tokens times KV heads, and times rows
        room = min(2_000_000 // (longest * kv), 520_000_000 // (longest * heads * draft))
        if fp32:   # its rate is an eighth of the tensor cores' and less
            room = min(room, 30_000_000 // (longest * heads * draft))
            longest, shortest = (longest, shortest) if room else (min(longest, 1500), min(shortest, 1500))
        least = draft if rng.random() < 0.4 else rng.randint(0, draft)
        return {"op": op, "sequences": _log_int(rng, 1, min(128, max(1, room))), "shortest": shortest,
                "longest": longest, "least": least, "draft": draft, "q_heads": heads, "kv_heads": kv,
                "mask": rng.random() < 0.7, "fp32": fp32, "dim": dim}
    sequences = _log_int(rng, 1, min(128, max(1, 2_000_000 // (longest * kv))))
    c = {"op": op, "sequences": sequences, "shortest": shortest, "longest": longest, "kv_heads": kv}
    if op == "select":
        budget = _log_int(rng, 1, longest)
        sinks = rng.choice([0, min(4, budget)])
        return {**c, "budget": budget, "sinks": sinks, "recent": rng.randint(0, budget - sinks) // rng.choice([1, 4])}
    c.update(dim=rng.choice([64, 128, 128, 256]), type=rng.choice(["bf16", "bf16", "fp32", "fp8"]))
    if rng.random() < 0.5:
        draft = _log_int(rng, 1, min(64, shortest))
        return {**c, "budget": rng.randint(1, min(draft, 16)), "draft": draft}
    return {**c, "budget": _log_int(rng, 1, longest), "draft": 0}


def _lengths(case):
    """Sequence lengths: even steps of the logarithm from shortest to longest."""
    n, lo, hi = case["sequences"], case["shortest"], case["longest"]
    return [min(hi, max(lo, round(lo * (hi / lo) ** ((i + 0.5) / n)))) for i in range(n)]


def _drafted(case):
    """Drafted tokens of each sequence, from least to draft in turn."""
    span = case["draft"] - case["least"] + 1
    return [case["least"] + (7 * i + span - 1) % span for i in range(case["sequences"])]


# ------------------------------------------------------------------- inputs
def _rows(shape, gen, dev, outliers):
    """N(0, 1) with a few large channels, as keys have them."""
    x = torch.randn(shape, generator=gen, device=dev)
    if outliers:
        gain = torch.ones(shape[-1], device=dev)
        gain[:: max(1, shape[-1] // 4)] = 3.0
        x *= gain
    return x


def _pool(blocks, heads, dim, gen, dev, dtype, outliers):
    """A filled pool, built some blocks at a time."""
    pool = torch.empty((blocks, heads, BS, dim), dtype=dtype, device=dev)
    for at in range(0, blocks, 8192):
        n = min(8192, blocks - at)
        x = _rows((n, heads, BS, dim), gen, dev, outliers)
        pool[at:at + n] = x.to(torch.float8_e4m3fn).view(torch.uint8) if dtype is torch.uint8 else x.to(dtype)
    return pool


def _tree_mask(counts, pick):
    """Each drafted token sees itself and its ancestors: a random earlier token or the context is its parent."""
    bits = []
    for n in counts:
        seen = []
        for i in range(n):
            parent = pick.randint(max(-1, i - 6), i - 1)
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        bits += [x - (1 << 64) if x >> 63 else x for x in seen]
    return bits


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    pick = random.Random(seed)
    lens, hkv = _lengths(case), case["kv_heads"]
    order = list(range(len(lens)))
    pick.shuffle(order)
    lens = [lens[i] for i in order]
    batch, longest = len(lens), max(lens)
    s = {"case": case, "longest": longest, "lens": torch.tensor(lens, dtype=torch.int32, device=dev)}
    if case["op"] != "select":
        per_seq = [-(-n // BS) for n in lens]
        used = sum(per_seq)
        blocks = used + max(1, used // 32)
        host = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32).cpu()
        table = torch.zeros((batch, max(per_seq)), dtype=torch.int32)
        at = 0
        for i, n in enumerate(per_seq):
            table[i, :n] = host[at:at + n]
            at += n
        s["block_table"] = table.to(dev)
        name = case["type"] if case["op"] == "compact" else "fp32" if case["fp32"] else "bf16"
        dtype = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.uint8}[name]
        s["k_cache"] = _pool(blocks, hkv, case["dim"], gen, dev, dtype, True)
        if case["op"] != "weights":
            s["v_cache"] = _pool(blocks, hkv, case["dim"], gen, dev, dtype, False)
    # running sums: heavy-tailed, some tokens never looked at, room for tokens to come
    width = longest + 37
    if case["op"] != "tree":
        w = torch.exp(2 * torch.randn((batch, hkv, width), generator=gen, device=dev) - 4)
        w *= torch.rand((batch, hkv, width), generator=gen, device=dev) > 0.1
        w *= (torch.arange(width, device=dev) < s["lens"][:, None])[:, None]
        if case["op"] == "weights":   # as many such steps before gave: a row's weights sum to one
            w *= 4 * case["draft"] * case["q_heads"] / hkv / longest
        s["weights"] = w
    if case["op"] in ("tree", "weights"):
        counts = _drafted(case)
        rows, hq, d = sum(counts), case["q_heads"], case["dim"]
        offsets = [0]
        for n in counts:
            offsets.append(offsets[-1] + n)
        s["rows"], s["scale"] = rows, d ** -0.5
        s["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=dev)
        s["mask"] = torch.tensor(_tree_mask(counts, pick), dtype=torch.int64, device=dev) if case["mask"] else None
        s["q"] = torch.randn((rows, hq, d), generator=gen, device=dev).to(s["k_cache"].dtype)
        if case["op"] == "tree":
            s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((rows, hq), device=dev)
        else:
            s["lse"] = _lse(s)
    elif case["op"] == "select":
        s["kept"] = torch.zeros((batch, hkv, case["budget"]), dtype=torch.int32, device=dev)
        s["kept_lens"] = torch.zeros(batch, dtype=torch.int32, device=dev)
    elif case["draft"]:
        # an accepted path: ascending drafted tokens, the same in every head
        n = case["budget"]
        first = s["lens"] - case["draft"]
        path = torch.rand((batch, case["draft"]), generator=gen, device=dev).topk(n, 1).indices.sort(1).values
        s["first"] = first
        s["kept"] = (first[:, None] + path)[:, None].to(torch.int32).contiguous()
        s["kept_lens"] = torch.randint(0, n + 1, (batch,), generator=gen, device=dev).to(torch.int32)
    else:
        # another set in every head: four first tokens, an eighth last ones and any between
        n = case["budget"]
        place = torch.arange(longest, device=dev)
        rank = torch.rand((batch, hkv, longest), generator=gen, device=dev)
        rank += 2 * ((place < 4) | (place >= s["lens"][:, None] - n // 8))[:, None]
        rank = rank.masked_fill((place >= s["lens"][:, None])[:, None], -1)
        at = rank.topk(min(n, longest), 2).indices
        at = at.masked_fill(rank.gather(2, at) < 0, longest).sort(2).values
        s["first"], s["kept"] = None, at.to(torch.int32).contiguous()
        s["kept_lens"] = s["lens"].clamp(max=n)
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program keeps for the library's calls: the attention's workspace."""
    from paged_kv_cache_104_gb300 import binding
    s["binding"] = binding
    c = s["case"]
    if c["op"] == "tree":
        s["workspace"] = binding.tree_workspace(c["q_heads"], c["kv_heads"], c["dim"], c["draft"], s["longest"])


# ------------------------------------------------------------ the plain forms
def _stored(s, which):
    """The pools' rows in the order of each sequence, float32 [sequences, KV heads, tokens, dim]."""
    x = s[which][s["block_table"].long()].transpose(1, 2).flatten(2, 3)
    return x[:, :, :s["longest"]].float()


def _padded(s):
    """Rows of q (and whether they are there) of each sequence: [sequences, drafted]."""
    off = s["offsets"].long()
    i = torch.arange(s["case"]["draft"], device=off.device)
    there = i < (off[1:] - off[:-1])[:, None]
    return (off[:-1, None] + i).clamp(max=max(s["rows"] - 1, 0)), there


def _scores(s):
    """Scaled products [sequences, KV heads, drafted, group, tokens], -inf where not visible; and what is visible."""
    case = s["case"]
    rows, there = _padded(s)
    hkv, g = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    q = s["q"].float()[rows].unflatten(2, (hkv, g)).permute(0, 2, 1, 3, 4)      # [b, hkv, t, g, d]
    score = (q.flatten(2, 3) @ _stored(s, "k_cache").transpose(2, 3)).unflatten(2, q.shape[2:4]) * s["scale"]
    n = (s["offsets"][1:] - s["offsets"][:-1]).long()
    place = torch.arange(s["longest"], device=q.device) - (s["lens"].long() - n)[:, None]   # [b, tokens]: which draft
    i = torch.arange(case["draft"], device=q.device)
    if s["mask"] is None:
        seen = place[:, None] <= i[:, None]
    else:
        bit = (s["mask"][rows][:, :, None] >> place.clamp(0, 63)[:, None]) & 1
        seen = (place < 0)[:, None] | (bit == 1)
    seen = seen & (place < n[:, None])[:, None] & there[:, :, None]             # [b, t, tokens]
    return score.masked_fill_(~seen[:, None, :, None], -math.inf), rows, there


def _back(x, rows, there, s):
    """[sequences, KV heads, drafted, group, ...] to rows of q."""
    x = x.transpose(1, 2)[there].flatten(1, 2)
    return torch.zeros((s["rows"],) + x.shape[1:], device=x.device).index_copy_(0, rows[there], x)


def _lse(s):
    score, rows, there = _scores(s)
    top = score.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0)
    return _back(torch.log(torch.exp(score.sub_(top)).sum(-1)) + top[..., 0], rows, there, s)


def _plain(s):
    case = s["case"]
    if case["op"] == "tree":
        score, rows, there = _scores(s)
        top = score.amax(-1, keepdim=True)
        top = top.masked_fill(top == -math.inf, 0)
        p = score.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        place = torch.arange(s["longest"], device=p.device)
        v = _stored(s, "v_cache").masked_fill_((place >= s["lens"][:, None])[:, None, :, None], 0)
        out = (p.flatten(2, 3) @ v).unflatten(2, p.shape[2:4]) / total.clamp(min=1e-38)
        s["out"].copy_(_back(out, rows, there, s))
        s["lse"].copy_(_back(torch.log(total[..., 0]) + top[..., 0], rows, there, s))
    elif case["op"] == "weights":
        score, rows, there = _scores(s)
        lse = s["lse"][rows].unflatten(2, (case["kv_heads"], -1)).transpose(1, 2)
        p = torch.exp(score.sub_(lse.masked_fill(lse == -math.inf, 0)[..., None]))
        s["weights"][:, :, :s["longest"]] += p.sum((2, 3))
    elif case["op"] == "select":
        place = torch.arange(s["longest"], device=s["lens"].device)
        n, want = s["lens"].long()[:, None], case["budget"]
        w = s["weights"][:, :, :s["longest"]]
        always = ((place < case["sinks"]) | (place >= n - case["recent"]))[:, None]
        w = torch.where(always, math.inf, w).masked_fill((place >= n)[:, None], -math.inf)
        order = torch.sort(w, dim=2, descending=True, stable=True).indices[:, :, :want]
        order = order.masked_fill(order >= n[:, :, None], s["longest"]).sort(2).values
        order = order.masked_fill(order == s["longest"], 0)
        s["kept"][:, :, :order.shape[2]] = order.to(torch.int32)
        s["kept_lens"].copy_(s["lens"].clamp(max=want))
    else:
        kept, n = s["kept"].long(), s["kept_lens"].long()
        batch, hkv = n.shape[0], case["kv_heads"]
        i = torch.arange(kept.shape[2], device=n.device)
        first = s["lens"].long() * 0 if s["first"] is None else s["first"].long()
        b, h, i = (i < n[:, None])[:, None].expand(batch, hkv, -1).nonzero(as_tuple=True)
        src, dst = kept.expand(batch, hkv, -1)[b, h, i], first[b] + i
        from_block, to_block = s["block_table"][b, src // BS].long(), s["block_table"][b, dst // BS].long()
        for pool in (s["k_cache"], s["v_cache"]):
            pool[to_block, h, dst % BS] = pool[from_block, h, src % BS]
        moved = s["weights"][b, h, src]
        place = torch.arange(s["weights"].shape[2], device=n.device)
        behind = (place >= (first + n)[:, None]) & (place < s["lens"][:, None])
        s["weights"][b, h, dst] = moved
        s["weights"].masked_fill_(behind[:, None], 0)


# ------------------------------------------------------------------- the pass
def _own(s):
    case, b = s["case"], s["binding"]
    if case["op"] == "tree":
        b.paged_tree_attention(s["out"], s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["lens"], s["offsets"],
                               s["mask"], s["longest"], case["draft"], s["scale"], s["workspace"], s["lse"])
    elif case["op"] == "weights":
        b.kv_add_weights(s["weights"], s["q"], s["k_cache"], s["block_table"], s["lens"], s["offsets"], s["mask"],
                         s["lse"], s["longest"], case["draft"], s["scale"])
    elif case["op"] == "select":
        b.kv_select(s["kept"], s["kept_lens"], s["weights"], s["lens"], s["longest"], case["sinks"], case["recent"])
    else:
        b.kv_compact(s["k_cache"], s["v_cache"], s["block_table"], s["lens"], s["kept"], s["kept_lens"], s["first"],
                     s["weights"])


def run(s):
    if own:
        _own(s)
    else:
        _plain(s)
    op = s["case"]["op"]
    if op == "tree":
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weights":
        return {"weights": s["weights"]}
    if op == "select":
        return {"kept": s["kept"], "kept_lens": s["kept_lens"]}
    k, v = s["k_cache"], s["v_cache"]
    if s["case"]["type"] == "fp8":
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    return {"k": k, "v": v, "weights": s["weights"]}


def work(case):
    lens, hkv = _lengths(case), case["kv_heads"]
    if case["op"] in ("tree", "weights"):
        counts, d, hq = _drafted(case), case["dim"], case["q_heads"]
        size = 4 if case["fp32"] else 2
        # a sequence without drafted tokens needs nothing; the mask's holes among the drafted are not counted out
        lens = [n if m else 0 for n, m in zip(lens, counts)]
        cells = sum(n * m - m * (m - 1) // 2 for n, m in zip(lens, counts)) * hq
        rows = sum(counts)
        table = sum(4 * -(-n // BS) for n in lens)
        if case["op"] == "tree":
            moved = 2 * size * d * hkv * sum(lens) + rows * hq * (2 * size * d + 4)
            return {"bytes": moved + table + 8 * rows * case["mask"], "flops": 4 * d * cells}
        moved = (size * d + 8) * hkv * sum(lens) + rows * hq * (size * d + 4)
        return {"bytes": moved + table + 8 * rows * case["mask"], "flops": 2 * d * cells}
    if case["op"] == "select":
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": 4 * hkv * (sum(lens) + kept) + 8 * len(lens), "flops": hkv * sum(lens)}
    row = case["dim"] * {"bf16": 2, "fp32": 4, "fp8": 1}[case["type"]]
    if case["draft"]:   # half the most on average; the drafted tokens' sums are written
        moved = len(lens) * case["budget"] / 2
        return {"bytes": hkv * (moved * (4 * row + 4) + 4 * case["draft"] * len(lens)) + 4 * moved + 12 * len(lens),
                "flops": 1}
    # what stays moves up (all but the rows ahead of the first gap); the sums are written up to the old length
    moved = sum(min(n, case["budget"]) for n in lens if n > case["budget"])
    return {"bytes": hkv * (moved * (4 * row + 8) + 4 * sum(lens)) + 8 * len(lens), "flops": 1}


# ----------------------------------------------------------- exact, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    lens = s["lens"].tolist()
    hkv = case["kv_heads"]

    def rows_of(which, b, h):
        ids = s["block_table"][b, :-(-lens[b] // BS)].long()
        return s[which][ids, h].flatten(0, 1)[:lens[b]]

    if case["op"] in ("tree", "weights"):
        off, g = s["offsets"].tolist(), case["q_heads"] // hkv
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
        weights = s["weights"].double() if case["op"] == "weights" else None
        for b, n in enumerate(lens):
            m = off[b + 1] - off[b]
            if not m:
                continue
            seen = torch.ones((m, n), dtype=torch.bool)
            seen[:, n - m:] = torch.ones(m, m).tril().bool()
            if s["mask"] is not None:
                word = s["mask"][off[b]:off[b + 1]].tolist()
                seen[:, n - m:] = torch.tensor([[(x >> j) & 1 == 1 for j in range(m)] for x in word])
            seen = seen.cuda()
            for h in range(hkv):
                q = s["q"][off[b]:off[b + 1], h * g:(h + 1) * g].double()
                score = torch.einsum("tgd,nd->tgn", q, rows_of("k_cache", b, h).double()) * s["scale"]
                score = torch.where(seen[:, None], score, -math.inf)
                if weights is None:
                    lse[off[b]:off[b + 1], h * g:(h + 1) * g] = torch.logsumexp(score, -1)
                    out[off[b]:off[b + 1], h * g:(h + 1) * g] = (
                        torch.softmax(score, -1).nan_to_num() @ rows_of("v_cache", b, h).double())
                else:
                    given = s["lse"][off[b]:off[b + 1], h * g:(h + 1) * g].double()
                    weights[b, h, :n] += torch.exp(score - given[..., None]).nan_to_num().sum((0, 1))
        return {"out": out, "lse": lse} if weights is None else {"weights": weights}
    if case["op"] == "select":
        return None   # whole numbers only
    weights = s["weights"].double()
    values = {"k": "k_cache", "v": "v_cache"}
    pools = {}
    for name, which in values.items():
        pool = s[which].view(torch.float8_e4m3fn) if case["type"] == "fp8" else s[which]
        pools[name] = pool.double()
    for b, n in enumerate(lens):
        m = int(s["kept_lens"][b])
        start = 0 if s["first"] is None else int(s["first"][b])
        table = s["block_table"][b].long()
        for h in range(hkv):
            src = s["kept"][b, min(h, s["kept"].shape[1] - 1), :m].long()
            dst = torch.arange(start, start + m, device="cuda")
            for name in values:
                pool = pools[name]
                pool[table[dst // BS], h, dst % BS] = pool[table[src // BS], h, src % BS].clone()
            line = weights[b, h].clone()
            weights[b, h, start:n] = 0
            weights[b, h, start:start + m] = line[src]
    return {**pools, "weights": weights}
