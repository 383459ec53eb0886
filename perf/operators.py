"""Cases of the operators that rotate positions on the way into the paged
cache, and of the block-scaled 8-bit cache with the attention that reads it.

  rope          kv_append_rope: q and k rotated by their positions, k and v
                scattered into the bf16 or fp32 pools
  append8       kv_append_fp8_block: the same into E4M3 pools with one
                power-of-two scale per block of 16 tokens and KV head
  decode8       paged_decode_attention_fp8_block: one query per sequence
  prefill8      chunked_prefill_attention_fp8_block: a prompt chunk

``own`` False: the plain forms, elementary torch operations in fp32 (fp64
where values are rounded to E4M3).  ``own`` True: the library's calls.
Pools are [blocks, KV heads, 16, head_dim], block scales [blocks, KV heads]
bytes e that stand for 2^(e - 127).
"""
import math
import random

import numpy as np
import torch

own = False

BS = 16                  # tokens per cache block
MAX_CODE = 448.0         # largest E4M3 value
E_MIN, E_MAX = -126, 119  # block scale exponents


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one sequence's new token: the launch-bound end of a decode step
        {"name": "rope, one token", "op": "rope", "tokens": 1, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "axes": 1, "cycle": False, "fp32": False, "positions": 32768},
        # a decode step of 128 sequences
        {"name": "rope, 128 sequences", "op": "rope", "tokens": 128, "q_heads": 32, "kv_heads": 8, "dim": 128,
         "rot": 128, "interleaved": False, "axes": 1, "cycle": False, "fp32": False, "positions": 131072},
        # four prompt chunks of 2,048 tokens with image patches: time, height and width
        {"name": "rope, 8192 tokens, three axes", "op": "rope", "tokens": 8192, "q_heads": 32, "kv_heads": 8,
         "dim": 128, "rot": 128, "interleaved": False, "axes": 3, "cycle": False, "fp32": False,
         "positions": 32768},
        # an odd chunk into fp32 pools, half of each head rotated, adjacent pairs
        {"name": "rope, 777 tokens, fp32, partial", "op": "rope", "tokens": 777, "q_heads": 16, "kv_heads": 2,
         "dim": 128, "rot": 64, "interleaved": True, "axes": 1, "cycle": False, "fp32": True,
         "positions": 8192},
        # the new tokens of 128 running sequences: each continues a block
        {"name": "append8, 128 sequences", "op": "append8", "sequences": 128, "tokens": 1, "first_row": -1,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "axes": 1,
         "cycle": False, "positions": 131072},
        # a prompt chunk of 2,048 tokens that starts in the middle of a block
        {"name": "append8, chunk of 2048", "op": "append8", "sequences": 1, "tokens": 2048, "first_row": 5,
         "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "interleaved": False, "axes": 1,
         "cycle": False, "positions": 32768},
        # one short conversation: latency
        {"name": "decode8, one sequence of 777", "op": "decode8", "sequences": 1, "shortest": 777,
         "longest": 777, "q_heads": 32, "kv_heads": 8},
        # the even batch of the llama8b_decode workload, after its append
        {"name": "decode8, 64 sequences of 2301", "op": "decode8", "sequences": 64, "shortest": 2301,
         "longest": 2301, "q_heads": 32, "kv_heads": 8},
        # long documents, eight query heads to a KV head
        {"name": "decode8, 8 sequences of 32001, group 8", "op": "decode8", "sequences": 8, "shortest": 32001,
         "longest": 32001, "q_heads": 64, "kv_heads": 8},
        # the ragged batch of the default workload: lengths from 128 to 32,768
        {"name": "decode8, 128 ragged sequences", "op": "decode8", "sequences": 128, "shortest": 128,
         "longest": 32768, "q_heads": 32, "kv_heads": 8},
        # the last piece of a short prompt, two KV heads
        {"name": "prefill8, 77 over 500", "op": "prefill8", "chunk": 77, "prior": 500, "q_heads": 8,
         "kv_heads": 2},
        # the default workload's prompt chunk: 2,048 tokens over 4,096 cached ones
        {"name": "prefill8, 2048 over 4096", "op": "prefill8", "chunk": 2048, "prior": 4096, "q_heads": 32,
         "kv_heads": 8},
    ]


def _log_int(rng, low, high):
    """An integer in [low, high], spread evenly over its logarithm."""
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return {"q_heads": kv * rng.choice([1, 2, 4, 8]), "kv_heads": kv}


def _rotation(rng, dim):
    axes = rng.choice([1, 1, 2, 3])
    return {"dim": dim, "rot": rng.choice([dim, dim, dim // 2]), "interleaved": rng.random() < 0.4, "axes": axes,
            "cycle": axes > 1 and rng.random() < 0.4, "positions": rng.choice([4096, 32768, 131072])}


def draw(rng):
    op = rng.choice(["rope", "append8", "decode8", "decode8", "prefill8"])
    if op == "rope":
        c = {"op": op, "tokens": _log_int(rng, 1, 4096), **_heads(rng)}
        return {**c, **_rotation(rng, rng.choice([64, 80, 128, 128, 256])), "fp32": rng.random() < 0.3}
    if op == "append8":
        if rng.random() < 0.5:
            c = {"op": op, "sequences": _log_int(rng, 1, 512), "tokens": 1, "first_row": -1}
        else:
            c = {"op": op, "sequences": rng.choice([1, 1, 2, 5]), "tokens": _log_int(rng, 2, 2048 // 5),
                 "first_row": rng.randrange(BS)}
        return {**c, **_heads(rng), **_rotation(rng, rng.choice([64, 128, 128]))}
    if op == "decode8":
        longest = _log_int(rng, 1, 32768)
        shortest = longest if rng.random() < 0.3 else _log_int(rng, 1, longest)
        heads = _heads(rng)
        # within the largest listed batch: cached tokens times query heads
        most = max(1, 24_000_000 // (longest * heads["q_heads"]))
        return {"op": op, "sequences": _log_int(rng, 1, min(192, most)), "shortest": shortest, "longest": longest,
                **heads}
    return {"op": op, "chunk": _log_int(rng, 1, 2048), "prior": rng.choice([0, 1]) * _log_int(rng, 1, 4096),
            **_heads(rng)}


def _lengths(case):
    """Sequence lengths: even steps of the logarithm from shortest to longest."""
    n, lo, hi = case["sequences"], case["shortest"], case["longest"]
    return [min(hi, max(lo, round(lo * (hi / lo) ** ((i + 0.5) / n)))) for i in range(n)]


def _pair_axis(case):
    """The position axis of each rotated pair: sections of the pairs, or the axes in turn."""
    pairs, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return [0] * pairs
    if case["cycle"]:
        return [i % axes for i in range(pairs)]
    first = pairs // (axes + 1)
    rest = [first + (pairs - first) * k // (axes - 1) for k in range(axes)]
    return [0 if i < first else 1 + sum(i >= r for r in rest[1:]) for i in range(pairs)]


# ------------------------------------------------------------------- inputs
def _table(case, dev):
    """cos and sin of position times frequency, float32 [positions, rot]."""
    half = case["rot"] // 2
    freq = 500000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    angle = torch.arange(case["positions"], dtype=torch.float64, device=dev)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _positions(case, tokens, gen, dev):
    """One sequence's positions follow each other; a batch's are anywhere. Further axes are a patch's row and column."""
    top = case["positions"]
    if case.get("sequences", 2) > 1 or tokens == 1:
        p = torch.randint(0, top, (tokens,), generator=gen, device=dev)
    else:
        p = torch.arange(tokens, device=dev) + int(torch.randint(0, top - tokens + 1, (1,), generator=gen, device=dev))
    rest = [torch.randint(0, min(top, 256), (tokens,), generator=gen, device=dev) for _ in range(case["axes"] - 1)]
    return torch.stack([p, *rest]).to(torch.int32).contiguous()


def _kv(shape, gen, dev, outliers):
    """N(0, 1) with a few large channels, as keys have them."""
    x = torch.randn(shape, generator=gen, device=dev)
    if outliers:
        gain = torch.ones(shape[-1], device=dev)
        gain[:: max(1, shape[-1] // 4)] = 6.0
        x *= gain
    return x.to(torch.bfloat16)


def _times2(x, e):
    """x times 2^e exactly, e whole numbers in [-300, 300] (torch.ldexp takes its power from an inexact pow)."""
    p = ((e.long() + 1023) << 52).view(torch.float64)
    return (x.double() * p).to(x.dtype)


def _codes(x):
    """E4M3 codes and scale bytes of blocks x [n, heads, 16, dim]."""
    amax = x.float().abs().amax((2, 3))
    m, e = torch.frexp(amax)                     # amax = m 2^e, m in [0.5, 1)
    e = (e - 9 + (m > 0.875)).clamp(E_MIN, E_MAX)
    q = _times2(x.float(), -e[:, :, None, None]).clamp(-MAX_CODE, MAX_CODE)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _pool8(blocks, heads, gen, dev, outliers, dim=128):
    """A filled block-scaled pool, built some blocks at a time; a block's size differs from its neighbours'."""
    codes = torch.empty((blocks, heads, BS, dim), dtype=torch.uint8, device=dev)
    scale = torch.empty((blocks, heads), dtype=torch.uint8, device=dev)
    for at in range(0, blocks, 8192):
        n = min(8192, blocks - at)
        x = _kv((n, heads, BS, dim), gen, dev, outliers)
        x = x * torch.exp2(torch.randn((n, heads, 1, 1), generator=gen, device=dev) * 0.5).to(torch.bfloat16)
        codes[at:at + n], scale[at:at + n] = _codes(x)
    return codes, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    pick = random.Random(seed)
    hq, hkv = case["q_heads"], case["kv_heads"]
    s = {"case": case, "scale": 128 ** -0.5}
    if case["op"] in ("rope", "append8"):
        per = case["tokens"]
        n = per * case.get("sequences", 1)
        d = case["dim"]
        s["q"] = torch.randn((n, hq, d), generator=gen, device=dev)
        s["k"] = _kv((n, hkv, d), gen, dev, True)
        s["v"] = _kv((n, hkv, d), gen, dev, False)
        dtype = torch.float32 if case.get("fp32") else torch.bfloat16
        s["q"], s["k"], s["v"] = (s[x].to(dtype) for x in "qkv")
        s["q_out"] = torch.zeros_like(s["q"])
        s["table"], s["positions"] = _table(case, dev), _positions(case, n, gen, dev)
        s["pair_axis"] = _pair_axis(case)
        s["axis"] = torch.tensor(s["pair_axis"], device=dev)
        # where the tokens go: consecutive rows of a sequence's blocks, the blocks anywhere in the pool
        if case["op"] == "rope" or case["first_row"] >= 0:
            first = case.get("first_row", 0)
            rows = [[first + i for i in range(per)] for _ in range(case.get("sequences", 1))]
        else:
            rows = [[pick.randrange(BS)] for _ in range(case["sequences"])]
        need = sum((r[-1] // BS) + 1 for r in rows)
        blocks = need + max(1, need // 16)
        ids = list(range(blocks))
        pick.shuffle(ids)
        slots, at = [], 0
        for r in rows:
            slots += [ids[at + i // BS] * BS + i % BS for i in r]
            at += r[-1] // BS + 1
        s["slots"] = torch.tensor(slots, dtype=torch.int64, device=dev)
        if case["op"] == "rope":
            s["k_cache"], s["v_cache"] = (torch.zeros((blocks, hkv, BS, d), dtype=dtype, device=dev) for _ in "kv")
        else:
            s["k_cache"], s["k_scale"] = _pool8(blocks, hkv, gen, dev, True, d)
            s["v_cache"], s["v_scale"] = _pool8(blocks, hkv, gen, dev, False, d)
    else:
        lens = _lengths(case) if case["op"] == "decode8" else [case["prior"] + case["chunk"]]
        if case["op"] == "decode8":
            pick.shuffle(lens)
        per_seq = [-(-n // BS) for n in lens]
        used = sum(per_seq)
        blocks = used + max(1, used // 32)
        ids = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
        table = torch.zeros((len(lens), max(per_seq)), dtype=torch.int32)
        at = 0
        host = ids.cpu()
        for i, n in enumerate(per_seq):
            table[i, :n] = host[at:at + n]
            at += n
        s["block_table"] = table.to(dev)
        s["k_cache"], s["k_scale"] = _pool8(blocks, hkv, gen, dev, True)
        s["v_cache"], s["v_scale"] = _pool8(blocks, hkv, gen, dev, False)
        s["lens"], s["total"], s["longest"] = torch.tensor(lens, dtype=torch.int32, device=dev), sum(lens), max(lens)
        rows = len(lens) if case["op"] == "decode8" else case["chunk"]
        s["q"] = torch.randn((rows, hq, 128), generator=gen, device=dev).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        if case["op"] == "prefill8":
            s["row"] = s["block_table"][0].contiguous()
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program keeps for the library's calls: the rotation's description, the decode's workspace."""
    from paged_kv_cache_104_gb300 import binding
    s["binding"] = binding
    case = s["case"]
    if "table" in s:
        s["rope"] = binding.Rope(s["table"], interleaved=case["interleaved"], pair_axis=s["pair_axis"])
    elif case["op"] == "decode8":
        s["workspace"] = binding.decode_workspace(case["sequences"], case["q_heads"], 128, s["longest"])


# ------------------------------------------------------------ the plain forms
def _rotate(x, s, dtype):
    """x [n, heads, dim] rotated by its positions, in dtype."""
    case, half = s["case"], s["case"]["rot"] // 2
    x = x.to(dtype)
    at = s["positions"].long()[s["axis"]].T                         # [n, pairs]
    pair = torch.arange(half, device=x.device)
    cos = s["table"][at, pair].to(dtype)[:, None]
    sin = s["table"][at, pair + half].to(dtype)[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * half:]], -1)


def _e4m3(y):
    """y (fp64) to the nearest E4M3 value, ties to the even code."""
    y = y.clamp(-MAX_CODE, MAX_CODE)
    e = torch.frexp(y)[1].clamp(min=-5) - 4                         # 2^e: the step at y
    return _times2(torch.round(_times2(y, -e)), e)


def _append8(new, codes, scale, slots):
    """New rows (fp64 [n, heads, dim]) into a block-scaled pool."""
    blk, row = slots // BS, slots % BS
    first = torch.full((codes.shape[0],), BS, device=slots.device).scatter_reduce(0, blk, row, "amin")
    touched, fresh = first < BS, first == 0
    amax = new.abs().amax(-1)                                       # [n, heads]
    top = torch.zeros(scale.shape, dtype=amax.dtype, device=amax.device)
    top = top.scatter_reduce(0, blk[:, None].expand_as(amax), amax, "amax")
    m, e = torch.frexp(top)
    e = (e - 9 + (m > 0.875)).clamp(E_MIN, E_MAX)
    old = scale.to(torch.int32) - 127
    e = torch.where(touched[:, None], torch.where(fresh[:, None], e, torch.maximum(e, old)), old)
    value = codes.view(torch.float8_e4m3fn).to(torch.float32).double()
    again = _e4m3(_times2(value, (old - e)[:, :, None, None]))  # older rows at the new scale
    keep = torch.arange(BS, device=slots.device)[None] < first[:, None]
    value = torch.where((keep & touched[:, None])[:, None, :, None], again, value)
    value[blk, :, row] = _e4m3(_times2(new, -e[blk][:, :, None]))
    codes.copy_(value.float().to(torch.float8_e4m3fn).view(torch.uint8))
    scale.copy_((e + 127).to(torch.uint8))


def _gather(codes, scale, blk, row):
    """Stored tokens as float32 [n, heads, dim]."""
    x = codes[blk, :, row].view(torch.float8_e4m3fn).float()
    return x * (scale[blk].to(torch.int32) << 23).view(torch.float32)[:, :, None]


def _plain(s):
    case = s["case"]
    hq, hkv = case["q_heads"], case["kv_heads"]
    g = hq // hkv
    if case["op"] == "rope":
        blk, row = s["slots"] // BS, s["slots"] % BS
        s["q_out"].copy_(_rotate(s["q"], s, torch.float32))
        s["k_cache"][blk, :, row] = _rotate(s["k"], s, torch.float32).to(s["k"].dtype)
        s["v_cache"][blk, :, row] = s["v"]
        return
    if case["op"] == "append8":
        s["q_out"].copy_(_rotate(s["q"], s, torch.float32))
        _append8(_rotate(s["k"], s, torch.float64), s["k_cache"], s["k_scale"], s["slots"])
        _append8(s["v"].double(), s["v_cache"], s["v_scale"], s["slots"])
        return
    q = s["q"].float().reshape(-1, hkv, g, 128)
    if case["op"] == "prefill8":
        pos = torch.arange(s["total"], device=q.device)
        blk, row = s["row"][pos // BS].long(), pos % BS
        k, v = (_gather(s[c + "_cache"], s[c + "_scale"], blk, row) for c in "kv")
        score = torch.einsum("chgd,nhd->hgcn", q, k) * s["scale"]
        seen = pos <= case["prior"] + torch.arange(case["chunk"], device=q.device)[:, None]
        score = score.masked_fill(~seen, -math.inf)
        p = torch.exp(score - score.amax(-1, keepdim=True))
        out = torch.einsum("hgcn,nhd->chgd", p / p.sum(-1, keepdim=True), v)
        s["out"].copy_(out.reshape(s["out"].shape))
        return
    # decode: all sequences' tokens in one row, sums by sequence
    lens, batch = s["lens"].long(), case["sequences"]
    seq = torch.repeat_interleave(torch.arange(batch, device=q.device), lens, output_size=s["total"])
    pos = torch.arange(s["total"], device=q.device) - (lens.cumsum(0) - lens)[seq]
    blk, row = s["block_table"][seq, pos // BS].long(), pos % BS
    k = _gather(s["k_cache"], s["k_scale"], blk, row)
    score = (k[:, :, None] * q[seq]).sum(-1) * s["scale"]           # [n, hkv, g]
    del k
    top = torch.full((batch, hkv, g), -math.inf, device=q.device)
    top = top.scatter_reduce(0, seq[:, None, None].expand_as(score), score, "amax")
    p = torch.exp(score - top[seq])
    v = _gather(s["v_cache"], s["v_scale"], blk, row)
    total = torch.zeros_like(top).index_add_(0, seq, p)
    out = torch.zeros((batch, hkv, g, 128), device=q.device).index_add_(0, seq, p[..., None] * v[:, :, None])
    s["out"].copy_((out / total[..., None]).reshape(s["out"].shape))


# ------------------------------------------------------------------- the pass
def _own(s):
    case, b = s["case"], s["binding"]
    if case["op"] == "rope":
        b.kv_append_rope(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], s["positions"],
                         s["rope"])
    elif case["op"] == "append8":
        b.kv_append_fp8_block(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["slots"],
                              q_out=s["q_out"], q=s["q"], positions=s["positions"], rope=s["rope"])
    elif case["op"] == "decode8":
        b.paged_decode_attention_fp8_block(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                           s["block_table"], s["lens"], s["longest"], s["scale"], s["workspace"])
    else:
        b.chunked_prefill_attention_fp8_block(s["out"], s["q"], s["k_cache"], s["v_cache"], s["k_scale"],
                                              s["v_scale"], s["row"], case["prior"], s["scale"])


def run(s):
    if own:
        _own(s)
    else:
        _plain(s)
    op = s["case"]["op"]
    if op == "rope":
        return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
    if op == "append8":
        codes, scales = torch.float8_e4m3fn, torch.float8_e8m0fnu
        return {"q": s["q_out"], "k": s["k_cache"].view(codes), "v": s["v_cache"].view(codes),
                "k_scale": s["k_scale"].view(scales), "v_scale": s["v_scale"].view(scales)}
    return {"out": s["out"]}


def work(case):
    hq, hkv = case["q_heads"], case["kv_heads"]
    if case["op"] in ("rope", "append8"):
        n = case["tokens"] * case.get("sequences", 1)
        d, rot, axes = case["dim"], case["rot"], case["axes"]
        size = 4 if case.get("fp32") else 2
        out = size if case["op"] == "rope" else 1
        per = d * (2 * size * hq + 2 * (size + out) * hkv) + 4 * rot + 4 * axes + 8
        # a block's scales; the older rows of a continued block are read only where its scale grows
        blocks = 0 if case["op"] == "rope" else case["sequences"] * -(-case["tokens"] // BS)
        return {"bytes": n * per + 4 * hkv * blocks, "flops": 3 * n * rot * (hq + hkv)}
    if case["op"] == "decode8":
        lens = _lengths(case)
        tokens, rows = sum(lens), len(lens)
        blocks = sum(-(-n // BS) for n in lens)
        flops = 4 * 128 * hq * tokens
    else:
        tokens, rows = case["prior"] + case["chunk"], case["chunk"]
        blocks = -(-tokens // BS)
        flops = 4 * 128 * hq * (case["chunk"] * case["prior"] + rows * (rows + 1) // 2)
    return {"bytes": 2 * hkv * (128 * tokens + blocks) + 4 * blocks + 4 * 128 * hq * rows, "flops": flops}


# ----------------------------------------------------------- exact, in 64 bits
def _numbers():
    """The value of each E4M3 code, from the format's fields."""
    code = np.arange(256)
    exp, man = (code >> 3) & 15, code & 7
    v = np.where(exp == 0, man / 8 * 2.0 ** -6, (1 + man / 8) * 2.0 ** (exp - 7.0))
    v[(code & 127) == 127] = np.nan
    return np.where(code > 127, -v, v)


def _nearest(y):
    """The nearest of the format's values: of two equally near ones that with the even code."""
    grid = _numbers()[:127]
    a = np.minimum(np.abs(y), MAX_CODE)
    hi = np.searchsorted(grid, a).clip(1, 126)
    lo = hi - 1
    up = (grid[hi] - a < a - grid[lo]) | ((grid[hi] - a == a - grid[lo]) & (hi % 2 == 0))
    return np.copysign(grid[np.where(up, hi, lo)], y)


def _turned(x, s):
    """The rotation as a product of complex numbers."""
    case = s["case"]
    half, n = case["rot"] // 2, x.shape[0]
    table, pos = s["table"].cpu().numpy().astype(np.float64), s["positions"].cpu().numpy()
    turn = np.empty((n, half), np.complex128)
    for i, axis in enumerate(s["pair_axis"]):
        turn[:, i] = table[pos[axis], i] + 1j * table[pos[axis], half + i]
    y = x.double().cpu().numpy().copy()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["interleaved"] else (
        slice(0, half), slice(half, 2 * half))
    z = (y[..., first] + 1j * y[..., second]) * turn[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_append8(new, codes, scale, slots):
    pool = _numbers()[codes.cpu().numpy()]
    e = scale.cpu().numpy().astype(np.int64) - 127
    by_block = {}
    for t, slot in enumerate(slots.tolist()):
        by_block.setdefault(slot // BS, []).append(t)
    for b, tokens in by_block.items():
        rows = np.array([slots[t] % BS for t in tokens])
        x = new[tokens].transpose(1, 0, 2)                          # [heads, rows, dim]
        with np.errstate(divide="ignore"):
            need = np.ceil(np.log2(np.abs(x).max((1, 2)) / MAX_CODE)).clip(E_MIN, E_MAX).astype(np.int64)
        first = rows.min()
        now = need if first == 0 else np.maximum(need, e[b])
        pool[b, :, :first] = _nearest(pool[b, :, :first] * 2.0 ** (e[b] - now)[:, None, None])
        pool[b][:, rows] = _nearest(x * 2.0 ** -now[:, None, None].astype(np.float64))
        e[b] = now
    return pool, 2.0 ** e


def _exact_attention(q, k, v, scale, seen=None):
    """softmax(scale q k^T) v in fp64: q [rows, hq, d], k and v [n, hkv, d], seen [rows, n]."""
    g = q.shape[1] // k.shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    for h in range(q.shape[1]):
        w = q[:, h].double() @ k[:, h // g].T * scale
        if seen is not None:
            w[~seen] = -math.inf
        out[:, h] = torch.softmax(w, -1) @ v[:, h // g]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "append8"):
        q, k, v = _turned(s["q"], s), _turned(s["k"], s), s["v"].double().cpu().numpy()
        slots = s["slots"].cpu().numpy()
        if case["op"] == "append8":
            kc, ks = _exact_append8(k, s["k_cache"], s["k_scale"], slots)
            vc, vs = _exact_append8(v, s["v_cache"], s["v_scale"], slots)
            return {"q": q, "k": kc, "v": vc, "k_scale": ks, "v_scale": vs}
        kc, vc = (s[c].double().cpu().numpy() for c in ("k_cache", "v_cache"))
        kc[slots // BS, :, slots % BS], vc[slots // BS, :, slots % BS] = k, v
        return {"q": q, "k": kc, "v": vc}
    value = torch.tensor(_numbers(), device="cuda")

    def stored(which, b):
        n = int(s["lens"][b])
        ids = s["block_table"][b, :-(-n // BS)].long()
        x = value[s[which + "_cache"][ids].long()] * 2.0 ** (s[which + "_scale"][ids].double() - 127)[:, :, None, None]
        return x.transpose(1, 2).flatten(0, 1)[:n]                  # [n, hkv, d]

    if case["op"] == "prefill8":
        last = case["prior"] + torch.arange(case["chunk"], device="cuda")
        seen = torch.arange(s["total"], device="cuda")[None] <= last[:, None]
        return {"out": _exact_attention(s["q"], stored("k", 0), stored("v", 0), s["scale"], seen)}
    return {"out": torch.cat([_exact_attention(s["q"][b:b + 1], stored("k", b), stored("v", b), s["scale"])
                              for b in range(case["sequences"])])}
