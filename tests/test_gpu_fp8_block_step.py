"""A serving run over the block-scaled cache, as an engine makes it: a prompt
in two chunks (rotated and quantised on the way in, each chunk's attention over
what is stored), then decode steps of a batch.  And the same run over the bf16
pools with kv_append_rope.  Everything is compared with fp64: the rotation and
the quantiser of the oracle, its attention over the stored values.

The rotated queries are rounded to bf16 by the append and the attention is held
to its own bound on them, so one bound covers a step: block_cases' for the
block-scaled cache, 2e-2 (the other bf16 tests') for the bf16 one."""
import numpy as np
import pytest
import torch

import block_cases as C
import oracle
import rope_cases as R
from oracle import fp8_block as FB
from oracle import rope as O
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5
HQ, HKV, D = 16, 4, 128


class _Stored:
    """block_cases.Pools of what the GPU holds now."""

    def __init__(self, codes, scale):
        self.codes, self.scale = [c.cpu() for c in codes], [s.cpu() for s in scale]

    def values(self, which):
        return torch.from_numpy(FB.dequantize(self.codes[which].numpy(), self.scale[which].numpy()))


def _new(t, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(t, h, D, generator=g).to(torch.bfloat16) for h in (HQ, HKV, HKV))


def _check_pool(codes, scale, want, blk, row):
    """The rows just written against the oracle's exact ones: half a step of
    E4M3 at the block's scale (the rotation's fp32 error is far below)."""
    got = FB.dequantize(codes.cpu().numpy(), scale.cpu().numpy())[blk, :, row]
    unit = np.exp2(scale.cpu().numpy().astype(float) - 127)[blk][:, :, None]
    bound = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * unit) * (1 + 2.0 ** -10) + 2.0 ** -20
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_prompt_then_steps_over_the_block_scaled_cache(interleaved):
    lens = [300, 45, 160, 1]                        # prompts; sequence 0 arrives in two chunks
    steps = 3
    table, nb = C.tables([n + steps for n in lens], 3)
    cs = R.table(512, D)
    rope = B.Rope(cs.cuda(), interleaved)
    codes = [torch.zeros(nb, HKV, 16, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scale = [torch.zeros(nb, HKV, dtype=torch.uint8, device="cuda") for _ in "kv"]
    dev_table = table.cuda()

    def append(q, k, v, slots, pos):
        qo = torch.empty_like(q).cuda()
        B.kv_append_fp8_block(k.cuda(), v.cuda(), *codes, *scale, slots.cuda(), q_out=qo, q=q.cuda(),
                              positions=pos.cuda(), rope=rope)
        turned = O.rotate(k.double().numpy(), cs.numpy(), pos.numpy(), interleaved)
        blk, row = (slots // 16).numpy(), (slots % 16).numpy()
        _check_pool(codes[0], scale[0], turned, blk, row)
        _check_pool(codes[1], scale[1], v.double().numpy(), blk, row)
        want = O.rotate(q.double().numpy(), cs.numpy(), pos.numpy(), interleaved)
        assert (np.abs(qo.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18).all()
        return qo

    def slots_of(seq, first, n):
        p = torch.arange(first, first + n)
        return table[seq, p // 16].long() * 16 + p % 16, p.to(torch.int32)

    for seq, n in enumerate(lens):
        for first, count in ([(0, 187), (187, 113)] if seq == 0 else [(0, n)]):
            q, k, v = _new(count, 10 * seq + first)
            slots, pos = slots_of(seq, first, count)
            qo = append(q, k, v, slots, pos)
            out = torch.empty_like(qo)
            B.chunked_prefill_attention_fp8_block(out, qo, *codes, *scale, dev_table[seq].contiguous(), first, SCALE)
            torch.cuda.synchronize()
            held = _Stored(codes, scale)
            used = table[seq, :-(-(first + count) // 16)].long()
            kv = [held.values(i)[used] for i in (0, 1)]
            args = (torch.arange(len(used), dtype=torch.int32), first, SCALE)
            ref = oracle.chunked_prefill(qo.cpu().double(), kv[0], kv[1], *args)
            ref_abs = oracle.chunked_prefill(qo.cpu().double(), kv[0], kv[1].abs(), *args)
            err = (out.cpu().double() - ref).abs() - C.bound(ref, ref_abs, 2.0 ** -11 + 2.0 ** -13)
            # weights below f16's range: 2^-25 of the largest V scale's 448 each
            assert bool((err <= (first + count) * 2.0 ** -25 * 448 * 2.0 ** -6).all()), float(err.max())
    now = list(lens)
    for step in range(steps):
        q, k, v = _new(len(lens), 1000 + step)
        where = [slots_of(s, n, 1) for s, n in enumerate(now)]
        slots, pos = (torch.cat([w[i] for w in where]) for i in (0, 1))
        qo = append(q, k, v, slots, pos)
        now = [n + 1 for n in now]
        out = C.decode(codes + scale, qo.cpu(), table, now, SCALE)
        C.check_decode(_Stored(codes, scale), qo.cpu(), table, now, SCALE, out)
    assert B.get_device_error() == 0


def test_prompt_then_step_over_the_bf16_cache():
    n, first = 200, 130
    table, nb = C.tables([n + 1], 4)
    cs = R.table(512, D)
    rope = B.Rope(cs.cuda(), pair_axis=[0] * 20 + [1] * 22 + [2] * 22)
    kc, vc = (torch.zeros(nb, HKV, 16, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    row = table[0].cuda()
    for at, count in ((0, first), (first, n - first), (n, 1)):
        q, k, v = _new(count, at)
        p = torch.arange(at, at + count)
        slots = table[0, p // 16].long() * 16 + p % 16
        pos = torch.stack([p, p % 14, p // 14]).to(torch.int32)
        qo = torch.empty_like(q).cuda()
        B.kv_append_rope(qo, q.cuda(), k.cuda(), v.cuda(), kc, vc, slots.cuda(), pos.cuda(), rope)
        out = torch.empty_like(qo)
        if at < n:
            B.chunked_prefill_attention(out, qo, kc, vc, row, at, SCALE)
            torch.cuda.synchronize()
            ref = oracle.chunked_prefill(qo.cpu(), kc.cpu(), vc.cpu(), table[0], at, SCALE)
        else:
            lens = torch.tensor([n + 1], dtype=torch.int32)
            B.paged_decode_attention(out, qo, kc, vc, row[None].contiguous(), lens.cuda(), n + 1, SCALE)
            torch.cuda.synchronize()
            ref = oracle.paged_decode(qo.cpu(), kc.cpu(), vc.cpu(), table, lens, SCALE)
        assert float((out.cpu().double() - ref).abs().max()) <= 2e-2
        want = O.rotate(k.double().numpy(), cs.numpy(), pos.numpy(), False, [0] * 20 + [1] * 22 + [2] * 22)
        held = kc.cpu()[slots // 16, :, slots % 16].double().numpy()
        assert (np.abs(held - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18).all()
    assert B.get_device_error() == 0


def test_step_captured_whole_and_replayed():
    """Append and decode of one step in one graph, replayed for the next token
    with the inputs' buffers refilled."""
    lens = [40, 700]
    table, nb = C.tables([n + 2 for n in lens], 5)
    cs = B.Rope(R.table(1024, D).cuda())
    pools = C.Pools(nb, HKV, 5)
    q0, k0, v0 = _new(2, 1)
    q1, k1, v1 = _new(2, 2)

    def state():
        return [t.clone() for t in pools.cuda()]

    def fill(buf, q, k, v, at):
        p = torch.tensor([n + at for n in lens])
        slots = table[torch.arange(2), p // 16].long() * 16 + p % 16
        for b, x in zip(buf, (q, k, v, slots, p.to(torch.int32)[None], (p + 1).to(torch.int32))):
            b.copy_(x)

    dev = table.cuda()
    ws = B.decode_workspace_fp8_block(2, HQ, HKV, D, 702)
    out = torch.zeros(2, HQ, D, dtype=torch.bfloat16, device="cuda")

    def step(buf, st):
        q, k, v, slots, pos, sl = buf
        B.kv_append_fp8_block(k, v, st[0], st[1], st[2], st[3], slots, q_out=q, q=q, positions=pos, rope=cs)
        B.paged_decode_attention_fp8_block(out, q, *st, dev, sl, 702, SCALE, ws)

    buf = [torch.zeros(s, dtype=t, device="cuda") for s, t in (
        ((2, HQ, D), torch.bfloat16), ((2, HKV, D), torch.bfloat16), ((2, HKV, D), torch.bfloat16),
        ((2,), torch.int64), ((1, 2), torch.int32), ((2,), torch.int32))]
    st, want = state(), []
    for at, (q, k, v) in enumerate(((q0, k0, v0), (q1, k1, v1))):
        fill(buf, q, k, v, at)
        step(buf, st)
        torch.cuda.synchronize()
        want.append(out.clone())
    ref = [t.clone() for t in st]
    for t, x in zip(st, state()):
        t.copy_(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(buf, st)
    for at, (q, k, v) in enumerate(((q0, k0, v0), (q1, k1, v1))):
        fill(buf, q, k, v, at)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[at])
    assert all(torch.equal(a, b) for a, b in zip(st, ref)) and B.get_device_error() == 0


def test_two_threads_on_streams_of_their_own():
    """Append, prefill and decode of two sequences' pools at once, from two host
    threads, give what each gives alone."""
    import threading
    cs = R.table(512, D).cuda()
    n = 300
    table, nb = C.tables([n], 6)
    pos = torch.arange(n)
    slots = (table[0, pos // 16].long() * 16 + pos % 16).cuda()
    row, pos32 = table[0].cuda(), pos.to(torch.int32).cuda()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    inputs = [[x.cuda() for x in _new(n, 60 + i)] for i in range(2)]

    def work(i, out, stream, times):
        q, k, v = inputs[i]
        rope = B.Rope(cs, bool(i))
        with torch.cuda.stream(stream):
            codes = [torch.zeros(nb, HKV, 16, D, dtype=torch.uint8, device="cuda") for _ in "kv"]
            scale = [torch.zeros(nb, HKV, dtype=torch.uint8, device="cuda") for _ in "kv"]
            ws = B.decode_workspace_fp8_block(1, HQ, HKV, D, n)
            qo, pre, dec = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q[:1])
            for _ in range(times):
                B.kv_append_fp8_block(k, v, *codes, *scale, slots, q_out=qo, q=q, positions=pos32, rope=rope)
                B.chunked_prefill_attention_fp8_block(pre, qo, *codes, *scale, row, 0, SCALE)
                B.paged_decode_attention_fp8_block(dec, qo[-1:], *codes, *scale, row[None], lens, n, SCALE, ws)
            out[i] = [qo, pre, dec, *codes, *scale]

    alone, both = {}, {}
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        work(i, alone, streams[i], 1)
        torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i, both, streams[i], 30)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(alone[i], both[i]))
