"""kv_append_rope on the GPU against the fp64 oracle.

Bounds.  A rotated element is fma(a, c, -fl(b s)) (or with the terms swapped)
of exact a, b and the table's fp32 c, s, |c|, |s| <= 1 + 2^-24: one product
rounding, one fma rounding, 2^-24 of at most |a| + |b| each, so the fp32
result is within 2^-23 (|a| + |b|) of the fp64 one; the bf16 store adds half a
step, 2^-8 relative to the value.  Values are copied bit for bit."""
import numpy as np
import pytest
import torch

import rope_cases as R
from oracle import rope as O
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu

FILL = 7.0


def _bits(t):
    return t.view(torch.int16) if t.element_size() == 2 else t.view(torch.int32)


def _check_rotated(got, x, cs, pos, rot, interleaved, axis, dtype):
    want = O.rotate(x.double().numpy(), cs.numpy(), pos.numpy(), interleaved, axis)
    bound = 2.0 ** -23 * O.magnitude(x.double().numpy(), rot, interleaved)
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * (np.abs(want) + bound)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= bound + 1e-45).all(), float((err - bound).max())
    assert torch.equal(_bits(got.cpu()[..., rot:].contiguous()), _bits(x[..., rot:].contiguous()))


def _run(t, hq, hkv, d, rot, interleaved, axes, in_turn, dtype, seed=1):
    cs = R.table(997, rot)
    axis = None if axes == 1 else R.sections(rot, axes, in_turn)
    q, k, v, pos = R.draw(t, hq, hkv, d, dtype, seed, axes)
    nb = t // 16 + 3
    slots = R.scattered_slots(t, nb, seed)
    kc, vc = (torch.full((nb, hkv, 16, d), FILL, dtype=dtype, device="cuda") for _ in "kv")
    qo = torch.full((t, hq, d), FILL, dtype=dtype, device="cuda")
    rope = B.Rope(cs.cuda(), interleaved, axis)
    B.kv_append_rope(qo, q.cuda(), k.cuda(), v.cuda(), kc, vc, slots.cuda(), pos.cuda(), rope)
    torch.cuda.synchronize()
    assert B.get_device_error() == 0
    kc, vc = kc.cpu(), vc.cpu()
    blk, row = slots // 16, slots % 16
    _check_rotated(qo, q, cs, pos, rot, interleaved, axis, dtype)
    _check_rotated(kc[blk, :, row], k, cs, pos, rot, interleaved, axis, dtype)
    assert torch.equal(_bits(vc[blk, :, row]), _bits(v))
    other = torch.ones(nb, 16, dtype=torch.bool)
    other[blk, row] = False
    for c in (kc, vc):
        assert bool((c.permute(0, 2, 1, 3)[other] == FILL).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 64), (64, 16), (80, 80), (80, 40), (96, 90),
                                   (256, 256), (24, 2), (512, 256)])
def test_shapes(d, rot, interleaved, dtype):
    _run(37, 6, 3, d, rot, interleaved, 1, False, dtype, seed=d + rot)


@pytest.mark.parametrize("axes,in_turn", [(2, False), (3, False), (3, True), (4, True)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_axes(axes, in_turn, interleaved, dtype):
    _run(21, 8, 2, 128, 96, interleaved, axes, in_turn, dtype, seed=axes)


@pytest.mark.parametrize("t,hq,hkv", [(1, 32, 8), (1, 1, 1), (2, 64, 8), (129, 5, 5), (2049, 8, 1), (300, 70, 7)])
def test_counts(t, hq, hkv):
    _run(t, hq, hkv, 128, 128, False, 1, False, torch.bfloat16, seed=t)


def test_columns_of_one_projection_and_in_place():
    """q, k, v as columns of one [T, (Hq + 2 Hkv) D] tensor, q rotated in place."""
    t, hq, hkv, d = 50, 8, 2, 128
    cs = R.table(997, d)
    q, k, v, pos = R.draw(t, hq, hkv, d, torch.bfloat16, 5)
    qkv = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).cuda()
    qs, ks, vs = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    slots = R.scattered_slots(t, 8, 5)
    kc, vc = (torch.zeros(8, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    B.kv_append_rope(qs, qs, ks, vs, kc, vc, slots.cuda(), pos.cuda(), B.Rope(cs.cuda()))
    torch.cuda.synchronize()
    _check_rotated(qs.contiguous(), q, cs, pos, d, False, None, torch.bfloat16)
    assert torch.equal(ks.cpu(), k) and torch.equal(vs.cpu(), v)
    _check_rotated(kc.cpu()[slots // 16, :, slots % 16], k, cs, pos, d, False, None, torch.bfloat16)
    assert torch.equal(vc.cpu()[slots // 16, :, slots % 16], v)


def test_no_queries_matches_with_queries():
    t, hkv, d = 33, 4, 128
    cs = R.table(997, d).cuda()
    q, k, v, pos = (x.cuda() for x in R.draw(t, 8, hkv, d, torch.bfloat16, 6))
    slots = R.scattered_slots(t, 5, 6).cuda()
    a, b, c, e = (torch.zeros(5, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    B.kv_append_rope(torch.empty_like(q), q, k, v, a, b, slots, pos, B.Rope(cs))
    B.kv_append_rope(None, None, k, v, c, e, slots, pos, B.Rope(cs))
    assert torch.equal(a, c) and torch.equal(b, e)


def test_zero_angle_is_kv_append():
    """Position 0 turns nothing: pools and queries as kv_append leaves them, bit for bit."""
    t, hkv, d = 40, 2, 128
    q, k, v, pos = (x.cuda() for x in R.draw(t, 4, hkv, d, torch.bfloat16, 8))
    slots = R.scattered_slots(t, 6, 8).cuda()
    a, b, c, e = (torch.zeros(6, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    qo = torch.empty_like(q)
    B.kv_append_rope(qo, q, k, v, a, b, slots, torch.zeros_like(pos), B.Rope(R.table(997, d).cuda()))
    B.kv_append(k, v, c, e, slots)
    assert torch.equal(a, c) and torch.equal(b, e) and torch.equal(qo, q)


def test_padding_and_bad_entries_are_skipped_whole():
    t, hq, hkv, d = 12, 4, 2, 128
    q, k, v, pos = R.draw(t, hq, hkv, d, torch.bfloat16, 9)
    slots = R.scattered_slots(t, 4, 9)
    slots[3] = -1
    pos[0, 3] = -5                                   # a padding token's position is not looked at
    pool = torch.full((4, hkv, 16, d), FILL, dtype=torch.bfloat16, device="cuda")

    def call(slots, pos):
        kc, vc = pool.clone(), pool.clone()
        qo = torch.full((t, hq, d), FILL, dtype=torch.bfloat16, device="cuda")
        B.kv_append_rope(qo, q.cuda(), k.cuda(), v.cuda(), kc, vc, slots.cuda(), pos.cuda(),
                         B.Rope(R.table(997, d).cuda()))
        return qo.cpu(), kc.cpu(), vc.cpu(), B.get_device_error()

    qo, kc, vc, err = call(slots, pos)
    assert err == 0 and bool((qo[3] == FILL).all()) and bool((qo[2] != FILL).any())
    for bad_slot, bad_pos, code in ((4 * 16, 1, 1), (None, 997, 6), (None, -1, 6)):
        s2, p2 = slots.clone(), pos.clone()
        if bad_slot is not None:
            s2[5] = bad_slot
        p2[0, 5] = bad_pos
        q2, k2, v2, err = call(s2, p2)
        assert err == code and B.get_device_error() == 0
        assert bool((q2[5] == FILL).all())
        keep = torch.arange(t) != 5
        assert torch.equal(q2[keep], qo[keep])
        b, r = int(slots[5]) // 16, int(slots[5]) % 16
        assert bool((k2[b, :, r] == FILL).all()) and bool((v2[b, :, r] == FILL).all())


def test_empty_and_other_stream_and_graph():
    t, hkv, d = 20, 2, 128
    cs = B.Rope(R.table(997, d).cuda())
    q, k, v, pos = (x.cuda() for x in R.draw(t, 4, hkv, d, torch.bfloat16, 10))
    slots = R.scattered_slots(t, 4, 10).cuda()
    ref = [torch.zeros(4, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    got = [x.clone() for x in ref]
    qr, qg = torch.zeros_like(q), torch.zeros_like(q)
    B.kv_append_rope(qr[:0], q[:0], k[:0], v[:0], *ref, slots[:0], pos[:, :0].contiguous(), cs)
    assert not bool(ref[0].any())
    B.kv_append_rope(qr, q, k, v, *ref, slots, pos, cs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            B.kv_append_rope(qg, q, k, v, *got, slots, pos, cs)
    torch.cuda.synchronize()
    assert not bool(got[0].any())                    # captured, not run
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qg, qr) and torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    q.mul_(2)                                        # a replay reads the buffers anew
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qg, qr * 2)


@pytest.mark.parametrize("t,hq,hkv,d,rot,dtype", [
    (8300, 32, 8, 128, 128, torch.bfloat16), (4300, 32, 8, 128, 64, torch.float32), (2500, 32, 8, 96, 96, torch.bfloat16),
    (9001, 30, 3, 128, 20, torch.bfloat16), (1100, 128, 1, 128, 128, torch.bfloat16)])
@pytest.mark.parametrize("in_place", [False, True])
def test_large_batches_equal_small_ones(t, hq, hkv, d, rot, dtype, in_place):
    """Several heads to a thread, and loads and stores that stream: bit for bit
    what pieces of 300 tokens give."""
    rope = B.Rope(R.table(997, rot).cuda(), False, R.sections(rot, 3))
    q, k, v, pos = (x.cuda() for x in R.draw(t, hq, hkv, d, dtype, 9, 3))
    nb = t // 16 + 3
    slots = R.scattered_slots(t, nb, 9).cuda()
    got = []
    for step in (t, 300):
        kc, vc = (torch.full((nb, hkv, 16, d), FILL, dtype=dtype, device="cuda") for _ in "kv")
        src = q.clone()
        qo = src if in_place else torch.empty_like(q)
        for i in range(0, t, step):
            s = slice(i, i + step)
            B.kv_append_rope(qo[s], src[s], k[s], v[s], kc, vc, slots[s], pos[:, s].contiguous(), rope)
        torch.cuda.synchronize()
        got.append((qo, kc, vc))
    assert B.get_device_error() == 0
    assert all(torch.equal(_bits(a), _bits(b)) for a, b in zip(*got))
    assert not torch.equal(_bits(got[0][0]), _bits(q))
