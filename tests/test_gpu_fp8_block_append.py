"""kv_append_fp8_block on the GPU against the oracle's quantiser.

Codes and scale bytes equal the oracle's bit for bit, with a rotation too: the
keys' one rounding is that of the fp64 rotation.  (test_rotated asks for less:
the fp32 rotation, within 2^-23 (|a| + |b|) of the fp64 one, and half a step of
E4M3, 2^-4 relative to the rounded value's binade or 2^-10 of the scale below
the normal range.)"""
import numpy as np
import pytest
import torch

import rope_cases as R
from oracle import fp8_block as FB
from oracle import rope as O
from paged_kv_cache_104_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _pools(nb, hkv, d, seed):
    """Pools that hold something everywhere: any finite code, plausible scales."""
    g = torch.Generator().manual_seed(300 + seed)
    codes = torch.randint(0, 127, (2, nb, hkv, 16, d), generator=g)
    codes += 128 * torch.randint(0, 2, codes.shape, generator=g)
    scale = 127 + torch.randint(-9, -5, (2, nb, hkv), generator=g)
    return codes.to(torch.uint8), scale.to(torch.uint8)


def _append(k, v, codes, scale, slots, **kw):
    c, s = codes.cuda(), scale.cuda()
    B.kv_append_fp8_block(k.cuda(), v.cuda(), c[0], c[1], s[0], s[1], slots.cuda(), **kw)
    torch.cuda.synchronize()
    return c.cpu(), s.cpu()


def _oracle(k, v, codes, scale, slots):
    c, s = codes.numpy().copy(), scale.numpy().copy()
    for i, x in enumerate((k, v)):
        FB.append_pool(x.double().numpy(), c[i], s[i], slots.tolist())
    return c, s


def _same(got, want):
    assert np.array_equal(got[1].numpy(), want[1])
    assert np.array_equal(got[0].numpy(), want[0])


@pytest.mark.parametrize("pieces", [[(0, 1)], [(7, 1)], [(15, 1)], [(15, 2)], [(0, 16)], [(0, 17)], [(5, 100)],
                                    [(i % 16, 1) for i in range(40)], [(3, 200), (0, 5), (15, 33), (9, 1)]])
@pytest.mark.parametrize("hkv,d", [(8, 128), (1, 128), (3, 64), (5, 16), (2, 112)])
def test_bit_exact_without_rotation(pieces, hkv, d):
    t = sum(n for _, n in pieces)
    nb = sum((f + n - 1) // 16 + 1 for f, n in pieces) + 2
    _, k, v, _ = R.draw(t, 1, hkv, d, torch.bfloat16, t + d)
    k = k * torch.exp2(torch.randint(-6, 7, (t, hkv, 1), generator=torch.Generator().manual_seed(t))).bfloat16()
    codes, scale = _pools(nb, hkv, d, t)
    slots = R.run_slots(pieces, nb, t)
    got = _append(k, v, codes, scale, slots)
    assert B.get_device_error() == 0
    _same(got, _oracle(k, v, codes, scale, slots))


def test_token_by_token_follows_the_scale_up():
    """A sequence's rows appended one at a time, each larger than the last."""
    hkv, d = 2, 128
    _, k, v, _ = R.draw(20, 1, hkv, d, torch.bfloat16, 3)
    k = (k * torch.exp2(torch.arange(20) - 10.0)[:, None, None]).bfloat16()
    codes, scale = _pools(3, hkv, d, 3)
    slots = R.run_slots([(0, 20)], 3, 3)
    c, s, oc, os_ = codes, scale, codes, scale
    for t in range(20):
        c, s = _append(k[t:t + 1], v[t:t + 1], c, s, slots[t:t + 1])
        a, b = _oracle(k[t:t + 1], v[t:t + 1], oc, os_, slots[t:t + 1])
        oc, os_ = torch.from_numpy(a), torch.from_numpy(b)
        _same((c, s), (a, b))


def test_special_values():
    hkv, d = 2, 64
    inf, nan = float("inf"), float("nan")
    k = torch.zeros(6, hkv, d)
    k[0, 0, :4] = torch.tensor([inf, -inf, nan, 1.0])
    k[1, 0, :3] = torch.tensor([-0.0, 1e-30, 3e38])          # a scale near the largest
    k[2, 1, 5] = 1e-40                                       # a subnormal alone
    k[3, 0] = nan                                            # nothing finite
    k[4, 0, :8] = torch.tensor([448., 449., 464., 465., 480., 1e4, -448., 26.5])
    k = k.bfloat16()
    codes, scale = _pools(7, hkv, d, 4)
    for slots in ([0, 16, 32, 48, 64, 80], [3, 19, 35, 51, 67, 83], [0, 1, 2, 3, 4, 5]):
        slots = torch.tensor(slots)
        got = _append(k, -k, codes, scale, slots)
        want = _oracle(k, -k, codes, scale, slots)
        assert B.get_device_error() == 0
        assert np.array_equal(got[1].numpy(), want[1])
        g, w = got[0].numpy().copy(), want[0].copy()
        g[(g & 0x7F) == 0x7F] = 0x7F                         # the sign of a NaN code is not specified
        w[(w & 0x7F) == 0x7F] = 0x7F
        assert np.array_equal(g, w)


@pytest.mark.parametrize("byte", [0, 1, 2, 240, 246, 253, 254, 255])
def test_continued_block_with_an_unusual_scale(byte):
    hkv, d = 1, 32
    _, k, v, _ = R.draw(2, 1, hkv, d, torch.bfloat16, 5)
    codes, scale = _pools(2, hkv, d, 5)
    scale[:] = byte
    slots = torch.tensor([9, 10])
    _same(_append(k, v, codes, scale, slots), _oracle(k, v, codes, scale, slots))


def test_order_errors_padding_and_bad_slots():
    hkv, d = 2, 128
    _, k, v, _ = R.draw(6, 1, hkv, d, torch.bfloat16, 6)
    codes, scale = _pools(4, hkv, d, 6)
    ok = torch.tensor([-1, 20, 21, -1, 0, 40])
    _same(_append(k, v, codes, scale, ok), _oracle(k, v, codes, scale, ok))
    assert B.get_device_error() == 0
    # (slots, the ones that are carried out, code): a gap, a return, a repeat, a step back, beyond the pool
    for slots, done, code in (([0, 2, 20, 21, 40, 41], [0, -1, 20, 21, 40, 41], 7),
                              ([0, 20, 21, 1, 40, 41], [0, 20, 21, -1, 40, 41], 7),
                              ([5, 5, 20, -1, -1, 5], [5, -1, 20, -1, -1, -1], 7),
                              ([5, 4, 20, 21, 22, 23], [5, -1, 20, 21, 22, 23], 7),
                              ([0, 64, 20, 21, 40, 41], [0, -1, 20, 21, 40, 41], 1)):
        got = _append(k, v, codes, scale, torch.tensor(slots))
        assert B.get_device_error() == code
        _same(got, _oracle(k, v, codes, scale, torch.tensor(done)))


@pytest.mark.parametrize("d,rot,interleaved,axes", [(128, 128, False, 1), (128, 128, True, 1), (128, 64, False, 3),
                                                    (64, 32, True, 2), (128, 96, False, 2)])
@pytest.mark.parametrize("pieces", [[(i % 16, 1) for i in range(30)], [(5, 130), (0, 20)]])
def test_rotated(d, rot, interleaved, axes, pieces):
    t, hq, hkv = sum(n for _, n in pieces), 6, 3
    nb = sum((f + n - 1) // 16 + 1 for f, n in pieces) + 1
    cs = R.table(997, rot)
    axis = None if axes == 1 else R.sections(rot, axes, axes == 3)
    q, k, v, pos = R.draw(t, hq, hkv, d, torch.bfloat16, t + rot, axes)
    codes, scale = _pools(nb, hkv, d, t)
    slots = R.run_slots(pieces, nb, t)
    qo = torch.zeros_like(q).cuda()
    c, s = _append(k, v, codes, scale, slots, q=q.cuda(), q_out=qo, positions=pos.cuda(),
                   rope=B.Rope(cs.cuda(), interleaved, axis))
    assert B.get_device_error() == 0
    turned = O.rotate(k.double().numpy(), cs.numpy(), pos.numpy(), interleaved, axis)
    oc, os_ = codes.numpy().copy(), scale.numpy().copy()
    FB.append_pool(turned, oc[0], os_[0], slots.tolist())
    FB.append_pool(v.double().numpy(), oc[1], os_[1], slots.tolist())
    assert np.array_equal(s.numpy(), os_)                    # no amax here is within fp32 rounding of a border
    assert np.array_equal(c[1].numpy(), oc[1])
    blk, row = slots // 16, slots % 16
    new = torch.zeros(nb, 16, dtype=torch.bool)
    new[blk, row] = True
    kept = ~new.numpy()[:, None, :, None] & np.ones_like(oc[0], bool)
    assert np.array_equal(c[0].numpy()[kept], oc[0][kept])   # other rows exactly as the oracle has them
    got = FB.dequantize(c[0].numpy(), s[0].numpy())[blk, :, row]
    unit = np.exp2(s[0].numpy().astype(float) - 127)[blk][:, :, None]
    fp32 = 2.0 ** -23 * O.magnitude(k.double().numpy(), rot, interleaved)
    # half a step is at most 2^-4 of the value's own binade, 2^-10 units below the normal range
    bound = np.maximum(2.0 ** -4 * (np.abs(turned) + fp32), 2.0 ** -10 * unit) + fp32
    assert (np.abs(got - turned) <= bound).all()
    # the queries: as the 16-bit append rotates them
    ref = torch.zeros_like(qo)
    pool = torch.zeros(nb, hkv, 16, d, dtype=torch.bfloat16, device="cuda")
    B.kv_append_rope(ref, q.cuda(), k.cuda(), v.cuda(), pool, pool.clone(), slots.cuda(), pos.cuda(),
                     B.Rope(cs.cuda(), interleaved, axis))
    assert torch.equal(qo, ref)


def _rotated_exactly(k, cs, pos, interleaved, codes, scale, slots):
    """The key pool against the oracle's codes of the fp64 rotation (NaN: of either sign)."""
    c, s = _append(k, k, codes, scale, slots, positions=pos.cuda(), rope=B.Rope(cs.cuda(), interleaved))
    assert B.get_device_error() == 0
    oc, os_ = codes[0].numpy().copy(), scale[0].numpy().copy()
    with np.errstate(invalid="ignore"):
        FB.append_pool(O.rotate(k.double().numpy(), cs.numpy(), pos.numpy(), interleaved), oc, os_, slots.tolist())
    got = c[0].numpy().copy()
    for x in (got, oc):
        x[(x & 0x7F) == 0x7F] = 0x7F
    assert np.array_equal(s[0].numpy(), os_)
    assert np.array_equal(got, oc)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("outlier", [1.0, 200.0])        # 200: most codes are subnormal
def test_rotated_codes_are_those_of_the_exact_keys(interleaved, outlier):
    """Of two million codes some lie where fp32 falls on the other side of a middle."""
    t, hkv, d = 2040, 8, 128
    _, k, _, pos = R.draw(t, 1, hkv, d, torch.bfloat16, 21)
    k[:, :, 5] *= outlier
    codes, scale = _pools(131, hkv, d, 21)
    _rotated_exactly(k, R.table(997, d), pos, interleaved, codes, scale, R.run_slots([(7, t)], 131, 21))


@pytest.mark.parametrize("tokens", [1, 40])              # a head to a CTA, and four
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_values_beside_the_middle_of_two_codes(interleaved, tokens):
    hkv, d = 72 if tokens == 40 else 2, 32
    first, second = O.pair_columns(d, interleaved)
    k = torch.zeros(tokens, hkv, d)
    cs = torch.zeros(4, d)
    cs[:, :d // 2], cs[:, d // 2:] = 1.0, 2.0 ** -20
    # middles: of normal codes, beside the subnormal ones, of those, of 0 and the least
    middle = [1.0625, 1.1875, 248.0, -1.9375, 2.0 ** -6 * 1.0625, 2.0 ** -7 + 2.0 ** -10, 3 * 2.0 ** -10, -5 * 2.0 ** -10,
              2.0 ** -10, 15 * 2.0 ** -10, 13 * 2.0 ** -10]
    for i, m in enumerate(middle):
        k[:, :, first[i]] = m
        k[:, :, second[i]] = 2.0 ** -18 * m * (1 if i % 2 else -1)    # m -+ 2^-38 m
    k[:, :, first[13]] = 400.0                                        # the scale is 1
    k[:, :, first[14]], k[:, :, second[14]] = 1.5, 1.5
    k[:, :, second[15]] = 0.0
    cs[1] = -cs[1]
    cs[2, 14], cs[2, d // 2 + 14] = 1.0 + 2.0 ** -23, 1.0             # cancels to 1.5 * 2^-23
    cs[3, 14], cs[3, d // 2 + 14] = 1.0 + 2.0 ** -8, 1.0 - 2.0 ** -24
    k = k.bfloat16()
    pos = (torch.arange(tokens) % 4).to(torch.int32)[None]
    codes, scale = _pools(5, hkv, d, 22)
    for at in range(4):
        _rotated_exactly(k, cs, (pos + at) % 4, interleaved, codes, scale, R.run_slots([(0, tokens)], 5, 22))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotated_infinities_and_nan(interleaved):
    t, hkv, d = 20, 2, 64
    _, k, _, pos = R.draw(t, 1, hkv, d, torch.bfloat16, 23)
    k[3, 0, 1], k[4, 1, 40], k[5, 0, 33], k[6, 0, 2] = float("inf"), -float("inf"), float("inf"), float("nan")
    k[7, 1, 9], k[8, 0, 10] = 3e38, -3e38
    codes, scale = _pools(3, hkv, d, 23)
    _rotated_exactly(k, R.table(997, d), pos, interleaved, codes, scale, R.run_slots([(4, t)], 3, 23))


def test_bad_position_skips_the_rest_of_its_run():
    hkv, d = 2, 128
    q, k, v, pos = R.draw(8, 4, hkv, d, torch.bfloat16, 11)
    codes, scale = _pools(3, hkv, d, 11)
    slots = torch.tensor([3, 4, 5, 6, 7, 8, 32, 33])
    rope = B.Rope(R.table(997, d).cuda())

    def call(pos, slots):
        qo = torch.zeros_like(q).cuda()
        c, s = _append(k, v, codes, scale, slots, q=q.cuda(), q_out=qo, positions=pos.cuda(), rope=rope)
        return c, s, qo.cpu(), B.get_device_error()

    bad = pos.clone()
    bad[0, 2] = 997
    c, s, qo, err = call(bad, slots)
    done = slots.clone()
    done[2:6] = -1
    c2, s2, qo2, err2 = call(pos, done)
    assert (err, err2) == (6, 0) and torch.equal(c, c2) and torch.equal(s, s2)
    assert not bool(qo[2].any()) and torch.equal(qo[:2], qo2[:2]) and torch.equal(qo[6:], qo2[6:])


def test_strided_in_place_graph_and_stream():
    t, hq, hkv, d = 45, 8, 2, 128
    q, k, v, pos = R.draw(t, hq, hkv, d, torch.bfloat16, 12)
    codes, scale = _pools(5, hkv, d, 12)
    slots = R.run_slots([(2, 45)], 5, 12)
    rope = B.Rope(R.table(997, d).cuda())
    qo = torch.zeros_like(q).cuda()
    want = _append(k, v, codes, scale, slots, q=q.cuda(), q_out=qo, positions=pos.cuda(), rope=rope)
    qkv = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1).cuda()
    qs, ks, vs = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    c, s, sl, ps = codes.cuda(), scale.cuda(), slots.cuda(), pos.cuda()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        B.kv_append_fp8_block(ks, vs, c[0], c[1], s[0], s[1], sl, q=qs, q_out=qs, positions=ps, rope=rope)
    torch.cuda.synchronize()
    assert torch.equal(c.cpu(), codes)               # captured, not run
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.cpu(), want[0]) and torch.equal(s.cpu(), want[1])
    assert torch.equal(qs, qo) and torch.equal(ks.cpu(), k)


def test_no_tokens():
    codes, scale = _pools(2, 2, 128, 13)
    k = torch.zeros(0, 2, 128, dtype=torch.bfloat16)
    c, s = _append(k, k, codes, scale, torch.zeros(0, dtype=torch.int64))
    assert torch.equal(c, codes) and torch.equal(s, scale)
