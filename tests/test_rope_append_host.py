"""The rotating and block-scaled appends without a GPU: what the oracle says
about small cases worked by hand, what the library refuses on the host, what
the binding refuses, and the debug mode's checks."""
import ctypes

import numpy as np
import pytest
import torch

import rope_cases as R
from oracle import fp8 as F
from oracle import fp8_block as FB
from oracle import rope as O
from paged_kv_cache_104_gb300 import binding as B
from paged_kv_cache_104_gb300 import validate as V


# ----------------------------------------------------------------- oracle pins
def test_oracle_rotation_by_hand():
    cs = np.array([[1.0, 1.0, 0.0, 0.0], [0.0, -1.0, 1.0, 0.0]])   # position 1: 90 and 180 degrees
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    assert O.rotate(x, cs, [[0]]).tolist() == x.tolist()
    assert O.rotate(x, cs, [[1]])[0, 0].tolist() == [-3.0, -2.0, 1.0, -4.0, 5.0]
    assert O.rotate(x, cs, [[1]], interleaved=True)[0, 0].tolist() == [-2.0, 1.0, -3.0, -4.0, 5.0]
    assert O.rotate(x, cs, [[0], [1]], pair_axis=[0, 1])[0, 0].tolist() == [1.0, -2.0, 3.0, -4.0, 5.0]


def test_oracle_rotation_keeps_lengths_and_relative_angles():
    cs = R.table(50, 32).numpy()
    x = np.random.default_rng(0).standard_normal((1, 1, 32))
    y = np.random.default_rng(1).standard_normal((1, 1, 32))
    assert np.isclose(np.linalg.norm(O.rotate(x, cs, [[17]])), np.linalg.norm(x), rtol=1e-6)
    near = [float((O.rotate(x, cs, [[p]]) * O.rotate(y, cs, [[p + 5]])).sum()) for p in (0, 9, 31)]
    assert np.allclose(near, near[0], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (224.1, 0), (1.0, -8), (1.75, -8),
                                    (1.76, -7), (0.0, -126), (1e-45, -126), (3e38, 119), (448.0 * 2.0 ** 119, 119)])
def test_oracle_exponent(amax, e):
    assert FB.exponent(amax) == e


def test_oracle_continues_and_restarts_blocks():
    pool, scale = np.zeros((2, 1, 16, 4), np.uint8), np.zeros((2, 1), np.uint8)
    FB.append_pool(np.full((1, 1, 4), 448.0), pool, scale, [16])          # block 1, row 0
    assert scale[1, 0] == 127 and F.decode(pool[1, 0, 0]).tolist() == [448.0] * 4
    FB.append_pool(np.full((1, 1, 4), 1000.0), pool, scale, [17])         # the scale grows by 4
    assert scale[1, 0] == 129
    assert FB.dequantize(pool, scale)[1, 0, :2].tolist() == [[448.0] * 4, [1024.0] * 4]
    FB.append_pool(np.full((1, 1, 4), 1.0), pool, scale, [18])            # and never shrinks
    assert scale[1, 0] == 129 and FB.dequantize(pool, scale)[1, 0, 2].tolist() == [1.0] * 4
    FB.append_pool(np.full((1, 1, 4), 1.0), pool, scale, [16])            # but with a new block
    assert scale[1, 0] == 127 - 8
    assert FB.runs([5, 6, 7, -1, 8, 15, 16, 17]) == [[0, 3], [4, 1], [5, 1], [6, 2]]


# -------------------------------------------------------------- host refusals
def _args(**kw):
    a = dict(q_out=0x1000, q=0x2000, k_new=0x3000, v_new=0x4000, k_cache=0x5000, v_cache=0x6000, k_scale=0x7000,
             v_scale=0x8000, slot_mapping=0x9000, num_tokens=4, num_blocks=8, q_out_stride=0, q_stride=0,
             k_stride=0, v_stride=0, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, dtype=1,
             cos_sin=0xa000, num_positions=64, positions=0xb000, num_axes=1, rot_dim=128, interleaved=0,
             pair_axis=None)
    a.update(kw)
    return B.RopeAppendArgs(**a)


BAD = [
    (dict(dtype=9), 2), (dict(num_tokens=-1), 1), (dict(num_blocks=0), 1), (dict(num_kv_heads=0), 1),
    (dict(head_dim=0), 1), (dict(block_size=8), 5), (dict(num_tokens=1 << 31), 3),
    (dict(k_new=None), 1), (dict(v_new=None), 1), (dict(k_cache=None), 1), (dict(v_cache=None), 1),
    (dict(slot_mapping=None), 1), (dict(slot_mapping=0x9004), 1), (dict(q=0x2008), 1), (dict(k_cache=0x5002), 1),
    (dict(cos_sin=0xa004), 1), (dict(positions=None), 1), (dict(positions=0xb002), 1), (dict(num_positions=0), 1),
    (dict(num_axes=0), 1), (dict(num_axes=5), 1), (dict(num_axes=2), 1),          # two axes need pair_axis
    (dict(rot_dim=0), 1), (dict(rot_dim=63), 1), (dict(rot_dim=130), 1),
    (dict(q=None), 1), (dict(q_out=None), 1), (dict(num_q_heads=0), 1),
    (dict(q_stride=1000), 1), (dict(k_stride=8), 1), (dict(v_stride=260), 1), (dict(q_out_stride=-1024), 1),
    (dict(q_out=0x2000, q_stride=2048), 1),                                        # in place, two strides
]


@pytest.mark.parametrize("kw,status", BAD + [(dict(head_dim=100, rot_dim=100), 5), (dict(head_dim=520), 5),
                                             (dict(head_dim=512, rot_dim=258), 5), (dict(cos_sin=None), 1)])
def test_rope_append_refuses(kw, status):
    assert B.load().pkv_kv_append_rope(ctypes.byref(_args(**kw)), None) == status


@pytest.mark.parametrize("kw,status", BAD + [(dict(dtype=0), 5), (dict(k_scale=None), 1), (dict(v_scale=None), 1),
                                             (dict(cos_sin=None), 1), (dict(head_dim=136), 5),
                                             (dict(head_dim=256), 5), (dict(head_dim=120, rot_dim=64), 5),
                                             (dict(rot_dim=72), 5), (dict(rot_dim=20), 5)])
def test_block_append_refuses(kw, status):
    assert B.load().pkv_kv_append_fp8_block(ctypes.byref(_args(**kw)), None) == status


def test_axes_beyond_their_number_and_null_args():
    ax = (ctypes.c_uint8 * 64)(*([0] * 63 + [2]))
    a = _args(num_axes=2, pair_axis=ctypes.addressof(ax))
    assert B.load().pkv_kv_append_rope(ctypes.byref(a), None) == 1
    assert B.load().pkv_kv_append_rope(None, None) == 1
    assert B.load().pkv_kv_append_fp8_block(None, None) == 1


def test_no_tokens_is_a_no_op():
    empty = dict(num_tokens=0, k_new=None, v_new=None, q=None, q_out=None)
    assert B.load().pkv_kv_append_rope(ctypes.byref(_args(**empty)), None) == 0
    assert B.load().pkv_kv_append_fp8_block(ctypes.byref(_args(**empty)), None) == 0


def _tensors(t=4, dtype=torch.bfloat16, pool=torch.bfloat16):
    q, k, v, pos = R.draw(t, 8, 2, 128, dtype, 1)
    kc, vc = torch.zeros(4, 2, 16, 128, dtype=pool), torch.zeros(4, 2, 16, 128, dtype=pool)
    return q, k, v, kc, vc, R.scattered_slots(t, 4, 1), pos


def test_binding_refuses_before_the_library():
    q, k, v, kc, vc, slots, pos = _tensors()
    rope = B.Rope(R.table(64, 128))
    with pytest.raises(B.PagedKVError, match="no rope"):
        B.kv_append_rope(q, q, k, v, kc, vc, slots, pos, None)
    with pytest.raises(TypeError):
        B.kv_append_rope(q, q, k, v, kc.half(), vc.half(), slots, pos, rope)
    sc = torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(B.PagedKVError, match="the pools are torch.bfloat16"):
        B.kv_append_fp8_block(k, v, kc, vc, sc, sc, slots)
    k8 = kc.to(torch.uint8)
    with pytest.raises(B.PagedKVError, match="queries need a rope"):
        B.kv_append_fp8_block(k, v, k8, k8, sc, sc, slots, q=q, q_out=q)


def test_binding_refuses_tensors_off_the_device(monkeypatch):
    q, k, v, kc, vc, slots, pos = _tensors()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(B.PagedKVError, match="current CUDA device"):
        B.kv_append_rope(q, q, k, v, kc, vc, slots, pos, B.Rope(R.table(64, 128)))


ROPE_BAD = {
    "v_cache": lambda a: a["vc"].float(), "vc": lambda a: a["vc"][:3], "slots": lambda a: a["slots"].int(),
    "slots2": lambda a: a["slots"][:, None], "k": lambda a: a["k"].float(), "k2": lambda a: a["k"][:3],
    "v": lambda a: a["v"].transpose(1, 2), "v2": lambda a: a["v"].expand(4, 2, 128)[:, :, ::2],
    "q": lambda a: a["q"][:, :, :64], "q2": lambda a: None, "qo": lambda a: a["qo"][:3], "qo2": lambda a: None,
    "pos": lambda a: a["pos"].long(), "pos2": lambda a: a["pos"][:, :3], "pos3": lambda a: None,
    "pos4": lambda a: a["pos"].expand(2, 4), "kc": lambda a: a["kc"].transpose(0, 1),
}


@pytest.mark.parametrize("which", sorted(ROPE_BAD))
def test_binding_names_the_tensor(which, monkeypatch):
    """Shape, type and layout refusals, with the tensors' device left aside."""
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)   # CPU tensors answer get_device() with -1
    q, k, v, kc, vc, slots, pos = _tensors()
    a = dict(qo=q.clone(), q=q, k=k, v=v, kc=kc, vc=vc, slots=slots, pos=pos)
    key = {"v_cache": "vc"}.get(which, which.rstrip("234"))
    a[key] = ROPE_BAD[which](a)
    name = {"kc": "k_cache", "vc": "v_cache", "slots": "slot_mapping", "k": "k_new", "v": "v_new", "q": "q",
            "qo": "q_out|q is", "pos": "positions"}[key]
    with pytest.raises(B.PagedKVError, match=name):
        B.kv_append_rope(a["qo"], a["q"], a["k"], a["v"], a["kc"], a["vc"], a["slots"], a["pos"],
                         B.Rope(R.table(64, 128)))


@pytest.mark.parametrize("ks,vs,name", [(lambda s: s[:3], lambda s: s, "k_scale"), (lambda s: s, lambda s: s.float(), "v_scale"),
                                        (lambda s: s, lambda s: s.T.contiguous().T, "v_scale")])
def test_binding_names_the_scale(ks, vs, name, monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    _, k, v, kc, _, slots, _ = _tensors()
    k8, sc = kc.to(torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(B.PagedKVError, match=name):
        B.kv_append_fp8_block(k, v, k8, k8.clone(), ks(sc), vs(sc), slots)


@pytest.mark.parametrize("make", [
    lambda: B.Rope(R.table(8, 16).double()), lambda: B.Rope(R.table(8, 16).T), lambda: B.Rope(torch.zeros(8)),
    lambda: B.Rope(R.table(8, 16), pair_axis=[0] * 7), lambda: B.Rope(R.table(8, 16), pair_axis=[0] * 7 + [4]),
    lambda: B.Rope(R.table(8, 16), pair_axis=[0] * 7 + [-1])])
def test_rope_refuses(make):
    with pytest.raises(B.PagedKVError):
        make()


# ------------------------------------------------------------------ debug mode
def test_run_and_position_checks():
    V.check_runs(torch.tensor([5, 6, 7, -1, 32, 33]), 4, 16)
    V.check_runs(R.run_slots([(3, 40), (0, 1), (15, 2)], 8, 1), 8, 16)
    for slots in ([5, 7], [6, 5], [5, -1, 6], [5, 40, 6], [0, 1, 2, 15]):
        with pytest.raises(V.ValidationError, match="returns to block"):
            V.check_runs(torch.tensor(slots), 4, 16)
    with pytest.raises(V.ValidationError, match="more than once"):
        V.check_runs(torch.tensor([5, 5]), 4, 16)
    slots = torch.tensor([1, -1, 2])
    V.check_positions(torch.tensor([[0, 99, 9], [3, -1, 0]], dtype=torch.int32), slots, 10)
    with pytest.raises(V.ValidationError, match="position 10 of token 2"):
        V.check_positions(torch.tensor([0, 0, 10], dtype=torch.int32), slots, 10)


def test_debug_mode_names_the_entry(monkeypatch):
    monkeypatch.setattr(B, "_device_of", lambda fn, t: -1)
    q, k, v, kc, vc, slots, pos = _tensors()
    rope = B.Rope(R.table(64, 128))
    sc = torch.zeros(4, 2, dtype=torch.uint8)
    k8 = kc.to(torch.uint8)
    B.set_debug(True)
    try:
        with pytest.raises(B.PagedKVError, match="outside the pool"):
            B.kv_append_rope(q, q, k, v, kc, vc, torch.tensor([0, 1, 2, 64]), pos % 64, rope)
        with pytest.raises(B.PagedKVError, match="position"):
            B.kv_append_rope(q, q, k, v, kc, vc, torch.tensor([0, 1, 2, 3]), pos + 64, rope)
        with pytest.raises(B.PagedKVError, match="returns to block"):
            B.kv_append_fp8_block(k, v, k8, k8, sc, sc, torch.tensor([0, 1, 3, 2]))
        with pytest.raises(B.PagedKVError, match="needs positions"):
            B.kv_append_rope(q, q, k, v, kc, vc, slots, None, rope)
        with pytest.raises(B.PagedKVError, match="positions is"):
            B.kv_append_rope(q, q, k, v, kc, vc, slots, pos[:, :3].contiguous(), rope)
    finally:
        B.set_debug(False)


def test_packed_arguments_are_the_structure():
    values = list(range(1, 28))
    assert bytes(B.RopeAppendArgs(*values)) == B._ROPE_APPEND.pack(*values)
