"""Refusals of the operators around the 4-bit cache: everything that is checked
on the host fails before any CUDA call, so this runs without a GPU."""
import ctypes

import numpy as np
import pytest

from tests import kv4_helpers as ref

A = 1 << 20   # a fake address, aligned; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from gemm_w4a16_gemv_gb300 import build
    import gemm_w4a16_gemv_gb300 as w4
    handle = ctypes.CDLL(build.build())
    for n, (args, res) in w4.SIGNATURES.items():
        getattr(handle, n).argtypes, getattr(handle, n).restype = args, res
    return handle


def _vary(call, good, cases):
    for change, code in cases:
        args = dict(good, **change)
        assert call(**args) == code, (change, code)


def test_plan_refusals(lib):
    def call(ctx, new, B, table, maxb, free, nfree, bs, T, seq, cu, pos, slots, taken):
        return lib.kv4_plan(ctx, new, B, table, maxb, free, nfree, bs, T, seq, cu, pos, slots, taken, None)
    good = dict(ctx=A, new=A, B=4, table=A, maxb=10, free=A, nfree=5, bs=16, T=4, seq=A, cu=A, pos=A, slots=A, taken=A)
    _vary(call, good, [({"ctx": None}, 1), ({"table": None}, 1), ({"taken": None}, 1), ({"free": None}, 1),
                       ({"pos": None}, 1), ({"slots": None}, 1), ({"B": 0}, 1), ({"B": 8193}, 2), ({"T": -1}, 1),
                       ({"T": (1 << 24) + 1}, 2), ({"maxb": 0}, 1), ({"maxb": 1 << 30}, 2), ({"nfree": -1}, 1),
                       ({"bs": 15}, 2), ({"bs": 8}, 2), ({"bs": 48}, 2), ({"bs": 512}, 2), ({"ctx": A + 2}, 3),
                       ({"slots": A + 4}, 3), ({"cu": A + 1}, 3)])


ROPE = dict(q=A, sq=1024, k=A, sk=512, wq=A, wk=A, cs=A, P=100, rot=128, pos=A, T=3, Hq=8, Hkv=4, D=128, eps=1e-6,
            off=0.0, inter=0)


def _rope_cases():
    return [({"q": None}, 1), ({"k": None}, 1), ({"pos": None}, 1), ({"T": -1}, 1), ({"D": 96}, 2), ({"D": 512}, 2),
            ({"sq": 1016}, 1), ({"sk": 515}, 1), ({"sq": (1 << 30) + 8}, 1), ({"rot": 8}, 2), ({"rot": 136}, 2),
            ({"rot": 40}, 2), ({"P": 0}, 1), ({"q": A + 8}, 3), ({"k": A + 2}, 3), ({"wq": A + 4}, 3),
            ({"cs": A + 4}, 3), ({"pos": A + 2}, 3), ({"eps": -1.0}, 1), ({"eps": float("nan")}, 1), ({"Hq": 2000}, 2),
            ({"T": (1 << 24) + 1}, 2), ({"Hkv": -1}, 1)]


def test_norm_rope_refusals(lib):
    def call(q, sq, k, sk, wq, wk, cs, P, rot, pos, T, Hq, Hkv, D, eps, off, inter, qo=A, ko=A):
        return lib.w4a16_qk_norm_rope(q, sq, k, sk, wq, wk, cs, P, rot, pos, qo, ko, T, Hq, Hkv, D, eps, off, inter, None)
    _vary(call, ROPE, _rope_cases() + [({"qo": None}, 1), ({"ko": A + 8}, 3), ({"T": 0}, 0), ({"T": 0, "q": None}, 0),
                                       ({"Hq": 0, "Hkv": 0}, 0)])


def test_append_refusals(lib):
    def call(q, sq, k, sk, wq, wk, cs, P, rot, pos, T, Hq, Hkv, D, eps, off, inter, v=A, sv=512, slots=A, qo=A, cache=A,
             nb=10, bs=16):
        return lib.kv4_append(q, sq, k, sk, v, sv, wq, wk, cs, P, rot, pos, slots, qo, cache, nb, bs, T, Hq, Hkv, D, eps,
                              off, inter, None)
    _vary(call, ROPE, _rope_cases() + [({"v": None}, 1), ({"sv": 504}, 1), ({"slots": None}, 1), ({"slots": A + 4}, 3),
                                       ({"cache": None}, 1), ({"cache": A + 8}, 3), ({"nb": 0}, 1), ({"bs": 20}, 2),
                                       ({"Hkv": 0}, 1), ({"qo": None}, 1), ({"T": 0}, 0)])


def test_gather_refusals(lib):
    def call(cache, nb, bs, slots, k, v, T, H, D):
        return lib.kv4_gather(cache, nb, bs, slots, k, v, T, H, D, None)
    good = dict(cache=A, nb=4, bs=16, slots=A, k=A, v=A, T=3, H=2, D=64)
    _vary(call, good, [({"cache": None}, 1), ({"k": None}, 1), ({"v": A + 2}, 3), ({"slots": A + 4}, 3), ({"T": -1}, 1),
                       ({"T": 0}, 0), ({"H": 0}, 1), ({"D": 80}, 2), ({"bs": 17}, 2), ({"nb": -1}, 1),
                       ({"T": 1 << 24, "H": 1024}, 2)])


def test_attention_refusals(lib):
    need = lib.kv4_attention_scratch_bytes(16, 8, 256)
    assert need > 0 and need % 256 == 0
    assert lib.kv4_attention_scratch_bytes(16, 3, 256) == 0 and lib.kv4_attention_scratch_bytes(16, 8, 100) == 0

    def call(q, sq, cache, nb, bs, table, maxb, seq, cu, B, out, T, Hq, Hkv, D, scale, w, s, mn, scr, sb):
        return lib.kv4_attention(q, sq, cache, nb, bs, table, maxb, seq, cu, B, out, T, Hq, Hkv, D, scale, w, s, mn, scr,
                                 sb, None)
    good = dict(q=A, sq=4096, cache=A, nb=9, bs=16, table=A, maxb=5, seq=A, cu=A, B=2, out=A, T=2, Hq=16, Hkv=8, D=256,
                scale=0.1, w=0, s=0, mn=1, scr=A, sb=need)
    _vary(call, good, [({"q": None}, 1), ({"cache": None}, 1), ({"table": None}, 1), ({"seq": None}, 1),
                       ({"cu": None}, 1), ({"out": None}, 1), ({"scr": None}, 1), ({"sb": need - 1}, 1),
                       ({"scr": A + 128}, 3), ({"q": A + 2}, 3), ({"cache": A + 8}, 3), ({"seq": A + 2}, 3),
                       ({"sq": 4088}, 1), ({"sq": 4097}, 1), ({"Hkv": 3}, 1), ({"Hq": 0}, 1), ({"D": 192}, 2),
                       ({"bs": 24}, 2), ({"B": 0}, 1), ({"B": 9000}, 2), ({"T": -2}, 1), ({"w": -1}, 1), ({"s": -1}, 1),
                       ({"mn": 0}, 1), ({"scale": float("inf")}, 1), ({"scale": float("nan")}, 1), ({"nb": 0}, 1),
                       ({"maxb": 0}, 1), ({"maxb": 1 << 28}, 2), ({"T": 0}, 0)])


def test_sample_refusals(lib):
    def call(x, dt, st, R, V, u, T, k, p, m, out):
        return lib.w4a16_sample(x, dt, st, R, V, u, T, k, p, m, out, None)
    good = dict(x=A, dt=1, st=1000, R=3, V=1000, u=A, T=A, k=A, p=A, m=A, out=A)
    _vary(call, good, [({"x": None}, 1), ({"u": None}, 1), ({"out": None}, 1), ({"dt": 2}, 1), ({"st": 999}, 1),
                       ({"R": -1}, 1), ({"R": 0}, 0), ({"V": 0}, 1), ({"R": (1 << 20) + 1}, 2),
                       ({"V": (1 << 18) + 1, "st": 1 << 19}, 2), ({"x": A + 1}, 3), ({"x": A + 2, "dt": 0}, 3),
                       ({"k": A + 2}, 3), ({"out": A + 1}, 3)])


def test_binding_checks_tensors():
    import torch
    import gemm_w4a16_gemv_gb300 as w4
    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    cache = z(2, 2, 1, 18 * 64, dt=torch.uint8)
    slots = z(3, dt=torch.int64)
    with pytest.raises(ValueError, match="must be \\[3, 2, 64\\]"):
        w4.kv4_append(z(3, 1, 64), z(3, 2, 64), cache, slots)
    with pytest.raises(TypeError, match="slots"):
        w4.kv4_append(z(3, 2, 64), z(3, 2, 64), cache, slots.int())
    with pytest.raises(ValueError, match="contiguous"):
        w4.kv4_append(z(3, 64, 2).transpose(1, 2), z(3, 2, 64), cache, slots)
    with pytest.raises(ValueError, match="cache must be"):
        w4.kv4_gather(z(2, 2, 100, dt=torch.uint8), slots)
    with pytest.raises(ValueError, match="needs positions"):
        w4.w4a16_qk_norm_rope(z(3, 2, 64), z(3, 2, 64), None, None, z(9, 64, dt=torch.float32), None)
    with pytest.raises(ValueError, match="num_tokens"):
        i = z(3, dt=torch.int32)
        w4.kv4_plan(i, i, z(3, 4, dt=torch.int32), i, 16)
    with pytest.raises(TypeError, match="float32 or"):
        w4.w4a16_sample(z(2, 9, dt=torch.float16), z(2, dt=torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        w4.w4a16_sample(z(2, 9), z(2, dt=torch.float32), stream=0)
    with pytest.raises(ValueError, match="multiple of 16"):
        w4.kv4_cache(2, 1, 24, 64)


def test_reference_quantiser_and_layout():
    # the helpers' own pins: a worked group, and write then read of a tile
    x = np.zeros((1, 64))
    x[0, :4] = [-1.5, 0.0, 6.0, 0.75]
    q, s, z = ref.quantise(x)
    assert s[0, 0] == np.float16(0.5) and z[0, 0] == 3
    assert q[0, :4].tolist() == [0, 3, 15, 5] and (q[0, 4:] == 3).all()   # 0.75 / 0.5 = 1.5 rounds to the even 2
    c = ref.Cache(2, 1, 32, 64)
    c.append(x.reshape(1, 1, 64), x.reshape(1, 1, 64) * 2, [37])
    assert c.values(0, 37, 0)[:4].tolist() == [-1.5, 0, 6, 1] and c.values(1, 37, 0)[2] == 12
    assert c.raw[1, 0, 0, (37 % 16) * 32] == 0x30 and (c.raw[0] == 0).all()


def test_reference_attention_against_a_worked_case():
    c = ref.Cache(1, 1, 16, 64)
    one = np.float16(1)
    for j, (kv, vv) in enumerate([(8, 1), (9, 2), (8, 4)]):
        c.put(0, j, 0, np.full(64, kv, np.uint8), [one], [np.float16(8)])
        c.put(1, j, 0, np.full(64, vv, np.uint8), [one], [np.float16(0)])
    q = np.full((1, 1, 64), 1.0)
    table = np.array([[0]])
    out, tol = ref.attention(q, c, table, [3], [0, 1], np.log(2) / 64)
    assert np.allclose(out, (1 + 2 * 2 + 4) / 4) and (tol > 0).all()       # weights 1, 2, 1
    out, _ = ref.attention(q, c, table, [3], [0, 1], np.log(2) / 64, window=1, sinks=1)
    assert np.allclose(out, 2.5)
