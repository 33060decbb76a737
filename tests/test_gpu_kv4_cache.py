"""Block tables and slot maps, head norms with rotation, and the 4-bit cache's
write and read-back against plain references."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests.gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


def _i32(torch, v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _plan_ref(ctx, new, table, free, bs, cap):
    table = table.copy()
    pos, slots = np.full(cap, -1), np.full(cap, -1, np.int64)
    cu, taken, t = [0], 0, 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        held, want = -(-c // bs), -(-(c + n) // bs)
        for i in range(held, want):
            table[b, i] = free[taken] if taken < len(free) else -1
            taken += 1
        for i in range(n):
            if t < cap:
                pos[t] = c + i
                blk = table[b, (c + i) // bs]
                slots[t] = blk * bs + (c + i) % bs if blk >= 0 else -1
            t += 1
        cu.append(min(t, cap))
    return np.array(ctx) + np.array(new), cu, pos, slots, taken, table


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("case", ["one", "decode", "mixed", "idle", "many", "padded"])
def test_plan(bs, case):
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(bs)
    B = {"one": 1, "many": 3001}.get(case, 37)
    ctx = rng.integers(0, 4 * bs, B)
    ctx[0] = 0
    new = {"one": np.array([1]), "decode": np.ones(B, int), "many": rng.integers(0, 4, B)}.get(case)
    if new is None:
        new = rng.integers(0, 3 * bs, B)
    if case == "idle":
        new[rng.random(B) < 0.5] = 0
        new[-5:] = 0
    width = int(-(-(ctx + new).max() // bs)) + 2
    held = -(-ctx // bs)
    ids = rng.permutation(int(held.sum()) + int((-(-(ctx + new) // bs) - held).sum()) + 5)
    table = np.full((B, width), -7)
    at = 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    free = ids[at:]
    total = int(new.sum())
    cap = total + 100 if case == "padded" else total
    dt, df = _i32(torch, table), _i32(torch, free)
    p = w4.kv4_plan(_i32(torch, ctx), _i32(torch, new), dt, df, bs, num_tokens=cap)
    torch.cuda.synchronize()
    ends, cu, pos, slots, taken, want = _plan_ref(ctx, new, table, free, bs, cap)
    assert np.array_equal(p.seq_lens.cpu(), ends) and np.array_equal(p.cu_new.cpu(), cu)
    assert np.array_equal(p.positions.cpu(), pos) and np.array_equal(p.slots.cpu(), slots)
    assert int(p.taken) == taken and np.array_equal(dt.cpu(), want)
    assert w4.w4a16_check_device_error() == 0


def test_plan_short_of_blocks_and_out_of_range_lengths():
    torch, w4 = cuda_or_skip()
    ctx, new = [16, 3, 0], [1, 40, 20]
    table = np.full((3, 4), -1)
    table[0, 0], table[1, 0] = 9, 8
    dt = _i32(torch, table)
    p = w4.kv4_plan(_i32(torch, ctx), _i32(torch, new), dt, _i32(torch, [5, 6]), 16, num_tokens=61)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    ends, cu, pos, slots, taken, want = _plan_ref(ctx, new, table, [5, 6], 16, 61)
    assert int(p.taken) == taken == 5 and np.array_equal(dt.cpu(), want)
    assert np.array_equal(p.slots.cpu(), slots) and np.array_equal(p.positions.cpu(), pos)
    # a negative length counts as none, a row that is too short keeps what fits
    dt = _i32(torch, np.full((2, 2), -1))
    p = w4.kv4_plan(_i32(torch, [-4, 30]), _i32(torch, [1, 5]), dt, _i32(torch, [3, 4, 5]), 16, num_tokens=6)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    assert p.slots.tolist()[0] == 3 * 16 and p.slots.tolist()[3:] == [-1, -1, -1]
    # more tokens than there is room for
    p = w4.kv4_plan(_i32(torch, [0]), _i32(torch, [9]), _i32(torch, [[-1]]), _i32(torch, [0]), 16, num_tokens=4)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    assert p.cu_new.tolist() == [0, 4] and p.slots.tolist() == [0, 1, 2, 3]
    assert w4.w4a16_check_device_error() == 0


def _rope_table(P, rot):
    a = np.arange(P)[:, None] * 10000.0 ** (-2 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def _qkv(torch, T, Hq, Hkv, D, seed, pad=0):
    """q, k, v as slices of one fused row, on the device and as float64."""
    g = torch.Generator().manual_seed(seed)
    row = (torch.randn(T, (Hq + 2 * Hkv) * D + pad, generator=g) * 2).to(torch.bfloat16)
    d = row.cuda()
    cut = [0, Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D]
    dev = [d[:, a:b].unflatten(1, (-1, D)) if b > a else d[:, a:b].reshape(T, 0, D) for a, b in zip(cut, cut[1:])]
    host = [row[:, a:b].double().numpy().reshape(T, -1, D) for a, b in zip(cut, cut[1:])]
    return dev, host


ROPE = [  # T, Hq, Hkv, D, rot, interleaved, norm
    (1, 16, 8, 256, 256, False, True), (3, 16, 8, 256, 128, False, True), (37, 7, 1, 128, 128, True, True),
    (5, 4, 4, 64, 64, False, True), (5, 4, 4, 64, 16, True, True), (2, 3, 5, 128, 48, False, True),
    (9, 1, 1, 256, 240, True, False), (129, 16, 8, 256, 256, True, True), (4, 8, 2, 128, 0, False, True),
    (1000, 5, 2, 64, 32, False, False), (4, 2, 1, 64, 48, False, True), (300, 64, 4, 128, 112, False, True)]


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm", ROPE)
def test_qk_norm_rope(T, Hq, Hkv, D, rot, inter, norm):
    # one BF16 rounding (2^-8 of the result at most: 8 significant bits) and binary32 steps: the sum of D
    # squares, rsqrt, two products and the rotation, together below 2^-17 of
    # the rotated pair's magnitude (D / 2 + 10 roundings of 2^-24)
    torch, w4 = cuda_or_skip()
    (q, k, _), (hq, hk, _) = _qkv(torch, T, Hq, Hkv, D, T + D, pad=8)
    rng = np.random.default_rng(rot)
    P = 77
    cs = _rope_table(P, rot) if rot else None
    pos = rng.integers(0, P, T)
    wq, wk = (ref.bf16(rng.normal(1, 0.3, D)) for _ in range(2))
    dw = lambda w: torch.tensor(w, dtype=torch.bfloat16, device="cuda") if norm else None
    qo, ko = w4.w4a16_qk_norm_rope(q, k, dw(wq), dw(wk), torch.tensor(cs, device="cuda") if rot else None,
                                   _i32(torch, pos) if rot else None, eps=1e-5, weight_offset=0.5, interleaved=inter)
    torch.cuda.synchronize()
    for out, x, w in ((qo, hq, wq), (ko, hk, wk)):
        want, size = ref.norm_rope(x, w if norm else None, cs, pos, 1e-5, 0.5, inter)
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * size + 1e-30)
    assert w4.w4a16_check_device_error() == 0


def test_qk_norm_rope_padding_and_bad_positions():
    torch, w4 = cuda_or_skip()
    (q, k, _), _ = _qkv(torch, 4, 2, 1, 64, 1)
    cs = torch.tensor(_rope_table(10, 64), device="cuda")
    full, _ = w4.w4a16_qk_norm_rope(q, k, None, None, cs, _i32(torch, [0, 1, 2, 9]))
    qo, ko = w4.w4a16_qk_norm_rope(q, k, None, None, cs, _i32(torch, [0, -1, 2, 9]))
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 0     # a padding row is no error
    assert not qo[1].any() and not ko[1].any()
    assert torch.equal(qo[[0, 2, 3]], full[[0, 2, 3]])
    qo, ko = w4.w4a16_qk_norm_rope(q, k, None, None, cs, _i32(torch, [0, 10, 2, 9]))
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    assert not qo[1].any() and torch.equal(qo[[0, 2, 3]], full[[0, 2, 3]])


def test_qk_norm_rope_in_place_and_zero_rows():
    torch, w4 = cuda_or_skip()
    (q, k, _), _ = _qkv(torch, 5, 4, 2, 128, 3)
    q, k = q.contiguous(), k.contiguous()
    q[2] = 0   # the norm of zeros stays zero
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    qo, ko = w4.w4a16_qk_norm_rope(q, k, w, w, None, None)
    w4.w4a16_qk_norm_rope(q, k, w, w, None, None, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and torch.equal(k, ko) and not q[2].any()
    e = w4.w4a16_qk_norm_rope(q[:0], k[:0], w, w, None, None)
    assert e[0].shape == (0, 4, 128)


@pytest.mark.parametrize("T,Hkv,D,bs", [(1, 8, 256, 16), (50, 3, 128, 32), (17, 1, 64, 64), (33, 2, 256, 128), (300, 2, 64, 256)])
def test_append_is_the_formula_bit_for_bit(T, Hkv, D, bs):
    torch, w4 = cuda_or_skip()
    (_, k, v), (_, hk, hv) = _qkv(torch, T, 1, Hkv, D, T * D)
    # groups at the edges of the formula: all equal, all of one sign, zeros,
    # tiny, huge and a tie of the extremes
    for t, f in enumerate([lambda x: x * 0 + 3, np.abs, lambda x: -np.abs(x), lambda x: x * 0, lambda x: x * 2.0 ** -30,
                           lambda x: x * 2.0 ** 30]):
        if t < T:
            for d, h in ((k, hk), (v, hv)):
                h[t] = ref.bf16(f(h[t]))
                d[t] = torch.tensor(h[t], device="cuda").to(torch.bfloat16)
    rng = np.random.default_rng(T)
    blocks = -(-T // bs) + 3
    slots = rng.permutation(blocks * bs)[:T]
    if T > 10:
        slots[7] = -1
    cache = w4.kv4_cache(blocks, Hkv, bs, D)
    cache.fill_(0xA5)
    want = ref.Cache(blocks, Hkv, bs, D, 0xA5)
    ds = torch.tensor(slots, device="cuda")
    w4.kv4_append(k, v, cache, ds)
    gk, gv = w4.kv4_gather(cache, ds)
    torch.cuda.synchronize()
    want.append(hk, hv, slots)
    assert np.array_equal(cache.cpu().numpy(), want.raw)     # and nothing outside the slots
    for part, got in ((0, gk), (1, gv)):
        got = got.double().cpu().numpy()
        for t in range(T):
            for h in range(Hkv):
                w = ref.bf16(want.values(part, int(slots[t]), h)) if slots[t] >= 0 else 0
                assert np.array_equal(got[t, h], np.broadcast_to(w, D))
    assert w4.w4a16_check_device_error() == 0


def test_append_of_nan_and_infinite_values_stays_in_its_group():
    torch, w4 = cuda_or_skip()
    (_, k, v), _ = _qkv(torch, 2, 1, 1, 128, 5)
    plain = w4.kv4_cache(1, 1, 16, 128)
    w4.kv4_append(k, v, plain, torch.arange(2, device="cuda"))
    a, _ = w4.kv4_gather(plain, torch.arange(2, device="cuda"))
    k[0, 0, 5], k[0, 0, 9] = float("nan"), float("inf")
    cache = w4.kv4_cache(1, 1, 16, 128)
    w4.kv4_append(k, v, cache, torch.arange(2, device="cuda"))
    b, _ = w4.kv4_gather(cache, torch.arange(2, device="cuda"))
    torch.cuda.synchronize()
    assert torch.isfinite(b.float()).all()
    assert torch.equal(a[0, 0, 64:], b[0, 0, 64:]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm", ROPE)
def test_fused_append_equals_norm_rope_then_append(T, Hq, Hkv, D, rot, inter, norm):
    torch, w4 = cuda_or_skip()
    (q, k, v), _ = _qkv(torch, T, Hq, Hkv, D, 2 * T + D)
    g = torch.Generator().manual_seed(1)
    cs = torch.tensor(_rope_table(50, rot), device="cuda") if rot else None
    pos = torch.randint(0, 50, (T,), generator=g, dtype=torch.int32).cuda() if rot else None
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() if norm else None for _ in range(2))
    slots = torch.randperm(T + 40, generator=g)[:T].cuda()
    a, b = (w4.kv4_cache((T + 40) // 16 + 1, Hkv, 16, D) for _ in range(2))
    q1 = w4.kv4_append(k, v, a, slots, q=q, q_weight=wq, k_weight=wk, cos_sin=cs, positions=pos, interleaved=inter)
    q2, k2 = w4.w4a16_qk_norm_rope(q, k, wq, wk, cs, pos, interleaved=inter)
    w4.kv4_append(k2, v, b, slots)
    torch.cuda.synchronize()
    assert torch.equal(q1, q2) and torch.equal(a, b)
    assert w4.w4a16_check_device_error() == 0


def test_slots_past_the_cache_are_refused_on_the_device():
    torch, w4 = cuda_or_skip()
    (_, k, v), _ = _qkv(torch, 3, 1, 2, 64, 9)
    cache = w4.kv4_cache(2, 2, 16, 64)
    w4.kv4_append(k, v, cache, torch.tensor([1, 32, 1 << 40], device="cuda"))
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    gk, gv = w4.kv4_gather(cache, torch.tensor([1, 32, -5], device="cuda"))
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    assert gk[0].any() and not gk[1:].any() and not gv[1:].any()
    assert w4.w4a16_check_device_error() == 0


def test_cache_offsets_past_32_bits():
    # the last pages of a cache of more than 2^32 bytes
    torch, w4 = cuda_or_skip()
    blocks = (1 << 32) // (8 * 18 * 256) + 20
    cache = torch.empty(blocks, 8, 1, 18 * 256, dtype=torch.uint8, device="cuda")
    (q, k, v), (hq, hk, hv) = _qkv(torch, 32, 16, 8, 256, 4)
    slots = torch.arange(32, device="cuda") + (blocks - 2) * 16
    w4.kv4_append(k, v, cache, slots)
    gk, gv = w4.kv4_gather(cache, slots)
    small = w4.kv4_cache(2, 8, 16, 256)
    w4.kv4_append(k, v, small, slots - (blocks - 2) * 16)
    args = [_i32(torch, [32]), _i32(torch, [0, 32]), w4.kv4_attention_scratch(16, 8, 256)]
    o1 = w4.kv4_attention(q, cache, _i32(torch, [[blocks - 2, blocks - 1]]), *args)
    o2 = w4.kv4_attention(q, small, _i32(torch, [[0, 1]]), *args)
    torch.cuda.synchronize()
    assert torch.equal(cache[blocks - 2:], small) and torch.equal(o1, o2)
    sk, sv = w4.kv4_gather(small, slots - (blocks - 2) * 16)
    assert torch.equal(gk, sk) and torch.equal(gv, sv)
    assert w4.w4a16_check_device_error() == 0
