"""Refusals of the operators for long contexts in the 4-bit cache: everything
that is checked on the host fails before any CUDA call, so this runs without a
GPU."""
import pytest
import torch

from tests.test_kv4_host import A, _vary, lib  # noqa: F401

GRID = [({"T": -1}, 1), ({"Hkv": 0}, 1), ({"D": 96}, 2), ({"D": 512}, 2), ({"bs": 8}, 2), ({"bs": 48}, 2), ({"nb": 0}, 1),
        ({"nb": 1 << 31}, 1), ({"T": (1 << 24) + 1}, 2), ({"T": 0}, 0)]
ROWS = [({"q": None}, 1), ({"q": A + 8}, 3), ({"sq": 4088}, 1), ({"sq": 4100}, 1), ({"sq": (1 << 30) + 8}, 1),
        ({"Hq": 12}, 1), ({"Hq": 2048, "sq": 1 << 20}, 2), ({"Hq": 0}, 1)]


def test_bounds_refusals(lib):
    def call(cache, nb, bs, slots, bounds, T, Hkv, D):
        return lib.kv4_bounds(cache, nb, bs, slots, bounds, T, Hkv, D, None)
    good = dict(cache=A, nb=9, bs=16, slots=A, bounds=A, T=3, Hkv=8, D=256)
    _vary(call, good, GRID + [({"cache": None}, 1), ({"slots": None}, 1), ({"bounds": None}, 1), ({"cache": A + 8}, 3),
                              ({"slots": A + 4}, 3), ({"bounds": A + 8}, 3), ({"Hkv": 2000}, 2)])


def test_select_refusals(lib):
    def call(q, sq, bounds, nb, bs, table, maxb, seq, cu, B, T, Hq, Hkv, D, top, first, recent, tables, lens):
        return lib.kv4_select(q, sq, bounds, nb, bs, table, maxb, seq, cu, B, T, Hq, Hkv, D, top, first, recent, tables,
                              lens, None)
    good = dict(q=A, sq=4096, bounds=A, nb=9, bs=16, table=A, maxb=20, seq=A, cu=A, B=3, T=3, Hq=16, Hkv=8, D=256, top=8,
                first=1, recent=2, tables=A, lens=A)
    _vary(call, good, GRID + ROWS + [
        ({"bounds": None}, 1), ({"bounds": A + 8}, 3), ({"table": None}, 1), ({"seq": None}, 1), ({"cu": A + 2}, 3),
        ({"tables": None}, 1), ({"lens": None}, 1), ({"lens": A + 1}, 3), ({"tables": A + 2}, 3), ({"top": 0}, 1),
        ({"top": 2}, 1), ({"first": -1}, 1), ({"recent": 0}, 1), ({"first": 0x7fffffff}, 1), ({"top": 32769}, 2),
        ({"maxb": 32769}, 2), ({"maxb": 0}, 1), ({"maxb": 1 << 62}, 2), ({"B": 0}, 1), ({"B": 4097}, 2)])
    assert call(**dict(good, Hq=264, sq=1 << 18)) == 2      # 33 query heads to a key head
    # more CTAs than a grid has
    assert call(**dict(good, T=1 << 24, Hq=1024, Hkv=1024, sq=1 << 18)) == 2


def test_sparse_attention_refusals(lib):
    need = lib.kv4_attention_scratch_bytes(16, 8, 256)

    def call(q, sq, cache, nb, bs, tables, top, lens, out, T, Hq, Hkv, D, scale, scratch, bytes):
        return lib.kv4_sparse_attention(q, sq, cache, nb, bs, tables, top, lens, out, T, Hq, Hkv, D, scale, scratch, bytes,
                                        None)
    good = dict(q=A, sq=4096, cache=A, nb=9, bs=16, tables=A, top=4, lens=A, out=A, T=3, Hq=16, Hkv=8, D=256, scale=0.1,
                scratch=A, bytes=need)
    _vary(call, good, GRID + ROWS + [
        ({"cache": None}, 1), ({"cache": A + 8}, 3), ({"tables": None}, 1), ({"tables": A + 2}, 3), ({"lens": None}, 1),
        ({"out": None}, 1), ({"out": A + 8}, 3), ({"scratch": None}, 1), ({"scratch": A + 128}, 3), ({"bytes": need - 1}, 1),
        ({"top": 0}, 1), ({"top": 1 << 30}, 2), ({"scale": float("nan")}, 1), ({"scale": float("inf")}, 1)])


def test_prefix_attention_refusals(lib):
    size = lib.kv4_prefix_attention_scratch_bytes
    need = size(3, 3, 2, 16, 8, 256)
    assert need > lib.kv4_attention_scratch_bytes(16, 8, 256) and need % 256 == 0
    for bad in ((-1, 3, 2, 16, 8, 256), (3, 0, 1, 16, 8, 256), (3, 4097, 2, 16, 8, 256), (3, 3, 0, 16, 8, 256),
                (3, 3, 4, 16, 8, 256), (3, 3, 2, 0, 8, 256), (3, 3, 2, 16, 0, 256), (3, 3, 2, 12, 8, 256),
                (3, 3, 2, 16, 8, 96), ((1 << 24) + 1, 3, 2, 16, 8, 256), (3, 3, 2, 2048, 8, 256)):
        assert size(*bad) == 0, bad
    # a scratch for more serves for less
    for T, B, N in ((4, 3, 2), (3, 4, 2), (3, 3, 3), (50, 40, 9)):
        assert size(T, B, N, 16, 8, 256) >= need

    def call(q, sq, cache, nb, bs, table, maxb, seq, cu, B, lens, groups, N, out, T, Hq, Hkv, D, scale, most, widest, scratch,
             bytes):
        return lib.kv4_prefix_attention(q, sq, cache, nb, bs, table, maxb, seq, cu, B, lens, groups, N, out, T, Hq, Hkv, D,
                                        scale, most, widest, scratch, bytes, None)
    good = dict(q=A, sq=4096, cache=A, nb=9, bs=16, table=A, maxb=4, seq=A, cu=A, B=3, lens=A, groups=A, N=2, out=A, T=3,
                Hq=16, Hkv=8, D=256, scale=0.1, most=1, widest=2, scratch=A, bytes=need)
    _vary(call, good, GRID + ROWS + [
        ({"cache": None}, 1), ({"cache": A + 8}, 3), ({"table": None}, 1), ({"seq": None}, 1), ({"cu": A + 2}, 3),
        ({"lens": None}, 1), ({"groups": None}, 1), ({"groups": A + 2}, 3), ({"out": A + 2}, 3), ({"scratch": None}, 1),
        ({"scratch": A + 128}, 3), ({"bytes": need - 1}, 1), ({"most": 0}, 1), ({"widest": 0}, 1), ({"N": 0}, 1),
        ({"N": 4}, 1), ({"B": 4097}, 2), ({"maxb": 1 << 30}, 2), ({"scale": float("inf")}, 1)])


def test_binding_refuses_shapes_types_and_places():
    import gemm_w4a16_gemv_gb300 as w4
    q, cache = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 1, 18 * 64, dtype=torch.uint8)
    i32 = dict(dtype=torch.int32)
    table, lens, cu = torch.zeros(2, 3, **i32), torch.ones(2, **i32), torch.arange(3, **i32)
    bounds, scratch = torch.zeros(3, 2, 144, dtype=torch.uint8), torch.zeros(64, dtype=torch.uint8)
    groups, slots = torch.tensor([0, 2], **i32), torch.zeros(2, dtype=torch.int64)
    one = torch.ones(1, **i32)
    with pytest.raises(ValueError, match="expected CUDA"):
        w4.kv4_bounds(cache, slots, bounds)
    with pytest.raises(TypeError, match="slots"):
        w4.kv4_bounds(cache, slots.int(), bounds)
    with pytest.raises(ValueError, match="bounds"):
        w4.kv4_bounds(cache, slots, bounds[:2])
    with pytest.raises(ValueError, match="expected CUDA"):
        w4.kv4_select(q, bounds, table, lens, cu, 16, 3)
    with pytest.raises(ValueError, match="bounds"):
        w4.kv4_select(q, bounds[..., :100], table, lens, cu, 16, 3)
    with pytest.raises(ValueError, match="top"):
        w4.kv4_select(q, bounds, table, lens, cu, 16, 0)
    with pytest.raises(ValueError, match="block_table"):
        w4.kv4_select(q, bounds, table[:1], lens, cu, 16, 3)
    with pytest.raises(TypeError, match="lens"):
        w4.kv4_select(q, bounds, table, lens, cu, 16, 3, lens=lens.long())
    with pytest.raises(ValueError, match="cu_new"):
        w4.kv4_select(q, bounds, table, lens, cu[:2], 16, 3)
    tables = torch.zeros(2, 2, 3, **i32)
    with pytest.raises(ValueError, match="expected CUDA"):
        w4.kv4_sparse_attention(q, cache, tables, lens, scratch)
    with pytest.raises(ValueError, match="tables"):
        w4.kv4_sparse_attention(q, cache, tables[:, :1], lens, scratch)
    with pytest.raises(ValueError, match="heads of 64"):
        w4.kv4_sparse_attention(q, torch.zeros(3, 2, 1, 18 * 128, dtype=torch.uint8), tables, lens, scratch)
    with pytest.raises(TypeError, match="scratch"):
        w4.kv4_sparse_attention(q, cache, tables, lens, scratch.float())
    with pytest.raises(ValueError, match="expected CUDA"):
        w4.kv4_prefix_attention(q, cache, table, lens, cu, one, groups, scratch)
    with pytest.raises(ValueError, match="cu_groups"):
        w4.kv4_prefix_attention(q, cache, table, lens, cu, one, lens[:1], scratch)
    with pytest.raises(TypeError, match="prefix_lens"):
        w4.kv4_prefix_attention(q, cache, table, lens, cu, one.long(), groups, scratch)
    with pytest.raises(ValueError, match="heads and elements"):
        w4.kv4_prefix_attention(q.transpose(0, 1).contiguous().transpose(0, 1), cache, table, lens, cu, one, groups, scratch)
