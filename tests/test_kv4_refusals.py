"""Further refusals of the operators around the 4-bit cache that are checked on
the host."""
import pytest

from tests.gpu_helpers import cuda_or_skip
from tests.test_kv4_host import A, _vary, lib  # noqa: F401


def test_table_widths_past_64_bits_in_slots(lib):
    # max_blocks * block_size wraps around to a small number
    def plan(maxb, bs):
        return lib.kv4_plan(A, A + 4096, 4, A + (1 << 21), maxb, A + (2 << 21), 5, bs, 4, A + (3 << 21), A + (4 << 21),
                            A + (5 << 21), A + (6 << 21), A + (7 << 21), None)

    def attention(maxb, bs):
        return lib.kv4_attention(A, 4096, A, 9, bs, A, maxb, A, A, 2, A, 2, 16, 8, 256, 0.1, 0, 0, 1, A,
                                 lib.kv4_attention_scratch_bytes(16, 8, 256), None)
    for bs in (16, 64, 256):
        for maxb in ((1 << 64) // bs + 1, (1 << 63) - 1, (1 << 62) + 5, (1 << 31) // bs):
            assert plan(maxb, bs) == 2 and attention(maxb, bs) == 2, (maxb, bs)


def test_plan_refuses_outputs_over_its_inputs(lib):
    # bytes of each array for 4 requests, a table of 4 x 10, 5 free blocks, 6 tokens
    sizes = dict(ctx=16, new=16, table=160, free=20, seq=16, cu=20, pos=24, slots=48, taken=4)
    at = {n: A + 4096 * i for i, n in enumerate(sizes)}

    def call(**change):
        p = dict(at, **change)
        return lib.kv4_plan(p["ctx"], p["new"], 4, p["table"], 10, p["free"], 5, 16, 6, p["seq"], p["cu"], p["pos"],
                            p["slots"], p["taken"], None)
    outputs = ("table", "seq", "cu", "pos", "slots", "taken")
    for o in outputs:
        for other in sizes:
            if other == o:
                continue
            for shift in (0, 8, -8):      # the same address, and a part of either in the other
                place = at[other] + shift
                over = place < at[other] + sizes[other] and at[other] < place + sizes[o]
                assert call(**{o: place}) == (1 if over else call()), (o, other, shift)
            # side by side is no overlap
            assert call(**{o: at[other] + -(-sizes[other] // 8) * 8}) == call()
    assert call() in (0, 4)               # (4: no device here)


@pytest.mark.gpu
def test_plan_in_place_is_refused_by_the_binding():
    torch, w4 = cuda_or_skip()
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, new = torch.tensor([3, 20], **i32), torch.ones(2, **i32)
    out = w4.kv4_plan_buffers(2, 2)._replace(seq_lens=ctx)
    with pytest.raises(w4.W4A16Error, match="overlap"):
        w4.kv4_plan(ctx, new, torch.full((2, 4), -1, **i32), torch.arange(8, **i32), 16, out=out)
