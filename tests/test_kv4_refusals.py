"""Further refusals of the operators around the 4-bit cache that are checked on
the host, and the binding without its host extension: no GPU is needed."""
import pytest

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
